// dl_layer.cuh -- parameters and launchers of the operators around the
// recurrent step: the short convolution, the selective state space scan and
// the residual RMS norm.
#pragma once

#include <cuda_runtime.h>

#include "dl_common.cuh"
#include "dl_launch.cuh"
#include "dl_seqs.cuh"

namespace dl {

// Defined in dl_api.cu: the process's launch counter and the error word of
// kernels that run without a state (null when it cannot be had).
void count_launches(int n);
int* shared_err_word();

struct ConvParams {
  const void* x;      // [T, C] rows of ldx elements
  const float* w;     // [C, W]
  const float* bias;  // [C] or null
  const void* h0;     // [n, W-1, C] or null
  void* h1;           // [n, W-1, C] or null; may be h0
  void* y;            // [T, C] rows of ldy elements
  long long ldx, ldy;
  int C;
  int silu;
};

// bf16: element type; vec: whether four channels can be accessed at a time.
cudaError_t launch_conv_prompt(const ConvParams& p, int n, const int32_t* starts, int W, bool bf16,
                               bool vec, cudaStream_t s);
cudaError_t launch_conv_step(const ConvParams& p, int B, int W, bool bf16, bool vec, cudaStream_t s);

struct SsmParams {
  const void* q;
  const void* k;
  const void* v;
  const float* dt;
  const float* a;     // [H]
  const float* d;     // [H] or null
  const float* bias;  // [H] or null
  const float* S0;    // [n, H, DV, DK] or null
  float* S1;          // [n, H, DV, DK] or null; may be S0
  void* o;
  int* err;
  long long ldq, ldk, ldv, lddt, ldo;
  int H, G;
  int softplus;
};

cudaError_t launch_ssm_step(const SsmParams& p, int B, int dk, int dv, bool bf16, cudaStream_t s);

// How a prompt call is cut along its sequences, and the workspace that takes.
struct SsmPlan {
  int tile_tokens;
  size_t bytes;
};
// Workspace of the largest launch of a call: where some sequence is cut, every
// tile's state and its decay.
size_t ssm_tile_bytes(int H, int dk, int dv, int n, const int32_t* starts, int tile_tokens);

// bf16 rows, on the tensor cores.
SsmPlan plan_ssm(int H, int G, int dk, int dv, int n, const int32_t* starts, int sms);
cudaError_t launch_ssm_chunked(const SsmParams& p, int n, const int32_t* starts, int dk, int dv,
                               const SsmPlan& plan, void* ws, cudaStream_t s);
// fp32 rows, or no rows at all.
SsmPlan plan_ssm_scan(int H, int dk, int dv, int n, const int32_t* starts, int sms);
cudaError_t launch_ssm_scan(const SsmParams& p, int n, const int32_t* starts, int dk, int dv,
                            const SsmPlan& plan, void* ws, cudaStream_t s);
// Own states of the tiles of sequences seq0 .. -> states they enter with.
template <typename Table>
cudaError_t launch_ssm_join(const SsmParams& p, float* ws, const float* wdecay, const Table& tab, int seq0,
                            int n, int dk, int dv, cudaStream_t s);

constexpr int kOutF32 = 0, kOutBF16 = 1, kOutE4M3 = 2;

struct NormParams {
  const void* x;
  const void* res;   // or null
  const float* w;    // [D]
  void* res_out;     // or null
  void* out;
  float* scales;     // [rows, ceil(D / 128)] or [rows]; e4m3 only
  long long rows, ldx, ldr, ldro, ldo;
  int D;
  int block;         // 128 or 0 (one scale per row)
  float eps;
};

cudaError_t launch_norm(const NormParams& p, bool bf16, int out, bool vec, cudaStream_t s);

// log(1 + e^x) without overflow.
__device__ __forceinline__ float softplusf(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

}  // namespace dl
