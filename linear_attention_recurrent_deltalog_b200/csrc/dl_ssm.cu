// dl_ssm.cu -- the selective state space recurrence, one head's fp32 state S
// (d_v x d_k) at a time:
//     dt = softplus(dt_raw + bias_h),  S <- e^{dt a_h} S + dt v k^T,
//     o = S q + d_h v
// for single tokens and, token by token, for packed prompts.  A warp owns 16
// rows of the state in registers (WarpRows' geometry: a lane holds four
// neighbouring key channels of each of its rows), and the 16 row sums S q
// finish in one butterfly.
#include "dl_layer.cuh"

namespace dl {

namespace {

template <typename T>
__device__ __forceinline__ float4 load4_any(const T* p) { return load4(p); }

__device__ __forceinline__ float step_dt(const SsmParams& p, float raw, int h) {
  if (p.bias != nullptr) raw += p.bias[h];
  return p.softplus ? softplusf(raw) : raw;
}

// One step of the warp's rows: s is updated, and the finished sum o of row
// `jl` (relative to the warp's first) is returned; lanes l and l^1 hold the
// same row.
template <int DK>
__device__ __forceinline__ float rows_step(float4 (&s)[WarpRows<DK>::NV], float4 k4, float4 q4,
                                           float alpha, float dt, const float* v, int lane,
                                           int& jl) {
  using W = WarpRows<DK>;
  const int rsub = lane / W::LPR;
  float part[W::NV];
#pragma unroll
  for (int i = 0; i < W::NV; ++i) {
    const float u = dt * v[i * W::RPI + rsub];
    s[i].x = fmaf(u, k4.x, alpha * s[i].x);
    s[i].y = fmaf(u, k4.y, alpha * s[i].y);
    s[i].z = fmaf(u, k4.z, alpha * s[i].z);
    s[i].w = fmaf(u, k4.w, alpha * s[i].w);
    part[i] = dot4(s[i], q4);
  }
  jl = reduced_index<W::NV, W::LPR>(lane) * W::RPI + rsub;
  return reduce_rows<W::NV, W::LPR>(part, lane);
}

// -------------------------------------------------------------- one token
//
// Bound by HBM: the state is read and written once.  One CTA per head, a
// warp per 16 rows; every lane issues all its loads before it needs one.
template <int DK, int DV, typename T>
__global__ void __launch_bounds__(2 * DV)
dl_ssm_step_kernel(const SsmParams p) {
  using W = WarpRows<DK>;
  __shared__ float sv[DV];
  const long long b = blockIdx.x / unsigned(p.H);
  const int h = int(blockIdx.x % unsigned(p.H));
  const int g = h / (p.H / p.G);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = gemv_col<DK>(lane), rsub = lane / W::LPR;
  float* S = p.S1 + (size_t(b) * p.H + h) * size_t(DV) * DK + size_t(warp * 16) * DK;
  float4 s[W::NV];
#pragma unroll
  for (int i = 0; i < W::NV; ++i)
    s[i] = *reinterpret_cast<const float4*>(S + size_t(i * W::RPI + rsub) * DK + c0);
  const float4 k4 = load4_any(static_cast<const T*>(p.k) + b * p.ldk + g * DK + c0);
  const float4 q4 = load4_any(static_cast<const T*>(p.q) + b * p.ldq + g * DK + c0);
  if (lane < 16)
    sv[warp * 16 + lane] = to_f(static_cast<const T*>(p.v)[b * p.ldv + h * DV + warp * 16 + lane]);
  const float dt = step_dt(p, p.dt[b * p.lddt + h], h);
  const float alpha = expf(dt * p.a[h]);
  __syncwarp();
  int jl;
  const float o = rows_step<DK>(s, k4, q4, alpha, dt, sv + warp * 16, lane, jl);
#pragma unroll
  for (int i = 0; i < W::NV; ++i)
    *reinterpret_cast<float4*>(S + size_t(i * W::RPI + rsub) * DK + c0) = s[i];
  if ((lane & 1) == 0) {
    const int j = warp * 16 + jl;
    const float d = p.d != nullptr ? p.d[h] : 0.f;
    static_cast<T*>(p.o)[b * p.ldo + h * DV + j] = Elem<T>::from_f(fmaf(d, sv[j], o));
  }
}

// ------------------------------------------------------- prompts, in order
//
// One CTA per sequence and head walks the tokens with the whole state in
// registers, kScanTile tokens staged in shared memory at a time.  Bound by
// the fp32 pipe (3 operations per state element and token).
constexpr int kScanTile = 16;

template <int DK, int DV, typename T, typename Table>
__global__ void __launch_bounds__(2 * DV)
dl_ssm_scan_kernel(const SsmParams p, const __grid_constant__ Table seqs, int seq0) {
  using W = WarpRows<DK>;
  constexpr int NT = 2 * DV;
  __shared__ __align__(16) float sk[kScanTile][DK];
  __shared__ __align__(16) float sq[kScanTile][DK];
  __shared__ float sv[kScanTile][DV];
  __shared__ float sdt[kScanTile], sal[kScanTile];
  const int sl = int(blockIdx.x / unsigned(p.H));
  const int h = int(blockIdx.x % unsigned(p.H));
  const int g = h / (p.H / p.G);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c0 = gemv_col<DK>(lane), rsub = lane / W::LPR;
  const size_t off = ((size_t(seq0) + sl) * p.H + h) * size_t(DV) * DK + size_t(warp * 16) * DK;
  const int begin = seqs.start[sl], end = seqs.start[sl + 1];
  const float d = p.d != nullptr ? p.d[h] : 0.f;
  const float a = p.a[h];
  float4 s[W::NV];
#pragma unroll
  for (int i = 0; i < W::NV; ++i)
    s[i] = p.S0 != nullptr
               ? *reinterpret_cast<const float4*>(p.S0 + off + size_t(i * W::RPI + rsub) * DK + c0)
               : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = begin; t0 < end; t0 += kScanTile) {
    const int nt = min(kScanTile, end - t0);
    __syncthreads();
    for (int i = tid; i < nt * DK; i += NT) {
      const long long t = t0 + i / DK;
      sk[i / DK][i % DK] = to_f(static_cast<const T*>(p.k)[t * p.ldk + g * DK + i % DK]);
      sq[i / DK][i % DK] = to_f(static_cast<const T*>(p.q)[t * p.ldq + g * DK + i % DK]);
    }
    for (int i = tid; i < nt * DV; i += NT) {
      const long long t = t0 + i / DV;
      sv[i / DV][i % DV] = to_f(static_cast<const T*>(p.v)[t * p.ldv + h * DV + i % DV]);
    }
    if (tid < nt) {
      const float dt = step_dt(p, p.dt[(long long)(t0 + tid) * p.lddt + h], h);
      sdt[tid] = dt;
      sal[tid] = expf(dt * a);
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const float4 k4 = load4(&sk[t][c0]), q4 = load4(&sq[t][c0]);
      int jl;
      const float o = rows_step<DK>(s, k4, q4, sal[t], sdt[t], &sv[t][warp * 16], lane, jl);
      if ((lane & 1) == 0) {
        const int j = warp * 16 + jl;
        static_cast<T*>(p.o)[(long long)(t0 + t) * p.ldo + h * DV + j] =
            Elem<T>::from_f(fmaf(d, sv[t][j], o));
      }
    }
  }
  if (p.S1 != nullptr) {
#pragma unroll
    for (int i = 0; i < W::NV; ++i)
      *reinterpret_cast<float4*>(p.S1 + off + size_t(i * W::RPI + rsub) * DK + c0) = s[i];
  }
}

struct RunStep {
  const SsmParams& p;
  int B;
  cudaStream_t s;
  template <int DK, int DV, typename T>
  cudaError_t run() const {
    dl_ssm_step_kernel<DK, DV, T><<<unsigned(B) * unsigned(p.H), 2 * DV, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
  }
};

struct RunScan {
  const SsmParams& p;
  int n;
  const int32_t* starts;
  cudaStream_t s;
  template <int DK, int DV, typename T, int NS>
  cudaError_t range(int s0, int m) const {
    SeqTable<NS> tab;
    fill_seqs(tab, starts, s0, m, 1 << 30);
    dl_ssm_scan_kernel<DK, DV, T, SeqTable<NS>>
        <<<unsigned(m) * unsigned(p.H), 2 * DV, 0, s>>>(p, tab, s0);
    count_launches(1);
    return cudaGetLastError();
  }
  template <int DK, int DV, typename T>
  cudaError_t run() const {
    if (n <= kSmallSeqs) return range<DK, DV, T, kSmallSeqs>(0, n);
    for (int s0 = 0; s0 < n; s0 += kLargeSeqs) {
      const cudaError_t e =
          range<DK, DV, T, kLargeSeqs>(s0, n - s0 < kLargeSeqs ? n - s0 : kLargeSeqs);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
};

}  // namespace

cudaError_t launch_ssm_step(const SsmParams& p, int B, int dk, int dv, bool bf16, cudaStream_t s) {
  return dispatch_shape(Shape{dk, dv, bf16 ? 1 : 0, 1}, RunStep{p, B, s});
}

cudaError_t launch_ssm_scan(const SsmParams& p, int n, const int32_t* starts, int dk, int dv,
                            bool bf16, cudaStream_t s) {
  return dispatch_shape(Shape{dk, dv, bf16 ? 1 : 0, 1}, RunScan{p, n, starts, s});
}

}  // namespace dl
