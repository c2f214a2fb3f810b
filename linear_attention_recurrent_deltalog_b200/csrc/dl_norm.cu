// dl_norm.cu -- root-mean-square norm of x (+ residual) rows,
//     h = x + res,  n = h / sqrt(mean(h^2) + eps) * w,
// written as fp32, bf16, or e4m3 codes with one fp32 scale per row or per
// block of 128 channels (scale = amax / 448, code = e4m3(n * 448 / amax),
// blocks below 2^-120 stored as zeros with scale 0).  Bound by HBM: x and
// res are read once, res_out, the codes and the scales written once.  A team
// of TPR threads owns a row and keeps it in registers (fp32) between the sum
// of squares and the output; thread i takes 8 consecutive channels of each
// TPR * 8, so a 128-channel block belongs to 16 neighbouring lanes.
#include <cuda_fp8.h>

#include "dl_layer.cuh"

namespace dl {

namespace {

template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, bool vec, float (&v)[8]) {
  if (vec) {
    load_f<8>(p, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < left ? to_f(p[e]) : 0.f;
}

__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, int left, bool vec, const float (&v)[8]) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bf2(v[0], v[1]), bf2(v[2], v[3]), bf2(v[4], v[5]), bf2(v[6], v[7]));
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = __float2bfloat16_rn(v[e]);
}
__device__ __forceinline__ void store8(float* p, int left, bool vec, const float (&v)[8]) {
  if (vec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = v[e];
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3* p, int left, bool vec, const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE,
                                                 __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  if (vec) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    return;
  }
  uint8_t* b = reinterpret_cast<uint8_t*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) b[e] = uint8_t(w[e >> 2] >> (8 * (e & 3)));
}

// The larger magnitude; a NaN on either side stays.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum or maximum over a team of TPR threads (whole warps).
template <int TPR, bool MAX>
__device__ __forceinline__ float team_reduce(float x, float* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    x = MAX ? max_nan(x, y) : x + y;
  }
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sm[warp] = x;
    __syncthreads();
    x = sm[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) x = MAX ? max_nan(x, sm[i]) : x + sm[i];
  }
  return x;
}

template <typename T, typename TO, int TPR, int V, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
dl_norm_kernel(const NormParams p) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;  // rows a CTA covers
  __shared__ float red[2][TPR / 32];
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
  const int i = threadIdx.x % TPR;
  if (TPR == 32 && row >= p.rows) return;  // whole warps only
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* res = p.res != nullptr ? static_cast<const T*>(p.res) + row * p.ldr : nullptr;
  float h[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * TPR + i) * 8;
    if (c < p.D) {
      load8(x + c, p.D - c, VEC, h[v]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] = 0.f;
    }
  }
  if (res != nullptr) {
    float r[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + i) * 8;
      if (c < p.D) load8(res + c, p.D - c, VEC, r[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + i) * 8;
      if (c < p.D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] += r[v][e];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[v][e], h[v][e], ss);
  if (p.res_out != nullptr) {
    T* ro = static_cast<T*>(p.res_out) + row * p.ldro;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + i) * 8;
      if (c < p.D) store8(ro + c, p.D - c, VEC, h[v]);
    }
  }
  ss = team_reduce<TPR, false>(ss, red[0]);
  const float r = 1.f / sqrtf(ss / float(p.D) + p.eps);
  float rowmax = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * TPR + i) * 8;
    if (c >= p.D) continue;
    float w[8];
    load8(p.w + c, p.D - c, VEC, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[v][e] = h[v][e] * r * w[e];
  }
  TO* out = static_cast<TO*>(p.out) + row * p.ldo;
  if constexpr (std::is_same<TO, __nv_fp8_e4m3>::value) {
    float m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      m[v] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m[v] = max_nan(m[v], fabsf(h[v][e]));
      rowmax = max_nan(rowmax, m[v]);
    }
    if (p.block == 0) {
      rowmax = team_reduce<TPR, true>(rowmax, red[1]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m[v] = max_nan(m[v], __shfl_xor_sync(0xffffffffu, m[v], o));
    }
    const int nblk = p.block == 0 ? 1 : (p.D + 127) / 128;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + i) * 8;
      if (c >= p.D) continue;
      const float amax = p.block == 0 ? rowmax : m[v];
      const bool zero = amax < kTinyAmax;
      const float inv = zero ? 0.f : __fdiv_rn(448.f, amax);
      if (p.block == 0 ? c == 0 : c % 128 == 0)
        p.scales[row * nblk + (p.block == 0 ? 0 : c / 128)] = zero ? 0.f : __fdiv_rn(amax, 448.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] *= inv;
      store8(out + c, p.D - c, VEC, h[v]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * TPR + i) * 8;
      if (c < p.D) store8(out + c, p.D - c, VEC, h[v]);
    }
  }
}

template <typename T, typename TO, int TPR, int V, bool VEC>
cudaError_t norm_t(const NormParams& p, cudaStream_t s) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  const long long grid = (p.rows + kRows - 1) / kRows;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  dl_norm_kernel<T, TO, TPR, V, VEC><<<unsigned(grid), TPR < 128 ? 128 : TPR, 0, s>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

// The team and the 8-channel pieces a thread holds, by the row's length.
template <typename T, typename TO, bool VEC>
cudaError_t norm_by_length(const NormParams& p, cudaStream_t s) {
  if (p.D <= 256) return norm_t<T, TO, 32, 1, VEC>(p, s);
  if (p.D <= 1024) return norm_t<T, TO, 32, 4, VEC>(p, s);
  if (p.D <= 2048) return norm_t<T, TO, 128, 2, VEC>(p, s);
  if (p.D <= 4096) return norm_t<T, TO, 128, 4, VEC>(p, s);
  if (p.D <= 8192) return norm_t<T, TO, 256, 4, VEC>(p, s);
  return norm_t<T, TO, 512, 4, VEC>(p, s);
}

template <typename T, typename TO>
cudaError_t norm_by_access(const NormParams& p, bool vec, cudaStream_t s) {
  return vec ? norm_by_length<T, TO, true>(p, s) : norm_by_length<T, TO, false>(p, s);
}

template <typename T>
cudaError_t norm_by_out(const NormParams& p, int out, bool vec, cudaStream_t s) {
  switch (out) {
    case kOutF32: return norm_by_access<T, float>(p, vec, s);
    case kOutBF16: return norm_by_access<T, __nv_bfloat16>(p, vec, s);
    default: return norm_by_access<T, __nv_fp8_e4m3>(p, vec, s);
  }
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, bool bf16, int out, bool vec, cudaStream_t s) {
  return bf16 ? norm_by_out<__nv_bfloat16>(p, out, vec, s) : norm_by_out<float>(p, out, vec, s);
}

}  // namespace dl
