// dl_norm.cu -- root-mean-square norm of x (+ residual) rows,
//     h = x + res,  n = h / sqrt(mean(h^2) + eps) * w,
// written as fp32, bf16, or e4m3 codes with one fp32 scale per row or per
// block of 128 channels (scale = amax / 448, code = e4m3(n * 448 / amax),
// blocks below 2^-120 stored as zeros with scale 0).  Bound by HBM: x and
// res are read once, res_out, the codes and the scales written once (8192 rows of
// 4096, bf16 to e4m3 with the residual: 40 us, 5.9 TB/s, 0.90 of a copy's rate;
// 53 with one row a CTA and w read anew for each).
//
// A team of TPR threads owns a row and keeps it in registers (fp32) between
// the sum of squares and the output; a 128-channel block belongs to 16
// neighbouring lanes, 8 channels each.  The grid holds as many teams as run
// at once: each walks down the rows with its part of w in registers and the
// next row's loads in flight while it finishes this one.
#include <cuda_fp8.h>

#include "dl_layer.cuh"

namespace dl {

namespace {

// Eight channels of a row as they lie in memory.  VEC: one or two 16-byte
// accesses; else element by element, 16 channels apart, so that the 16 lanes
// of a block touch neighbours.
template <typename T, bool VEC>
struct Raw8 {
  T e[8];
  __device__ __forceinline__ void load(const T* row, int c, int D) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < D) e[i] = row[c + 16 * i];
  }
  __device__ __forceinline__ float get(int i) const { return to_f(e[i]); }
};
template <>
struct Raw8<__nv_bfloat16, true> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int c, int D) {
    if (c < D) r = *reinterpret_cast<const uint4*>(row + c);
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 4 ? (i < 2 ? r.x : r.y) : (i < 6 ? r.z : r.w);
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <>
struct Raw8<float, true> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* row, int c, int D) {
    if (c < D) {
      a = reinterpret_cast<const float4*>(row + c)[0];
      b = reinterpret_cast<const float4*>(row + c)[1];
    }
  }
  __device__ __forceinline__ float get(int i) const {
    const float4 v = i < 4 ? a : b;
    return (i & 2) ? ((i & 1) ? v.w : v.z) : ((i & 1) ? v.y : v.x);
  }
};

__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The same eight channels on the way out.
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    if (c < D)
      *reinterpret_cast<uint4*>(row + c) =
          make_uint4(bf2(v[0], v[1]), bf2(v[2], v[3]), bf2(v[4], v[5]), bf2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < D) row[c + 16 * i] = __float2bfloat16_rn(v[i]);
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* row, int c, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    if (c < D) {
      reinterpret_cast<float4*>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < D) row[c + 16 * i] = v[i];
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_fp8_e4m3* row, int c, int D, const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE,
                                                 __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  if constexpr (VEC) {
    if (c < D) *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
  } else {
    uint8_t* b = reinterpret_cast<uint8_t*>(row);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < D) b[c + 16 * i] = uint8_t(w[i >> 2] >> (8 * (i & 3)));
  }
}

constexpr float kSmallAmax = 0x1p-64f, kSmallUp = 0x1p64f;

// The larger magnitude; a NaN on either side stays.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum or maximum over a team of TPR threads: lanes of a warp, or a CTA.
template <int TPR, bool MAX>
__device__ __forceinline__ float team_reduce(float x, float* sm) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
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

template <int TPR>
constexpr int kNormThreads = TPR < 128 ? 128 : TPR;

// CTAs an SM must hold: 768 threads of 80 registers keep 48 KB of bf16 loads
// in flight; fp32 rows (twice the bytes a thread) and odd ones take 128
// registers and 512 threads.
template <typename T, int TPR, bool VEC>
constexpr int kNormCtas = (sizeof(T) == 2 && VEC ? 768 : 512) / kNormThreads<TPR>;

template <typename T, typename TO, int TPR, int V, bool VEC>
__global__ void __launch_bounds__(kNormThreads<TPR>, kNormCtas<T, TPR, VEC>)
dl_norm_kernel(const NormParams p) {
  constexpr bool kCodes = std::is_same<TO, __nv_fp8_e4m3>::value;
  constexpr int kRows = kNormThreads<TPR> / TPR;  // rows a CTA covers at a time
  // two sets, used in turn: a thread may still read one when another writes the next row's
  __shared__ float red[2][2][TPR / 32 + 1];
  const int i = threadIdx.x % TPR;
  const int D = p.D;
  int c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = VEC ? (v * TPR + i) * 8 : (v * TPR + (i & ~15)) * 8 + (i & 15);
  const long long step = (long long)gridDim.x * kRows;
  long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
  // the row of the warp's first team: every lane takes the same turns
  long long lead = TPR < 32 ? (long long)blockIdx.x * kRows + (threadIdx.x & ~31) / TPR : row;
  Raw8<T, VEC> x[V], r[V];
  auto fetch = [&](long long at) {
    if (at >= p.rows) return;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v].load(static_cast<const T*>(p.x) + at * p.ldx, c[v], D);
    if (p.res != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) r[v].load(static_cast<const T*>(p.res) + at * p.ldr, c[v], D);
    }
  };
  fetch(row);
  float w[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    Raw8<float, VEC> t;
    t.load(p.w, c[v], D);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[v][e] = (VEC ? c[v] : c[v] + 16 * e) < D ? t.get(e) : 0.f;
  }
  const int nblk = p.block == 0 ? 1 : (D + 127) / 128;
  for (int turn = 0; lead < p.rows; lead += step, row += step, turn ^= 1) {
    const bool live = TPR >= 32 || row < p.rows;
    float h[V][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float t = x[v].get(e);
        if (p.res != nullptr) t += r[v].get(e);
        h[v][e] = live && (VEC ? c[v] : c[v] + 16 * e) < D ? t : 0.f;
        ss = fmaf(h[v][e], h[v][e], ss);
      }
    fetch(row + step);
    if (p.res_out != nullptr && live) {
      T* ro = static_cast<T*>(p.res_out) + row * p.ldro;
#pragma unroll
      for (int v = 0; v < V; ++v) store8<VEC>(ro, c[v], D, h[v]);
    }
    ss = team_reduce<TPR, false>(ss, red[turn][0]);
    const float rn = 1.f / sqrtf(ss / float(D) + p.eps);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] = h[v][e] * rn * w[v][e];
    TO* out = static_cast<TO*>(p.out) + row * p.ldo;
    if constexpr (kCodes) {
      float m[V], rowmax = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        m[v] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m[v] = max_nan(m[v], fabsf(h[v][e]));
        rowmax = max_nan(rowmax, m[v]);
      }
      if (p.block == 0) {
        rowmax = team_reduce<TPR, true>(rowmax, red[turn][1]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m[v] = max_nan(m[v], __shfl_xor_sync(0xffffffffu, m[v], o));
      }
      if (!live) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float amax = p.block == 0 ? rowmax : m[v];
        const bool zero = amax < kTinyAmax;
        // 448 / amax leaves fp32's range from amax = 1.75 * 2^-120 down: small
        // blocks are brought up by a power of two first, which rounds nothing
        const bool small = amax < kSmallAmax;
        if (small) {
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] *= kSmallUp;
        }
        const float inv = zero ? 0.f : __fdiv_rn(448.f, small ? amax * kSmallUp : amax);
        const int first = VEC ? c[v] : c[v] - (i & 15) + (i & 15) * 8;  // as if it held 8 neighbours
        if (p.block == 0 ? first == 0 : (first % 128 == 0 && first < D))
          p.scales[row * nblk + (p.block == 0 ? 0 : first / 128)] = zero ? 0.f : __fdiv_rn(amax, 448.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] *= inv;
        store8<VEC>(out, c[v], D, h[v]);
      }
    } else if (live) {
#pragma unroll
      for (int v = 0; v < V; ++v) store8<VEC>(out, c[v], D, h[v]);
    }
  }
}

template <typename T, typename TO, int TPR, int V, bool VEC>
cudaError_t norm_t(const NormParams& p, cudaStream_t s) {
  constexpr int kRows = kNormThreads<TPR> / TPR;
  static std::atomic<int> per_sm{0};
  auto kern = dl_norm_kernel<T, TO, TPR, V, VEC>;
  int n = per_sm.load(std::memory_order_relaxed);
  if (n == 0) {
    const cudaError_t e =
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kNormThreads<TPR>, 0);
    if (e != cudaSuccess) return e;
    per_sm.store(n, std::memory_order_relaxed);
  }
  const long long most = (long long)n * sm_count();
  if (most <= 0) return cudaErrorInvalidConfiguration;
  const long long need = (p.rows + kRows - 1) / kRows;
  kern<<<unsigned(need < most ? need : most), kNormThreads<TPR>, 0, s>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

// The team and the 8-channel pieces a thread holds, by the row's length: the
// smallest team that holds a row in two pieces a thread (one below 257, where a
// warp or half of one is enough, and between 513 and 1024), since lanes without
// channels cost as much as others and the root is a team's work.  bf16 rows with the
// residual to e4m3, 2^23 channels in all, in us for this team and the others that
// hold the row (threads x pieces):
//     128    16x1 11.7   32x1 20.3   32x2 28.4
//     256    32x1 11.4   32x2 15.5   64x1 19.5   128x1 33.0
//     512    32x2 10.2   64x1 11.7   128x1 18.7
//     1024   128x1 11.3  64x2 10.6   128x2 15.6  32x4 18.8
//     2048   128x2 10.5  256x1 11.7  256x2 15.8
//     4096   256x2 10.9  512x1 15.3  512x2 18.5
//     8192   512x2 12.5  512x4 17.7
// The other types order alike (fp32 rows of 767: 32x4 42, 128x1 20, 64x2 19).
template <typename T, typename TO, bool VEC>
cudaError_t norm_by_length(const NormParams& p, cudaStream_t s) {
  if (p.D <= 128) return norm_t<T, TO, 16, 1, VEC>(p, s);
  if (p.D <= 256) return norm_t<T, TO, 32, 1, VEC>(p, s);
  if (p.D <= 512) return norm_t<T, TO, 32, 2, VEC>(p, s);
  if (p.D <= 1024) return norm_t<T, TO, 128, 1, VEC>(p, s);
  if (p.D <= 2048) return norm_t<T, TO, 128, 2, VEC>(p, s);
  if (p.D <= 4096) return norm_t<T, TO, 256, 2, VEC>(p, s);
  if (p.D <= 8192) return norm_t<T, TO, 512, 2, VEC>(p, s);
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
