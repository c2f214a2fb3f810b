// dl_conv.cu -- the short depthwise causal convolution of a token's channels,
//     y[t, c] = act(bias[c] + sum_j w[c, j] x[t - W + 1 + j, c]),
// for packed prompts and for single tokens.  Rows before a sequence's first
// token come from its state (its last W - 1 input rows, oldest first).  Two
// flops a byte: bound by HBM.  A thread owns VEC neighbouring channels (16
// bytes) and walks down the tokens of its tile with the last W - 1 rows in
// registers, so an input row is read once, but for the W - 1 rows at the
// head of a tile.
#include "dl_layer.cuh"

namespace dl {

namespace {

constexpr int kConvThreads = 256;

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1)
    v[0] = to_f(p[0]);
  else
    load_f<VEC>(p, v);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    p[0] = Elem<T>::from_f(v[0]);
  } else {
    uint4 r;
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      r = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      r = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
    }
    *reinterpret_cast<uint4*>(p) = r;
  }
}

template <int VEC, int W>
struct Taps {
  float w[VEC][W], b[VEC];
  __device__ __forceinline__ Taps(const ConvParams& p, int c) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[e][j] = p.w[size_t(c + e) * W + j];
      b[e] = p.bias != nullptr ? p.bias[c + e] : 0.f;
    }
  }
};

// x / (1 + e^-x): __expf and __fdividef are within a few ulp here, below the
// rounding of either output type's tolerance; e^-x = inf gives -0.
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }

// One output row from the W rows old[0 .. W-2], cur.
template <int VEC, int W>
__device__ __forceinline__ void taps_row(const Taps<VEC, W>& t, const float (&old)[W - 1][VEC],
                                         const float (&cur)[VEC], bool act, float (&y)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float s = t.b[e];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = fmaf(t.w[e][j], old[j][e], s);
    s = fmaf(t.w[e][W - 1], cur[e], s);
    y[e] = act ? silu(s) : s;
  }
}

template <int VEC, int W>
__device__ __forceinline__ void shift(float (&old)[W - 1][VEC], const float (&cur)[VEC]) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) old[j][e] = old[j + 1][e];
#pragma unroll
  for (int e = 0; e < VEC; ++e) old[W - 2][e] = cur[e];
}

// Row `r` of the state of sequence s (zeros without one).
template <typename T, int VEC, int W>
__device__ __forceinline__ void state_row(const ConvParams& p, const void* h, size_t s, int r, int c,
                                          float (&v)[VEC]) {
  if (h == nullptr) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = 0.f;
    return;
  }
  load_vec<T, VEC>(static_cast<const T*>(h) + (s * (W - 1) + r) * size_t(p.C) + c, v);
}

template <typename T, int VEC, int W, int TILE, typename Table>
__global__ void __launch_bounds__(kConvThreads)
dl_conv_prompt_kernel(const ConvParams p, const __grid_constant__ Table seqs, int seq0, int nvec,
                      long long total) {
  const long long id = (long long)blockIdx.x * kConvThreads + threadIdx.x;
  if (id >= total) return;
  const int tile = int(id / nvec);
  const int c = int(id % nvec) * VEC;
  const int sl = seqs.find(tile);
  const int begin = seqs.start[sl], end = seqs.start[sl + 1];
  const int first = tile - seqs.tile0[sl];
  const int t0 = begin + first * TILE;
  const int t1 = min(t0 + TILE, end);
  const size_t s = size_t(seq0) + size_t(sl);
  const T* x = static_cast<const T*>(p.x) + c;
  T* y = static_cast<T*>(p.y) + c;
  const Taps<VEC, W> taps(p, c);
  float old[W - 1][VEC];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int t = t0 - (W - 1) + j;
    if (t >= begin)
      load_vec<T, VEC>(x + (long long)t * p.ldx, old[j]);
    else
      state_row<T, VEC, W>(p, p.h0, s, W - 1 + t - begin, c, old[j]);
  }
  // The first tile's thread is the only one to read these channels' old
  // state, so it also writes the new one and h1 may be h0.
  if (first == 0 && p.h1 != nullptr) {
    float nh[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int t = end - (W - 1) + j;
      if (t >= begin)
        load_vec<T, VEC>(x + (long long)t * p.ldx, nh[j]);
      else
        state_row<T, VEC, W>(p, p.h0, s, W - 1 + t - begin, c, nh[j]);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_vec<T, VEC>(static_cast<T*>(p.h1) + (s * (W - 1) + j) * size_t(p.C) + c, nh[j]);
  }
  constexpr int U = 8;  // rows in flight
  int t = t0;
  for (; t + U <= t1; t += U) {
    float cur[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) load_vec<T, VEC>(x + (long long)(t + u) * p.ldx, cur[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float o[VEC];
      taps_row<VEC, W>(taps, old, cur[u], p.silu != 0, o);
      store_vec<T, VEC>(y + (long long)(t + u) * p.ldy, o);
      shift<VEC, W>(old, cur[u]);
    }
  }
  for (; t < t1; ++t) {
    float cur[VEC], o[VEC];
    load_vec<T, VEC>(x + (long long)t * p.ldx, cur);
    taps_row<VEC, W>(taps, old, cur, p.silu != 0, o);
    store_vec<T, VEC>(y + (long long)t * p.ldy, o);
    shift<VEC, W>(old, cur);
  }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads)
dl_conv_step_kernel(const ConvParams p, int nvec, long long total) {
  const long long id = (long long)blockIdx.x * kConvThreads + threadIdx.x;
  if (id >= total) return;
  const size_t b = size_t(id / nvec);
  const int c = int(id % nvec) * VEC;
  float old[W - 1][VEC], cur[VEC], o[VEC];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) state_row<T, VEC, W>(p, p.h0, b, j, c, old[j]);
  load_vec<T, VEC>(static_cast<const T*>(p.x) + (long long)b * p.ldx + c, cur);
  const Taps<VEC, W> taps(p, c);
  taps_row<VEC, W>(taps, old, cur, p.silu != 0, o);
  store_vec<T, VEC>(static_cast<T*>(p.y) + (long long)b * p.ldy + c, o);
  shift<VEC, W>(old, cur);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    store_vec<T, VEC>(static_cast<T*>(p.h1) + (b * (W - 1) + j) * size_t(p.C) + c, old[j]);
}

template <typename T, int VEC, int W, int TILE, int NS>
cudaError_t conv_prompt_range(const ConvParams& p, const int32_t* starts, int s0, int n,
                              cudaStream_t s) {
  SeqTable<NS> tab;
  const int nvec = p.C / VEC;
  const long long total = fill_seqs(tab, starts, s0, n, TILE) * nvec;
  const long long grid = (total + kConvThreads - 1) / kConvThreads;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  dl_conv_prompt_kernel<T, VEC, W, TILE, SeqTable<NS>>
      <<<unsigned(grid), kConvThreads, 0, s>>>(p, tab, s0, nvec, total);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int VEC, int W, int TILE>
cudaError_t conv_prompt_tiled(const ConvParams& p, int n, const int32_t* starts, cudaStream_t s) {
  if (n <= kSmallSeqs) return conv_prompt_range<T, VEC, W, TILE, kSmallSeqs>(p, starts, 0, n, s);
  for (int s0 = 0; s0 < n; s0 += kLargeSeqs) {
    const int m = n - s0 < kLargeSeqs ? n - s0 : kLargeSeqs;
    const cudaError_t e = conv_prompt_range<T, VEC, W, TILE, kLargeSeqs>(p, starts, s0, m, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int VEC, int W>
cudaError_t conv_prompt_t(const ConvParams& p, int n, const int32_t* starts, cudaStream_t s) {
  return conv_prompt_tiled<T, VEC, W, 32>(p, n, starts, s);
}

template <typename T, int VEC, int W>
cudaError_t conv_step_t(const ConvParams& p, int B, cudaStream_t s) {
  const int nvec = p.C / VEC;
  const long long total = (long long)B * nvec;
  const long long grid = (total + kConvThreads - 1) / kConvThreads;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  dl_conv_step_kernel<T, VEC, W><<<unsigned(grid), kConvThreads, 0, s>>>(p, nvec, total);
  count_launches(1);
  return cudaGetLastError();
}

// f.run<T, VEC, W>() for the runtime type, access width and filter width.
template <typename T, int VEC, typename F>
cudaError_t by_width(int W, F&& f) {
  switch (W) {
    case 2: return f.template run<T, VEC, 2>();
    case 3: return f.template run<T, VEC, 3>();
    default: return f.template run<T, VEC, 4>();
  }
}
template <typename F>
cudaError_t by_type(int W, bool bf16, bool vec, F&& f) {
  if (bf16)
    return vec ? by_width<__nv_bfloat16, 8>(W, f) : by_width<__nv_bfloat16, 1>(W, f);
  return vec ? by_width<float, 4>(W, f) : by_width<float, 1>(W, f);
}

struct RunPrompt {
  const ConvParams& p;
  int n;
  const int32_t* starts;
  cudaStream_t s;
  template <typename T, int VEC, int W>
  cudaError_t run() const { return conv_prompt_t<T, VEC, W>(p, n, starts, s); }
};
struct RunStep {
  const ConvParams& p;
  int B;
  cudaStream_t s;
  template <typename T, int VEC, int W>
  cudaError_t run() const { return conv_step_t<T, VEC, W>(p, B, s); }
};

}  // namespace

cudaError_t launch_conv_prompt(const ConvParams& p, int n, const int32_t* starts, int W, bool bf16,
                               bool vec, cudaStream_t s) {
  return by_type(W, bf16, vec, RunPrompt{p, n, starts, s});
}

cudaError_t launch_conv_step(const ConvParams& p, int B, int W, bool bf16, bool vec, cudaStream_t s) {
  return by_type(W, bf16, vec, RunStep{p, B, s});
}

}  // namespace dl
