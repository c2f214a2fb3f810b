// dl_conv.cu -- the short depthwise causal convolution of a token's channels,
//     y[t, c] = act(bias[c] + sum_j w[c, j] x[t - W + 1 + j, c]),
// for packed prompts and for single tokens.  Rows before a sequence's first
// token come from its state (its last W - 1 input rows, oldest first).  Two
// flops a byte: bound by memory (T = 8192, C = 4352, W = 4, bf16: 31 us in a
// replayed graph, 4.7 TB/s of rows in and out; fewer instructions or reciprocals, or
// rows further ahead, made it no faster, and the 8-byte accesses alone do not hold
// it: fp32 rows of the same bytes, 16 at a time, take as long, both 29 without the
// activation).  A thread owns VEC neighbouring channels: four where the rows allow
// 8-byte (bf16) or 16-byte (fp32) accesses, else one.
// Eight bf16 channels a thread were slower: their taps (fp32, 128 bytes a
// thread at W = 4) and the rows in flight leave room for a third of the warps.
// A prompt's thread walks down the tokens of its tile with the last W - 1 rows
// in registers, so an input row is read once, but for the W - 1 rows at the
// head of a tile; a step's thread takes several sequences, so that the taps
// are read once for all of them (B = 512, C = 4352: 5.4 us, 41 with eight channels
// and one sequence a thread).
#include "dl_layer.cuh"

namespace dl {

namespace {

constexpr int kConvThreads = 256;

// VEC channels of a row as they lie in memory.
template <typename T, int VEC>
struct Raw {
  T e[VEC];
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 r;
};
template <>
struct Raw<float, 4> {
  float4 r;
};

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
  return *reinterpret_cast<const Raw<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> zero_raw() {
  Raw<T, VEC> z;
  memset(&z, 0, sizeof(z));
  return z;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 4>& x, float (&v)[4]) {
  v[0] = __uint_as_float(x.r.x << 16);
  v[1] = __uint_as_float(x.r.x & 0xffff0000u);
  v[2] = __uint_as_float(x.r.y << 16);
  v[3] = __uint_as_float(x.r.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const Raw<float, 4>& x, float (&v)[4]) {
  v[0] = x.r.x;
  v[1] = x.r.y;
  v[2] = x.r.z;
  v[3] = x.r.w;
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw<T, 1>& x, float (&v)[1]) {
  v[0] = to_f(x.e[0]);
}

__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store_vec(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[1]) {
  p[0] = Elem<T>::from_f(v[0]);
}

// The taps of channels c .. c + VEC - 1: VEC * W neighbouring floats.
template <int VEC, int W>
struct Taps {
  float w[VEC * W], b[VEC];
  __device__ __forceinline__ Taps(const ConvParams& p, int c) {
    const float* src = p.w + size_t(c) * W;
    if constexpr (VEC == 4) {
      load_f<VEC * W>(src, w);
      if (p.bias != nullptr) {
        load_f<VEC>(p.bias + c, b);
        return;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC * W; ++j) w[j] = src[j];
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) b[e] = p.bias != nullptr ? p.bias[c + e] : 0.f;
  }
};

// x / (1 + e^-x).  For bf16 rows with the hardware's exponential and reciprocal:
// the rounding of x log2(e) leaves the exponential right to |x| units of 2^-24 or
// so (60 at x = -60), far below the output's 2^-9.  Their forms that flush
// denormals need no scaling around them (a third of the kernel's instructions
// otherwise); from x = -87.3 down (|y| < 2^-119) the result is -0.
__device__ __forceinline__ float silu(float x, __nv_bfloat16) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return x * r;
}
// For fp32 rows right to a few units of 2^-24 wherever the result is normal: e^-|x|
// cannot overflow, and its product with x comes before the quotient's.  The
// divisor lies in [1, 2], so one Newton step makes the reciprocal whole (T = 8192,
// C = 2176: 31 us; 39 with the library's rounded reciprocal, 29.5 with bf16's form).
__device__ __forceinline__ float silu(float x, float) {
  const float e = expf(-fabsf(x)), d = 1.f + e;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  r = fmaf(r, fmaf(-d, r, 1.f), r);
  return x * (x < 0.f ? e : 1.f) * r;
}

// One output row from the W rows old[0 .. W-2], cur.
template <typename T, int VEC, int W>
__device__ __forceinline__ void taps_row(const Taps<VEC, W>& t, const float (&old)[W - 1][VEC],
                                         const float (&cur)[VEC], bool act, float (&y)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float s = t.b[e];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = fmaf(t.w[e * W + j], old[j][e], s);
    s = fmaf(t.w[e * W + W - 1], cur[e], s);
    y[e] = act ? silu(s, T{}) : s;
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
__device__ __forceinline__ Raw<T, VEC> state_row(const ConvParams& p, size_t s, int r, int c) {
  if (p.h0 == nullptr) return zero_raw<T, VEC>();
  return load_raw<T, VEC>(static_cast<const T*>(p.h0) + (s * (W - 1) + r) * size_t(p.C) + c);
}

constexpr int kRowsInFlight = 4;

template <typename T, int VEC, int W, typename Table>
__global__ void __launch_bounds__(kConvThreads, sizeof(T) == 2 ? 3 : 2)
dl_conv_prompt_kernel(const ConvParams p, const __grid_constant__ Table seqs, int seq0, unsigned nvec,
                      unsigned total, int tile_rows) {
  const unsigned id = blockIdx.x * unsigned(kConvThreads) + threadIdx.x;
  if (id >= total) return;
  const int tile = int(id / nvec);
  const int c = int(id % nvec) * VEC;
  const int sl = seqs.find(tile);
  const int begin = seqs.start[sl], end = seqs.start[sl + 1];
  const int first = tile - seqs.tile0[sl];
  const int t0 = begin + first * tile_rows;
  const int t1 = min(t0 + tile_rows, end);
  const size_t s = size_t(seq0) + size_t(sl);
  const T* x = static_cast<const T*>(p.x) + c;
  T* y = static_cast<T*>(p.y) + c;
  constexpr int U = kRowsInFlight;
  Raw<T, VEC> next[U];
  auto fetch = [&](int t) {
    const T* src = x + (long long)t * p.ldx;
    if (t + U <= t1) {
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = load_raw<T, VEC>(src + u * p.ldx);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t + u < t1) next[u] = load_raw<T, VEC>(src + u * p.ldx);
    }
  };
  fetch(t0);
  const Taps<VEC, W> taps(p, c);
  float old[W - 1][VEC];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int t = t0 - (W - 1) + j;
    unpack(t >= begin ? load_raw<T, VEC>(x + (long long)t * p.ldx)
                      : state_row<T, VEC, W>(p, s, W - 1 + t - begin, c),
           old[j]);
  }
  // The first tile's thread is the only one to read these channels' old
  // state, so it also writes the new one and h1 may be h0.
  if (first == 0 && p.h1 != nullptr) {
    Raw<T, VEC> nh[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int t = end - (W - 1) + j;
      nh[j] = t >= begin ? load_raw<T, VEC>(x + (long long)t * p.ldx)
                         : state_row<T, VEC, W>(p, s, W - 1 + t - begin, c);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      *reinterpret_cast<Raw<T, VEC>*>(static_cast<T*>(p.h1) + (s * (W - 1) + j) * size_t(p.C) + c) = nh[j];
  }
  for (int t = t0; t < t1; t += U) {
    Raw<T, VEC> cur[U];
#pragma unroll
    for (int u = 0; u < U; ++u) cur[u] = next[u];
    fetch(t + U);
    float o[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float in[VEC];
      unpack(cur[u], in);
      taps_row<T, VEC, W>(taps, old, in, p.silu != 0, o[u]);
      shift<VEC, W>(old, in);
    }
    T* dst = y + (long long)t * p.ldy;
    if (t + U <= t1) {
#pragma unroll
      for (int u = 0; u < U; ++u) store_vec(dst + u * p.ldy, o[u]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t + u < t1) store_vec(dst + u * p.ldy, o[u]);
    }
  }
}

// One token of `rows` sequences (b0, b0 + 1, ..) per thread.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads)
dl_conv_step_kernel(const ConvParams p, int B, unsigned nvec, unsigned total, int rows) {
  const unsigned id = blockIdx.x * unsigned(kConvThreads) + threadIdx.x;
  if (id >= total) return;
  const int c = int(id % nvec) * VEC;
  const int b0 = int(id / nvec) * rows, b1 = min(b0 + rows, B);
  const Taps<VEC, W> taps(p, c);
  constexpr int U = 4;  // sequences in flight
  const T* x = static_cast<const T*>(p.x) + c;
  T* y = static_cast<T*>(p.y) + c;
  for (int b = b0; b < b1; b += U) {
    Raw<T, VEC> r[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u >= b1) continue;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) r[u][j] = state_row<T, VEC, W>(p, size_t(b + u), j, c);
      r[u][W - 1] = load_raw<T, VEC>(x + (long long)(b + u) * p.ldx);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u >= b1) continue;
      float old[W - 1][VEC], in[VEC], o[VEC];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) unpack(r[u][j], old[j]);
      unpack(r[u][W - 1], in);
      taps_row<T, VEC, W>(taps, old, in, p.silu != 0, o);
      store_vec(y + (long long)(b + u) * p.ldy, o);
      T* h = static_cast<T*>(p.h1) + size_t(b + u) * (W - 1) * size_t(p.C) + c;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        *reinterpret_cast<Raw<T, VEC>*>(h + size_t(j) * size_t(p.C)) = r[u][j + 1];
    }
  }
}

// Threads that fill the device once.
long long one_wave() { return (long long)(sm_count() > 0 ? sm_count() : 1) * 3 * kConvThreads; }

template <typename T, int VEC, int W, int NS>
cudaError_t conv_prompt_range(const ConvParams& p, const int32_t* starts, int s0, int n,
                              cudaStream_t s) {
  SeqTable<NS> tab;
  const int nvec = p.C / VEC;
  // Tiles that fill whole waves of threads, 96 rows at most (T = 8192, C = 4352:
  // 32 us at 80 rows, 35 at 32, 41 at 8), 8 at least: a tile re-reads W - 1 rows.
  const long long rows = (long long)starts[s0 + n] - starts[s0];
  const long long deep = (rows * nvec + one_wave() - 1) / one_wave();  // rows a thread in one wave
  const long long waves = (deep + 95) / 96;
  int tile = waves == 0 ? 8 : int((deep + waves * 8 - 1) / (waves * 8)) * 8;
  long long total = fill_seqs(tab, starts, s0, n, tile) * nvec;
  for (int i = 0; i < 4 && tile > 8 && total > waves * one_wave(); ++i) {  // the sequences' last, short tiles
    tile += 8;
    total = fill_seqs(tab, starts, s0, n, tile) * nvec;
  }
  if (total > 0xffffffffLL - kConvThreads) return cudaErrorInvalidConfiguration;
  const unsigned grid = unsigned((total + kConvThreads - 1) / kConvThreads);
  dl_conv_prompt_kernel<T, VEC, W, SeqTable<NS>>
      <<<grid, kConvThreads, 0, s>>>(p, tab, s0, unsigned(nvec), unsigned(total), tile);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int VEC, int W>
cudaError_t conv_prompt_t(const ConvParams& p, int n, const int32_t* starts, cudaStream_t s) {
  if (n <= kSmallSeqs) return conv_prompt_range<T, VEC, W, kSmallSeqs>(p, starts, 0, n, s);
  for (int s0 = 0; s0 < n; s0 += kLargeSeqs) {
    const int m = n - s0 < kLargeSeqs ? n - s0 : kLargeSeqs;
    const cudaError_t e = conv_prompt_range<T, VEC, W, kLargeSeqs>(p, starts, s0, m, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int VEC, int W>
cudaError_t conv_step_t(const ConvParams& p, int B, cudaStream_t s) {
  const int nvec = p.C / VEC;
  // as many sequences a thread as leave half a wave of threads, at most 8
  long long rows = (long long)B * nvec / (one_wave() / 2);
  rows = rows < 1 ? 1 : (rows > 8 ? 8 : rows);
  const long long total = (B + rows - 1) / rows * nvec;
  if (total > 0xffffffffLL - kConvThreads) return cudaErrorInvalidConfiguration;
  const unsigned grid = unsigned((total + kConvThreads - 1) / kConvThreads);
  dl_conv_step_kernel<T, VEC, W>
      <<<grid, kConvThreads, 0, s>>>(p, B, unsigned(nvec), unsigned(total), int(rows));
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
    return vec ? by_width<__nv_bfloat16, 4>(W, f) : by_width<__nv_bfloat16, 1>(W, f);
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
