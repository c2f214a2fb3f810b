// dl_ssm.cu -- the selective state space recurrence, one head's fp32 state S
// (d_v x d_k) at a time:
//     dt = softplus(dt_raw + bias_h),  S <- e^{dt a_h} S + dt v k^T,
//     o = S q + d_h v
// for single tokens and, token by token, for packed prompts of fp32 rows.
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
// Bound by HBM: the state is read and written once (B = 256, H = 64, d = 128 x 64:
// 160 us, 6.75 TB/s: a torch copy of 2 GB runs at 6.55, the fastest stream measured
// at 6.83).  One CTA per head; a warp
// owns 16 rows of the state in registers (WarpRows' geometry: a lane holds four
// neighbouring key channels of each of its rows) and issues all its loads before
// it needs one, and the 16 row sums S q finish in one butterfly.
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
// For fp32 rows (on the tensor cores each product would be three to nine).  Rows
// of the state are independent, so a warp takes few of them, four, and walks
// down the tokens with its part in registers: four key channels a lane, all
// four rows at d_k = 128, two of them at 64.  (Eight lanes a row needed fewer
// shuffles for the row sums S q but four times the reads of k and q, and those
// bounded it.)  Bound by the fp32 pipe (3 operations per state element and
// token) where the rows fill the device and by the instructions of one warp,
// 70 a token, where they do not (T = 2048, H = 64, d = 128 x 64: 285 us, 19
// TFLOP/s; H = 4, cut: 50 us).  A CTA (16
// rows) stages kScanTile tokens in shared memory, the next tile in flight.
// Sequences too few to fill the device are cut into tiles along their length:
// a first launch (STATES) forms every tile's own state from zero and
// dl_ssm_join_kernel turns those into the states the tiles enter with.
constexpr int kScanTile = 16;
constexpr int kScanRows = 16;  // rows of the state a CTA covers
constexpr int kScanThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

// 16 bytes to shared memory; zeros where there is no token.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16u : 0u)
               : "memory");
}

struct ScanTiles {
  float* ws;       // [tiles, H, DK, DV]
  float* wdecay;   // [tiles, H] log2 of a tile's whole decay
  int tile_tokens;
};

template <int DK, int DV, bool STATES, typename Table>
__global__ void __launch_bounds__(kScanThreads)
dl_ssm_scan_kernel(const SsmParams p, const ScanTiles cut, const __grid_constant__ Table seqs, int seq0) {
  constexpr int NR = DK / 32;             // rows a lane holds four channels of
  constexpr int kCols = DK / 4;           // lanes a row
  constexpr int kParts = DV / kScanRows;  // CTAs a head
  __shared__ __align__(16) float sk[2][kScanTile][DK];
  __shared__ __align__(16) float sq[2][kScanTile][STATES ? 4 : DK];
  __shared__ __align__(16) float sv[2][kScanTile][kScanRows];
  __shared__ __align__(16) float so[kScanTile][kScanRows];
  __shared__ float2 sdt[2][kScanTile];    // dt, e^{dt a}
  const int part = int(blockIdx.x % unsigned(kParts));
  const int h = int(blockIdx.x / unsigned(kParts) % unsigned(p.H));
  const int tile = int(blockIdx.x / unsigned(kParts * p.H));
  const int sl = seqs.find(tile);
  const int first_tile = seqs.tile0[sl], ntiles = seqs.tile0[sl + 1] - first_tile;
  const bool last_tile = tile - first_tile == ntiles - 1;
  if (STATES && last_tile) return;  // nobody enters from a last tile's own state
  const int begin = seqs.start[sl] + (tile - first_tile) * cut.tile_tokens;
  const int end = last_tile ? seqs.start[sl + 1] : begin + cut.tile_tokens;
  const int g = h / (p.H / p.G);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = warp * 4 + lane / kCols * NR, c0 = lane % kCols * 4;  // this lane's rows (of 16) and channels
  const int row = part * kScanRows + r0;
  const size_t user = ((size_t(seq0) + sl) * p.H + h) * size_t(DV) * DK + size_t(row) * DK + c0;
  const size_t tiled = (size_t(tile) * p.H + h) * size_t(DV) * DK + size_t(c0) * DV + row;
  const float* q = static_cast<const float*>(p.q) + g * DK;
  const float* k = static_cast<const float*>(p.k) + g * DK;
  const float* v = static_cast<const float*>(p.v) + h * DV + part * kScanRows;
  float* o = static_cast<float*>(p.o) + h * DV + part * kScanRows;
  const float a = p.a[h];
  const float d = !STATES && p.d != nullptr ? p.d[h] : 0.f;

  auto stage = [&](int t0, int b) {  // rows t0 .. of k, q and v
    for (int i = tid; i < kScanTile * (DK / 4); i += kScanThreads) {
      const int t = i / (DK / 4), c = i % (DK / 4) * 4;
      const bool there = t0 + t < end;
      const long long at = there ? t0 + t : begin;
      copy16(&sk[b][t][c], k + at * p.ldk + c, there);
      if (!STATES) copy16(&sq[b][t][STATES ? 0 : c], q + at * p.ldq + c, there);
    }
    if (tid < kScanTile * kScanRows / 4) {
      const int t = tid / (kScanRows / 4), c = tid % (kScanRows / 4) * 4;
      const bool there = t0 + t < end;
      copy16(&sv[b][t][c], v + (there ? t0 + t : begin) * p.ldv + c, there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto raw_dt = [&](int t0) {
    return tid < kScanTile && t0 + tid < end ? p.dt[(long long)(t0 + tid) * p.lddt + h] : 0.f;
  };
  float forgot = 0.f;  // this thread's tokens' log2 decays (STATES)
  auto put_dt = [&](int t0, int b, float raw) {  // behind the end the state stays as it is
    if (tid >= kScanTile) return;
    const float dt = t0 + tid < end ? step_dt(p, raw, h) : 0.f;
    sdt[b][tid] = make_float2(dt, expf(dt * a));
    if (STATES) forgot += dt * a * kLog2e;
  };

  float4 s[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (STATES) continue;
    const float* w = cut.ws + tiled + i;
    if (ntiles > 1)
      s[i] = make_float4(w[0], w[DV], w[2 * DV], w[3 * DV]);
    else if (p.S0 != nullptr)
      s[i] = *reinterpret_cast<const float4*>(p.S0 + user + size_t(i) * DK);
  }
  if (begin < end) {
    stage(begin, 0);
    put_dt(begin, 0, raw_dt(begin));
  }
  float raw = raw_dt(begin + kScanTile);
  for (int t0 = begin, b = 0; t0 < end; t0 += kScanTile, b ^= 1) {
    const bool more = t0 + kScanTile < end;
    if (more) {
      stage(t0 + kScanTile, b ^ 1);
      put_dt(t0 + kScanTile, b ^ 1, raw);
      raw = raw_dt(t0 + 2 * kScanTile);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const int groups = min((end - t0 + 7) / 8, kScanTile / 8);
    for (int e = 0; e < groups; ++e) {
      float sum[8 * NR];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = e * 8 + j;
        const float2 step = sdt[b][t];
        const float4 kt = load4(&sk[b][t][c0]);
        float vt[NR];
        load_small<NR>(&sv[b][t][r0], vt);
        float4 qt = kt;
        if (!STATES) qt = load4(&sq[b][t][STATES ? 0 : c0]);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float u = step.x * vt[i];
          s[i].x = fmaf(u, kt.x, step.y * s[i].x);
          s[i].y = fmaf(u, kt.y, step.y * s[i].y);
          s[i].z = fmaf(u, kt.z, step.y * s[i].z);
          s[i].w = fmaf(u, kt.w, step.y * s[i].w);
          sum[j * NR + i] = dot4(s[i], qt);
        }
      }
      if (!STATES) {
        // eight tokens' sums at once: each exchange halves what a lane holds, until
        // it is one row's of one token (one token at a time the shuffles wait for
        // one another, 150 cycles a token)
#pragma unroll
        for (int n = 8 * NR, x = kCols / 2; n > 1; n >>= 1, x >>= 1)
#pragma unroll
          for (int i = 0; i < n / 2; ++i) {
            const bool upper = (lane & x) != 0;
            const float give = upper ? sum[i] : sum[i + n / 2];
            sum[i] = (upper ? sum[i + n / 2] : sum[i]) + __shfl_xor_sync(0xffffffffu, give, x);
          }
        so[e * 8 + lane % kCols / NR][r0 + lane % NR] = sum[0];
      }
    }
    __syncthreads();
    if (!STATES && tid < kScanTile * kScanRows / 4) {
      const int t = tid / (kScanRows / 4), c = tid % (kScanRows / 4) * 4;
      const float4 y = load4(&so[t][c]), x = load4(&sv[b][t][c]);
      if (t0 + t < end)
        *reinterpret_cast<float4*>(o + (long long)(t0 + t) * p.ldo + c) =
            make_float4(fmaf(d, x.x, y.x), fmaf(d, x.y, y.y), fmaf(d, x.z, y.z), fmaf(d, x.w, y.w));
    }
  }
  if (STATES) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float* w = cut.ws + tiled + i;
      w[0] = s[i].x;
      w[DV] = s[i].y;
      w[2 * DV] = s[i].z;
      w[3 * DV] = s[i].w;
    }
    if (part == 0 && warp == 0) {
      forgot = warp_sum(forgot);
      if (lane == 0) cut.wdecay[size_t(tile) * p.H + h] = forgot;
    }
  } else if (last_tile && p.S1 != nullptr) {
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<float4*>(p.S1 + user + size_t(i) * DK) = s[i];
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

template <int DK, int DV, int NS>
cudaError_t scan_range(const SsmParams& p, int s0, int n, const int32_t* starts, const SsmPlan& plan,
                       void* ws, cudaStream_t s) {
  SeqTable<NS> tab;
  const long long tiles = fill_seqs(tab, starts, s0, n, plan.tile_tokens);
  const long long grid = tiles * p.H * (DV / kScanRows);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  float* w = static_cast<float*>(ws);
  const ScanTiles cut{w, w + size_t(tiles) * p.H * DV * DK, plan.tile_tokens};
  if (tiles > n) {
    dl_ssm_scan_kernel<DK, DV, true, SeqTable<NS>><<<unsigned(grid), kScanThreads, 0, s>>>(p, cut, tab, s0);
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_ssm_join(p, cut.ws, cut.wdecay, tab, s0, n, DK, DV, s);
    if (e != cudaSuccess) return e;
  }
  dl_ssm_scan_kernel<DK, DV, false, SeqTable<NS>><<<unsigned(grid), kScanThreads, 0, s>>>(p, cut, tab, s0);
  count_launches(1);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t scan_all(const SsmParams& p, int n, const int32_t* starts, const SsmPlan& plan, void* ws,
                     cudaStream_t s) {
  if (n <= kSmallSeqs) return scan_range<DK, DV, kSmallSeqs>(p, 0, n, starts, plan, ws, s);
  for (int s0 = 0; s0 < n; s0 += kLargeSeqs) {
    const int m = n - s0 < kLargeSeqs ? n - s0 : kLargeSeqs;
    const cudaError_t e = scan_range<DK, DV, kLargeSeqs>(p, s0, m, starts, plan, ws, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_ssm_step(const SsmParams& p, int B, int dk, int dv, bool bf16, cudaStream_t s) {
  return dispatch_shape(Shape{dk, dv, bf16 ? 1 : 0, 1}, RunStep{p, B, s});
}

// Tile length: with two CTAs an SM most of the latency is hidden, so a call
// takes about its tokens spread over as many, or its longest sequence.  Where the
// latter is three times the former or more, sequences are cut to the former's
// length (the cut reads k and v twice and costs two launches).  Both sides, in us
// (median of replayed graphs; ratio: the longest to the spread):
//     ratio 4.6, T = 2048 H = 16 d = 128 x 64     209 whole, 147 in 3, 124 in 4 (taken)
//     ratio 4.6, T = 300 H = 16 d = 64 x 64       26 whole, 20.5 in 4 (taken)
//     ratio 2.8, T = 517 (3) H = 16 d = 64 x 64   29 whole (taken), 29 in 2
//     ratio 2.4, T = 2048 (8) H = 8 d = 128 x 64  72 whole (taken), 93 in 2
//     ratio 2.3, T = 2048 H = 32 d = 128 x 64     211 whole (taken), 215 in 2
// Finer cuts than the spread gain in those (25 us in 6, 65 in 6, 182 in 8), less
// surely below (ratio 1.2: 283 whole and 324 in 4 at H = 64 d = 128 x 64, 201 and 190
// at H = 32 d = 64 x 128).
SsmPlan plan_ssm_scan(int H, int dk, int dv, int n, const int32_t* starts, int sms) {
  constexpr long long kMinTile = 64;
  long long longest = 0;
  for (int i = 0; i < n; ++i) {
    const long long t = (long long)starts[i + 1] - starts[i];
    longest = t > longest ? t : longest;
  }
  const long long total = n > 0 ? (long long)starts[n] - starts[0] : 0;
  const long long spread = total * H * (dv / kScanRows) / (2LL * sms);
  long long parts = longest / (spread > kMinTile ? spread : kMinTile);
  if (parts < 3) parts = 1;
  const long long len = (longest + parts - 1) / parts;
  const long long tile = (len + kScanTile - 1) / kScanTile * kScanTile;
  SsmPlan plan{};
  plan.tile_tokens = parts > 1 ? int(tile) : 1 << 30;
  plan.bytes = ssm_tile_bytes(H, dk, dv, n, starts, plan.tile_tokens);
  return plan;
}

cudaError_t launch_ssm_scan(const SsmParams& p, int n, const int32_t* starts, int dk, int dv,
                            const SsmPlan& plan, void* ws, cudaStream_t s) {
  if (dk == 128)
    return dv == 64 ? scan_all<128, 64>(p, n, starts, plan, ws, s) : scan_all<128, 128>(p, n, starts, plan, ws, s);
  return dv == 64 ? scan_all<64, 64>(p, n, starts, plan, ws, s) : scan_all<64, 128>(p, n, starts, plan, ws, s);
}

}  // namespace dl
