// dl_ssm_tc.cu -- the selective state space scan of packed bf16 prompts on
// the tensor cores, 128 tokens at a time.
//
// With lambda_j = dt_j a (log2 units), s_t = sum_{j>t} lambda_j over the
// chunk's tokens and tot = lambda_0 + s_0, a chunk that enters with state S
// gives (rows t, i: tokens; p: value rows; n: key channels)
//     o_t   = 2^{tot - s_t} (S q_t) + sum_{i<=t} M_ti v_i,
//     M_ti  = (q_t . k_i) dt_i 2^{s_i - s_t}   (+ d_h on the diagonal),
//     S'    = 2^{tot} S + sum_i (2^{s_i} dt_i v_i) k_i^T.
// Every exponent is <= 0, whatever the decays are.  As MMAs (fp32
// accumulators in TMEM):
//     G = Q K^T            [t, i]   A, B from shared memory, K-major
//     Y = Q S^T            [t, p]   B: the state as bf16, written by its owners
//     Y += M V             [t, p]   A: M as bf16 in TMEM, B: V, MN-major
//     D = K^T (w o V)      [n, p]   A: K, MN-major, B: w o V in three bf16 parts
// Rounding: the state is carried in fp32 registers (one thread per key
// channel and 64 value rows) and w o V enters D as hi + mid + lo, all 24 bits,
// so S' is right to fp32 rounding; only what feeds the bf16 output o is rounded
// to bf16 on the way, each term once (M, or the state that q reads), which
// is of the size of o's own rounding.
//
// A CTA owns 128 value columns (two neighbouring heads of a group at d_v = 64,
// which share G and the loads of q and k; one head at 128) and walks the
// chunks of one tile of one sequence.  Long sequences are cut into tiles when
// there are too few CTAs: a first launch (STATES) forms every tile's own state
// from zero, dl_ssm_join_kernel turns those into the state each tile enters
// with, and the main launch starts from them.
//
// Warps 0-7: element work (warp w reaches TMEM lanes 32 (w mod 4) ..; w / 4
// picks the 64 value columns).  Warp 8: TMA.  Warp 9: MMA issue.  Warps 10,
// 11: dt, decays and their sums, one chunk ahead.
#include <cuda.h>

#include "dl_layer.cuh"
#include "dl_tmem.cuh"

namespace dl {

namespace {

constexpr int kQ = 128;             // tokens per chunk
constexpr int kThreads = 384;
constexpr int kComputeWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
// Decay factors below 2^-150 are 0 in fp32: clamping there keeps the sums finite.
constexpr float kMinLambda = -150.f;

// TMEM columns
constexpr uint32_t kColG = 0, kColY = 128, kColD = 256, kColM = 384;

template <int DK>
struct TcLayout {
  static constexpr uint32_t kKBlocks = DK / 64;                 // 64-column boxes of q and k
  static constexpr uint32_t kBox = kQ * 128;                    // bytes of a box
  static constexpr uint32_t offQ = 0;
  static constexpr uint32_t offK = offQ + kKBlocks * kBox;
  static constexpr uint32_t offV = offK + kKBlocks * kBox;      // two stages of two boxes
  static constexpr uint32_t offW = offV + 4 * kBox;             // 3 parts x 2 boxes x 64 rows
  static constexpr uint32_t kWPart = kBox;                      // bytes of one part
  static constexpr uint32_t offS = offW + 3 * kWPart;           // 2 boxes of DK rows
  static constexpr uint32_t kSBox = DK * 128;
  static constexpr uint32_t offF = offS + 2 * kSBox;            // s, h, w: [2][2][128] each
  static constexpr uint32_t kF = 2 * 2 * kQ * 4;
  static constexpr uint32_t offT = offF + 3 * kF;               // tot [2][2]
  static constexpr uint32_t offBar = offT + 16;
  static constexpr uint32_t total = offBar + 32 * 8 + 16 + 1024;  // + alignment of the base
};

enum Bar {
  kFullQ, kFullK, kFullV0, kFullV1, kWts0, kWts1, kWtsFree0, kWtsFree1, kG, kWA, kWB, kDA, kDB, kMReady,
  kY, kSReady, kYFree, kBars
};

struct TcParams {
  const float* dt;
  const float* a;
  const float* d;
  const float* bias;
  const float* S0;
  float* S1;
  __nv_bfloat16* o;
  float* ws;        // [tiles, H, DV, DK]: STATES writes a tile's own state, main reads its entry state
  float* wdecay;    // [tiles, H] log2 of a tile's whole decay
  int* err;
  long long lddt, ldo;
  int H, G, softplus;
  int pairs;        // CTAs per tile
  int tile_tokens;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// Descriptors of 128-byte swizzled operands: boxes of 128-byte rows (64 bf16).
//   K-major (rows: M or N index): 8-row groups 1024 bytes apart; a K step of
//     16 is 32 bytes further along the rows.
//   MN-major (rows: K index): 8-row groups 1024 bytes apart (stride offset),
//     the next 64 M or N indices `lbo` bytes away; a K step of 16 is two groups.
__device__ __forceinline__ uint64_t desc_sw128(const void* start, uint32_t lbo) {
  uint64_t d = uint64_t((smem_u32(start) >> 4) & 0x3FFFu);
  d |= uint64_t((lbo >> 4) & 0x3FFFu) << 16;
  d |= uint64_t(1024u >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// D[tmem] (+)= A B with A in TMEM (lane = row, a column = two K elements).
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                        uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight bf16 (two per word) times w, each product as three bf16 parts whose
// sum is the fp32 product: the upper 16 bits are cut off twice (exact
// remainders), the last part is rounded.
__device__ __forceinline__ void weigh8(uint4 x, float w, uint4& hi, uint4& mid, uint4& lo) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t o0[4], o1[4], o2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(in[i] << 16) * w;
    const float b = __uint_as_float(in[i] & 0xffff0000u) * w;
    o0[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    const float ra = a - __uint_as_float(__float_as_uint(a) & 0xffff0000u);
    const float rb = b - __uint_as_float(__float_as_uint(b) & 0xffff0000u);
    o1[i] = __byte_perm(__float_as_uint(ra), __float_as_uint(rb), 0x7632);
    o2[i] = pack_bf(ra - __uint_as_float(__float_as_uint(ra) & 0xffff0000u),
                    rb - __uint_as_float(__float_as_uint(rb) & 0xffff0000u));
  }
  hi = make_uint4(o0[0], o0[1], o0[2], o0[3]);
  mid = make_uint4(o1[0], o1[1], o1[2], o1[3]);
  lo = make_uint4(o2[0], o2[1], o2[2], o2[3]);
}

// One arrival per warp once all its lanes are done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <int DK, int DV, bool STATES, typename Table>
__global__ void __launch_bounds__(kThreads, 1)
dl_ssm_chunk_kernel(const TcParams p, const __grid_constant__ Table seqs, int seq0,
                    const __grid_constant__ CUtensorMap mapQ,
                    const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapV) {
  using L = TcLayout<DK>;
  constexpr int kHeads = 128 / DV;  // heads a CTA covers
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sQ = smem + L::offQ;
  unsigned char* sK = smem + L::offK;
  unsigned char* sV = smem + L::offV;
  unsigned char* sW = smem + L::offW;
  unsigned char* sS = smem + L::offS;
  float* fS = reinterpret_cast<float*>(smem + L::offF);  // [buf][head][token]
  float* fH = fS + 2 * 2 * kQ;
  float* fW = fH + 2 * 2 * kQ;
  float* fT = reinterpret_cast<float*>(smem + L::offT);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::offBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = int(blockIdx.x / unsigned(p.pairs));
  const int pair = int(blockIdx.x % unsigned(p.pairs));
  const int sl = seqs.find(tile);
  const int first_tile = seqs.tile0[sl], ntiles = seqs.tile0[sl + 1] - first_tile;
  const int seq_end = seqs.start[sl + 1];
  const int begin = seqs.start[sl] + (tile - first_tile) * p.tile_tokens;
  const int end = min(begin + p.tile_tokens, seq_end);
  const bool last_tile = tile - first_tile == ntiles - 1;
  if (STATES && last_tile) return;  // nobody enters from a last tile's own state
  const int nch = (end - begin + kQ - 1) / kQ;
  // heads: pairs run through the heads of a group
  const int hpg = p.H / p.G, ppg = (hpg + kHeads - 1) / kHeads;
  const int g = pair / ppg;
  const int h0 = g * hpg + (pair % ppg) * kHeads;
  const int hend = (g + 1) * hpg;
  const size_t seq = size_t(seq0) + size_t(sl);

  if (warp == 0) tmem_alloc(tmem_slot, 512);
  if (tid == 32) {
    for (int i = 0; i < kBars; ++i) {
      uint32_t n = 1;
      if (i == kWts0 || i == kWts1) n = kHeads;
      if (i == kWtsFree0 || i == kWtsFree1 || i == kWA || i == kWB || i == kMReady || i == kSReady ||
          i == kYFree)
        n = kComputeWarps;
      mbar_init(&bars[i], n);
    }
    fence_mbar_init();
    *abort_flag = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int errh = int(seq) * p.H + h0;
// One thread's wait, and a whole warp's (which gives up as one).
#define DL_WAIT(bar, parity)                            \
  if (!mbar_wait(&bars[bar], (parity), p.err, errh)) { \
    *abort_flag = 1;                                    \
    break;                                              \
  }
#define DL_WAIT_WARP(bar, parity)                                                              \
  if (!__all_sync(0xffffffffu, mbar_wait(&bars[bar], (parity), p.err, errh))) { \
    *abort_flag = 1;                                                                           \
    break;                                                                                     \
  }

  if (warp == 8) {
    // ------------------------------------------------------------- copies
    if (lane == 0) {
      for (int c = 0; c < nch; ++c) {
        const int t0 = begin + c * kQ;
        // q was read last by chunk c - 1's first MMAs, k and the other value
        // stage by its last ones
        if (c > 0 && !STATES) DL_WAIT(kG, (c - 1) & 1);
        if (!STATES) {
          mbar_arrive_expect_tx(&bars[kFullQ], L::kKBlocks * L::kBox);
          for (uint32_t b = 0; b < L::kKBlocks; ++b)
            tma_load_2d(sQ + b * L::kBox, &mapQ, g * DK + int(b) * 64, t0, &bars[kFullQ]);
        }
        if (c == 0) {
          mbar_arrive_expect_tx(&bars[kFullK], L::kKBlocks * L::kBox);
          for (uint32_t b = 0; b < L::kKBlocks; ++b)
            tma_load_2d(sK + b * L::kBox, &mapK, g * DK + int(b) * 64, t0, &bars[kFullK]);
          mbar_arrive_expect_tx(&bars[kFullV0], 2 * L::kBox);
          for (uint32_t b = 0; b < 2; ++b)
            tma_load_2d(sV + b * L::kBox, &mapV, h0 * DV + int(b) * 64, t0, &bars[kFullV0]);
        }
        if (c > 0) {
          DL_WAIT(kDB, (c - 1) & 1);
          mbar_arrive_expect_tx(&bars[kFullK], L::kKBlocks * L::kBox);
          for (uint32_t b = 0; b < L::kKBlocks; ++b)
            tma_load_2d(sK + b * L::kBox, &mapK, g * DK + int(b) * 64, t0, &bars[kFullK]);
        }
        if (c + 1 < nch) {  // the other value stage: chunk c - 1 is done with it
          const int sn = (c + 1) & 1;
          mbar_arrive_expect_tx(&bars[kFullV0 + sn], 2 * L::kBox);
          for (uint32_t b = 0; b < 2; ++b)
            tma_load_2d(sV + (2 * sn + b) * L::kBox, &mapV, h0 * DV + int(b) * 64, t0 + kQ,
                        &bars[kFullV0 + sn]);
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // --------------------------------------------------------------- MMAs
    if (lane == 0) {
      constexpr uint32_t idG = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idY = idesc_bf16(128, 128, false, true);
      constexpr uint32_t idM = idesc_bf16(128, DV == 64 ? 64 : 128, false, true);
      constexpr uint32_t idD = idesc_bf16(128, 128, true, true);
      for (int c = 0; c < nch; ++c) {
        const uint32_t ph = uint32_t(c) & 1u;
        const unsigned char* v = sV + (c & 1) * 2 * L::kBox;
        if (!STATES) {
          DL_WAIT(kFullQ, ph);
        }
        DL_WAIT(kFullK, ph);
        if (!STATES) {
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            umma_f16(tmem + kColG, desc_sw128(sQ + (ks / 4) * L::kBox + (ks % 4) * 32, 16),
                     desc_sw128(sK + (ks / 4) * L::kBox + (ks % 4) * 32, 16), idG, ks > 0);
          DL_WAIT(kSReady, ph);
          if (c > 0) DL_WAIT(kYFree, (c - 1) & 1);
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            umma_f16(tmem + kColY, desc_sw128(sQ + (ks / 4) * L::kBox + (ks % 4) * 32, 16),
                     desc_sw128(sS + ks * 2048, L::kSBox), idY, ks > 0);
          umma_commit(&bars[kG]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          DL_WAIT(half ? kWB : kWA, ph);
          tc_fence_after();
#pragma unroll
          for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_f16(tmem + kColD, desc_sw128(sK + half * 8192 + ks * 2048, L::kBox),
                       desc_sw128(sW + part * L::kWPart + ks * 2048, 8192), idD,
                       half + part + ks > 0);
          umma_commit(&bars[half ? kDB : kDA]);
          if (half == 0 && !STATES) {
            DL_WAIT(kMReady, ph);
            tc_fence_after();
#pragma unroll
            for (int hd = 0; hd < kHeads; ++hd)
#pragma unroll
              for (int ks = 0; ks < kQ / 16; ++ks)
                umma_ts(tmem + kColY + hd * 64, tmem + kColM + hd * 64 + ks * 8,
                        desc_sw128(v + hd * L::kBox + ks * 2048, L::kBox), idM, true);
            umma_commit(&bars[kY]);
          }
        }
        if (*abort_flag) break;
      }
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ------------------------------------------------------------- decays
    const int hs = warp - 10;
    const int h = h0 + hs;
    if (hs < kHeads) {
      const bool live = h < hend;
      const float a2 = live ? p.a[h] * kLog2e : 0.f;
      const float bias = live && p.bias != nullptr ? p.bias[h] : 0.f;
      for (int c = 0; c < nch; ++c) {
        const int buf = c & 1;
        const int t0 = begin + c * kQ + lane * 4;
        float dt[4], lam[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dt[e] = 0.f;
          if (live && t0 + e < end) {
            const float raw = p.dt[(long long)(t0 + e) * p.lddt + h] + bias;
            dt[e] = p.softplus ? softplusf(raw) : raw;
          }
          lam[e] = fmaxf(dt[e] * a2, kMinLambda);
        }
        // sums over the tokens behind each one
        const float own = (lam[0] + lam[1]) + (lam[2] + lam[3]);
        float inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float y = __shfl_down_sync(0xffffffffu, inc, o);
          if (lane + o < 32) inc += y;
        }
        float behind = __shfl_down_sync(0xffffffffu, inc, 1);
        if (lane == 31) behind = 0.f;
        float s[4];
        s[3] = behind;
        s[2] = s[3] + lam[3];
        s[1] = s[2] + lam[2];
        s[0] = s[1] + lam[1];
        if (c >= 2) DL_WAIT_WARP(kWtsFree0 + buf, ((c >> 1) - 1) & 1);
        const int at = (buf * 2 + hs) * kQ + lane * 4;
        *reinterpret_cast<float4*>(fS + at) = make_float4(s[0], s[1], s[2], s[3]);
        *reinterpret_cast<float4*>(fH + at) =
            make_float4(s[0] + log2f(dt[0]), s[1] + log2f(dt[1]), s[2] + log2f(dt[2]),
                        s[3] + log2f(dt[3]));
        *reinterpret_cast<float4*>(fW + at) =
            make_float4(exp2f(s[0]) * dt[0], exp2f(s[1]) * dt[1], exp2f(s[2]) * dt[2],
                        exp2f(s[3]) * dt[3]);
        if (lane == 0) fT[buf * 2 + hs] = s[0] + lam[0];
        warp_arrive(&bars[kWts0 + buf], lane);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------- element work
    const int wg = warp >> 2, quarter = warp & 3;
    const int hs = DV == 64 ? wg : 0;       // head slot of this thread's columns
    const int h = h0 + hs;
    const bool live = h < hend;
    const int row = quarter * 32 + lane;    // token of M and Y, key channel of D
    const int col0 = DV == 64 ? 0 : wg * 64;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const bool owns = row < DK;             // has a key channel of the state
    const size_t tile_off = ((ntiles > 1 ? size_t(tile) : seq) * p.H + h) * size_t(DV) * DK +
                            size_t(col0) * DK + row;
    float S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
    float decay = 0.f;  // log2 of everything forgotten in this tile (STATES)
    const float* in = STATES ? nullptr : (ntiles > 1 ? p.ws : p.S0);
    if (in != nullptr && live && owns) {
#pragma unroll
      for (int i = 0; i < 64; ++i) S[i] = in[tile_off + size_t(i) * DK];
    }
    const float dskip = !STATES && live && p.d != nullptr ? p.d[h] : 0.f;
    auto put_state = [&]() {
      if (!owns) return;
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) {
        const uint4 r = make_uint4(pack_bf(S[8 * ch], S[8 * ch + 1]), pack_bf(S[8 * ch + 2], S[8 * ch + 3]),
                                   pack_bf(S[8 * ch + 4], S[8 * ch + 5]), pack_bf(S[8 * ch + 6], S[8 * ch + 7]));
        *reinterpret_cast<uint4*>(sS + wg * L::kSBox + row * 128 + ((ch ^ (row & 7)) << 4)) = r;
      }
    };
    // w o V of 64 tokens: this group's box, 4 sixteen-byte pieces a thread;
    // rows from `len` on may hold anything and count as zeros
    auto weigh_half = [&](const unsigned char* v, const float* w, int half, int len) {
      const int t = (quarter * 32 + lane);
      const unsigned char* src = v + wg * L::kBox + half * 8192;
      unsigned char* dst = sW + wg * 8192;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = (t >> 3) + 16 * j, off = r * 128 + (t & 7) * 16;
        uint4 x = *reinterpret_cast<const uint4*>(src + off);
        if (half * 64 + r >= len) x = make_uint4(0u, 0u, 0u, 0u);
        uint4 hi, mid, lo;
        weigh8(x, w[half * 64 + r], hi, mid, lo);
        *reinterpret_cast<uint4*>(dst + off) = hi;
        *reinterpret_cast<uint4*>(dst + L::kWPart + off) = mid;
        *reinterpret_cast<uint4*>(dst + 2 * L::kWPart + off) = lo;
      }
    };
    if (!STATES) {
      put_state();
      fence_async_smem();
      warp_arrive(&bars[kSReady], lane);
      // the blocks of M above the diagonal stay zero for good
      uint32_t z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = 0u;
#pragma unroll
      for (int cb = 0; cb < 4; ++cb)
        if (DV == 64 || (cb & 1) == wg) tmem_st16(tmem + kColM + hs * 64 + cb * 16 + lanes, z);
      tmem_wait_st();
    }
    for (int c = 0; c < nch; ++c) {
      const uint32_t ph = uint32_t(c) & 1u;
      const int buf = c & 1;
      const int t0 = begin + c * kQ;
      const int len = min(kQ, end - t0);
      unsigned char* v = sV + buf * 2 * L::kBox;
      const float* ws_ = fS + (buf * 2 + hs) * kQ;
      const float* wh = fH + (buf * 2 + hs) * kQ;
      const float* ww = fW + (buf * 2 + hs) * kQ;
      DL_WAIT_WARP(kWts0 + buf, (c >> 1) & 1);
      DL_WAIT_WARP(kFullV0 + buf, (c >> 1) & 1);
      if (len < kQ) {
        // rows behind the sequence may hold anything: zeros for the sums over
        // tokens (G's columns there are masked)
        DL_WAIT_WARP(kFullK, ph);
        for (int i = tid; i < (kQ - len) * 8; i += kComputeWarps * 32) {
          const int off = (len + (i >> 3)) * 128 + (i & 7) * 16;
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          for (uint32_t b = 0; b < L::kKBlocks; ++b) *reinterpret_cast<uint4*>(sK + b * L::kBox + off) = zero;
          for (uint32_t b = 0; b < 2; ++b) *reinterpret_cast<uint4*>(v + b * L::kBox + off) = zero;
        }
      }
      weigh_half(v, ww, 0, len);
      fence_async_smem();
      tc_fence_before();
      warp_arrive(&bars[kWA], lane);
      const float tot = fT[buf * 2 + hs];
      if (!STATES) {
        const float st = ws_[row];
        DL_WAIT_WARP(kG, ph);
        tc_fence_after();
        // Y *= 2^{tot - s_t}
        const float grow = ex2(tot - st);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float y[32];
          const uint32_t at = tmem + kColY + wg * 64 + b * 32 + lanes;
          tmem_ld32(at, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] *= grow;
          tmem_st32(at, y);
        }
        // M, up to the diagonal block (at d_v = 128 the groups take turns)
#pragma unroll 1
        for (int cb = DV == 64 ? 0 : wg; cb <= quarter; cb += DV == 64 ? 1 : 2) {
          float x[32];
          tmem_ld32(tmem + kColG + cb * 32 + lanes, x);
          tmem_wait_ld();
          const float4* hp = reinterpret_cast<const float4*>(wh + cb * 32);
          uint32_t m[16];
          if (cb < quarter) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 hc = hp[i];
              m[2 * i] = pack_bf(x[4 * i] * ex2(hc.x - st), x[4 * i + 1] * ex2(hc.y - st));
              m[2 * i + 1] = pack_bf(x[4 * i + 2] * ex2(hc.z - st), x[4 * i + 3] * ex2(hc.w - st));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 hc = hp[i];
              const float e[4] = {hc.x, hc.y, hc.z, hc.w};
              float r[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int j = 4 * i + k;
                r[k] = j <= lane ? x[j] * ex2(e[k] - st) : 0.f;
                if (j == lane) r[k] += dskip;
              }
              m[2 * i] = pack_bf(r[0], r[1]);
              m[2 * i + 1] = pack_bf(r[2], r[3]);
            }
          }
          tmem_st16(tmem + kColM + hs * 64 + cb * 16 + lanes, m);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bars[kMReady], lane);
      }
      DL_WAIT_WARP(kDA, ph);
      weigh_half(v, ww, 1, len);
      fence_async_smem();
      warp_arrive(&bars[kWB], lane);
      DL_WAIT_WARP(kDB, ph);
      tc_fence_after();
      {
        const float keep = exp2f(tot);
        decay += tot;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x[32];
          tmem_ld32(tmem + kColD + wg * 64 + b * 32 + lanes, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) S[b * 32 + i] = fmaf(S[b * 32 + i], keep, x[i]);
        }
      }
      if (!STATES) {
        put_state();
        fence_async_smem();
        tc_fence_before();
        warp_arrive(&bars[kSReady], lane);
      }
      warp_arrive(&bars[kWtsFree0 + buf], lane);
      if (!STATES) {
        DL_WAIT_WARP(kY, ph);
        tc_fence_after();
        __nv_bfloat16* o = p.o + (long long)(t0 + row) * p.ldo + h * DV + col0;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float y[32];
          tmem_ld32(tmem + kColY + wg * 64 + b * 32 + lanes, y);
          tmem_wait_ld();
          if (live && row < len) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(o + b * 32 + i * 8) =
                  make_uint4(pack_bf(y[8 * i], y[8 * i + 1]), pack_bf(y[8 * i + 2], y[8 * i + 3]),
                             pack_bf(y[8 * i + 4], y[8 * i + 5]), pack_bf(y[8 * i + 6], y[8 * i + 7]));
          }
        }
        tc_fence_before();
        warp_arrive(&bars[kYFree], lane);
      }
    }
    if (*abort_flag == 0 && live && owns) {
      float* out = STATES ? p.ws : (last_tile ? p.S1 : nullptr);
      if (out != nullptr) {
        const size_t off = STATES ? tile_off
                                  : (seq * p.H + h) * size_t(DV) * DK + size_t(col0) * DK + row;
#pragma unroll
        for (int i = 0; i < 64; ++i) out[off + size_t(i) * DK] = S[i];
      }
      if (STATES && row == 0 && col0 == 0) p.wdecay[size_t(tile) * p.H + h] = decay;
    }
  }
#undef DL_WAIT
#undef DL_WAIT_WARP
  __syncthreads();
  if (*abort_flag) {  // let copies and MMAs in flight end before the memory is given back
    const long long t = clock64();
    while (clock64() - t < kWaitCycles / 16) {
    }
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

// Turns the tiles' own states into the states they enter with, in place:
// E_0 = S0, E_{j+1} = 2^{decay_j} E_j + own_j, one thread per four elements.
template <typename Table>
__global__ void __launch_bounds__(256)
dl_ssm_join_kernel(const float* S0, float* ws, const float* wdecay, const __grid_constant__ Table seqs,
                   int seq0, int H, int tile_floats) {
  const int per = tile_floats / 1024;  // blocks per head
  const int sl = int(blockIdx.x / unsigned(H * per));
  const int rest = int(blockIdx.x % unsigned(H * per));
  const int h = rest / per;
  const int at = (rest % per) * 1024 + threadIdx.x * 4;
  const int j0 = seqs.tile0[sl], j1 = seqs.tile0[sl + 1];
  if (j1 - j0 < 2) return;
  float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
  if (S0 != nullptr)
    e = *reinterpret_cast<const float4*>(S0 + ((size_t(seq0) + sl) * H + h) * size_t(tile_floats) + at);
  for (int j = j0; j < j1; ++j) {
    float4* w = reinterpret_cast<float4*>(ws + (size_t(j) * H + h) * size_t(tile_floats) + at);
    if (j + 1 == j1) {
      *w = e;
      break;
    }
    const float4 own = *w;
    const float k = exp2f(wdecay[size_t(j) * H + h]);
    *w = e;
    e = make_float4(fmaf(e.x, k, own.x), fmaf(e.y, k, own.y), fmaf(e.z, k, own.z), fmaf(e.w, k, own.w));
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<void*> cache{nullptr};
  void* f = cache.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    cache.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeFn>(f);
}

// Rows of `cols` bf16, boxes of 64 columns x 128 rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, long long rows, int cols, long long ld) {
  EncodeFn f = encode_fn();
  if (f == nullptr) return false;
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows > 0 ? rows : 1)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {64, kQ};
  const cuuint32_t step[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool STATES, int NS>
cudaError_t launch_chunk(const TcParams& p, const SeqTable<NS>& tab, int seq0, unsigned grid,
                         const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  auto kern = dl_ssm_chunk_kernel<DK, DV, STATES, SeqTable<NS>>;
  const cudaError_t e = prepare_kernel(kern, done);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, TcLayout<DK>::total, s>>>(p, tab, seq0, q, k, v);
  count_launches(1);
  return cudaGetLastError();
}

template <int DK, int DV, int NS>
cudaError_t launch_range(const SsmParams& sp, TcParams p, int seq0, int n, const int32_t* starts,
                         const SsmPlan& plan, void* ws, cudaStream_t s) {
  SeqTable<NS> tab;
  const long long tiles = fill_seqs(tab, starts, seq0, n, plan.tile_tokens);
  const long long grid = tiles * p.pairs;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  p.ws = static_cast<float*>(ws);
  p.wdecay = p.ws + size_t(tiles) * p.H * DV * DK;
  CUtensorMap q, k, v;
  const long long rows = starts[seq0 + n];
  if (!encode_rows(&q, sp.q, rows, p.G * DK, sp.ldq) || !encode_rows(&k, sp.k, rows, p.G * DK, sp.ldk) ||
      !encode_rows(&v, sp.v, rows, p.H * DV, sp.ldv))
    return cudaErrorInvalidValue;
  if (tiles > n) {
    cudaError_t e = launch_chunk<DK, DV, true, NS>(p, tab, seq0, unsigned(grid), q, k, v, s);
    if (e != cudaSuccess) return e;
    const long long blocks = (long long)n * p.H * (DV * DK / 1024);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    dl_ssm_join_kernel<SeqTable<NS>><<<unsigned(blocks), 256, 0, s>>>(
        sp.S0, p.ws, p.wdecay, tab, seq0, p.H, DV * DK);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_chunk<DK, DV, false, NS>(p, tab, seq0, unsigned(grid), q, k, v, s);
}

template <int DK, int DV>
cudaError_t launch_tc(const SsmParams& sp, const TcParams& p, int n, const int32_t* starts,
                      const SsmPlan& plan, void* ws, cudaStream_t s) {
  if (n <= kSmallSeqs) return launch_range<DK, DV, kSmallSeqs>(sp, p, 0, n, starts, plan, ws, s);
  for (int s0 = 0; s0 < n; s0 += kLargeSeqs) {
    const int m = n - s0 < kLargeSeqs ? n - s0 : kLargeSeqs;
    const cudaError_t e = launch_range<DK, DV, kLargeSeqs>(sp, p, s0, m, starts, plan, ws, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int cta_pairs(int H, int G, int dv) {
  const int heads = 128 / dv, hpg = H / G;
  return G * ((hpg + heads - 1) / heads);
}

}  // namespace

// Tile length: one CTA runs per SM, and a cut tile costs a second walk over
// its k and v (about kStatesCost of a full one), so take the length whose
// waves of CTAs finish first.
SsmPlan plan_ssm(int H, int G, int dk, int dv, int n, const int32_t* starts, int sms) {
  constexpr double kStatesCost = 0.4, kTileCost = 1.0;  // in chunks
  const int pairs = cta_pairs(H, G, dv);
  long long longest = 0;
  for (int i = 0; i < n; ++i) {
    const long long c = ((long long)starts[i + 1] - starts[i] + kQ - 1) / kQ;
    longest = c > longest ? c : longest;
  }
  SsmPlan best{};
  best.tile_tokens = 0;
  double best_cost = 0;
  for (const int parts : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32, 48, 64}) {
    if (parts > 1 && parts > longest) break;
    const long long len = longest > 0 ? (longest + parts - 1) / parts : 1;  // chunks a tile
    long long tiles = 0, chunks = 0, cut = 0;
    for (int i = 0; i < n; ++i) {
      const long long c = ((long long)starts[i + 1] - starts[i] + kQ - 1) / kQ;
      const long long t = c > len ? (c + len - 1) / len : 1;
      tiles += t;
      chunks += c;
      cut += (t - 1) * len;
    }
    // all work spread evenly, but never less than the longest tile
    const double even = double(pairs) * (double(chunks) + kTileCost * double(tiles)) / sms;
    const double one = double(len) + kTileCost;
    double cost = even > one ? even + 0.5 * one : one;
    if (cut > 0) {
      const double ev = double(pairs) * kStatesCost * double(cut) / sms;
      const double on = kStatesCost * double(len) + kTileCost;
      cost += (ev > on ? ev + 0.5 * on : on) + 2 * kTileCost;
    }
    if (best.tile_tokens == 0 || cost < 0.98 * best_cost) {
      best.tile_tokens = int(len * kQ < (1 << 30) ? len * kQ : (1 << 30));
      best_cost = cost;
    }
    if (parts == 1 && even >= 4 * one) break;  // more than enough CTAs
  }
  // workspace of the largest launch range
  long long most = 0;
  bool any = false;
  const int step = n <= kSmallSeqs ? (n > 0 ? n : 1) : kLargeSeqs;
  for (int s0 = 0; s0 < n; s0 += step) {
    long long tiles = 0;
    const int m = n - s0 < step ? n - s0 : step;
    for (int i = s0; i < s0 + m; ++i) {
      const long long len = (long long)starts[i + 1] - starts[i];
      tiles += len > best.tile_tokens ? (len + best.tile_tokens - 1) / best.tile_tokens : 1;
    }
    any = any || tiles > m;
    most = tiles > most ? tiles : most;
  }
  best.bytes = any ? size_t(most) * H * (size_t(dv) * dk + 1) * 4 : 0;
  return best;
}

cudaError_t launch_ssm_chunked(const SsmParams& sp, int n, const int32_t* starts, int dk, int dv,
                               const SsmPlan& plan, void* ws, cudaStream_t s) {
  TcParams p{};
  p.dt = sp.dt;
  p.a = sp.a;
  p.d = sp.d;
  p.bias = sp.bias;
  p.S0 = sp.S0;
  p.S1 = sp.S1;
  p.o = static_cast<__nv_bfloat16*>(sp.o);
  p.err = sp.err;
  p.lddt = sp.lddt;
  p.ldo = sp.ldo;
  p.H = sp.H;
  p.G = sp.G;
  p.softplus = sp.softplus;
  p.pairs = cta_pairs(sp.H, sp.G, dv);
  p.tile_tokens = plan.tile_tokens;
  if (dk == 128) return dv == 64 ? launch_tc<128, 64>(sp, p, n, starts, plan, ws, s)
                                 : launch_tc<128, 128>(sp, p, n, starts, plan, ws, s);
  return dv == 64 ? launch_tc<64, 64>(sp, p, n, starts, plan, ws, s)
                  : launch_tc<64, 128>(sp, p, n, starts, plan, ws, s);
}

}  // namespace dl
