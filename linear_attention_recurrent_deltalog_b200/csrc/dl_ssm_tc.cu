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
//     Z = M V              [t, p]   A: M as bf16 in TMEM, B: V, MN-major
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
// Warps 0-7: element work on M, the state and o (warp w reaches TMEM lanes
// 32 (w mod 4) ..; w / 4 picks the 64 value columns).  Warps 8-11: w o V, 16
// tokens at a time.  Warp 12: TMA.  Warp 13: MMA issue.  Warps 14, 15: dt,
// decays and their sums, one chunk ahead.  In turn the tensor cores run
// G, Y, D, Z = M V of a chunk; M is formed while Y and D run, the state moves on
// and o is written while Z and the next G run.
#include <cuda.h>

#include "dl_layer.cuh"
#include "dl_tmem.cuh"

namespace dl {

namespace {

constexpr int kQ = 128;             // tokens per chunk
constexpr int kThreads = 512;
constexpr int kElemWarps = 8, kWeighWarps = 4;
constexpr int kPiece = 16;          // tokens of w o V staged at a time
constexpr int kPieces = kQ / kPiece;
constexpr float kLog2e = 1.4426950408889634f;
// Decay factors below 2^-150 are 0 in fp32: clamping there keeps the sums finite.
constexpr float kMinLambda = -150.f;

// TMEM columns.  M takes G's place block by block: tokens 32 b .. 32 b + 31 of
// head slot s are the 16 columns at kColG + 32 b + 16 s.
constexpr uint32_t kColG = 0, kColY = 128, kColZ = 256, kColD = 384;

template <int DK>
struct TcLayout {
  static constexpr uint32_t kKBlocks = DK / 64;                 // 64-column boxes of q and k
  static constexpr uint32_t kBox = kQ * 128;                    // bytes of a box
  static constexpr uint32_t kK = kKBlocks * kBox;
  static constexpr uint32_t offQ = 0;
  static constexpr uint32_t offK = offQ + kK;                   // two stages
  static constexpr uint32_t offV = offK + 2 * kK;               // two stages of two boxes
  static constexpr uint32_t offW = offV + 4 * kBox;             // two stages x 3 parts x 2 boxes x 16 rows
  static constexpr uint32_t kWBox = kPiece * 128;
  static constexpr uint32_t kWPart = 2 * kWBox;
  static constexpr uint32_t kWStage = 3 * kWPart;
  static constexpr uint32_t offS = offW + 2 * kWStage;          // 2 boxes of DK rows
  static constexpr uint32_t kSBox = DK * 128;
  // per token, [2 buffers][2 heads][128] floats: s, dt, w; and the column
  // factors of M's blocks below the diagonal ones, 32 + 64 + 96 per head
  static constexpr uint32_t offF = offS + 2 * kSBox;
  static constexpr uint32_t kF = 2 * 2 * kQ * 4;
  static constexpr uint32_t kCols = 192;
  static constexpr uint32_t offC = offF + 3 * kF;
  static constexpr uint32_t offT = offC + 2 * 2 * kCols * 4;    // tot [2][2]
  static constexpr uint32_t offBar = offT + 16;
  static constexpr uint32_t total = offBar + 32 * 8 + 16 + 1024;  // + alignment of the base
};
static_assert(TcLayout<128>::total <= kMaxSmemOptIn, "shared memory of a CTA");

enum Bar {
  kFullQ, kFullK0, kFullK1, kFullV0, kFullV1, kWts0, kWts1, kWtsFree0, kWtsFree1, kWFull0, kWFull1,
  kWFree0, kWFree1, kG, kY, kD0, kD1, kZ0, kZ1, kMReady, kSReady, kYFree0, kYFree1,
  kPair0, kPair1, kPair2, kPair3, kBars
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

// The MMA warp runs as one, with the issue itself predicated on one lane
// (`lead`): operands then stay in uniform registers.  Issued from a branch of
// one lane instead, each MMA cost 180 cycles, three times its run time.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// D[tmem] (+)= A B, both from shared memory.
__device__ __forceinline__ void umma_ss(uint32_t lead, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(adesc),
      "l"(bdesc), "r"(idesc), "r"(uint32_t(accumulate)), "r"(lead)
      : "memory");
}
// D[tmem] (+)= A B with A in TMEM (lane = row, a column = two K elements).
__device__ __forceinline__ void umma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                        uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem), "r"(a_tmem),
      "l"(bdesc), "r"(idesc), "r"(uint32_t(accumulate)), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void umma_done(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
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

__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Eight bf16 (two per word) times w, each product as three bf16 parts whose
// sum is the fp32 product: the upper 16 bits are cut off twice (exact
// remainders), the last part is rounded.
__device__ __forceinline__ void weigh8(uint4 x, float w, uint4& hi, uint4& mid, uint4& lo) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t o0[4], o1[4], o2[4];
  const uint64_t w2 = f2_pack(w, w), minus = f2_pack(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    const uint64_t y =
        f2_mul(f2_pack(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xffff0000u)), w2);
    f2_unpack(y, a, b);
    o0[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    const uint64_t r = f2_fma(f2_pack(__uint_as_float(__float_as_uint(a) & 0xffff0000u),
                                      __uint_as_float(__float_as_uint(b) & 0xffff0000u)),
                              minus, y);
    f2_unpack(r, a, b);
    o1[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    const uint64_t r2 = f2_fma(f2_pack(__uint_as_float(__float_as_uint(a) & 0xffff0000u),
                                       __uint_as_float(__float_as_uint(b) & 0xffff0000u)),
                               minus, r);
    f2_unpack(r2, a, b);
    o2[i] = pack_bf(a, b);
  }
  hi = make_uint4(o0[0], o0[1], o0[2], o0[3]);
  mid = make_uint4(o1[0], o1[1], o1[2], o1[3]);
  lo = make_uint4(o2[0], o2[1], o2[2], o2[3]);
}

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// 8 element warps of 168, 4 of 96, 4 of 72: 64,512 of the 65,536 the block starts with (128 each).
constexpr int kElemRegs = 168, kWeighRegs = 96, kCtrlRegs = 72;
static_assert(kElemWarps * 32 * kElemRegs + kWeighWarps * 32 * kWeighRegs + 4 * 32 * kCtrlRegs <=
                  kThreads * 128,
              "register shares");

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
  float* fDt = fS + 2 * 2 * kQ;
  float* fW = fDt + 2 * 2 * kQ;
  float* fC = reinterpret_cast<float*>(smem + L::offC);
  float* fT = reinterpret_cast<float*>(smem + L::offT);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::offBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the warp's: uniform registers
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
      if (i == kWtsFree0 || i == kWtsFree1) n = kElemWarps + kWeighWarps;
      if (i == kWFull0 || i == kWFull1) n = kWeighWarps;
      if (i >= kPair0) n = 2;
      if (i == kMReady || i == kSReady || i == kYFree0 || i == kYFree1) n = kElemWarps;
      mbar_init(&bars[i], n);
    }
    fence_mbar_init();
    *abort_flag = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int errh = int(seq) * p.H + h0;
// One thread's wait, and a whole warp's (which gives up as one).
#define DL_WAIT(bar, parity)                            \
  if (!mbar_wait(&bars[bar], (parity), p.err, errh)) { \
    *abort_flag = 1;                                    \
    goto done;                                          \
  }
#define DL_WAIT_WARP(bar, parity)                                               \
  if (!__all_sync(0xffffffffu, mbar_wait(&bars[bar], (parity), p.err, errh))) { \
    *abort_flag = 1;                                                            \
    goto done;                                                                  \
  }

  if (warp >= 12) {
    give_registers<kCtrlRegs>();
    if (warp == 12) {
      // ----------------------------------------------------------- copies
      if (lane == 0) {
        auto copy = [&](unsigned char* dst, const CUtensorMap* map, uint32_t boxes, int x, int c, int bar) {
          mbar_arrive_expect_tx(&bars[bar], boxes * L::kBox);
          for (uint32_t b = 0; b < boxes; ++b)
            tma_load_2d(dst + b * L::kBox, map, x + int(b) * 64, begin + c * kQ, &bars[bar]);
        };
        auto copy_q = [&](int c) { copy(sQ, &mapQ, L::kKBlocks, g * DK, c, kFullQ); };
        auto copy_k = [&](int c) { copy(sK + (c & 1) * L::kK, &mapK, L::kKBlocks, g * DK, c, kFullK0 + (c & 1)); };
        auto copy_v = [&](int c) { copy(sV + (c & 1) * 2 * L::kBox, &mapV, 2, h0 * DV, c, kFullV0 + (c & 1)); };
        if (!STATES && nch > 0) copy_q(0);
        for (int c = 0; c < 2 && c < nch; ++c) {
          copy_k(c);
          copy_v(c);
        }
        for (int c = 0; c + 1 < nch; ++c) {  // each buffer's last reader belongs to chunk c
          if (!STATES) {
            DL_WAIT(kY, c & 1);
            copy_q(c + 1);
          }
          if (c + 2 < nch) {
            DL_WAIT(kD0 + (c & 1), (c >> 1) & 1);
            copy_k(c + 2);
            // chunk c's values made room for its outputs on their way out
            if (!STATES) DL_WAIT(kYFree0 + (c & 1), (c >> 1) & 1);
            copy_v(c + 2);
          }
        }
      }
    } else if (warp == 13) {
      // ------------------------------------------------------------- MMAs
      {
        const uint32_t lead = elect_lane();
        constexpr uint32_t idG = idesc_bf16(128, 128, false, false);
        constexpr uint32_t idY = idesc_bf16(128, 128, false, true);
        constexpr uint32_t idM = idesc_bf16(128, DV == 64 ? 64 : 128, false, true);
        constexpr uint32_t idD = idesc_bf16(128, 128, true, true);
        for (int c = 0; c < nch; ++c) {
          const uint32_t ph = uint32_t(c) & 1u;
          const unsigned char* k = sK + ph * L::kK;
          const unsigned char* v = sV + ph * 2 * L::kBox;
          DL_WAIT_WARP(kFullK0 + ph, (c >> 1) & 1);
          if (!STATES) {
            DL_WAIT_WARP(kFullQ, ph);
            if (c > 0) DL_WAIT_WARP(kZ0 + ((c - 1) & 1), ((c - 1) >> 1) & 1);  // M, where G goes, is still being read
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks)
              umma_ss(lead, tmem + kColG, desc_sw128(sQ + (ks / 4) * L::kBox + (ks % 4) * 32, 16),
                       desc_sw128(k + (ks / 4) * L::kBox + (ks % 4) * 32, 16), idG, ks > 0);
            umma_done(lead, &bars[kG]);
            if (c > 0) DL_WAIT_WARP(kYFree0 + ((c - 1) & 1), ((c - 1) >> 1) & 1);
          }
          DL_WAIT_WARP(kSReady, ph);
          tc_fence_after();
          if (!STATES) {
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks)
              umma_ss(lead, tmem + kColY, desc_sw128(sQ + (ks / 4) * L::kBox + (ks % 4) * 32, 16),
                       desc_sw128(sS + ks * 2048, L::kSBox), idY, ks > 0);
            umma_done(lead, &bars[kY]);
          }
#pragma unroll 1
          for (int pc = 0; pc < kPieces; ++pc) {
            const int st = pc & 1;
            DL_WAIT_WARP(kWFull0 + st, (c * (kPieces / 2) + (pc >> 1)) & 1);
            tc_fence_after();
            const uint64_t a = desc_sw128(k + pc * (kPiece * 128), L::kBox);
#pragma unroll
            for (int part = 0; part < 3; ++part)
              umma_ss(lead, tmem + kColD, a, desc_sw128(sW + st * L::kWStage + part * L::kWPart, L::kWBox), idD,
                       pc + part > 0);
            umma_done(lead, &bars[kWFree0 + st]);
          }
          umma_done(lead, &bars[kD0 + ph]);
          if (!STATES) {
            DL_WAIT_WARP(kMReady, ph);
            tc_fence_after();
#pragma unroll
            for (int hd = 0; hd < kHeads; ++hd)
#pragma unroll
              for (int ks = 0; ks < kQ / 16; ++ks)
                umma_ts(lead, tmem + kColZ + hd * 64, tmem + kColG + (ks >> 1) * 32 + hd * 16 + (ks & 1) * 8,
                        desc_sw128(v + hd * L::kBox + ks * 2048, L::kBox), idM, ks > 0);
            umma_done(lead, &bars[kZ0 + ph]);
          }
        }
      }
    } else {
      // ----------------------------------------------------------- decays
      const int hs = warp - 14;
      const int h = h0 + hs;
      if (hs < kHeads) {
        const bool live = h < hend;
        const float a2 = live ? p.a[h] * kLog2e : 0.f;
        const float bias = live && p.bias != nullptr ? p.bias[h] : 0.f;
        float next[4];  // raw steps of the next chunk (the last row again behind the end)
        auto fetch = [&](int c) {
          if (!live || c >= nch) return;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            next[e] = p.dt[(long long)min(begin + c * kQ + lane * 4 + e, end - 1) * p.lddt + h];
        };
        fetch(0);
        for (int c = 0; c < nch; ++c) {
          const int buf = c & 1;
          const int t0 = begin + c * kQ + lane * 4;
          float dt[4], lam[4], raw[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) raw[e] = next[e] + bias;
          fetch(c + 1);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dt[e] = p.softplus ? softplusf(raw[e]) : raw[e];
            if (!live || t0 + e >= end) dt[e] = 0.f;
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
          *reinterpret_cast<float4*>(fDt + at) = make_float4(dt[0], dt[1], dt[2], dt[3]);
          *reinterpret_cast<float4*>(fW + at) =
              make_float4(exp2f(s[0]) * dt[0], exp2f(s[1]) * dt[1], exp2f(s[2]) * dt[2],
                          exp2f(s[3]) * dt[3]);
          if (!STATES) {
            // what brings token i to the first token of row block b = 1, 2, 3
            float* cols = fC + (buf * 2 + hs) * L::kCols;
#pragma unroll
            for (int b = 1; b < 4; ++b) {
              const float ref = __shfl_sync(0xffffffffu, s[0], 8 * b);
              if (lane < 8 * b)
                *reinterpret_cast<float4*>(cols + 16 * b * (b - 1) + lane * 4) =
                    make_float4(ex2(s[0] - ref) * dt[0], ex2(s[1] - ref) * dt[1],
                                ex2(s[2] - ref) * dt[2], ex2(s[3] - ref) * dt[3]);
            }
          }
          if (lane == 0) fT[buf * 2 + hs] = s[0] + lam[0];
          warp_arrive(&bars[kWts0 + buf], lane);
        }
      }
    }
  } else if (warp >= 8) {
    // -------------------------------------------------------------- w o V
    give_registers<kWeighRegs>();
    const int t = tid - kElemWarps * 32;               // 0 .. 127
    const int box = t >> 6, r = (t >> 3) & 7, off = r * 128 + (t & 7) * 16;
    for (int c = 0; c < nch; ++c) {
      const int buf = c & 1;
      const int len = min(kQ, end - (begin + c * kQ));
      unsigned char* v = sV + buf * 2 * L::kBox;
      const float* w = fW + (buf * 2 + (DV == 64 ? box : 0)) * kQ;
      DL_WAIT_WARP(kWts0 + buf, (c >> 1) & 1);
      DL_WAIT_WARP(kFullV0 + buf, (c >> 1) & 1);
      if (len < kQ) {
        // rows behind the sequence may hold anything: zeros for the sums over
        // tokens (G's columns there are masked)
        DL_WAIT_WARP(kFullK0 + buf, (c >> 1) & 1);
        for (int i = t; i < (kQ - len) * 8; i += kWeighWarps * 32) {
          const int at = (len + (i >> 3)) * 128 + (i & 7) * 16;
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          for (uint32_t b = 0; b < L::kKBlocks; ++b)
            *reinterpret_cast<uint4*>(sK + buf * L::kK + b * L::kBox + at) = zero;
          for (uint32_t b = 0; b < 2; ++b) *reinterpret_cast<uint4*>(v + b * L::kBox + at) = zero;
        }
      }
#pragma unroll 1
      for (int pc = 0; pc < kPieces; ++pc) {
        const int st = pc & 1, use = c * (kPieces / 2) + (pc >> 1);
        uint4 x[2];
        float wt[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = pc * kPiece + 8 * j + r;
          x[j] = *reinterpret_cast<const uint4*>(v + box * L::kBox + pc * (kPiece * 128) + j * 1024 + off);
          wt[j] = w[row];
          if (row >= len) x[j] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (use > 0) DL_WAIT_WARP(kWFree0 + st, (use - 1) & 1);
        unsigned char* dst = sW + st * L::kWStage + box * L::kWBox + off;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint4 hi, mid, lo;
          weigh8(x[j], wt[j], hi, mid, lo);
          *reinterpret_cast<uint4*>(dst + j * 1024) = hi;
          *reinterpret_cast<uint4*>(dst + L::kWPart + j * 1024) = mid;
          *reinterpret_cast<uint4*>(dst + 2 * L::kWPart + j * 1024) = lo;
        }
        fence_async_smem();
        warp_arrive(&bars[kWFull0 + st], lane);
      }
      warp_arrive(&bars[kWtsFree0 + buf], lane);
    }
  } else {
    // ------------------------------------------------------- element work
    take_registers<kElemRegs>();
    const int wg = warp >> 2, quarter = warp & 3;
    const int hs = DV == 64 ? wg : 0;       // head slot of this thread's columns
    const int h = h0 + hs;
    const bool live = h < hend;
    const int row = quarter * 32 + lane;    // token of M, Y and Z, key channel of D
    const int col0 = DV == 64 ? 0 : wg * 64;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const bool owns = row < DK;             // has a key channel of the state
    const size_t tile_off = ((ntiles > 1 ? size_t(tile) : seq) * p.H + h) * size_t(DV) * DK +
                            size_t(col0) * DK + row;
    float S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
    uint32_t pair_ph = 0;
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
    if (!STATES) {
      put_state();
      fence_async_smem();
    }
    warp_arrive(&bars[kSReady], lane);
    for (int c = 0; c < nch; ++c) {
      const uint32_t ph = uint32_t(c) & 1u;
      const int buf = c & 1;
      const int t0 = begin + c * kQ;
      const int len = min(kQ, end - t0);
      DL_WAIT_WARP(kWts0 + buf, (c >> 1) & 1);
      const float tot = fT[buf * 2 + hs];
      float grow = 0.f;
      if (!STATES) {
        const float* s = fS + (buf * 2 + hs) * kQ;
        const float st = s[row];
        grow = ex2(tot - st);
        const float far = ex2(s[quarter * 32] - st);
        const uint64_t far2 = f2_pack(far, far);
        DL_WAIT_WARP(kG, ph);
        tc_fence_after();
        constexpr int kStep = DV == 64 ? 1 : 2;  // at d_v = 128 the groups take turns
        int cb = DV == 64 ? 0 : wg;
        float x[32];
        tmem_ld32(tmem + kColG + cb * 32 + lanes, x);
        tmem_wait_ld();
        if (DV == 64) {
          tc_fence_before();
          warp_arrive(&bars[kPair0 + quarter], lane);
        }
#pragma unroll 1
        for (; cb <= quarter; cb += kStep) {
          uint32_t m[16];
          if (cb < quarter) {
            const ulonglong2* cf = reinterpret_cast<const ulonglong2*>(
                fC + (buf * 2 + hs) * L::kCols + 16 * quarter * (quarter - 1) + cb * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const ulonglong2 f = cf[i];
              float a, b;
              f2_unpack(f2_mul(f2_pack(x[4 * i], x[4 * i + 1]), f2_mul(f.x, far2)), a, b);
              m[2 * i] = pack_bf(a, b);
              f2_unpack(f2_mul(f2_pack(x[4 * i + 2], x[4 * i + 3]), f2_mul(f.y, far2)), a, b);
              m[2 * i + 1] = pack_bf(a, b);
            }
          } else {
            const ulonglong2* sp = reinterpret_cast<const ulonglong2*>(s + cb * 32);
            const ulonglong2* dp = reinterpret_cast<const ulonglong2*>(fDt + (buf * 2 + hs) * kQ + cb * 32);
            const uint64_t minus = f2_pack(-st, -st);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t sj = i & 1 ? sp[i >> 1].y : sp[i >> 1].x;
              const uint64_t dj = i & 1 ? dp[i >> 1].y : dp[i >> 1].x;
              float e0, e1, r0, r1;
              f2_unpack(f2_add(sj, minus), e0, e1);
              f2_unpack(f2_mul(f2_mul(f2_pack(ex2(e0), ex2(e1)), dj), f2_pack(x[2 * i], x[2 * i + 1])), r0, r1);
              if (2 * i == lane) r0 += dskip;
              if (2 * i + 1 == lane) r1 += dskip;
              m[i] = pack_bf(2 * i <= lane ? r0 : 0.f, 2 * i + 1 <= lane ? r1 : 0.f);
            }
          }
          // the next block, needed or not: a load under a condition could have its
          // registers copied before they arrive
          tmem_ld32(tmem + kColG + min(cb + kStep, 3) * 32 + lanes, x);
          if (DV == 64) {  // until the other head's warp has read these columns of G too
            DL_WAIT_WARP(kPair0 + quarter, pair_ph);
            pair_ph ^= 1u;
            tc_fence_after();
          }
          tmem_st16(tmem + kColG + cb * 32 + hs * 16 + lanes, m);
          tmem_wait_ld();
          if (DV == 64 && cb + kStep <= quarter) {
            tc_fence_before();
            warp_arrive(&bars[kPair0 + quarter], lane);
          }
        }
        {
          uint32_t z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0u;
          for (; cb < 4; cb += kStep) tmem_st16(tmem + kColG + cb * 32 + hs * 16 + lanes, z);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bars[kMReady], lane);
      }
      DL_WAIT_WARP(kD0 + ph, (c >> 1) & 1);
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
        put_state();  // Y, which reads the last one, was issued before D
        fence_async_smem();
      }
      tc_fence_before();
      warp_arrive(&bars[kSReady], lane);
      warp_arrive(&bars[kWtsFree0 + buf], lane);
      if (!STATES) {
        DL_WAIT_WARP(kZ0 + ph, (c >> 1) & 1);
        tc_fence_after();
        // through the warp's 32 rows of the value stage, whose last reader Z was,
        // so that 8 lanes write a row's 128 bytes (one row a lane kept the store
        // path busy for 3,000 cycles a chunk)
        unsigned char* mine = sV + (buf * 2 + wg) * L::kBox + quarter * 4096;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float y[32], z[32];
          tmem_ld32(tmem + kColY + wg * 64 + b * 32 + lanes, y);
          tmem_ld32(tmem + kColZ + wg * 64 + b * 32 + lanes, z);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_bf(fmaf(y[8 * i + 2 * k], grow, z[8 * i + 2 * k]),
                             fmaf(y[8 * i + 2 * k + 1], grow, z[8 * i + 2 * k + 1]));
            *reinterpret_cast<uint4*>(mine + lane * 128 + (((b * 4 + i) ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
        {
          const int r0 = lane >> 3, ch = lane & 7;
          __nv_bfloat16* o = p.o + (long long)(t0 + quarter * 32 + r0) * p.ldo + h * DV + col0 + ch * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = r0 + 4 * i;
            const uint4 w = *reinterpret_cast<const uint4*>(mine + r * 128 + ((ch ^ (r & 7)) << 4));
            if (live && quarter * 32 + r < len) *reinterpret_cast<uint4*>(o + (long long)(4 * i) * p.ldo) = w;
          }
        }
        fence_async_smem();
        tc_fence_before();
        warp_arrive(&bars[kYFree0 + ph], lane);
      }
    }
    if (live && owns) {
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
done:
  __syncwarp();
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
