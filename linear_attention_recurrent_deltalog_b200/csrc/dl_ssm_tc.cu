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
//     Y = grow o Y + M V   [t, p]   A: M as bf16 in TMEM, B: V, MN-major
//     D = (w o V)^T K      [p, n]   A: w o V in TMEM as three bf16 parts, B: K, MN-major
// Rounding: the state is carried in fp32 registers (one thread per value row)
// and w o V enters D as hi + mid + lo, all 24 bits, so S' is right to fp32
// rounding; only what feeds the bf16 output o is rounded to bf16 on the way, each
// term once (M, or the state that q reads), which is of the size of o's own
// rounding (0.0023 of o's norm in all, 0.0017 of it the output's).
//
// A work item is 128 value columns (two neighbouring heads of a group at d_v =
// 64, which share G and the loads of q and k; one head at 128) over the chunks of
// one tile of one sequence; a CTA an SM walks over its items, the next one's
// loads in flight.  Long sequences are cut into tiles when there are too few
// items: a first launch (STATES) forms every tile's own state from zero,
// dl_ssm_join_kernel turns those into the state each tile enters with, and the
// main launch starts from them.
//
// T = 8192, H = 64, d = 128 x 64, one sequence in four tiles: 114 us a pass in a row
// of passes.  Each launch alone, caches cold, under the profiler: 38 us for the
// states (2.4 a chunk), 7 for the join, 75 for the main launch (4.7 a chunk, 1.8 of
// them its MMAs').  What bounds a chunk is the element work: 4,490 of a
// scheduler's 8,100 cycles issue an instruction, the tensor pipe is busy for 0.38
// of them.  M and w o V are TMEM operands because shared memory is next: an MMA
// with both operands there reads 128 bytes a cycle, all it can deliver, and w o V
// there, written once and read with K three times over, cost 0.3 MB more a chunk.
//
// Warps 0-7: M and o (warp w reaches TMEM lanes 32 (w mod 4) ..).  Warps 8-11:
// the state, a value row a thread.  Warps 12-19: w o V, 16 tokens at a time.
// Warp 20: TMA.  Warp 21: MMA issue.  Warps 22, 23: dt, decays and their sums,
// one chunk ahead.  In turn the tensor cores run G, D with Y in its middle,
// M V; M is formed while D runs, the state moves on and o is written while M V
// and the next G run.  (With the state and M in the same warps, one after the
// other, a chunk took half as long again.)
#include <cuda.h>

#include <algorithm>

#include "dl_layer.cuh"
#include "dl_tmem.cuh"

namespace dl {

namespace {

constexpr int kQ = 128;             // tokens per chunk
constexpr int kElemWarps = 8, kStateWarps = 4, kWeighWarps = 8, kCtrlWarps = 4;
constexpr int kFirstState = kElemWarps, kFirstWeigh = kFirstState + kStateWarps,
              kFirstCtrl = kFirstWeigh + kWeighWarps;
constexpr int kThreads = 32 * (kFirstCtrl + kCtrlWarps);
constexpr int kPiece = 16;          // tokens of w o V staged at a time
constexpr int kPieces = kQ / kPiece;
constexpr float kLog2e = 1.4426950408889634f;
// Decay factors below 2^-150 are 0 in fp32: clamping there keeps the sums finite.
constexpr float kMinLambda = -150.f;

// TMEM columns.  M takes G's place block by block: tokens 32 b .. 32 b + 31 of
// head slot s are the 16 columns at kColG + 32 b + 16 s.  A stage of w o V is
// three parts of 8 columns (16 tokens, two a column).
constexpr int kStages = 4;
constexpr uint32_t kColG = 0, kColY = 128, kColW = 256, kColD = 384;
constexpr uint32_t kWPart = kPiece / 2, kWStage = 3 * kWPart;
static_assert(kColW + kStages * kWStage <= kColD, "TMEM columns");

template <int DK>
struct TcLayout {
  static constexpr uint32_t kKBlocks = DK / 64;                 // 64-column boxes of q, k and the state
  static constexpr uint32_t kBox = kQ * 128;                    // bytes of a box
  static constexpr uint32_t kK = kKBlocks * kBox;
  static constexpr uint32_t offQ = 0;
  static constexpr uint32_t offK = offQ + kK;                   // two stages
  static constexpr uint32_t offV = offK + 2 * kK;               // two stages of two boxes
  static constexpr uint32_t offS = offV + 4 * kBox;             // the state, 128 value rows
  // per token, [2 buffers][2 heads][128] floats: s, dt, w; and the column
  // factors of M's blocks below the diagonal ones, 32 + 64 + 96 per head
  static constexpr uint32_t offF = offS + kK;
  static constexpr uint32_t kF = 2 * 2 * kQ * 4;
  static constexpr uint32_t kCols = 192;
  static constexpr uint32_t offC = offF + 3 * kF;
  static constexpr uint32_t offT = offC + 2 * 2 * kCols * 4;    // tot [2][2]
  static constexpr uint32_t offBar = offT + 16;
  static constexpr uint32_t total = offBar + 40 * 8 + 16 + 1024;  // + alignment of the base
};
static_assert(TcLayout<128>::total <= kMaxSmemOptIn, "shared memory of a CTA");

enum Bar {
  kFullQ, kFullK0, kFullK1, kFullV0, kFullV1, kWts0, kWts1, kWtsFree0, kWtsFree1, kWFull0,
  kWFree0 = kWFull0 + kStages, kG = kWFree0 + kStages, kY, kD0, kD1, kZ0, kZ1, kMReady, kSReady, kSReady1,
  kYFree, kVFree0, kVFree1, kPair0, kBars = kPair0 + 4
};
static_assert(kBars <= 40, "barrier slots");

// The sequences of a launch, longest first, and the tiles they are cut into.
template <int N>
struct OrderedSeqs {
  int n;
  int seq[N], begin[N], end[N];  // place in the call, tokens
  int tile0[N + 1];
  __device__ __forceinline__ int index(int sl) const { return seq[sl]; }
  __device__ __forceinline__ int find(int tile) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile0[mid] <= tile)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
};

template <int N>
long long fill_ordered(OrderedSeqs<N>& t, const int32_t* starts, int s0, int n, int tile) {
  t.n = n;
  for (int i = 0; i < n; ++i) t.seq[i] = i;
  std::stable_sort(t.seq, t.seq + n, [&](int a, int b) {
    return starts[s0 + a + 1] - starts[s0 + a] > starts[s0 + b + 1] - starts[s0 + b];
  });
  long long tiles = 0;
  for (int i = 0; i < n; ++i) {
    t.begin[i] = starts[s0 + t.seq[i]];
    t.end[i] = starts[s0 + t.seq[i] + 1];
    t.tile0[i] = int(tiles);
    const long long len = (long long)t.end[i] - t.begin[i];
    tiles += len > tile ? (len + tile - 1) / tile : 1;
  }
  t.tile0[n] = int(tiles);
  return tiles;
}

struct TcParams {
  const float* dt;
  const float* a;
  const float* d;
  const float* bias;
  const float* S0;
  float* S1;
  __nv_bfloat16* o;
  float* ws;        // [tiles, H, DK, DV]: STATES writes a tile's own state, main reads its entry state
  float* wdecay;    // [tiles, H] log2 of a tile's whole decay
  int* err;
  long long lddt, ldo;
  int H, G, softplus;
  int pairs;        // work items per tile
  int hpg, ppg;     // heads and items of a group
  int tile_tokens;
  unsigned items;   // tiles * pairs
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x below the diagonal (j < lane), x + d on it, 0 above.  In assembly, because
// the compiler would branch around the exponential in x, once an element.
__device__ __forceinline__ float on_diagonal(float x, float d, int j, int lane) {
  float r;
  asm("{\n\t.reg .pred p, q;\n\t.reg .f32 y;\n\t"
      "setp.eq.s32 p, %3, %4;\n\t"
      "setp.gt.s32 q, %3, %4;\n\t"
      "selp.f32 y, %2, 0f00000000, p;\n\t"
      "add.rn.f32 y, y, %1;\n\t"
      "selp.f32 %0, 0f00000000, y, q;\n\t}"
      : "=f"(r)
      : "f"(x), "f"(d), "r"(j), "r"(lane));
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

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// A box of 32 rows on its way out, and the wait until its shared memory has been read.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
               "r"(x), "r"(y), "r"(smem_u32(src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
// 16 lanes x 32 columns: registers 4 b + 2 i, + 1 of lane l are columns 8 b +
// 2 (l mod 4), + 1 of TMEM lane 8 i + l / 4.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}

// mbar_wait with a long suspension: a waiting warp sleeps until its phase
// completes (or a millisecond has passed) and leaves the issue slots to others.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* err, int head) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    if (done) return true;
    if (clock64() - t0 > kWaitCycles) {
      if (err != nullptr && atomicCAS(err, 0, kDevErrTimeout) == 0) err[1] = head;
      return false;
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two bf16 values times two weights, each product as three bf16 parts whose
// sum is the fp32 product: the upper 16 bits are cut off twice (exact
// remainders), the last part is rounded.  21 cycles a scheduler; products and
// remainders in packed bf16 operations took 40, in packed fp32 ones no less.
__device__ __forceinline__ void weigh2(uint32_t v2, float2 w, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  float a = __uint_as_float(v2 << 16) * w.x, b = __uint_as_float(v2 & 0xffff0000u) * w.y;
  hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
  b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
  mid = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
  b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
  lo = pack_bf(a, b);
}

// Four 8 x 8 matrices of 16-bit elements, transposed: register m of lane l
// holds rows 2 (l mod 4), 2 (l mod 4) + 1 of column l / 4 of matrix m.
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t (&r)[4], const void* row_addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(row_addr))
               : "memory");
}
// 16 lanes x 8 columns: registers 0, 1 (2, 3) of lane l are column l mod 4 (4 +
// l mod 4) of TMEM lanes l / 4 and 8 + l / 4.
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Registers a thread starts with, and the share of each role.
constexpr int kStartRegs = 80, kElemRegs = 88, kStateRegs = 168, kWeighRegs = 48, kCtrlRegs = 40;
static_assert(kElemWarps * kElemRegs + kStateWarps * kStateRegs + kWeighWarps * kWeighRegs +
                      kCtrlWarps * kCtrlRegs <=
                  kThreads / 32 * kStartRegs,
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
                    const __grid_constant__ CUtensorMap mapV,
                    const __grid_constant__ CUtensorMap mapO) {
  using L = TcLayout<DK>;
  constexpr int kHeads = 128 / DV;  // heads a CTA covers
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sQ = smem + L::offQ;
  unsigned char* sK = smem + L::offK;
  unsigned char* sV = smem + L::offV;
  unsigned char* sS = smem + L::offS;
  float* fS = reinterpret_cast<float*>(smem + L::offF);  // [buf][head][token]
  float* fDt = fS + 2 * 2 * kQ;
  float* fW = fDt + 2 * 2 * kQ;
  float* fC = reinterpret_cast<float*>(smem + L::offC);
  float* fT = reinterpret_cast<float*>(smem + L::offT);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::offBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the warp's: uniform registers
  // Work item: a tile of a sequence and the heads of 128 value columns.
  struct Work {
    int tile, begin, end, nch;
    int g, h0, hend;
    bool cut, last;  // the sequence has several tiles; this is its last
    size_t seq;
  };
  auto work = [&](unsigned item) {
    Work w;
    w.tile = int(item / unsigned(p.pairs));
    const int pair = int(item - unsigned(w.tile) * unsigned(p.pairs));
    const int sl = seqs.find(w.tile);
    const int first = seqs.tile0[sl], ntiles = seqs.tile0[sl + 1] - first;
    w.begin = seqs.begin[sl] + (w.tile - first) * p.tile_tokens;
    w.end = w.begin + min(p.tile_tokens, seqs.end[sl] - w.begin);  // the sum stays an int32
    w.nch = (w.end - w.begin + kQ - 1) / kQ;
    w.cut = ntiles > 1;
    w.last = w.tile - first == ntiles - 1;
    // pairs run through the heads of a group
    w.g = p.G > 1 ? pair / p.ppg : 0;
    w.h0 = w.g * p.hpg + (pair - w.g * p.ppg) * kHeads;
    w.hend = (w.g + 1) * p.hpg;
    w.seq = size_t(seq0) + size_t(seqs.index(sl));
    return w;
  };
  // A CTA's items, every role's alike: items come longest first and every other
  // round of them is dealt in reverse, so that the CTAs' shares are even.  (In
  // STATES nobody needs a last tile.)
#define DL_ITEMS(w)                                                                              \
  for (unsigned round = 0, item = blockIdx.x; item < p.items;                                    \
       ++round, item = round * gridDim.x + ((round & 1u) ? gridDim.x - 1 - blockIdx.x : blockIdx.x)) \
    if (const Work w = work(item); !(STATES && w.last))

  // The state an item enters with, in the call or in the workspace; heads of an
  // item lie side by side in both.
  auto prefetch_state = [&](const Work& w, int at, int step) {
    const float* in = STATES ? nullptr : (w.cut ? p.ws + (size_t(w.tile) * p.H + w.h0) * size_t(DV) * DK
                              : p.S0 != nullptr ? p.S0 + (w.seq * p.H + w.h0) * size_t(DV) * DK : nullptr);
    if (in == nullptr) return;
    const int lines = min(kHeads, w.hend - w.h0) * (DV * DK / 32);
    for (int i = at; i < lines; i += step) prefetch_l2(in + size_t(i) * 32);
  };
  // what the roles ask for first is on its way while they are set up
  {
    const Work w = work(blockIdx.x);
    prefetch_state(w, tid, kThreads);
    if (tid < kQ && w.begin + tid < w.end) prefetch_l2(p.dt + (long long)(w.begin + tid) * p.lddt + w.h0);
    if (tid == kThreads - 1) {
      prefetch_map(&mapQ);
      prefetch_map(&mapK);
      prefetch_map(&mapV);
      prefetch_map(&mapO);
    }
  }
  if (warp == 0) tmem_alloc(tmem_slot, 512);
  if (tid == 32) {
    for (int i = 0; i < kBars; ++i) {
      uint32_t n = 1;
      if (i == kWts0 || i == kWts1) n = kHeads;
      if (i == kWtsFree0 || i == kWtsFree1) n = (STATES ? 0 : kElemWarps) + kStateWarps + kWeighWarps;
      if (i == kSReady || i == kSReady1) n = kStateWarps;
      if (i >= kWFull0 && i < kWFree0) n = kWeighWarps / 2;
      if (i >= kPair0) n = 2;
      if (i == kMReady || i == kYFree || i == kVFree0 || i == kVFree1) n = kElemWarps;
      mbar_init(&bars[i], n);
    }
    fence_mbar_init();
    *abort_flag = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int errh = int(blockIdx.x);
// One thread's wait, and a whole warp's (which gives up as one).
#define DL_WAIT(bar, parity)                            \
  if (!wait_phase(&bars[bar], (parity), p.err, errh)) { \
    *abort_flag = 1;                                    \
    goto done;                                          \
  }
#define DL_WAIT_WARP(bar, parity)                                               \
  if (!__all_sync(0xffffffffu, wait_phase(&bars[bar], (parity), p.err, errh))) { \
    *abort_flag = 1;                                                            \
    goto done;                                                                  \
  }

  if (warp >= kFirstCtrl) {
    give_registers<kCtrlRegs>();
    if (warp == kFirstCtrl) {
      // ----------------------------------------------------------- copies
      if (lane == 0) {
        auto copy = [&](unsigned char* dst, const CUtensorMap* map, uint32_t boxes, int x, int t, int bar) {
          mbar_arrive_expect_tx(&bars[bar], boxes * L::kBox);
          for (uint32_t b = 0; b < boxes; ++b)
            tma_load_2d(dst + b * L::kBox, map, x + int(b) * 64, t, &bars[bar]);
        };
        unsigned n = 0;
        DL_ITEMS(w) {
          for (int c = 0; c < w.nch; ++c, ++n) {
            const uint32_t ph = n & 1u;
            const int t = w.begin + c * kQ;
            // in the order in which the buffers come free: k's last reader is D of
            // the last chunk but one, the values' its outputs on their way out, q's
            // the last chunk's Y
            if (n > 1) DL_WAIT(kD0 + ph, ((n >> 1) - 1) & 1);
            copy(sK + ph * L::kK, &mapK, L::kKBlocks, w.g * DK, t, kFullK0 + ph);
            if (!STATES && n > 1) DL_WAIT(kVFree0 + ph, ((n >> 1) - 1) & 1);
            copy(sV + ph * 2 * L::kBox, &mapV, 2, w.h0 * DV, t, kFullV0 + ph);
            if (!STATES) {
              if (n > 0) DL_WAIT(kY, (n - 1) & 1);
              copy(sQ, &mapQ, L::kKBlocks, w.g * DK, t, kFullQ);
            }
          }
        }
      }
    } else if (warp == kFirstCtrl + 1) {
      // ------------------------------------------------------------- MMAs
      {
        const uint32_t lead = elect_lane();
        constexpr uint32_t idG = idesc_bf16(128, 128, false, false);
        constexpr uint32_t idY = idG;
        constexpr uint32_t idM = idesc_bf16(128, DV == 64 ? 64 : 128, false, true);
        constexpr uint32_t idD = idesc_bf16(128, DK, false, true);
        unsigned n = 0;
        DL_ITEMS(w)
        for (int c = 0; c < w.nch; ++c, ++n) {
          const uint32_t ph = n & 1u;
          const unsigned char* k = sK + ph * L::kK;
          const unsigned char* v = sV + ph * 2 * L::kBox;
          DL_WAIT_WARP(kFullK0 + ph, (n >> 1) & 1);
          if (!STATES) {
            DL_WAIT_WARP(kFullQ, ph);
            if (n > 0) DL_WAIT_WARP(kZ0 + (ph ^ 1u), ((n - 1) >> 1) & 1);  // M, where G goes, is still being read
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks)
              umma_ss(lead, tmem + kColG, desc_sw128(sQ + (ks / 4) * L::kBox + (ks % 4) * 32, 16),
                       desc_sw128(k + (ks / 4) * L::kBox + (ks % 4) * 32, 16), idG, ks > 0);
            umma_done(lead, &bars[kG]);
          }
          // STATES alternates between two accumulators (no G takes the other's
          // place): a chunk waits for the state to have taken up the last but one
          if (!STATES) DL_WAIT_WARP(kSReady, ph);
          if (STATES && n > 1) DL_WAIT_WARP(kSReady + ph, ((n >> 1) - 1) & 1);
          tc_fence_after();
          const uint32_t dcol = tmem + (STATES && ph ? kColG : kColD);
#pragma unroll 1
          for (int pc = 0; pc < kPieces; ++pc) {
            if (!STATES && pc == kPieces / 2) {  // by now the last chunk's Y has been read
              if (n > 0) DL_WAIT_WARP(kYFree, (n - 1) & 1);
              tc_fence_after();
#pragma unroll
              for (int ks = 0; ks < DK / 16; ++ks)
                umma_ss(lead, tmem + kColY, desc_sw128(sQ + (ks / 4) * L::kBox + (ks % 4) * 32, 16),
                        desc_sw128(sS + (ks / 4) * L::kBox + (ks % 4) * 32, 16), idY, ks > 0);
              umma_done(lead, &bars[kY]);
            }
            const int st = pc % kStages;
            DL_WAIT_WARP(kWFull0 + st, (n * (kPieces / kStages) + pc / kStages) & 1);
            tc_fence_after();
            const uint64_t kd = desc_sw128(k + pc * (kPiece * 128), L::kBox);
#pragma unroll
            for (int part = 0; part < 3; ++part)
              umma_ts(lead, dcol, tmem + kColW + st * kWStage + part * kWPart, kd, idD, pc + part > 0);
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
                umma_ts(lead, tmem + kColY + hd * 64, tmem + kColG + (ks >> 1) * 32 + hd * 16 + (ks & 1) * 8,
                        desc_sw128(v + hd * L::kBox + ks * 2048, L::kBox), idM, true);
            umma_done(lead, &bars[kZ0 + ph]);
          }
        }
      }
    } else {
      // ----------------------------------------------------------- decays
      const int hs = warp - kFirstCtrl - 2;
      if (hs < kHeads) {
        unsigned n = 0;
        DL_ITEMS(w) {
        const int h = w.h0 + hs;
        const bool live = h < w.hend;
        const float a2 = live ? p.a[h] * kLog2e : 0.f;
        const float bias = live && p.bias != nullptr ? p.bias[h] : 0.f;
        float next[4];  // raw steps of the next chunk (the last row again behind the end)
        auto fetch = [&](int c) {
          if (!live || c >= w.nch) return;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            next[e] = p.dt[(long long)min(w.begin + c * kQ + lane * 4 + e, w.end - 1) * p.lddt + h];
        };
        fetch(0);
        if (round > 0) prefetch_state(w, hs * 32 + lane, kHeads * 32);
        for (int c = 0; c < w.nch; ++c, ++n) {
          const int buf = int(n & 1u);
          const int t0 = w.begin + c * kQ + lane * 4;
          float dt[4], lam[4], raw[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) raw[e] = next[e] + bias;
          fetch(c + 1);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dt[e] = p.softplus ? softplusf(raw[e]) : raw[e];
            if (!live || t0 + e >= w.end) dt[e] = 0.f;
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
          if (n > 1) DL_WAIT_WARP(kWtsFree0 + buf, ((n >> 1) - 1) & 1);
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
    }
  } else if (warp >= kFirstWeigh) {
    // -------------------------------------------------------------- w o V
    give_registers<kWeighRegs>();
    const int odd = (warp - kFirstWeigh) >> 2;  // four warps take the even pieces, four the odd ones
    const int quarter = warp & 3;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const int head = DV == 64 ? quarter >> 1 : 0;
    // this lane's row of the matrices it points at: tokens r, 8 + r; 8 value columns each
    const int r = lane & 7, trow = (lane >> 4) * 8 + r, pblk = (lane >> 3) & 1;
    uint32_t at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      at[i] = (quarter >> 1) * L::kBox + trow * 128 + ((((quarter & 1) * 4 + i * 2 + pblk) ^ r) << 4);
    unsigned n = 0;
    DL_ITEMS(wk)
    for (int c = 0; c < wk.nch; ++c, ++n) {
      const int buf = int(n & 1u);
      const int len = min(kQ, wk.end - (wk.begin + c * kQ));
      unsigned char* v = sV + buf * 2 * L::kBox;
      const float2* w = reinterpret_cast<const float2*>(fW + (buf * 2 + head) * kQ) + (lane & 3);
      DL_WAIT_WARP(kWts0 + buf, (n >> 1) & 1);
      DL_WAIT_WARP(kFullV0 + buf, (n >> 1) & 1);
      if (len < kQ && odd == 0) {
        // rows behind the sequence may hold anything: zeros for the sums over
        // tokens (G's columns there are masked), in place before the first piece
        DL_WAIT_WARP(kFullK0 + buf, (n >> 1) & 1);
        for (int i = tid - kFirstWeigh * 32; i < (kQ - len) * 8; i += 128) {
          const int at = (len + (i >> 3)) * 128 + (i & 7) * 16;
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          for (uint32_t b = 0; b < L::kKBlocks; ++b)
            *reinterpret_cast<uint4*>(sK + buf * L::kK + b * L::kBox + at) = zero;
          for (uint32_t b = 0; b < 2; ++b) *reinterpret_cast<uint4*>(v + b * L::kBox + at) = zero;
        }
        fence_async_smem();
      }
#pragma unroll 1
      for (int pc = odd; pc < kPieces; pc += 2) {
        const int st = pc % kStages, use = int(n) * (kPieces / kStages) + pc / kStages;
        uint32_t x[2][4], part[3][2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) ldmatrix_x4_t(x[i], v + pc * (kPiece * 128) + at[i]);
        const float2 w0 = w[pc * (kPiece / 2)], w1 = w[pc * (kPiece / 2) + 4];
        if ((pc + 1) * kPiece > len) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int first = pc * kPiece + (j >> 1) * 8 + 2 * (lane & 3);
            const uint32_t keep = first >= len ? 0u : (first + 1 >= len ? 0xffffu : 0xffffffffu);
            x[0][j] &= keep;
            x[1][j] &= keep;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            weigh2(x[i][j], j < 2 ? w0 : w1, part[0][i][j], part[1][i][j], part[2][i][j]);
        if (use > 0) DL_WAIT_WARP(kWFree0 + st, (use - 1) & 1);
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tmem_st_16x8(tmem + kColW + st * kWStage + q * kWPart + lanes + (uint32_t(16 * i) << 16), part[q][i]);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bars[kWFull0 + st], lane);
      }
      warp_arrive(&bars[kWtsFree0 + buf], lane);
    }
  } else if (warp >= kFirstState) {
    // ---------------------------------------------------------- the state
    take_registers<kStateRegs>();
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;    // value row, lane of D
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const int hd = DV == 64 ? quarter >> 1 : 0;
    const int p0 = DV == 64 ? (quarter & 1) * 32 : quarter * 32;  // the warp's first row of its head
    // The state comes and goes through D's place in TMEM: global rows are
    // touched 32 bytes by 4 lanes, the registers hold a row a lane.
    unsigned n = 0;
    DL_ITEMS(w) {
    const bool owns = w.h0 + hd < w.hend;
    const size_t head_off = (w.seq * p.H + w.h0 + hd) * size_t(DV) * DK + size_t(p0) * DK;
    const size_t tile_off = (size_t(w.tile) * p.H + w.h0 + hd) * size_t(DV) * DK + p0 + lane;
    const size_t piece = head_off + size_t(lane >> 2) * DK + 2 * (lane & 3);
    float decay = 0.f;  // log2 of everything forgotten in this tile (STATES)
    float S[DK];
    if (STATES) {
#pragma unroll
      for (int i = 0; i < DK; ++i) S[i] = 0.f;
    } else {
      const bool ws = owns && w.cut, user = owns && !w.cut && p.S0 != nullptr;
      // all loads before the first store: one latency, not DK / 32
      float x[DK / 32][32];
      const uint32_t to = tmem + kColD + lanes;
      if (user) {
#pragma unroll
        for (int b = 0; b < DK / 32; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 v = *reinterpret_cast<const float2*>(
                p.S0 + piece + size_t((i >> 3) * 16 + (i & 1) * 8) * DK + b * 32 + ((i >> 1) & 3) * 8);
            x[b][2 * i] = v.x;
            x[b][2 * i + 1] = v.y;
          }
#pragma unroll
        for (int b = 0; b < DK / 32; ++b) {
          tmem_st_16x32(to + b * 32, *reinterpret_cast<float(*)[16]>(x[b]));
          tmem_st_16x32(to + b * 32 + (16u << 16), *reinterpret_cast<float(*)[16]>(x[b] + 16));
        }
      } else {
#pragma unroll
        for (int b = 0; b < DK / 32; ++b)
#pragma unroll
          for (int i = 0; i < 32; ++i) x[b][i] = ws ? p.ws[tile_off + size_t(b * 32 + i) * DV] : 0.f;
#pragma unroll
        for (int b = 0; b < DK / 32; ++b) tmem_st32(to + b * 32, x[b]);
      }
      tmem_wait_st();
#pragma unroll
      for (int b = 0; b < DK / 32; ++b)
        tmem_ld32(tmem + kColD + b * 32 + lanes, *reinterpret_cast<float(*)[32]>(S + 32 * b));
      tmem_wait_ld();
      tc_fence_before();
    }
    auto put8 = [&](int i) {  // eight channels as bf16
      *reinterpret_cast<uint4*>(sS + (i / 8) * L::kBox + row * 128 + (((i & 7) ^ (row & 7)) << 4)) =
          make_uint4(pack_bf(S[8 * i], S[8 * i + 1]), pack_bf(S[8 * i + 2], S[8 * i + 3]),
                     pack_bf(S[8 * i + 4], S[8 * i + 5]), pack_bf(S[8 * i + 6], S[8 * i + 7]));
    };
    if (!STATES) {
#pragma unroll
      for (int i = 0; i < DK / 8; ++i) put8(i);
      fence_async_smem();
    }
    if (!STATES && w.nch > 0) warp_arrive(&bars[kSReady], lane);
    for (int c = 0; c < w.nch; ++c, ++n) {
      const uint32_t ph = n & 1u;
      const int buf = int(ph);
      // the next item's state stands in for this one's last
      const bool goes_on = STATES || c + 1 < w.nch;
      DL_WAIT_WARP(kWts0 + buf, (n >> 1) & 1);
      const float tot = fT[buf * 2 + hd];
      const float keep = exp2f(tot);
      decay += tot;
      warp_arrive(&bars[kWtsFree0 + buf], lane);
      DL_WAIT_WARP(kD0 + ph, (n >> 1) & 1);
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < DK / 16; ++b) {
        float x[16];
        tmem_ld16(tmem + (STATES && ph ? kColG : kColD) + b * 16 + lanes, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) S[b * 16 + i] = fmaf(S[b * 16 + i], keep, x[i]);
        if (!STATES && goes_on) {  // Y, which reads the last one, was issued before D's end
          put8(2 * b);
          put8(2 * b + 1);
        }
      }
      if (!STATES) fence_async_smem();
      tc_fence_before();
      if (goes_on) warp_arrive(&bars[STATES ? kSReady + ph : kSReady], lane);
    }
    if (STATES) {
      if (owns) {
#pragma unroll
        for (int i = 0; i < DK; ++i) p.ws[tile_off + size_t(i) * DV] = S[i];
        if (p0 + lane == 0) p.wdecay[size_t(w.tile) * p.H + w.h0 + hd] = decay;
      }
    } else if (owns && w.last && p.S1 != nullptr) {
#pragma unroll
      for (int b = 0; b < DK / 32; ++b)
        tmem_st32(tmem + kColD + b * 32 + lanes, *reinterpret_cast<float(*)[32]>(S + 32 * b));
      tmem_wait_st();
      float x[DK / 32][32];
      const uint32_t from = tmem + kColD + lanes;
#pragma unroll
      for (int b = 0; b < DK / 32; ++b) {
        tmem_ld_16x32(from + b * 32, *reinterpret_cast<float(*)[16]>(x[b]));
        tmem_ld_16x32(from + b * 32 + (16u << 16), *reinterpret_cast<float(*)[16]>(x[b] + 16));
      }
      tmem_wait_ld();
#pragma unroll
      for (int b = 0; b < DK / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          *reinterpret_cast<float2*>(p.S1 + piece + size_t((i >> 3) * 16 + (i & 1) * 8) * DK + b * 32 +
                                     ((i >> 1) & 3) * 8) = make_float2(x[b][2 * i], x[b][2 * i + 1]);
    }
    }
  } else if (!STATES) {
    // ----------------------------------------------------------- M and o
    take_registers<kElemRegs>();
    const int wg = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;    // token
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    // Y: 64 value columns of head slot hs
    const int hs = DV == 64 ? wg : 0;
    const int col0 = DV == 64 ? 0 : wg * 64;
    unsigned n = 0;
    DL_ITEMS(w) {
    const int h = w.h0 + hs;
    const bool live = h < w.hend;
    const float dskip = live && p.d != nullptr ? p.d[h] : 0.f;
    for (int c = 0; c < w.nch; ++c, ++n) {
      const uint32_t ph = n & 1u;
      const int buf = int(ph);
      const int t0 = w.begin + c * kQ;
      const int len = min(kQ, w.end - t0);
      DL_WAIT_WARP(kWts0 + buf, (n >> 1) & 1);
      const float grow = ex2(fT[buf * 2 + hs] - fS[(buf * 2 + hs) * kQ + row]);
      float st[kHeads];
#pragma unroll
      for (int e = 0; e < kHeads; ++e) st[e] = fS[(buf * 2 + e) * kQ + row];
      DL_WAIT_WARP(kG, ph);
      tc_fence_after();
      if (n > 0) {  // by now the last chunk's outputs have left its value stage
        if (lane == 0) tma_store_read();
        warp_arrive(&bars[kVFree0 + (buf ^ 1)], lane);
      }
      // M's blocks below the diagonal are formed by one group for both heads
      // (at d_v = 64 the groups take turns, at 128 group 0 has them), so that
      // they can take G's place at once.  The diagonal one has two readers at
      // d_v = 64, each for its head, and goes in once both have read it.
      float x[32];
      uint32_t m[16];
      const uint32_t at = tmem + kColG + lanes;
      constexpr int kStep = kHeads;
      if (kHeads == 2 || wg == 1) {
        tmem_ld32(at + quarter * 32, x);
        tmem_wait_ld();
        if (kHeads == 2) {
          tc_fence_before();
          warp_arrive(&bars[kPair0 + quarter], lane);
        }
        const float4* sp = reinterpret_cast<const float4*>(fS + (buf * 2 + hs) * kQ + quarter * 32);
        const float4* dp = reinterpret_cast<const float4*>(fDt + (buf * 2 + hs) * kQ + quarter * 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 sc = sp[i], dc = dp[i];
          const float se[4] = {sc.x, sc.y, sc.z, sc.w}, de[4] = {dc.x, dc.y, dc.z, dc.w};
          float r[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            r[k] = on_diagonal(x[4 * i + k] * (ex2(se[k] - st[hs]) * de[k]), dskip, 4 * i + k, lane);
          m[2 * i] = pack_bf(r[0], r[1]);
          m[2 * i + 1] = pack_bf(r[2], r[3]);
        }
        if (kHeads == 2) {
          DL_WAIT_WARP(kPair0 + quarter, ph);
          tc_fence_after();
        }
        tmem_st16(at + quarter * 32 + 16 * hs, m);
      }
      if (kHeads == 2 || wg == 0) {
        float far[kHeads];
#pragma unroll
        for (int e = 0; e < kHeads; ++e) far[e] = ex2(fS[(buf * 2 + e) * kQ + quarter * 32] - st[e]);
        int cb = kHeads == 2 ? wg : 0;
#pragma unroll 1
        for (; cb < quarter; cb += kStep) {
          tmem_ld32(at + cb * 32, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kHeads; ++e) {
            const float4* cf = reinterpret_cast<const float4*>(
                fC + (buf * 2 + e) * L::kCols + 16 * quarter * (quarter - 1) + cb * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 f = cf[i];
              m[2 * i] = pack_bf(x[4 * i] * (f.x * far[e]), x[4 * i + 1] * (f.y * far[e]));
              m[2 * i + 1] = pack_bf(x[4 * i + 2] * (f.z * far[e]), x[4 * i + 3] * (f.w * far[e]));
            }
            tmem_st16(at + cb * 32 + 16 * e, m);
          }
        }
        if (cb == quarter) cb += kStep;
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i] = 0u;
        for (; cb < 4; cb += kStep)
#pragma unroll
          for (int e = 0; e < kHeads; ++e) tmem_st16(at + cb * 32 + 16 * e, m);
      }
      warp_arrive(&bars[kWtsFree0 + buf], lane);
      // Y as it enters the sum
      DL_WAIT_WARP(kY, ph);
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        tmem_ld32(tmem + kColY + wg * 64 + b * 32 + lanes, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] *= grow;
        tmem_st32(tmem + kColY + wg * 64 + b * 32 + lanes, x);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&bars[kMReady], lane);
      DL_WAIT_WARP(kZ0 + ph, (n >> 1) & 1);
      tc_fence_after();
      // through the warp's 32 rows of the value stage, whose last reader M V was:
      // whole boxes leave by TMA (a row a lane kept the store path busy for 3,000
      // cycles a chunk)
      unsigned char* out = sV + (buf * 2 + wg) * L::kBox + quarter * 4096;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        tmem_ld32(tmem + kColY + wg * 64 + b * 32 + lanes, x);
        tmem_wait_ld();
        if (b == 1) {
          tc_fence_before();
          warp_arrive(&bars[kYFree], lane);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(out + lane * 128 + (((4 * b + i) ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf(x[8 * i], x[8 * i + 1]), pack_bf(x[8 * i + 2], x[8 * i + 3]),
                         pack_bf(x[8 * i + 4], x[8 * i + 5]), pack_bf(x[8 * i + 6], x[8 * i + 7]));
      }
      fence_async_smem();
      __syncwarp();
      if (live && quarter * 32 + 32 <= len) {
        if (lane == 0) tma_store_2d(&mapO, h * DV + col0, t0 + quarter * 32, out);
      } else if (live) {  // rows behind the sequence stay as they are
        const int r0 = lane >> 3, ch = lane & 7;
        __nv_bfloat16* o = p.o + (long long)(t0 + quarter * 32 + r0) * p.ldo + h * DV + col0 + ch * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + 4 * i;
          if (quarter * 32 + r < len)
            *reinterpret_cast<uint4*>(o + (long long)(4 * i) * p.ldo) =
                *reinterpret_cast<const uint4*>(out + r * 128 + ((ch ^ (r & 7)) << 4));
        }
      }
    }
    }
  }
done:
  __syncwarp();
  if (!STATES && warp < kElemWarps && lane == 0) tma_store_read();
#undef DL_ITEMS
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
// E_0 = S0, E_{j+1} = 2^{decay_j} E_j + own_j, one thread per four value rows
// of a key channel (the workspace holds states as [d_k, d_v]).
template <typename Table>
__global__ void __launch_bounds__(256)
dl_ssm_join_kernel(const float* S0, float* ws, const float* wdecay, const __grid_constant__ Table seqs,
                   int seq0, int H, int dk, int dv) {
  const int floats = dk * dv, per = floats / 1024;  // blocks per head
  const int sl = int(blockIdx.x / unsigned(H * per));
  const int rest = int(blockIdx.x % unsigned(H * per));
  const int h = rest / per;
  const int at = (rest % per) * 1024 + threadIdx.x * 4;
  const int j0 = seqs.tile0[sl], j1 = seqs.tile0[sl + 1];
  if (j1 - j0 < 2) return;
  float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
  if (S0 != nullptr) {
    const float* src = S0 + ((size_t(seq0) + seqs.index(sl)) * H + h) * size_t(floats) + size_t(at % dv) * dk + at / dv;
    e = make_float4(src[0], src[dk], src[2 * dk], src[3 * dk]);
  }
  auto at_tile = [&](int j) { return reinterpret_cast<float4*>(ws + (size_t(j) * H + h) * size_t(floats) + at); };
  constexpr int U = 4;  // tiles in flight
  for (int j = j0; j + 1 < j1; j += U) {
    float4 own[U];
    float k[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j + u + 1 < j1) {
        own[u] = *at_tile(j + u);
        k[u] = exp2f(wdecay[size_t(j + u) * H + h]);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j + u + 1 < j1) {
        *at_tile(j + u) = e;
        e = make_float4(fmaf(e.x, k[u], own[u].x), fmaf(e.y, k[u], own[u].y), fmaf(e.z, k[u], own[u].z),
                        fmaf(e.w, k[u], own[u].w));
      }
  }
  *at_tile(j1 - 1) = e;
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

// Rows of `cols` bf16, boxes of 64 columns x `box_rows` rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, long long rows, int cols, long long ld, int box_rows) {
  EncodeFn f = encode_fn();
  if (f == nullptr) return false;
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows > 0 ? rows : 1)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {64, cuuint32_t(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool STATES, int NS>
cudaError_t launch_chunk(const TcParams& p, const OrderedSeqs<NS>& tab, int seq0, unsigned grid,
                         const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& o, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  auto kern = dl_ssm_chunk_kernel<DK, DV, STATES, OrderedSeqs<NS>>;
  // the roles' register shares add up against what the block starts with
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa{};
    const cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) < kStartRegs) return cudaErrorInvalidConfiguration;
  const cudaError_t e = prepare_kernel(kern, done);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, TcLayout<DK>::total, s>>>(p, tab, seq0, q, k, v, o);
  count_launches(1);
  return cudaGetLastError();
}

template <int DK, int DV, int NS>
cudaError_t launch_range(const SsmParams& sp, TcParams p, int seq0, int n, const int32_t* starts,
                         const SsmPlan& plan, void* ws, cudaStream_t s) {
  OrderedSeqs<NS> tab;
  const long long tiles = fill_ordered(tab, starts, seq0, n, plan.tile_tokens);
  const long long items = tiles * p.pairs;
  if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidConfiguration;
  const long long grid = items < sms ? items : sms;  // one CTA an SM
  p.items = unsigned(items);
  p.ws = static_cast<float*>(ws);
  p.wdecay = p.ws + size_t(tiles) * p.H * DV * DK;
  CUtensorMap q, k, v, o;
  const long long rows = starts[seq0 + n];
  if (!encode_rows(&q, sp.q, rows, p.G * DK, sp.ldq, kQ) || !encode_rows(&k, sp.k, rows, p.G * DK, sp.ldk, kQ) ||
      !encode_rows(&v, sp.v, rows, p.H * DV, sp.ldv, kQ) || !encode_rows(&o, sp.o, rows, p.H * DV, sp.ldo, 32))
    return cudaErrorInvalidValue;
  if (tiles > n) {
    cudaError_t e = launch_chunk<DK, DV, true, NS>(p, tab, seq0, unsigned(grid), q, k, v, o, s);
    if (e != cudaSuccess) return e;
    e = launch_ssm_join(sp, p.ws, p.wdecay, tab, seq0, n, DK, DV, s);
    if (e != cudaSuccess) return e;
  }
  return launch_chunk<DK, DV, false, NS>(p, tab, seq0, unsigned(grid), q, k, v, o, s);
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
// its k and v (kStatesCost of a full one: 2.4 of 4.7 us a chunk), so take the length whose
// waves of CTAs finish first.  One sequence, in us by parts (* taken), each point
// the median of replayed graphs:
//     T = 8192, H = 64, d = 128 x 64   243 whole, 138 in 3, 110 in 4*, 143 in 5, 114 in 10
//     T = 8192, H = 64, d = 64 x 64    231 whole, 131 in 3, 102 in 4*, 129 in 5, 102 in 10
//     T = 2048, H = 16, d = 64 x 64    62 whole, 34 in 4, 25 in 8 and more*
// At d_k = 64 D is half as wide and the same lengths win.  T = 6001 in 24 sequences
// stays whole (81, 117 in halves).  Three uneven sequences of 8192 tokens are where
// the estimate errs: 142 in 4 parts*, 122 in 5.
SsmPlan plan_ssm(int H, int G, int dk, int dv, int n, const int32_t* starts, int sms) {
  constexpr double kStatesCost = 0.5, kTileCost = 1.0;  // in chunks
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
  best.bytes = ssm_tile_bytes(H, dk, dv, n, starts, best.tile_tokens);
  return best;
}

size_t ssm_tile_bytes(int H, int dk, int dv, int n, const int32_t* starts, int tile_tokens) {
  long long most = 0;
  bool any = false;
  const int step = n <= kSmallSeqs ? (n > 0 ? n : 1) : kLargeSeqs;
  for (int s0 = 0; s0 < n; s0 += step) {
    long long tiles = 0;
    const int m = n - s0 < step ? n - s0 : step;
    for (int i = s0; i < s0 + m; ++i) {
      const long long len = (long long)starts[i + 1] - starts[i];
      tiles += len > tile_tokens ? (len + tile_tokens - 1) / tile_tokens : 1;
    }
    any = any || tiles > m;
    most = tiles > most ? tiles : most;
  }
  return any ? size_t(most) * H * (size_t(dv) * dk + 1) * 4 : 0;
}

template <typename Table>
cudaError_t launch_ssm_join(const SsmParams& p, float* ws, const float* wdecay, const Table& tab, int seq0,
                            int n, int dk, int dv, cudaStream_t s) {
  const long long blocks = (long long)n * p.H * (dv * dk / 1024);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  dl_ssm_join_kernel<Table><<<unsigned(blocks), 256, 0, s>>>(p.S0, ws, wdecay, tab, seq0, p.H, dk, dv);
  count_launches(1);
  return cudaGetLastError();
}
template cudaError_t launch_ssm_join(const SsmParams&, float*, const float*, const SeqTable<kSmallSeqs>&, int, int,
                                     int, int, cudaStream_t);
template cudaError_t launch_ssm_join(const SsmParams&, float*, const float*, const SeqTable<kLargeSeqs>&, int, int,
                                     int, int, cudaStream_t);

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
  p.hpg = sp.H / sp.G;
  p.ppg = p.pairs / sp.G;
  p.tile_tokens = plan.tile_tokens;
  if (dk == 128) return dv == 64 ? launch_tc<128, 64>(sp, p, n, starts, plan, ws, s)
                                 : launch_tc<128, 128>(sp, p, n, starts, plan, ws, s);
  return dv == 64 ? launch_tc<64, 64>(sp, p, n, starts, plan, ws, s)
                  : launch_tc<64, 128>(sp, p, n, starts, plan, ws, s);
}

}  // namespace dl
