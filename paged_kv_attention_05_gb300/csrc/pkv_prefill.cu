// Prefill / chunked-prefill attention (requests with more than one query
// token) on the 5th-generation tensor cores: tcgen05.mma with accumulators in
// tensor memory, K/V pages gathered by TMA through the block table.
//
// What it computes: "Tour: One forward pass", stop 10 — causal attention for
// the request's query rows over all of its keys (R3: 298 query rows, 298
// keys), the keys found through the block table; stop 3 — query row i sits
// at position num_computed + i, so a chunk that continues a cached prompt sees
// the cached keys plus its own causal triangle.  "vLLM 推理全流程深度解析",
// prefill section: lower-triangular causal mask; the FlashAttention idea of
// keeping the score tile on chip.  "vLLM MHA Code Path: From QKV to Paged KV
// Cache", "One Path Covers MHA, GQA, and MQA": query head h reads KV head
// h / (Hq / Hkv).
//
// GB300 design.  A work item is a 128-row query tile of one request for two
// query heads of the same KV head (one head when Hq / Hkv is odd): tiles "a"
// and "b" share every K/V tile.  A persistent grid (one CTA per SM, all 512
// TMEM columns) takes items from an atomic cursor, longest first.  Roles:
//   warp 0      producer: publishes the item in a two-slot ring, loads the two
//               Q tiles by TMA as soon as the previous item's last S = Q K^T
//               has consumed them, then the K and V tiles of 128 keys (8 pages
//               each, one 16-slot x 64-dim box per page and half, 128-byte
//               swizzle) into a 2-stage ring, K and V released separately; in
//               a request's last tile it zero-fills the V rows of keys past
//               seq_len so that no stale value (NaN) reaches P.V;
//   warp 1      allocates TMEM and issues every MMA from one thread, in the
//               order S_a(0) S_b(0) | PV_a(j) S_a(j+1) PV_b(j) S_b(j+1) ...:
//               S into TMEM, P taken from TMEM (the scores' columns,
//               overwritten with bf16 probabilities) and V from shared memory
//               (MN-major), O accumulating in TMEM; tcgen05.commit drives the
//               mbarriers.  Because one thread's MMAs complete in order, S(j+1)
//               being ready also means PV(j) is done;
//   warps 2-9   softmax, two warps per row quarter (one per 64-key half of
//               the scores), one query row per thread (TMEM lane = 32 *
//               (warp % 4) + lane = row), both query tiles in turn: scores ->
//               causal/length mask (only on tiles that cross the diagonal) ->
//               running max in the log2 domain -> exp2 -> row sum -> bf16 P
//               back into TMEM.  O is rescaled in TMEM only when a row's max
//               grows by more than 2^8 (exact, rare).  At the end of an item
//               each warp leaves its partial row sums in shared memory;
//   warps 10-13 epilogue: once O_x is final, read it out of TMEM in two
//               64-column halves, divide by the row sum, release O_x to the
//               next item's first P.V and write the bf16 rows to global memory
//               through a per-warp staging area (whole 64-byte row pieces).
// pkv_attention_scored runs instances with softmax warps of their own kind (8
// or 16, a set for each query tile; described there), whose key tiles start at
// the window's first page; the other roles are the same.
// pkv_attention_int4 runs an instance of 20 warps: the producer brings pages of
// codes and scales by bulk copies, four warps turn them into the fp16 K and V tiles,
// one finds the tiles' exponents (and these five with one more convert the query rows);
// the softmax is described there.  4 chunks of 2047 tokens of 64 heads on 8, after 4099
// (us; floor 423, pkv_attention on the same batch 630): 1267 with two warps that form
// bf16 tiles, 1083 with four and fp16 tiles, 940 with registers moved to the softmax and
// the tiles' loop rolled, 857 with a row per softmax thread, 843 with key codes in
// buffers of their own, 788 with codes taken as fp16 subnormals, 755 with the query rows
// converted by all six, 760 with V tiles scaled each by its own largest value (by that of
// all tiles so far, values far below it were lost).  What it has over pkv_attention's 630 is the forming of the
// tiles: beside it tensor pipe 49%, issue slots 53%, alu 43%.
// Every mbarrier wait is bounded; on expiry the kernel records
// PKV_DEV_ERR_TIMEOUT, stops issuing work, frees its TMEM and returns.
#include <cuda_fp16.h>

#include <type_traits>

#include "pkv_combine.cuh"
#include "pkv_device.cuh"
#include "pkv_int4.cuh"
#include "pkv_score.cuh"

namespace pkv {
namespace {

using namespace dev;

// Warps: producer, MMA issuer, softmax, four of epilogue.  8 softmax warps in
// the plain call (two a row quarter, both query tiles in turn) and in scored
// calls with a running maximum (one a row quarter and tile), 16 with a fixed
// reference (two a row quarter and tile).
__host__ __device__ constexpr int soft_warps(bool fixed_ref) { return fixed_ref ? 16 : 8; }
__host__ __device__ constexpr int threads_of(bool fixed_ref) {
  return 32 * (2 + soft_warps(fixed_ref) + 4);  // 448, 704
}
constexpr int kStages = 2;
constexpr int kTileK = 128;                       // keys per KV tile
constexpr int kHalfBytes = 128 * 128;             // 128 rows x 64 bf16
constexpr int kTileBytes = 2 * kHalfBytes;        // a Q, K or V tile: 32 KB
constexpr int kPageBoxBytes = 16 * 128;           // one 16-slot x 64-dim box
constexpr int kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;         // log2 units
constexpr float kMaxSum = 0x1p40f;                // scored calls: sum of a row over a pair of blocks
constexpr float kMaxSum16 = 0x1.fp15f;            // 4-bit calls: sum of a row over 64 columns
constexpr float kLift16 = 8.f;                    // and log2 of the largest weight at first

// shared-memory layout (offsets from a 1024-byte aligned base)
constexpr int kOffQ = 0;                          // Q_a | Q_b
constexpr int kOffK = kOffQ + 2 * kTileBytes;
constexpr int kOffV = kOffK + kStages * kTileBytes;
constexpr int kStageWarp = 32 * 64;               // epilogue staging: 32 rows x 64 bytes
constexpr int kOffStage = kOffV + kStages * kTileBytes;  // one staging area per epilogue warp
constexpr int kOffLsum = kOffStage + 4 * kStageWarp;  // [2 items][2 tiles][2 halves][128 rows]
constexpr int kOffBar = kOffLsum + 2 * 2 * 2 * 128 * 4;
enum {
  B_QF = 0,   // [2] Q tile loaded
  B_QE = 2,   // [2] Q tile consumed by the item's last S
  B_KF = 4,   // [2] K stage loaded
  B_KE = 6,   // [2] K stage free
  B_VF = 8,   // [2] V stage ready
  B_VT = 10,  // [2] V stage loaded (tail tiles: before the zero fill)
  B_VE = 12,  // [2] V stage free
  B_SF = 14,  // [2] S_x ready
  B_PF = 16,  // [2] P_x written
  B_OF = 18,  // [2] O_x final for the item
  B_OE = 20,  // [2] O_x read by the epilogue
  B_IF = 22,  // [2] item slot published
  B_IE = 24,  // [2] item slot released
  B_XP = 26,  // [4] exchange between the two softmax warps of a row quarter
  B_LF = 30,  // [2] row sums of tile x written for the epilogue, even items
  kNumBars = 32
};
constexpr int kOffItems = kOffBar + kNumBars * 8;  // 2 item slots
constexpr int kOffXch = kOffItems + 2 * 48;        // [4 quarters][2 slots][2 halves][32] floats
constexpr int kOffCtl = kOffXch + 4 * 2 * 2 * 32 * 4;  // TMEM address, abort flag
constexpr int kOffBarLF1 = kOffCtl + 16;           // [2] the same for odd items
constexpr int kSmemBytes = kOffBarLF1 + 16 + 1024;  // + alignment slack
// The instance for the cache of 4-bit codes: 20 warps (producer, MMA, two for the query
// rows; 8 of softmax; 4 of epilogue; two for K tiles, two for V tiles), the scales and
// zeros of the tiles, and the powers of two that its fp16 tiles are scaled by.  The
// softmax takes registers from the other warps: with the 96 that 640 threads have each
// it spills (999 against 870 us for 4 chunks of 2047 tokens, the tiles left zero); with the
// shares below 28 bytes still are.
constexpr int kThreadsI4 = 640;
constexpr int kRegsLaunch = 96, kRegsSoft = 120, kRegsEpi = 96, kRegsFew = 72;
static_assert(256 * kRegsSoft + 128 * kRegsEpi + 256 * kRegsFew <= kThreadsI4 * kRegsLaunch,
              "the shares must fit what the block is launched with");
constexpr int kDequantWarps = 2;  // of K; of V; of Q
constexpr int kOffBarI4 = kOffBarLF1 + 16;
enum {
  I_KR = 0,   // [2] key codes of a tile loaded
  I_KT = 2,   // [2] and turned into its K tile
  I_QD = 4,   // [2] Q tile converted
  I_MR = 6,   // [4] scales and zeros of a tile loaded
  I_XR = 10,  // [4] and its exponents found
  kNumBarsI4 = 14
};
constexpr int kOffTileExp = kOffBarI4 + 8 * kNumBarsI4;  // [4 tiles] exponents of K and V (int2)
constexpr int kMetaBytes = kPage4 - kMeta4;
constexpr int kOffMeta = (kOffTileExp + 4 * 8 + 127) / 128 * 128;  // scales: see meta_offset
constexpr int kOffKRaw = kOffMeta + 2 * 8 * kMetaBytes;            // [2] key codes of a tile
constexpr int kSmemBytesI4 = kOffKRaw + 2 * 8 * kSide4 + 1024;
// The scales and zeros of tile c: of four tiles at a time, two where the plain softmax
// exchanges values.  The query rows' factors lie beside their row sums, in the places of
// the second warp of a row, which this softmax does not have.
static_assert(kOffXch % 16 == 0 && kOffCtl - kOffXch >= 2 * 8 * kMetaBytes, "room for two tiles");
__host__ __device__ constexpr int meta_offset(uint32_t c) {
  return (c & 2 ? kOffMeta : kOffXch) + (int)(c & 1) * 8 * kMetaBytes;
}
__host__ __device__ constexpr int qfac_offset(uint32_t it_cnt, int x) {
  return kOffLsum + (((int)(it_cnt & 1) * 2 + x) * 2 + 1) * 128 * 4;
}
// Where page p's value codes of a tile land in its stage: in the first half of the rows of
// the warp that turns them into the tile (half 0 of a row, 128 bytes each).
constexpr int kPagesPerWarp = 8 / kDequantWarps;
__host__ __device__ constexpr int raw_offset(int p) {
  return p / kPagesPerWarp * (128 / kDequantWarps * 128) + p % kPagesPerWarp * kSide4;
}
static_assert(kSmemBytesI4 <= 232448, "shared memory per CTA");

struct Item {
  int r, qt, ha, hb;  // hb < 0: single-tile item
  int g, q0, n, L;
  int ctx, nkv, base, prefix;  // first key of the tiles; keys every row sees (scored)
};

// What an instance does to the scores.  kFixedCap: fixed_reference() holds.
enum Cap { kNoCap, kAnyCap, kFixedCap };

// First key of the j-th tile an item processes.  With a distance bias the
// tiles run from the diagonal back: the bias falls with distance, so a row's
// maximum is found in its first tile and stays (forward, steep slopes would
// raise it, and rescale the output, at every tile).  Where a window cuts the
// first tile, it comes last: in the one after it every row sees all or most
// keys, so that the running maximum settles there.
template <bool kScored, bool kBias>
__device__ __forceinline__ int tile_key0(const Item& it, int j) {
  int t = j;
  if (kBias)
    t = it.nkv - 1 - j;
  else if (kScored && it.base > 0)
    t = j + 1 < it.nkv ? j + 1 : 0;
  return it.base + t * kTileK;
}

// a prefill entry written by the plan kernel, read through L2
__device__ __forceinline__ PreEntry load_entry(const PreEntry* p) {
  const int4 w0 = __ldcg(reinterpret_cast<const int4*>(p));
  const int4 w1 = __ldcg(reinterpret_cast<const int4*>(p) + 1);
  return PreEntry{w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}

// Shared-memory matrix descriptor: 128-byte swizzle, SBO = 1024 bytes
// (8-row groups), LBO as given (MN-major: distance between 64-element atoms).
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((1024 >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for tcgen05
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}

// Instruction descriptor, kind::f16: bf16 (or fp16) A and B, fp32 D, M = N = 128.
__host__ __device__ constexpr uint32_t idesc_16(bool b_mn_major, bool bf16) {
  return (1u << 4)                         // D format f32
         | ((bf16 ? 1u : 0u) << 7)         // A format
         | ((bf16 ? 1u : 0u) << 10)        // B format
         | ((b_mn_major ? 1u : 0u) << 16)  // B major-ness
         | ((128u >> 3) << 17)             // N
         | ((128u >> 4) << 24);            // M
}

// The MMA role runs on a whole converged warp, so that operands are
// warp-uniform values; one elected lane (the lowest, the same every time, so
// that its commits track all its MMAs) issues each instruction.
// D (TMEM) (+)= A (shared) * B (shared)
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D (TMEM) (+)= A (TMEM) * B (shared)
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          bar)
      : "memory");
}

#define PKV_LD32(taddr, v)                                                                     \
  asm volatile(                                                                                \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13," \
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"   \
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),   \
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]),            \
        "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),         \
        "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),         \
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]),         \
        "=f"(v[31])                                                                            \
      : "r"(taddr))

#define PKV_ST32(taddr, v)                                                                     \
  asm volatile(                                                                                \
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12," \
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n"  \
      ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]),        \
      "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]),         \
      "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]),     \
      "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]),     \
      "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])                              \
      : "memory")

#define PKV_ST32U(taddr, v)                                                                    \
  asm volatile(                                                                                \
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12," \
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n"  \
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),        \
      "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]),         \
      "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),     \
      "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]),     \
      "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])                              \
      : "memory")

#define PKV_ST16U(taddr, v)                                                                    \
  asm volatile(                                                                                \
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12," \
      "%13,%14,%15,%16};\n" ::"r"(taddr),                                                     \
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),  \
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),        \
      "r"(v[15])                                                                               \
      : "memory")

#define PKV_LD16(taddr, v)                                                                     \
  asm volatile(                                                                                \
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13," \
      "%14,%15}, [%16];\n"                                                                     \
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),   \
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]),            \
        "=f"(v[13]), "=f"(v[14]), "=f"(v[15])                                                  \
      : "r"(taddr))

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// Adds the bias -slope2 * (distance - from) to 32 columns (d0: distance of the
// first one's key; from: see bias_from) or, without a cap, forms s * lin + nm +
// bias.  Capped: the distances in four pairs stepped by eight columns, exact whole
// numbers.  Without a cap: the biases stepped instead (one operation less; three
// additions at most, whose roundings stay below 2^-22 of the bias).  kSym: a
// column past d0 counts its distance too.
template <bool kCapped, bool kSym>
__device__ __forceinline__ void bias32(float (&s)[32], const ScoreArgs& sp, float nm,
                                       float slope2, float d0, float from) {
  if (kSym) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      if (!kCapped)
        split(fma2(pair(s[i], s[i + 1]), sp.lin2, pair(nm, nm)), s[i], s[i + 1]);
#pragma unroll
      for (int k = i; k < i + 2; ++k) s[k] = fmaf(-slope2, fabsf((float)k - d0) - from, s[k]);
    }
    return;
  }
  f32x2 b[4];
  if (kCapped) {
    const f32x2 m = pair(slope2, slope2), e8 = pair(8.f, 8.f);
    const float e0 = from - d0;
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = pair(e0 + 2.f * k, e0 + (2.f * k + 1.f));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      split(fma2(b[i & 3], m, pair(s[2 * i], s[2 * i + 1])), s[2 * i], s[2 * i + 1]);
      if (i < 12) b[i & 3] = add2(b[i & 3], e8);
    }
    return;
  }
  const float b0 = fmaf(-slope2, d0, nm);
  const f32x2 b8 = pair(8.f * slope2, 8.f * slope2);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    b[k] = pair(fmaf(slope2, 2.f * k, b0), fmaf(slope2, 2.f * k + 1.f, b0));
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    split(fma2(pair(s[2 * i], s[2 * i + 1]), sp.lin2, b[i & 3]), s[2 * i], s[2 * i + 1]);
    if (i < 12) b[i & 3] = add2(b[i & 3], b8);
  }
}
// 32 raw products s = q.K (columns of one row) to logits in log2 units + nm,
// the cap by the given form.
template <Cap kCap, bool kBias, bool kSym, Form kForm>
__device__ __forceinline__ void logits32(float (&s)[32], const ScoreArgs& sp, float nm,
                                         float slope2, float d0, float from, float& big) {
  if (kCap != kNoCap) cap_values<kForm>(s, sp, nm, big);
  if (kBias) {
    bias32<kCap != kNoCap, kSym>(s, sp, nm, slope2, d0, from);
  } else if (kCap == kNoCap) {
    const f32x2 nm2 = pair(nm, nm);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      split(fma2(pair(s[2 * i], s[2 * i + 1]), sp.lin2, nm2), s[2 * i], s[2 * i + 1]);
  }
}
// The same, the form of the cap by the warp's visible scores.  kEdge: -inf
// outside low <= i <= lim (columns there may hold anything).
template <Cap kCap, bool kBias, bool kSym, bool kEdge>
__device__ __forceinline__ void logits32_any(float (&s)[32], const ScoreArgs& sp, float nm,
                                             int lim, int low, bool valid_row, float slope2,
                                             float d0, float from) {
  float big = 0.f;
  if (kCap == kNoCap) {
    logits32<kCap, kBias, kSym, kDeg2>(s, sp, nm, slope2, d0, from, big);
  } else {
    if (kEdge) {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = i <= lim && i >= low ? s[i] : 0.f;
    }
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      m0 = max3f(m0, fabsf(s[i]), fabsf(s[i + 1]));
      m1 = max3f(m1, fabsf(s[i + 2]), fabsf(s[i + 3]));
    }
    const float m = valid_row ? fmaxf(m0, m1) : 0.f;
    if (__all_sync(0xffffffffu, m * m <= sp.limit2)) {
      logits32<kCap, kBias, kSym, kDeg2>(s, sp, nm, slope2, d0, from, big);
    } else if (__all_sync(0xffffffffu, m * m <= sp.limit3)) {
      logits32<kCap, kBias, kSym, kDeg3>(s, sp, nm, slope2, d0, from, big);
    } else if (kCap == kAnyCap && __all_sync(0xffffffffu, m * sp.k <= 1.f)) {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = capped_poly(s[i], sp) + nm;
      if (kBias) bias32<true, kSym>(s, sp, nm, slope2, d0, from);
    } else {
      logits32<kCap, kBias, kSym, kExp>(s, sp, nm, slope2, d0, from, big);
    }
  }
  if (kEdge) {
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = i <= lim && i >= low ? s[i] : -INFINITY;
  }
}
// p = exp2(s), packed to bf16 pairs (P.V takes both its operands in V's type; a
// weight is off by 2^-8 of itself at most, as in the plain call); returns the sum
// of the rounded values: the weights that meet V then add up to the row sum they
// are divided by, so that a row that one key dominates is off by no rounding of
// its weight (2.0e-3 instead of 2.3e-3 relative error of the capped prefill's
// output, 1.7e-3 of it the output's own rounding).
__device__ __forceinline__ float exp32(const float (&s)[32], uint32_t (&p)[16]) {
  float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    p[i] = pack_bf16(fast_exp2(s[2 * i]), fast_exp2(s[2 * i + 1]));
    add_bf16x2(r[2 * (i & 1)], r[2 * (i & 1) + 1], p[i]);
  }
  return (r[0] + r[1]) + (r[2] + r[3]);
}
// 16 TMEM columns of fp32 (bf16 pairs) times alpha
__device__ __forceinline__ void rescale16(uint32_t t, float alpha) {
  float v[16];
  uint32_t u[16];
  PKV_LD16(t, v);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[i] * alpha);
  PKV_ST16U(t, u);
}
__device__ __forceinline__ void rescale16_f16(uint32_t t, float alpha) {
  float v[16];
  uint32_t u[16];
  PKV_LD16(t, v);
  tmem_wait_ld();
  const __half2 a2 = __float2half2_rn(alpha);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w = __float_as_uint(v[i]);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&w), a2);
    u[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  PKV_ST16U(t, u);
}
__device__ __forceinline__ void rescale16_bf16(uint32_t t, float alpha) {
  float v[16];
  uint32_t u[16];
  PKV_LD16(t, v);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w = __float_as_uint(v[i]);
    u[i] = pack_bf16(__uint_as_float(w << 16) * alpha, __uint_as_float(w & 0xFFFF0000u) * alpha);
  }
  PKV_ST16U(t, u);
}

// The instance for 4-bit caches runs on fp16 tiles: a cached value has up to 12
// significant bits (s with 8 times a code with 4, plus z), of which bf16 keeps 8 and
// fp16 11, and the same goes for the weights (outputs off by 3.0e-3 of their size with
// bf16 tiles, 1.7e-3 with these, of which the bf16 output is 1.6e-3).  What fp16 lacks
// in range, powers of two make up: each query row and each K and V tile have one, by which
// their largest value lies in [2^13, 2^14) (query rows) or
// [2^-7, 2^-6) (tiles, see dequant8): values down to 2^-7 of the largest keep all
// their bits, and what is below is off by 2^-18 of it at most.
__device__ __forceinline__ int q_exponent(uint32_t x) {
  return max((int)(x >> 23) - 127 - 13, -100);
}
__device__ __forceinline__ int tile_exponent(uint32_t x) {  // (of values up to 2^105)
  return min(max((int)(x >> 23) - 127 + 7, -100), 112);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The share of the block's registers that this warpgroup goes on with.
template <int kRegs, bool kMore>
__device__ __forceinline__ void take_regs() {
  if (kMore)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
// A word's eight codes to the fp16 values s * code + z, each rounded once.  A code in the
// last bits of a half is the subnormal code * 2^-24, four bits up code * 2^-20: nothing
// but a mask makes it the operand of the multiply-add (s: the row's scale times 2^24,
// below 2^16 as the tile's values are below 2^-6; t: times 2^20).
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t s, uint32_t t, uint32_t z) {
  uint32_t v[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const uint32_t c = (n < 2 ? w : w >> 8) & (n & 1 ? 0x00F000F0u : 0x000F000Fu);
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&c),
                              *reinterpret_cast<const __half2*>(n & 1 ? &t : &s),
                              *reinterpret_cast<const __half2*>(&z));
    v[n] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Rows 8 set .. + 7 of a Q tile to fp16 in place, their powers of two to fac.  Four lanes a
// row; a lane takes every fourth of its 16-byte pieces (in odd rows the two halves of a
// 128-byte line swapped: eight lanes meet eight bank groups).  `scale` gives the sign:
// the softmax takes its size.
__device__ __forceinline__ void convert_q(uint8_t* q, float* fac, int set, float scale) {
  const int lane = threadIdx.x & 31, row = 8 * set + (lane >> 2), tig = lane & 3;
  auto piece = [&](int i) {
    return reinterpret_cast<uint4*>(q + (i >> 1) * kHalfBytes + sw128(row, tig + 4 * ((i + row) & 1)));
  };
  __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const uint4 v = *piece(i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[k])));
  }
  float big = fmaxf(__low2float(m), __high2float(m));
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
  const int e = q_exponent(__float_as_uint(big));
  const float down = copysignf(pow2(-e), scale);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const uint4 v = *piece(i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = pack_f16(__uint_as_float(w[k] << 16) * down,
                      __uint_as_float(w[k] & 0xFFFF0000u) * down);
    *piece(i) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (tig == 0) fac[row] = pow2(e);
}

// kScored: a window, a prefix (runtime), and per instance a cap, a bias (kSym:
// that may meet keys after a row's position, with a prefix).  kI4: the cache of 4-bit
// codes (pkv_attention_int4): the producer brings a tile's pages as they are cached,
// and warps of their own turn them, and the query rows, into fp16 tiles.
template <bool kScored, Cap kCap, bool kBias, bool kSym, bool kI4 = false>
__global__ void __launch_bounds__(kI4 ? kThreadsI4 : threads_of(kCap == kFixedCap), 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, ArgsOf<kScored> a,
                   Workspace ws) {
  // This grid is the programmatic dependent of the decode grid, which
  // triggers it after its own wait for the plan kernel: the plan is complete
  // when any CTA here runs, so the items start without waiting for the decode
  // grid (which leaves some SMs to them, see pkv_decode.cu); what the plan and
  // the kernels before it wrote is read through L2 (ld.global.cg).  The split
  // decode results are merged at the end, once the decode grid has finished
  // (so this grid finishing implies that every kernel before it has).
  constexpr int kSoft = soft_warps(kCap == kFixedCap), kDeq = kI4 ? 3 * kDequantWarps : 0;
  constexpr int kThreads = kI4 ? kThreadsI4 : threads_of(kCap == kFixedCap);
  constexpr int kSoft0 = kI4 ? 4 : 2;  // the first softmax warp
  constexpr int kHalves = kScored ? kSoft / 8 : kI4 ? 1 : 2;  // softmax warps that share a row
  // (a scored call lets the next kernel, usually another call's plan or cache
  // write, set up meanwhile: everything before this kernel has finished or, as
  // the decode grid, writes only what those wait for)
  if (kScored) grid_dep_launch();
  const int n_pre = __ldcg(&ws.hdr->n_pre_entries);
  if (n_pre == 0) {  // a step without prefill work (every CTA agrees)
    // (a scored call reads its part of the plan before the wait)
    const int id = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    CombineStart start{};
    if (kScored) start = combine_start(ws, id);
    grid_dep_wait();
    if (!kScored) start = combine_start(ws, id);
    combine_splits(a, ws, id, gridDim.x * (kThreads / 32), start);
    return;
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  // row sums of tile x of item it_cnt written
  auto lf_bar = [&](uint32_t it_cnt, int x) {
    return (it_cnt & 1) ? sbase + kOffBarLF1 + 8u * (uint32_t)x : bar(B_LF + x);
  };
  auto i4_bar = [&](int i) { return sbase + kOffBarI4 + 8u * (uint32_t)i; };
  volatile int* ctl = reinterpret_cast<volatile int*>(smem + kOffCtl);
  volatile int* abort = ctl + 1;  // ctl[0] = TMEM base address
  auto wait = [&](uint32_t b, uint32_t parity) {
    return mbar_wait_warp(b, parity, abort, ws.err);
  };
  Item* items = reinterpret_cast<Item*>(smem + kOffItems);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.hq / a.hkv;
  // two heads of one KV head per item
  const bool pairs = (G % 2) == 0 && !((kScored || kI4) && single_head_items(a, n_pre, gridDim.x));
  const int per_entry = pairs ? a.hq / 2 : a.hq;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bar(i), 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(B_PF + x), 4 * kHalves);  // one arrival per softmax warp of the tile
      mbar_init(bar(B_OE + x), 4);  // one arrival per epilogue warp
      mbar_init(bar(B_LF + x), 4 * kHalves);  // one arrival per softmax warp of the tile
      mbar_init(sbase + kOffBarLF1 + 8 * x, 4 * kHalves);
      mbar_init(bar(B_IE + x), 1 + kSoft + 4 + kDeq);  // MMA warp, softmax, epilogue (and these)
      if (kI4) {  // one arrival per dequantising warp
        mbar_init(bar(B_KF + x), kDequantWarps);
        mbar_init(bar(B_VF + x), kDequantWarps);
        mbar_init(i4_bar(I_KR + x), 1);
        mbar_init(i4_bar(I_KT + x), kDequantWarps);
        mbar_init(i4_bar(I_QD + x), kDeq);
        for (int i = x; i < 4; i += 2) {
          mbar_init(i4_bar(I_MR + i), 1);
          mbar_init(i4_bar(I_XR + i), 1);
        }
      }
    }
    for (int i = 0; i < 4; ++i) mbar_init(bar(B_XP + i), 2);
    ctl[1] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     sbase + kOffCtl),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)ctl[0];
  const int n_items = n_pre * per_entry;
  // The Q tiles of item it_cnt to fp16, by the six warps that form tiles (w: 0 .. 5): the
  // query rows come when the item before has issued its last S, and the next S waits for
  // them; each warp has formed its share of the first K or V tile by then (the V tile after
  // the rows: 804 us for 4 chunks of 2047 tokens of 64 heads, so 762).
  auto query_rows = [&](const Item& it, uint32_t it_cnt, uint32_t (&q_cnt)[2], int w) {
    for (int x = 0; x < (it.hb >= 0 ? 2 : 1); ++x) {
      if (!wait(bar(B_QF + x), q_cnt[x]++ & 1)) return false;
      for (int set = w; set < 16; set += 6)
        convert_q(smem + kOffQ + x * kTileBytes,
                  reinterpret_cast<float*>(smem + qfac_offset(it_cnt, x)), set, a.scale);
      fence_async_smem();  // (read by the MMAs)
      __syncwarp();
      if (lane == 0) mbar_arrive(i4_bar(I_QD + x));
    }
    return true;
  };

  if (warp == 0) {
    if (kI4) take_regs<kRegsFew, false>();
    // ------------------------------ producer ------------------------------
    // Global loads are issued one step before their values are needed: the
    // next item's cursor and entry (which carries its request's lengths)
    // while the current item is being issued, and each tile's block ids one
    // tile ahead; a load only stalls at its first use.
    uint32_t tile_cnt = 0, vt_uses[kStages] = {0, 0}, qx_cnt[2] = {0, 0};
    // (a scored call without decode units has every CTA at once: the first
    // item of each is its index, and the cursor counts on from there)
    const bool own_first = kScored && __ldcg(&ws.hdr->n_dec_units) == 0;
    const int after = own_first ? (int)gridDim.x : 0;
    int w_nxt = (int)blockIdx.x;
    if (!own_first) {
      if (lane == 0) w_nxt = atomicAdd(&ws.hdr->pre_counter, 1);
      w_nxt = __shfl_sync(0xffffffffu, w_nxt, 0);
    }
    const PreEntry none{-1, 0, 0, 0, 0, 0, 0, 0};
    PreEntry e_nxt = w_nxt < n_items ? load_entry(ws.pre + w_nxt / per_entry) : none;
    for (uint32_t it_cnt = 0;; ++it_cnt) {
      const int slot = it_cnt & 1;
      const int w = w_nxt;
      const PreEntry e = e_nxt;
      const int q0 = e.q0, q1 = e.q0 + e.n, Lr = e.L;
      if (it_cnt >= 2 &&
          !wait(bar(B_IE + slot), ((it_cnt >> 1) - 1) & 1))
        break;
      if (w >= n_items || *abort) {
        if (lane == 0) {
          items[slot].r = -1;
          mbar_arrive(bar(B_IF + slot));
        }
        break;
      }
      Item it;
      {
        const int hp = w % per_entry;
        it.r = e.r;
        it.qt = e.qt;
        it.nkv = e.nkv;
        it.ha = pairs ? 2 * hp : hp;
        it.hb = pairs ? 2 * hp + 1 : -1;
        it.g = it.ha / G;
        it.q0 = q0;
        it.n = q1 - q0;
        it.L = Lr;
        it.ctx = Lr - it.n;
        it.base = kScored ? e.base : 0;
        it.prefix = kScored ? e.prefix : 0;
      }
      if (lane == 0) {
        items[slot] = it;
        mbar_arrive(bar(B_IF + slot));
      }
      // the next item's cursor and entry (consumed after this item)
      if (lane == 0) w_nxt = after + atomicAdd(&ws.hdr->pre_counter, 1);
      w_nxt = __shfl_sync(0xffffffffu, w_nxt, 0);
      e_nxt = w_nxt < n_items ? load_entry(ws.pre + w_nxt / per_entry) : none;
      const int* btrow = a.bt + (int64_t)it.r * a.bt_width;
      const int row0 = it.q0 + it.qt * kPreTileQ;
      // Q tiles, once the previous item's last S has read them
      bool ok = true;
      auto load_q = [&]() {
        for (int x = 0; x < 2 && ok; ++x) {
          const int h = x == 0 ? it.ha : it.hb;
          if (h < 0) continue;
          if (qx_cnt[x] > 0 &&
              !wait(bar(B_QE + x), (qx_cnt[x] - 1) & 1)) {
            ok = false;
            break;
          }
          qx_cnt[x]++;
          if (lane == 0) {
            const uint32_t qd = sbase + kOffQ + x * kTileBytes;
            mbar_expect_tx(bar(B_QF + x), kTileBytes);
            tma_load_3d(qd, &tm_q, bar(B_QF + x), 0, h, row0);
            tma_load_3d(qd + kHalfBytes, &tm_q, bar(B_QF + x), 64, h, row0);
          }
        }
      };
      if (!kI4) load_q();
      // lane p < pages(j) holds the block id of page p of tile j
      auto tile_key = [&](int j) { return tile_key0<kScored, kBias>(it, j); };
      auto tile_pages = [&](int key) { return min(8, (it.L - key + 15) / 16); };
      // first key any row of the item sees (its tiles start at this key's page)
      const int vlow = kScored ? first_key(it.ctx + it.qt * kPreTileQ, score_of(a).window) : 0;
      int blk_nxt = lane < tile_pages(tile_key(0)) ? __ldcg(btrow + (tile_key(0) >> 4) + lane) : 0;
      if constexpr (kI4) {
        // A tile's key codes into one of two buffers of their own, with its scales and
        // zeros, two tiles ahead of its value codes, which go into the V stage: the K
        // tile, formed when its stage is free, waits for no load.
        auto page_of = [&](int blk) {
          return reinterpret_cast<const uint8_t*>(a.kc) + ((int64_t)blk * a.hkv + it.g) * kPage4;
        };
        auto load_keys = [&](int j, uint32_t c) {  // the blocks of tile j, checked
          const int pages = tile_pages(tile_key(j));
          int blk = blk_nxt;
          if (j + 1 < it.nkv && lane < tile_pages(tile_key(j + 1)))
            blk_nxt = __ldcg(btrow + (tile_key(j + 1) >> 4) + lane);
          if (lane < pages && (blk < 0 || (int64_t)blk >= a.num_blocks)) {
            atomicOr(ws.err, PKV_DEV_ERR_BLOCK_ID);
            blk = 0;
          }
          if (c >= 2 && !wait(i4_bar(I_KT + (c & 1)), ((c >> 1) - 1) & 1)) {
            ok = false;
            return blk;
          }
          const uint32_t mbar = i4_bar(I_MR + (c & 3)), kbar = i4_bar(I_KR + (c & 1));
          if (lane == 0) {
            mbar_expect_tx(mbar, pages * kMetaBytes);
            mbar_expect_tx(kbar, pages * kSide4);
          }
          __syncwarp();
          if (lane < pages) {
            bulk_load(sbase + meta_offset(c) + lane * kMetaBytes, page_of(blk) + kMeta4, kMetaBytes,
                      mbar);
            bulk_load(sbase + kOffKRaw + ((c & 1) * 8 + lane) * kSide4, page_of(blk), kSide4, kbar);
          }
          return blk;
        };
        int blk = load_keys(0, tile_cnt), blk1 = 0;
        if (ok && it.nkv > 1) blk1 = load_keys(1, tile_cnt + 1);
        if (ok) load_q();
        for (int j = 0; ok && j < it.nkv; ++j) {
          const uint32_t c = tile_cnt++;
          const int s = c % kStages, pages = tile_pages(tile_key(j));
          if (c >= (uint32_t)kStages &&
              !wait(bar(B_VE + s), ((c / kStages) - 1) & 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_expect_tx(bar(B_VT + s), pages * kSide4);
          __syncwarp();
          if (lane < pages)
            bulk_load(sbase + kOffV + s * kTileBytes + raw_offset(lane), page_of(blk) + kSide4,
                      kSide4, bar(B_VT + s));
          // (V of tile c - 2 is done with: the scales of four tiles are enough)
          blk = blk1;
          if (j + 2 < it.nkv) blk1 = load_keys(j + 2, c + 2);
        }
      }
      for (int j = 0; !kI4 && ok && j < it.nkv; ++j) {
        const uint32_t c = tile_cnt++;
        const int s = c % kStages;
        const int key0 = tile_key(j);
        const int pages = tile_pages(key0);
        const bool tail = key0 + kTileK > it.L || (kScored && key0 < vlow);
        int blk = blk_nxt;
        if (j + 1 < it.nkv && lane < tile_pages(tile_key(j + 1)))
          blk_nxt = __ldcg(btrow + (tile_key(j + 1) >> 4) + lane);
        if (c >= (uint32_t)kStages &&
            !wait(bar(B_KE + s), ((c / kStages) - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane < pages && (blk < 0 || (int64_t)blk >= a.num_blocks)) {
          atomicOr(ws.err, PKV_DEV_ERR_BLOCK_ID);
          blk = 0;
        }
        const uint32_t kdst = sbase + kOffK + s * kTileBytes;
        if (lane == 0) mbar_expect_tx(bar(B_KF + s), pages * 2 * kPageBoxBytes);
        __syncwarp();
        if (lane < pages) {
          tma_load_4d(kdst + lane * kPageBoxBytes, &tm_k, bar(B_KF + s), 0, it.g, 0, blk);
          tma_load_4d(kdst + kHalfBytes + lane * kPageBoxBytes, &tm_k, bar(B_KF + s), 64, it.g,
                      0, blk);
        }
        if (c >= (uint32_t)kStages &&
            !wait(bar(B_VE + s), ((c / kStages) - 1) & 1)) {
          ok = false;
          break;
        }
        const uint32_t vdst = sbase + kOffV + s * kTileBytes;
        const uint32_t vbar = tail ? bar(B_VT + s) : bar(B_VF + s);
        if (lane == 0) mbar_expect_tx(vbar, pages * 2 * kPageBoxBytes);
        __syncwarp();
        if (lane < pages) {
          tma_load_4d(vdst + lane * kPageBoxBytes, &tm_v, vbar, 0, it.g, 0, blk);
          tma_load_4d(vdst + kHalfBytes + lane * kPageBoxBytes, &tm_v, vbar, 64, it.g, 0, blk);
        }
        if (tail) {
          // wait for the V boxes, zero the rows of keys >= seq_len (and, at a
          // window's start, of the keys no row sees), publish
          ok = wait(bar(B_VT + s), vt_uses[s] & 1);
          vt_uses[s]++;
          if (!ok) break;
          uint8_t* v = smem + kOffV + s * kTileBytes;
          auto zero_rows = [&](int z0, int z1) {
            for (int i = lane; i < (z1 - z0) * 16; i += 32) {
              const int row = z0 + (i >> 4), within = i & 15;
              *reinterpret_cast<uint4*>(v + (within >> 3) * kHalfBytes + row * 128 +
                                        (within & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          };
          zero_rows(min(it.L - key0, kTileK), kTileK);
          if (kScored) zero_rows(0, vlow - key0);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_VF + s));
        }
      }
      if (!ok) break;
    }
  } else if (warp == 1) {
    if (kI4) take_regs<kRegsFew, false>();
    // ------------------------------ MMA issuer ------------------------------
    // (the whole warp runs this, in step; see mma_ss)
    {
      const uint32_t id_s = idesc_16(false, !kI4), id_o = idesc_16(true, !kI4);
      uint32_t tile_cnt = 0, s_cnt[2] = {0, 0}, o_cnt[2] = {0, 0}, q_cnt[2] = {0, 0};
      // Operand descriptors of every buffer, built once: a descriptor's low
      // field is the address / 16, so a k-step's offset is added to it.
      const uint64_t dq0 = sdesc(sbase + kOffQ, 16), dq1 = sdesc(sbase + kOffQ + kTileBytes, 16);
      const uint64_t dk0 = sdesc(sbase + kOffK, 16), dk1 = sdesc(sbase + kOffK + kTileBytes, 16);
      const uint64_t dv0 = sdesc(sbase + kOffV, kHalfBytes);
      const uint64_t dv1 = sdesc(sbase + kOffV + kTileBytes, kHalfBytes);
      static_assert(kStages == 2, "one descriptor per stage");
      // S_x(c) = Q_x K_c^T
      auto issue_s = [&](int x, uint32_t c) {
        const uint64_t da = x ? dq1 : dq0, db = (c & 1) ? dk1 : dk0;
        const uint32_t d = tmem + x * 128;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
          mma_ss(d, da + off, db + off, id_s, kk > 0);
        }
        mma_commit(bar(B_SF + x));
        s_cnt[x]++;
      };
      // O_x (+)= P_x V_c  (P_x: bf16 pairs, keys 0-63 in columns 0-31 and keys
      // 64-127 in columns 64-95 of S_x: each half where its own scores were;
      // in a scored call each 32 keys where their scores were)
      auto issue_pv = [&](int x, uint32_t c, bool acc) {
        const uint64_t db = (c & 1) ? dv1 : dv0;
        const uint32_t d = tmem + 256 + x * 128, pa = tmem + x * 128;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(d,
                 pa + (kScored ? (kk >> 1) * 32 + (kk & 1) * 8 : (kk >> 2) * 64 + (kk & 3) * 8),
                 db + ((kk * 16 * 128) >> 4), id_o, (acc || kk > 0) ? 1u : 0u);
      };
      bool ok = true;
      for (uint32_t it_cnt = 0; ok; ++it_cnt) {
        const int slot = it_cnt & 1;
        if (!wait(bar(B_IF + slot), (it_cnt >> 1) & 1)) break;
        const Item it = items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IE + slot));
        if (it.r < 0) break;
        const int nx = it.hb >= 0 ? 2 : 1;
        for (int x = 0; x < nx && ok; ++x)
          ok = wait(kI4 ? i4_bar(I_QD + x) : bar(B_QF + x), q_cnt[x]++ & 1);
        const uint32_t c0 = tile_cnt;
        if (!ok || !wait(bar(B_KF + c0 % kStages), (c0 / kStages) & 1)) break;
        tc_fence_after();
        for (int x = 0; x < nx; ++x) issue_s(x, c0);
        mma_commit(bar(B_KE + c0 % kStages));
        if (it.nkv == 1)
          for (int x = 0; x < nx; ++x) mma_commit(bar(B_QE + x));
        for (int j = 0; j < it.nkv && ok; ++j) {
          const uint32_t c = c0 + j;
          const bool more = j + 1 < it.nkv;
          if (!wait(bar(B_VF + c % kStages), (c / kStages) & 1)) {
            ok = false;
            break;
          }
          for (int x = 0; x < nx; ++x) {
            if (!wait(bar(B_PF + x), (s_cnt[x] - 1) & 1) ||
                (j == 0 && o_cnt[x] > 0 &&
                 !wait(bar(B_OE + x), (o_cnt[x] - 1) & 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_pv(x, c, j > 0);
            if (x == nx - 1) mma_commit(bar(B_VE + c % kStages));  // every PV of V_c issued
            if (more) {
              // the next K tile is waited for only now, with PV_x already queued
              if (x == 0 && !wait(bar(B_KF + (c + 1) % kStages), ((c + 1) / kStages) & 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
              issue_s(x, c + 1);
            } else {
              mma_commit(bar(B_OF + x));  // O_x final: its epilogue need not wait for the other tile
              o_cnt[x]++;
            }
          }
          if (!ok) break;
          if (more) {
            mma_commit(bar(B_KE + (c + 1) % kStages));
            if (j + 2 == it.nkv)
              for (int x = 0; x < nx; ++x) mma_commit(bar(B_QE + x));
          }
        }
        if (!ok) break;
        tile_cnt += it.nkv;
      }
    }
    __syncwarp();
  } else if (kScored && warp < 2 + kSoft) {
    if constexpr (kScored) {
    // ------------- softmax of a scored call: a set of warps for each query tile -------------
    // The first half of the softmax warps serves tile a of every item, the
    // second tile b: the two tiles' softmaxes run beside each other.  P of a
    // block of 32 columns goes where its scores began (16 packed columns).
    //   Fixed reference: 16 warps, each 64 columns (hf) of its 32 rows in two
    //     rounds; nothing passes between the warps of a row.
    //   Running maximum: 8 warps, each its 32 rows whole, so that no row needs
    //     another warp's values.  Quick path: pairs of blocks that every row of
    //     the warp sees, the maximum at hand and the form of the cap foreseen:
    //     straight code, checked at its end, and redone if the check fails (P
    //     has not left the registers, the scores are still in TMEM).  Block
    //     path: any block, masks, new maxima, in a loop.
    // 8 prompts of 2048 tokens, 64 heads over 8, us with L2 flushed: without
    // options 476, bias 505, window of 1024 417; cap 50 with scores of rms 3
    // 531 (of rms 5, many past a quarter of the cap, 595; of rms 9, many past
    // half, 762), with a bias 618, with the window 445; cap 200 679 to 753; the
    // plain call 512 (with scores of rms 3 its repeated maxima take it to 658).
    // The floor is 285, with the window 214.  Bound by the chain S -> P -> P.V of
    // a tile: under cap 50 no pipe is active half of the time (tensor 45%, fma
    // 31, alu 28, XU 22; issue slots 47) and six of the twelve cycles between two
    // instructions of a warp are waits for data (long scoreboard); scores past
    // half of the cap lengthen it by the reciprocal and the second exponential
    // (XU 29%).  Measured and not kept, for the cap (526 at the
    // time, with row sums of the unrounded weights): a row's 128
    // or 64 columns in straight code with all of its forms in place (730 to
    // 2229: instruction-cache misses); two warps a row as in the plain call
    // (573); four warps a row and tile (566); a row per thread (530 to 608); a
    // quick path checked at its end with 16 warps (584); prefetched rounds of 16
    // columns (601).  For the bias: two warps a row that exchange maxima (718
    // to 825: 80 registers a thread spill).
    const int x = (warp - 2) / (4 * kHalves);  // my query tile
    const int hf = kHalves == 1 ? 0 : ((warp - 2) >> 2) & 1;
    const int b0 = 2 * hf;  // my first block of 32 columns
    const int qd = warp & 3;
    const int row = qd * 32 + lane;  // == TMEM lane
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    float* lsum = reinterpret_cast<float*>(smem + kOffLsum);
    const ScoreArgs& sp = score_of(a);
    const uint32_t t_s = tmem + x * 128 + 32 * b0 + lane_off;
    const uint32_t t_o = tmem + 256 + x * 128 + lane_off;
    uint32_t s_cnt = 0;
    // The quick path's form of the cap: the exponential for the next eight
    // items after a score past the polynomial's range; kBlocks: none.
    constexpr int kBlocks = 2;
    int form = kCap == kAnyCap && sp.limit3 < 0.f ? kBlocks : 0, hold = 0;
    bool ok = true;
    for (uint32_t it_cnt = 0; ok; ++it_cnt) {
      const int slot = it_cnt & 1;
      if (!wait(bar(B_IF + slot), (it_cnt >> 1) & 1)) break;
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_IE + slot));
      if (it.r < 0) break;
      if (x == 1 && it.hb < 0) continue;  // an item of one tile
      const int qrow = it.qt * kPreTileQ + row;  // row inside the request
      const bool valid_row = qrow < it.n;
      // rows past the request's take the last row's position; they take part
      // in no decision, and their results are dropped
      const int rpos = it.ctx + (valid_row ? qrow : it.n - 1);
      const int last = max(rpos, it.prefix - 1);           // last visible key
      const int first = first_key(rpos, sp.window);   // first visible key
      const float slope2 = kBias ? __ldg(sp.slopes + (x ? it.hb : it.ha)) * kLog2e : 0.f;
      // The reference (log2 units) that the exponentials are taken against:
      // fixed (see fixed_reference), or the running maximum, rounded up to a
      // whole number, so that rescaling is exact; it follows the scores only
      // when a block's sum passes kMaxSum: bf16 keeps its precision over fp32's
      // exponents, so a reference below the maximum costs none, and 2^40 leaves
      // the sums room to 2^127.
      float ref = kCap == kFixedCap ? 0.f : -INFINITY;
      const float from = kCap == kFixedCap ? bias_from(slope2, rpos, first, last) : 0.f;
      float l = 0.f;
      if (form == 1 && --hold <= 0) form = 0;
      for (int j = 0; j < it.nkv; ++j) {
        const int key0 = tile_key0<kScored, kBias>(it, j) + 32 * b0;  // key of my first column
        const int lim = last - key0, low = first - key0;  // low <= column <= lim is visible
        if (!wait(bar(B_SF + x), s_cnt++ & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if constexpr (kCap == kFixedCap) {
          // (one vote a tile, and a loop without masks for most: votes and
          // branches of a block's own cost a tenth)
          if (__all_sync(0xffffffffu, lim >= 63 && low <= 0)) {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              float s[32];
              uint32_t p[16];
              PKV_LD32(t_s + 32 * c, s);
              tmem_wait_ld();
              logits32_any<kCap, kBias, kSym, false>(s, sp, 0.f, 0, 0, valid_row, slope2,
                                                     (float)(rpos - key0 - 32 * c), from);
              l += exp32(s, p);
              PKV_ST16U(t_s + 32 * c, p);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              float s[32];
              uint32_t p[16];
              const int lc = lim - 32 * c, wc = low - 32 * c;
              if (__all_sync(0xffffffffu, lc < 0 || wc > 31)) {  // no row sees any
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = 0;
              } else {
                PKV_LD32(t_s + 32 * c, s);
                tmem_wait_ld();
                logits32_any<kCap, kBias, kSym, true>(s, sp, 0.f, lc, wc, valid_row, slope2,
                                                      (float)(rpos - key0 - 32 * c), from);
                l += exp32(s, p);
              }
              PKV_ST16U(t_s + 32 * c, p);
            }
          }
        } else {
          // blocks c1 .. c2 - 1 are seen whole by every row of the warp
          const int c1 = (__reduce_max_sync(0xffffffffu, low) + 31) >> 5;
          const int c2 = min(4, (__reduce_min_sync(0xffffffffu, lim) + 1) >> 5);
          uint32_t done = 0;  // blocks whose P is written
          bool tried = false;
          for (;;) {
            // the block path: before the quick one only where a row has no
            // maximum yet, after it whatever is left
            const bool have = __all_sync(0xffffffffu, ref != -INFINITY || !valid_row);
            if (tried || !have || form == kBlocks) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                if ((done >> c) & 1) continue;
                float s[32];
                uint32_t p[16];
                const int lc = lim - 32 * c, wc = low - 32 * c;
                if (__all_sync(0xffffffffu, lc < 0 || wc > 31)) {  // no row sees any
#pragma unroll
                  for (int i = 0; i < 16; ++i) p[i] = 0;
                } else {
                  PKV_LD32(t_s + 32 * c, s);
                  tmem_wait_ld();
                  logits32_any<kCap, kBias, kSym, true>(s, sp, 0.f, lc, wc, valid_row, slope2,
                                                        (float)(rpos - key0 - 32 * c), 0.f);
                  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                  for (int i = 0; i < 32; i += 4) {
                    m0 = max3f(m0, s[i], s[i + 1]);
                    m1 = max3f(m1, s[i + 2], s[i + 3]);
                  }
                  const float m = fmaxf(m0, m1);
                  const bool up = m > ref + kRescaleThreshold;
                  if (__any_sync(0xffffffffu, up)) {
                    // the reference moves up by k whole units (a row without
                    // one: everything so far of it is zero)
                    const float to = up ? ceilf(m) : ref;
                    const float k = up ? to - ref : 0.f;
                    const float alpha =
                        k < 126.f ? __int_as_float((127 - (int)k) << 23) : 0.f;
                    l *= alpha;
                    ref = to;
                    tmem_wait_st();
                    if (j > 0) {
                      // (PV of the tile before is complete: S of this one is)
#pragma unroll 1
                      for (int ch = 0; ch < 8; ++ch) rescale16(t_o + ch * 16, alpha);
                    }
#pragma unroll 1
                    for (int e = 0; e < 4; ++e)
                      if ((done >> e) & 1) rescale16_bf16(t_s + 32 * e, alpha);
                  }
                  const float r0 = ref == -INFINITY ? 0.f : ref;  // (no key seen yet)
#pragma unroll
                  for (int i = 0; i < 32; ++i) s[i] -= r0;
                  l += exp32(s, p);
                }
                PKV_ST16U(t_s + 32 * c, p);
                done |= 1u << c;
                // (the rest by the quick path, once each row has a maximum)
                if (!tried && form != kBlocks && c2 > c1 &&
                    __all_sync(0xffffffffu, ref != -INFINITY || !valid_row))
                  break;
              }
            }
            if (done == 15u) break;
            if (tried) continue;
            tried = true;
            // the quick path: pairs of blocks, none of them done yet
#pragma unroll 1
            for (int h = 0; h < 4 && form != kBlocks;) {
              if (h < c1 || h + 2 > c2 || ((done >> h) & 3) != 0) {
                h += 2;
                continue;
              }
              uint32_t p[2][16];
              float big = 0.f, sum = 0.f;
              auto go = [&](auto f) {
                float s[2][32];
                PKV_LD32(t_s + 32 * h, s[0]);
                PKV_LD32(t_s + 32 * h + 32, s[1]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  logits32<kCap, kBias, kSym, decltype(f)::value>(
                      s[c], sp, -ref, slope2, (float)(rpos - key0 - 32 * (h + c)), 0.f, big);
                  sum += exp32(s[c], p[c]);
                }
              };
              if (kCap == kNoCap || form == 0)
                go(std::integral_constant<Form, kDeg3>());
              else
                go(std::integral_constant<Form, kExp>());
              if (kCap != kNoCap && form == 0 &&
                  !__all_sync(0xffffffffu, big <= sp.limit3 || !valid_row)) {
                form = 1;
                hold = 8;
                continue;
              }
              // (past kMaxSum a new maximum is needed: the block path's)
              if (__all_sync(0xffffffffu, sum <= kMaxSum || !valid_row)) {
                l += sum;
                PKV_ST16U(t_s + 32 * h, p[0]);
                PKV_ST16U(t_s + 32 * h + 32, p[1]);
                done |= 3u << h;
              }
              h += 2;
            }
            if (done == 15u) break;
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PF + x));
      }
      if (!ok) break;
      // the row sums of the item, for the epilogue (see the plain call's)
      lsum[(((it_cnt & 1) * 2 + x) * 2 + hf) * 128 + row] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(lf_bar(it_cnt, x));
    }
    }
  } else if (kI4 && warp < kSoft0) {
    if constexpr (kI4) {
      take_regs<kRegsFew, false>();
      // ------------- the tiles' exponents; query rows with the warps below -------------
      uint32_t q_cnt[2] = {0, 0}, tile_cnt = 0;
      bool ok = true;
      for (uint32_t it_cnt = 0; ok; ++it_cnt) {
        const int slot = it_cnt & 1;
        if (!wait(bar(B_IF + slot), (it_cnt >> 1) & 1)) break;
        const Item it = items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IE + slot));
        if (it.r < 0) break;
        // tile j's exponents (the first of the two warps): the largest of |z| and
        // |z + 15 s| of its keys, and of its values.  The weights and their sum follow the
        // values': it counts as 2^-36 at least, and 2^-60 of those before it, which keeps
        // them in fp32's range for values of up to 2^60.
        constexpr int kLeast = 7 - 36;
        int vmax = kLeast;
        auto exponents = [&](int j) {
          const uint32_t c = tile_cnt + j;
          if (warp != 2) return;
          if (!wait(i4_bar(I_MR + (c & 3)), (c >> 2) & 1)) {
            ok = false;
            return;
          }
          uint32_t big[2] = {0, 0};
#pragma unroll
          for (int row = lane; row < 128; row += 32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t pair = *reinterpret_cast<const uint32_t*>(
                  smem + meta_offset(c) + (row >> 4) * kMetaBytes + 64 * i + 4 * (row & 15));
              const float sc = __uint_as_float(pair << 16);
              const float z = __uint_as_float(pair & 0xFFFF0000u);
              const float m = fmaxf(fabsf(z), fabsf(fmaf(15.f, sc, z)));
              if (row < it.L - j * kTileK) big[i] = max(big[i], __float_as_uint(m));
            }
          }
          const int kexp = tile_exponent(__reduce_max_sync(0xffffffffu, big[0]));
          const int e = tile_exponent(__reduce_max_sync(0xffffffffu, big[1]));
          const int vexp = max(max(e, kLeast), vmax - 60);
          vmax = max(vmax, e);
          if (lane == 0) {
            *reinterpret_cast<int2*>(smem + kOffTileExp + 8 * (c & 3)) = make_int2(kexp, vexp);
            mbar_arrive(i4_bar(I_XR + (c & 3)));
          }
        };
#pragma unroll 1
        for (int j = 0; ok && j < it.nkv; ++j) {
          exponents(j);
          if (ok && j == min(1, it.nkv - 1)) ok = query_rows(it, it_cnt, q_cnt, warp - 2);
        }
        tile_cnt += it.nkv;
      }
    }
  } else if (warp < kSoft0 + 8) {
    if constexpr (kI4) {
      take_regs<kRegsSoft, true>();
      // ------------- softmax of a 4-bit call: four warps for each query tile -------------
      // A row per thread, its 128 scores in two rounds of 64: nothing passes between
      // warps.  The scores are scaled by the powers of two of the row and of the K tile; a V
      // tile's, 2^ev, goes into its weights, w = 2^(x + ev - ref), so that a tile keeps its
      // values' bits whatever the size of the others'.  The reference (whole log2 units)
      // moves when the sum of a round passes 63488, close below fp16's largest number (with
      // 2^14, more often: 788 us for 760, see above), to where the largest weight is 2^8: far
      // enough above fp16's smallest that 2^19 keys' roundings to halves of 2^-24 are 2^-13
      // of the largest weight together.  The row's sum of 2^x is kept in units of the present
      // tile's, l 2^(ref - ev).  One loop for everything, on purpose: with the exponentials in
      // two places and both query tiles in one warp the kernel's roles did not fit the
      // instruction caches together, and all of them, the MMA's too, took two to three times
      // as long (4 chunks of 2047 tokens, 64 heads: 1368 us, 940 with the tiles' loop rolled).
      const int x = (warp - kSoft0) >> 2;
      const int qd = warp & 3;
      const int row = qd * 32 + lane;  // == TMEM lane
      const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
      const uint32_t t_s0 = tmem + x * 128 + lane_off, t_o = tmem + 256 + x * 128 + lane_off;
      float* lsum = reinterpret_cast<float*>(smem + kOffLsum);
      const float sl2 = fabsf(a.scale) * kLog2e;
      uint32_t s_cnt = 0, tile_cnt = 0;
      bool ok = true;
      for (uint32_t it_cnt = 0; ok; ++it_cnt) {
        const int slot = it_cnt & 1;
        if (!mbar_wait_warp(bar(B_IF + slot), (it_cnt >> 1) & 1, abort, ws.err)) break;
        const Item it = items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IE + slot));
        if (it.r < 0) break;
        if (x == 1 && it.hb < 0) {  // an item of one tile
          tile_cnt += it.nkv;
          continue;
        }
        const int qrow = it.qt * kPreTileQ + row;           // row inside the request
        const int qpos = qrow < it.n ? it.ctx + qrow : 0;   // last visible key
        float ref = -INFINITY, l = 0.f;
        int vexp = 0;
        for (int j = 0; j < it.nkv; ++j, ++tile_cnt) {
          if (!mbar_wait_warp(bar(B_SF + x), s_cnt++ & 1, abort, ws.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int2 te = *reinterpret_cast<const int2*>(smem + kOffTileExp + 8 * (tile_cnt & 3));
          // (never 0, so that a masked -inf stays one: zero rows have the smallest factors)
          const float f = fmaxf(
              sl2 * pow2(te.x) * reinterpret_cast<const float*>(smem + qfac_offset(it_cnt, x))[row],
              0x1p-126f);
          l *= pow2(min(te.y - vexp, 127));
          vexp = te.y;
          const float ev = (float)vexp;
          float o_alpha = 1.f;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int lim = qpos - j * kTileK - 64 * h;  // columns <= lim are visible
            const uint32_t t_s = t_s0 + 64 * h;
            float sv[64], sum;
            bool move = ref == -INFINITY;  // look for the maximum
#pragma unroll 1
            for (;;) {
              PKV_LD32(t_s + 0, (sv + 0));
              PKV_LD32(t_s + 32, (sv + 32));
              tmem_wait_ld();
              if (!__all_sync(0xffffffffu, lim >= 63)) {
#pragma unroll
                for (int i = 0; i < 64; ++i) sv[i] = (i <= lim) ? sv[i] : -INFINITY;
              }
              const bool any_move = __any_sync(0xffffffffu, move);
              if (any_move) {
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                for (int i = 0; i < 64; i += 4) {
                  m0 = max3f(m0, sv[i], sv[i + 1]);
                  m1 = max3f(m1, sv[i + 2], sv[i + 3]);
                }
                const float m = ceilf(fmaxf(m0, m1) * f) + ev - kLift16;
                const float to = move ? fmaxf(ref, m) : ref;
                const float alpha = ref == -INFINITY ? 0.f : fast_exp2(ref - to);
                ref = to;
                l *= alpha;
                o_alpha *= alpha;
                if (h == 1) {  // the weights of the first round
                  tmem_wait_st();
#pragma unroll 1
                  for (int ch = 0; ch < 2; ++ch) rescale16_f16(t_s0 + 16 * ch, alpha);
                }
              }
              // w = exp2(s * f + ev - ref), packed over sv[0 .. 31] (sv[2i], sv[2i + 1] are read
              // before sv[i] is written)
              float rs[4] = {0.f, 0.f, 0.f, 0.f};
              const float nm = ev - ref;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float x0, x1;
                fma2(x0, x1, sv[2 * i], sv[2 * i + 1], f, f, nm, nm);
                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                add2(rs[2 * (i & 1)], rs[2 * (i & 1) + 1], p0, p1);
                sv[i] = __uint_as_float(pack_f16(p0, p1));
              }
              sum = (rs[0] + rs[1]) + (rs[2] + rs[3]);
              if (any_move) break;
              move = !(sum <= kMaxSum16);
              if (!__any_sync(0xffffffffu, move)) break;
            }
            PKV_ST32(t_s, (sv + 0));  // 32 packed columns where my scores began
            l += sum;
          }
          if (j > 0 && __any_sync(0xffffffffu, o_alpha != 1.f)) {
            // (PV of the tile before is complete: S of this one is)
#pragma unroll 1
            for (int ch = 0; ch < 8; ++ch) rescale16(t_o + ch * 16, o_alpha);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_PF + x));
        }
        if (!ok) break;
        // the row's sum in units of the weights, for the epilogue
        lsum[((it_cnt & 1) * 2 + x) * 2 * 128 + row] = l * pow2(-vexp);
        __syncwarp();
        if (lane == 0) mbar_arrive(lf_bar(it_cnt, x));
      }
    }
    if constexpr (!kScored && !kI4) {
    // ------------------- softmax: two warps per row, a column half each -------------------
    // Warp w reads TMEM lanes 32 * (w % 4) .. + 31 (its 32 rows, one per
    // thread) and key columns 64 * hf .. 64 * hf + 63, hf = (w - 2) / 4, of
    // both query tiles of the item in turn; both warps of a row quarter (w and
    // w + 4) sit on the same SM sub-partition and work on the same tile at the
    // same time, so each tile's softmax takes half as long.  The warps of a
    // quarter exchange per-row values (the need for a max pass, the partial
    // maxima, the partial sums) through shared memory and a two-arrival
    // mbarrier, whose waits are bounded like every other.
    const int hf = (warp - kSoft0) >> 2;
    const int qd = warp & 3;
    const int row = qd * 32 + lane;  // == TMEM lane
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    float* xch = reinterpret_cast<float*>(smem + kOffXch);
    const float sl2 = a.scale * kLog2e;
    uint32_t s_cnt[2] = {0, 0}, x_cnt = 0;
    bool ok = true;
    // this lane's value out, the other warp's value for the same row back
    auto exchange = [&](float v) -> float {
      const int sl = x_cnt & 1;  // two slots: a slot is rewritten only after both read it
      xch[((qd * 2 + sl) * 2 + hf) * 32 + lane] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_XP + qd));
      if (!wait(bar(B_XP + qd), x_cnt & 1)) ok = false;
      x_cnt++;
      return xch[((qd * 2 + sl) * 2 + (1 - hf)) * 32 + lane];
    };
    float* lsum = reinterpret_cast<float*>(smem + kOffLsum);
    for (uint32_t it_cnt = 0; ok; ++it_cnt) {
      const int slot = it_cnt & 1;
      if (!wait(bar(B_IF + slot), (it_cnt >> 1) & 1)) break;
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_IE + slot));
      if (it.r < 0) break;
      const int nx = it.hb >= 0 ? 2 : 1;
      const int qrow = it.qt * kPreTileQ + row;  // row inside the request
      const bool valid_row = qrow < it.n;
      const int qpos = valid_row ? it.ctx + qrow : 0;  // last visible key
      float m_used[2] = {-INFINITY, -INFINITY}, l_part[2] = {0.f, 0.f};
      for (int j = 0; j < it.nkv && ok; ++j) {
        const int lim = qpos - j * kTileK - 64 * hf;  // my columns <= lim are visible
        const bool masked = !__all_sync(0xffffffffu, lim >= 63);
        for (int x = 0; x < nx && ok; ++x) {
          if (!wait(bar(B_SF + x), s_cnt[x]++ & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t t_s = tmem + x * 128 + 64 * hf + lane_off;
          // my 64 scores of the row in registers (one wait), then P in place
          float sv[64];
          auto load_scores = [&]() {
            PKV_LD32(t_s + 0, (sv + 0));
            PKV_LD32(t_s + 32, (sv + 32));
            tmem_wait_ld();
            if (masked) {
#pragma unroll
              for (int i = 0; i < 64; ++i) sv[i] = (i <= lim) ? sv[i] : -INFINITY;
            }
          };
          // p = exp2(s * scale * log2(e) - m) two columns at a time (packed
          // fp32 pairs for the multiply-add and the sums); the bf16 pairs are
          // packed over sv[0..31] (sv[2i], sv[2i+1] read before sv[i] is written)
          float rs[4];
          auto exp_pack = [&](float m) {
            rs[0] = rs[1] = rs[2] = rs[3] = 0.f;
            const float nm = -m;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x0, x1;
              fma2(x0, x1, sv[2 * i], sv[2 * i + 1], sl2, sl2, nm, nm);
              const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
              add2(rs[2 * (i & 1)], rs[2 * (i & 1) + 1], p0, p1);
              sv[i] = __uint_as_float(pack_bf16(p0, p1));
            }
          };
          load_scores();
          float alpha = 1.f;
          bool resc = false;
          // After the first tile, P is computed with the running max straight
          // away: no p exceeds 2^8 (the rescale threshold) while a half-row
          // sum does not, so the max pass is taken only when some half-row's
          // sum does (or is not finite) in either warp of the quarter.
          bool need_max = j == 0;
          if (!need_max) {
            exp_pack(m_used[x]);
            const float tot = (rs[0] + rs[1]) + (rs[2] + rs[3]);
            const float mine = (tot <= 256.f) ? 0.f : 1.f;
            const float other = exchange(mine);
            if (!ok) break;
            need_max = __any_sync(0xffffffffu, mine + other > 0.f);
            if (need_max) load_scores();
          }
          if (need_max) {
            // the row maximum over both halves: three-input max chains, then
            // the other warp's half through the exchange
            float mx[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = max3f(sv[k], sv[k + 4], sv[k + 8]);
#pragma unroll
            for (int i = 12; i < 60; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) mx[k] = max3f(mx[k], sv[i + k], sv[i + 4 + k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], sv[60 + k]);
            const float pm = fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]);
            const float po = exchange(pm);
            if (!ok) break;
            // (both warps form the same value: the halves in a fixed order)
            const float mt = (hf == 0 ? fmaxf(pm, po) : fmaxf(po, pm)) * sl2;
            resc = mt > m_used[x] + kRescaleThreshold;
            if (resc) {
              alpha = fast_exp2(m_used[x] - mt);  // 0 on the first tile
              m_used[x] = mt;
            }
            exp_pack(m_used[x]);
          }
          PKV_ST32(t_s, (sv + 0));  // P half: 32 packed columns where my scores began
          l_part[x] = l_part[x] * alpha + ((rs[0] + rs[1]) + (rs[2] + rs[3]));
          if (j > 0 && __any_sync(0xffffffffu, resc)) {
            // PV(j-1) is complete (S(j) is, and one thread's MMAs finish in
            // order); each warp rescales its own 64 output columns
            const uint32_t t_o = tmem + 256 + x * 128 + 64 * hf + lane_off;
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
              float ov[32];
              PKV_LD32(t_o + ch * 32, ov);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] *= alpha;
              PKV_ST32(t_o + ch * 32, ov);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_PF + x));
        }
      }
      if (!ok) break;
      // this warp's partial row sums of the item, for the epilogue warps
      // (one barrier per item parity: the softmax may finish the next item
      // before the epilogue has waited for this one, and one barrier would
      // then have completed two phases, which a parity wait cannot tell
      // apart from none)
      for (int x = 0; x < nx; ++x) {
        lsum[(((it_cnt & 1) * 2 + x) * 2 + hf) * 128 + row] = l_part[x];
        __syncwarp();
        if (lane == 0) mbar_arrive(lf_bar(it_cnt, x));
      }
    }
    }
  } else if (kI4 && warp >= kSoft0 + kSoft + 4) {
    if constexpr (kI4) {
      take_regs<kRegsFew, false>();
      // -------- 4-bit codes to fp16 tiles: two warps the K tiles, two the V tiles --------
      // Four lanes a row, 32 dimensions each: a 16-byte read, four 16-byte pieces written
      // where TMA would put them (128-byte swizzle).  The lanes of the upper half row take
      // another row of the eight, so that eight lanes meet eight different bank groups.  10
      // instructions a word of eight codes, 1600 a tile of keys and values; a loop of eight
      // rows a step (its eight steps in a row were 8 KB of code, see the softmax).
      const int side = (warp - kSoft0 - kSoft - 4) >> 1, dw = warp & 1;  // 1: V
      const int gid = lane >> 2, tig = lane & 3;
      constexpr int kWarpRows = 128 / kDequantWarps;
      const int lane_row = gid ^ (tig & 2);  // of eight
      const uint32_t src0 = (side ? raw_offset(kPagesPerWarp * dw) : kPagesPerWarp * dw * kSide4) +
                            lane_row * kRow4 + 16 * tig;
      uint32_t dst0[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst0[i] = (tig >> 1) * kHalfBytes + kWarpRows * dw * 128 +
                  sw128(lane_row, 4 * (tig & 1) + i);
      uint32_t tile_cnt = 0, q_cnt[2] = {0, 0};
      bool ok = true;
      for (uint32_t it_cnt = 0; ok; ++it_cnt) {
        const int slot = it_cnt & 1;
        if (!wait(bar(B_IF + slot), (it_cnt >> 1) & 1)) break;
        const Item it = items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IE + slot));
        if (it.r < 0) break;
        for (int j = 0; ok && j < it.nkv; ++j) {
          const uint32_t c = tile_cnt++;
          const int s = c % kStages;
          const int keys = it.L - j * kTileK;  // rows past these are zeroed
          const uint8_t* meta = smem + meta_offset(c);
          // scales, exponents, codes (the values' are in their stage), and a K stage's room
          if (!wait(i4_bar(I_MR + (c & 3)), (c >> 2) & 1) ||
              !wait(i4_bar(I_XR + (c & 3)), (c >> 2) & 1) ||
              !wait(side ? bar(B_VT + s) : i4_bar(I_KR + s), (c / kStages) & 1) ||
              (!side && c >= (uint32_t)kStages &&
               !wait(bar(B_KE + s), ((c / kStages) - 1) & 1))) {
            ok = false;
            break;
          }
          const int2 te = *reinterpret_cast<const int2*>(smem + kOffTileExp + 8 * (c & 3));
          uint8_t* stage = smem + (side ? kOffV : kOffK) + s * kTileBytes;
          const uint8_t* raw = side ? stage : smem + kOffKRaw + s * 8 * kSide4;
          const uint32_t* pairs =
              reinterpret_cast<const uint32_t*>(meta + kPagesPerWarp * dw * kMetaBytes) + 16 * side;
          const float down = pow2(-(side ? te.y : te.x));
          // eight rows a step, from the last: in the V stage a step overwrites codes of rows
          // behind its own only
          uint4 w = *reinterpret_cast<const uint4*>(raw + src0 + (kWarpRows / 8 - 1) * 8 * kRow4);
#pragma unroll 1
          for (int k = kWarpRows / 8 - 1; k >= 0; --k) {
            uint32_t pair = pairs[(k >> 1) * (kMetaBytes / 4) + 8 * (k & 1) + lane_row];
            if (kWarpRows * dw + 8 * k + lane_row >= keys) pair = 0;
            const float sc = __uint_as_float(pair << 16) * down;
            const float z = __uint_as_float(pair & 0xFFFF0000u) * down;
            const float sh = sc * 0x1p24f, sl = sc * 0x1p20f;
            const uint32_t s2 = pack_f16(sh, sh), t2 = pack_f16(sl, sl), z2 = pack_f16(z, z);
            const uint4 now = w;
            if (k > 0) w = *reinterpret_cast<const uint4*>(raw + src0 + (k - 1) * 8 * kRow4);
            __syncwarp();
            *reinterpret_cast<uint4*>(stage + dst0[0] + k * 1024) = dequant8(now.x, s2, t2, z2);
            *reinterpret_cast<uint4*>(stage + dst0[1] + k * 1024) = dequant8(now.y, s2, t2, z2);
            *reinterpret_cast<uint4*>(stage + dst0[2] + k * 1024) = dequant8(now.z, s2, t2, z2);
            *reinterpret_cast<uint4*>(stage + dst0[3] + k * 1024) = dequant8(now.w, s2, t2, z2);
          }
          fence_async_smem();  // (read by the MMAs)
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar((side ? B_VF : B_KF) + s));
            if (!side) mbar_arrive(i4_bar(I_KT + s));
          }
          if (j == 0) ok = query_rows(it, it_cnt, q_cnt, 2 + 2 * side + dw);
        }
      }
    }
  } else {
    if (kI4) take_regs<kRegsEpi, false>();
    // ------------------ epilogue: one warp per TMEM lane quarter ------------------
    // Warp w (four after the softmax) owns rows 32 * (w % 4) .. + 31 of both output tiles.  When
    // O_x is final (its last P.V done) and both partial row sums are in, the
    // warp reads the 128-column row block out of TMEM in two halves,
    // normalises them and packs them to bf16 in registers, and releases O_x as
    // soon as the second half is read (the next item's first P.V may then
    // overwrite it); each 32-column chunk goes out through the warp's staging
    // area in shared memory, so that each global store writes whole 64-byte
    // row pieces (8 rows x 4 lanes).
    // The softmax warps never wait for this work.
    const int qd = warp & 3;
    const int row = qd * 32 + lane;  // == TMEM lane
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const float* lsum = reinterpret_cast<const float*>(smem + kOffLsum);
    const uint32_t stg = sbase + kOffStage + (warp - kSoft0 - kSoft) * kStageWarp;
    uint32_t o_cnt[2] = {0, 0};
    for (uint32_t it_cnt = 0;; ++it_cnt) {
      const int slot = it_cnt & 1;
      if (!wait(bar(B_IF + slot), (it_cnt >> 1) & 1)) break;
      const Item it = items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_IE + slot));
      if (it.r < 0) break;
      const int nx = it.hb >= 0 ? 2 : 1;
      bool ok = true;
      for (int x = 0; x < nx && ok; ++x) {
        const uint32_t par = o_cnt[x]++ & 1;
        if (!wait(bar(B_OF + x), par) ||
            !wait(lf_bar(it_cnt, x), (it_cnt >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* ls = lsum + ((it_cnt & 1) * 2 + x) * 2 * 128;
        // the sums of the warps that shared the row
        const float inv = 1.f / (kHalves == 1 ? ls[row] : ls[row] + ls[128 + row]);
        const uint32_t t_o = tmem + 256 + x * 128 + lane_off;
        const int h = x == 0 ? it.ha : it.hb;
        const int row_base = it.qt * kPreTileQ + qd * 32;  // the warp's first row
        uint16_t* obase = a.out + (int64_t)it.q0 * a.out_stride + (int64_t)h * kHeadSize;
        // two 64-column halves; O_x is released once the second half is in
        // registers (the first half is already on its way out by then)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t held[32];  // 64 outputs of the row, bf16 pairs
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            float ov[16];
            PKV_LD16(t_o + half * 64 + ch * 16, ov);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              held[ch * 8 + i] = pack_bf16(ov[2 * i] * inv, ov[2 * i + 1] * inv);
          }
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_OE + x));
          }
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            // this lane's row: 16-byte piece k at slot k ^ ((lane >> 1) & 3), so
            // that eight lanes of a store phase hit eight different bank groups
#pragma unroll
            for (int k = 0; k < 4; ++k)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                               stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)),
                           "r"(held[cc * 16 + 4 * k]), "r"(held[cc * 16 + 4 * k + 1]),
                           "r"(held[cc * 16 + 4 * k + 2]), "r"(held[cc * 16 + 4 * k + 3])
                           : "memory");
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = i * 8 + (lane >> 2), c = lane & 3;
              uint4 v;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                           : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                           : "r"(stg + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4))
                           : "memory");
              const int qr = row_base + rr;
              if (qr < it.n)
                *reinterpret_cast<uint4*>(obase + (int64_t)qr * a.out_stride + half * 64 +
                                          cc * 32 + c * 8) = v;
            }
            __syncwarp();
          }
        }
      }
      if (!ok) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem),
                 "r"(kTmemCols));
  }
  // the split decode results, once the decode grid has finished
  grid_dep_wait();
  combine_splits(a, ws, blockIdx.x * (kThreads / 32) + warp, gridDim.x * (kThreads / 32));
}

// (K and V of 4-bit pages come by bulk copies: their maps are the query's, not used)
template <bool kScored, Cap kCap, bool kBias, bool kSym, bool kI4 = false>
cudaError_t launch_prefill_as(const ScoredArgs& a, const Workspace& ws, int sms, cudaStream_t st) {
  static std::atomic<bool> attr[kMaxAttrDevices];
  auto* kernel = prefill_kernel<kScored, kCap, kBias, kSym, kI4>;
  constexpr int kSmem = kI4 ? kSmemBytesI4 : kSmemBytes;
  constexpr int kThreads = kI4 ? kThreadsI4 : threads_of(kCap == kFixedCap);
  if (kI4) {  // (shares that the launch does not have would be waited for without end)
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_acquire) == 0) {
      cudaFuncAttributes fa;
      if (cudaError_t e = cudaFuncGetAttributes(&fa, kernel)) return e;
      regs.store(fa.numRegs, std::memory_order_release);
    }
    if (regs.load(std::memory_order_acquire) < kRegsLaunch) return cudaErrorInvalidConfiguration;
  }
  if (cudaError_t e = smem_attr_once(kernel, kSmem, attr)) return e;
  CUtensorMap tq, tk, tv;
  if (!make_rows_map(&tq, a.q, a.q_rows, a.hq, a.q_stride, 1, kPreTileQ)) return cudaErrorInvalidValue;
  if (kI4) {
    tk = tv = tq;
  } else if (!make_cache_map(&tk, a.kc, a.num_blocks, a.hkv) ||
             !make_cache_map(&tv, a.vc, a.num_blocks, a.hkv)) {
    return cudaErrorInvalidValue;
  }
  return launch_dependent(kernel, dim3(sms), dim3(kThreads), kSmem, st, tq, tk, tv, a, ws);
}

}  // namespace

cudaError_t launch_prefill(const ScoredArgs& a, const Workspace& ws, int sms, cudaStream_t st) {
  const ScoreArgs& sc = a.score;
  if (a.kv == kInt4) return launch_prefill_as<false, kNoCap, false, false, true>(a, ws, sms, st);
  if (!sc.on) return launch_prefill_as<false, kNoCap, false, false>(a, ws, sms, st);
  const bool bias = sc.slopes != nullptr, sym = bias && sc.prefix != nullptr;
  if (sc.softcap > 0.f) {
    if (dev::fixed_reference(a))
      return sym    ? launch_prefill_as<true, kFixedCap, true, true>(a, ws, sms, st)
             : bias ? launch_prefill_as<true, kFixedCap, true, false>(a, ws, sms, st)
                    : launch_prefill_as<true, kFixedCap, false, false>(a, ws, sms, st);
    return bias ? launch_prefill_as<true, kAnyCap, true, true>(a, ws, sms, st)
                : launch_prefill_as<true, kAnyCap, false, false>(a, ws, sms, st);
  }
  return sym    ? launch_prefill_as<true, kNoCap, true, true>(a, ws, sms, st)
         : bias ? launch_prefill_as<true, kNoCap, true, false>(a, ws, sms, st)
                : launch_prefill_as<true, kNoCap, false, false>(a, ws, sms, st);
}

}  // namespace pkv
