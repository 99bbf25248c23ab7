// Split-KV decode attention over the cache of 4-bit codes (pkv_attention_int4):
// requests of one query token, or a few.  Longer ones take the prefill kernel's
// instance for this cache; work units, split results and their merge are those of
// the bf16 path.
//
// Mathematics.  K_j = s_j c_j + z_j with codes c_j and the row's own scale and zero;
// for values t_j and y_j likewise.  A row's logits (log2 units, f = scale * log2 e):
//   x_j = f s_j (q . c_j) + f z_j (sum_d q_d),
// and with weights e_j = 2^(x_j - ref), over the keys:
//   out = (sum_j (e_j t_j) c_j + sum_j e_j y_j) / sum_j e_j,
// so that the products run on the codes, and scales and zeros are two multiply-adds a
// score and one a weight.
//
// GB300 design.  A page of a KV head is one record of 2176 bytes (keys, values,
// scales), one bulk copy into a ring of the warp's own; nothing else is read.  At
// 6.8 TB/s an SM gets a page every 93 cycles, 372 issue slots, of which the codes'
// way into the MMA operands may take a part:
//   * codes as fp16 numbers without an operation besides the mask: a nibble in the
//     low bits of a half is the subnormal c * 2^-24, one place up c * 2^-20, exact
//     either way.  A word and the word shifted by 8, each with two masks, are the
//     operands of 8 codes (five operations).  The power of two is undone in fp32:
//     2^-24 at the end, and the 16 between the two masks in the query (half of its
//     values are divided by 16), in the output by its rows.
//   * keys and output dimensions are the MMA's 16 rows and query rows its 8 columns
//     (S^T = K Q^T, O^T = V^T P^T): a step of 8 query rows, which groups of up to 8
//     heads need, takes half the MMAs and accumulators of query rows in the 16-row
//     operand.  P^T's operand is S^T's accumulator transposed, 8x8 by 8x8
//     (movmatrix).
//   * k order of S: a thread holds 32 consecutive dimensions of its two keys; the
//     16 keys of a page are the MMA rows in the order kappa(m), so that the key rows
//     that eight lanes read lie in different banks.
//   * query rows are scaled by a power of two, so that their largest value is
//     between 2^10 and 2^11 in fp16: values down to 2^-23 of it stay exact, smaller ones
//     are off by 2^-31 of it at most (half of the row is divided by 16 more).  Rows of up
//     to 2^110: the factor that undoes it, and the codes' 2^24, stays finite (applied to the
//     scales and zeros apart, for rows up to 2^127, it took 128 decodes of 8192 keys from
//     182.4 to 183.9 us, and lost keys above 2^104).
//   * weights: e_j t_j is rounded to fp16 (2^-11 of itself at most).  The
//     reference follows the largest e_j t_j of a row, not the largest e_j: fp16's range
//     then holds every weight that counts, however large or small the value rows'
//     scales.  It is moved only when a weight passes 2^14 (checked by one vote for
//     two pages, no exchange between the lanes otherwise).
//   * values come by ldmatrix, transposed: a register has a byte, two dimensions, of
//     four keys, so that a mask and a shift by 8 make MMA operands of it too.
// Keys past the unit's end get weight 0 and scale and zero 0.
//
// Two pages are taken at a time: their chains of dependent operations (S's products,
// the weights, P's transposition) run beside one another.  128 decodes of 8192 keys,
// 32 query heads on 8 | 32 decodes of 32,768 keys, 32 on one, us:
//   one page at a time, 8 | 8 warps               252 | 160
//   two pages, 12 | 8 warps                       202 |  99
//   and one MMA tile with 16 warps | two with 8   190 |  82
//   (with 20 | 10 warps, fewer registers          199 |  96
//   one page at a time with 16 | 12 warps         194 |  88
//   four tiles with 8 warps, one page                    87
//   the next pages' S before these ones' weights         90, spills
//   shifts by a high product, off the alu pipe    211 |  89)
//   values by transposed loads, one fence a stage 187 |  80
//   four pages a stage with two tiles             187 |  77
//   (with 12 warps and one | two pages at a time         81 | 84, spills)
//   three units a worker for four (the plan)      183 |  77
// The first is bound by HBM (6.2 TB/s of codes and scales, 0.92 of the copy rate) with
// the alu pipe, which takes the masks and shifts; the second by the latency of a
// step's chain, with two warps a scheduler, whose registers the tiles take (of about 2000
// cycles for two pages the tensor pipe is busy 1000, the alu pipe 900; asking for a
// stage's copies takes 300 to 400, waiting for them 120).  Asking for the next unit's
// pages while this one's last steps run, in the loop, cost more registers and code than
// it saved (189 | 86).
#include <cuda_fp16.h>

#include "pkv_int4.cuh"
#include "pkv_sched.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr uint32_t kNib0 = 0x000F000Fu, kNib1 = 0x00F000F0u;
constexpr float kMaxWeight = 16384.f;  // e_j t_j that the reference is kept for
// The scale of a value row without spread counts as this (its codes are zero), so that
// its e_j is held below 2^54 by the same bound; scales of others are above it.  (Zeros of up
// to 2^60: a unit's sum of e_j y_j stays finite.)
constexpr float kMinScale = 0x1p-40f;

// Instances: items of at most 8 * kTiles query rows.  The rings take what shared memory
// there is: 96 pages for the CTA's warps, in stages of kStagePages.
template <int kTiles>
struct Cfg4 {
  static constexpr int kWarps = kTiles == 1 ? 16 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStagePages = kTiles == 1 ? 2 : 4;
  static constexpr int kStages = 96 / kWarps / kStagePages;
  static constexpr int kWarpBytes = kStages * kStagePages * kPage4;
  static constexpr int kOffBar = kWarps * kWarpBytes;
  static constexpr int kOffCtl = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmem = kOffCtl + (2 + kWarps) * 4 + 128;  // (abort, items given out, first items)
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
// Two matrices of 16 rows of 16 bytes, transposed: lane l gives row l % 16 of matrix l / 16
// and receives, of the first (second) matrix in x, y (z, w), bytes 4 (l % 4) .. + 3 of
// columns l / 4 and l / 4 + 8.
__device__ __forceinline__ uint4 load_transposed(uint32_t addr) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(addr));
  return v;
}
// D += A(16x16, row) * B(16x8, col); fp16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the 8x8 matrix of b16 values that the warp holds, transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// One warp's ring: the stage its next step takes, and the parity of that step's wait.
struct Ring {
  uint32_t base, bars, stage, parity;
};

// Query rows row0 .. of a unit (nrows of them in all), at most 8 * kT, kSp pages a
// stage, two (32 keys) at a time.  Returns false when a wait gave up.
template <int kT>
__device__ __forceinline__ bool run_unit(const AttnArgs& a, const Workspace& ws, const DecUnit& un,
                                         int row0, Ring& ring, uint64_t pol,
                                         volatile int* abort) {
  constexpr int kStages = Cfg4<kT>::kStages, kSp = Cfg4<kT>::kStagePages, kPg = 2;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int G = a.hq / a.hkv;
  const int ug = un.gq & 0xFFFF;  // KV head
  const int qn = un.gq >> 16;     // query tokens of the request
  const int k0 = un.k0, k1 = un.k1;
  const int p0 = k0 / kBlockSize;
  const int npages = (k1 + kBlockSize - 1) / kBlockSize - p0, nstages = (npages + kSp - 1) / kSp;
  const int nrows = qn * G;

  // The ids of 32 pages, one per lane, and of the next 32.
  const int* btrow = table_row(a, un.r, ug) + p0;
  auto load_ids = [&](int p) {
    const uint8_t* page = nullptr;
    if (p + lane < npages) {
      int blk = __ldg(btrow + p + lane);
      if (blk < 0 || (int64_t)blk >= a.num_blocks) {
        atomicOr(ws.err, PKV_DEV_ERR_BLOCK_ID);
        blk = 0;
      }
      page = reinterpret_cast<const uint8_t*>(a.kc) + ((int64_t)blk * a.hkv + ug) * kPage4;
    }
    return page;
  };
  const uint8_t *ids = load_ids(0), *ids_next = load_ids(32);
  // pages kSp * j .. + kSp - 1 into stage st, each by the lane that holds its id; the stage's
  // last pages were taken by this warp already (program order; one lane's fence is for all:
  // with one by each lane that loads, 32 decodes of 32,768 keys took 82.5 us for 79.6)
  auto issue = [&](int j, uint32_t st) {
    const int first = kSp * j & 31;
    if (first == 0 && j > 0) {
      ids = ids_next;
      ids_next = load_ids(kSp * j + 32);
    }
    const uint32_t bar = ring.bars + 8 * st;
    if (lane == first) {
      fence_async_smem();
      mbar_expect_tx(bar, min(kSp, npages - kSp * j) * kPage4);
    }
    __syncwarp();
    if ((lane & ~(kSp - 1)) == first && ids != nullptr)
      bulk_load_hint(ring.base + (kSp * st + (lane & (kSp - 1))) * kPage4, ids, kPage4, bar, pol);
  };
  {
    uint32_t st = ring.stage;
    for (int j = 0; j < kStages && j < nstages; ++j) {
      issue(j, st);
      st = st + 1 == kStages ? 0 : st + 1;
    }
  }

  // Query rows: tile t has rows row0 + 8 t .. + 7 (token * G + head in group), a thread
  // dimensions 32 tig .. + 31 of row gid.  Operand pair 2 i + h of k-step order: word
  // i of the keys' codes, shifted by 8 h.
  uint32_t qb[kT][8][2];
  float fac[kT][2], off[kT][2];  // by the thread's two columns: f * 2^(24 + exponent), f * sum q
  int vis[kT][2];                // keys the column's row sees end here
  const float f = a.scale * kLog2e;
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    const int row = row0 + 8 * t + gid;
    uint4 raw[4] = {};
    if (row < nrows) {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (int64_t)(un.q0 + row / G) * a.q_stride + (int64_t)(ug * G + row % G) * kHeadSize +
          32 * tig);
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = __ldg(src + i);
    }
    float big = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        big = max3f(big, fabsf(lo16(w[j])), fabsf(hi16(w[j])));
        sum += lo16(w[j]) + hi16(w[j]);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    // q * 2^-ex, its largest value in [2^10, 2^11)
    const int ex = max((int)(__float_as_uint(big) >> 23) - 127 - 10, -100);
    const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
    const float rf = f * __uint_as_float((uint32_t)(127 + ex) << 23) * 0x1p24f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float m = j & 1 ? down * 0.0625f : down;
        qb[t][2 * i + (j >> 1)][j & 1] = pack_f16(lo16(w[j]) * m, hi16(w[j]) * m);
      }
    }
    const float rs = f * sum;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      fac[t][c] = __shfl_sync(0xffffffffu, rf, 4 * (2 * tig + c));
      off[t][c] = __shfl_sync(0xffffffffu, rs, 4 * (2 * tig + c));
      const int r = row0 + 8 * t + 2 * tig + c;
      vis[t][c] = min(k1, un.ctx + (r < nrows ? r / G : qn - 1) + 1);
    }
  }
  const int all_see = min(k1, un.ctx + 1);  // every row sees the keys before

  // o[t][d]: output dimensions of the thread's two MMA rows (see below), columns 2 tig,
  // + 1; sums of e and of e * zero over the thread's keys; the negative reference of
  // each column (0 and `unset` while a row has seen no key)
  float o[kT][8][4], l[kT][2], z[kT][2], nref[kT][2];
#pragma unroll
  for (int t = 0; t < kT; ++t) {
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][d][e] = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) l[t][c] = z[t][c] = nref[t][c] = 0.f;
  }
  uint32_t unset = (1u << 2 * kT) - 1;  // columns without a reference (the same in each gid)

  // MMA row m < 8 of a page's first (second) eight is its key kappa(m) (+ 8)
  const int key = ((gid >> 1) ^ (gid & 1)) + 4 * (gid & 1);
  const uint32_t at_k = ring.base + kRow4 * key + 16 * tig;
  const uint32_t at_m = ring.base + kMeta4 + 4 * key;
  // values, transposed: row 4 t + u of a matrix is the key that MMA column 2 t (u = 0), 2 t + 1
  // (u = 2), 2 t + 8 (u = 1), 2 t + 9 (u = 3) has
  const int vt = (lane >> 2) & 3, vkey = ((lane & 2) ? (vt ^ 1) + 4 : vt) + 8 * (lane & 1);
  const uint32_t at_v = ring.base + kSide4 + kRow4 * vkey + 16 * (lane >> 4);

  for (int j = 0; j < nstages; ++j) {
    if (!mbar_wait_warp(ring.bars + 8 * ring.stage, ring.parity, abort, ws.err)) return false;
#pragma unroll 1
    for (int half = 0; half < kSp; half += kPg) {
      if (kSp > kPg && half > 0 && kSp * j + half >= npages) break;
      const uint32_t st = (kSp * ring.stage + half) * kPage4;
      // S^T = K Q^T
      float acc[kPg][kT][4];
      uint32_t mk[kPg][2], mv[kPg][2];
#pragma unroll
      for (int g = 0; g < kPg; ++g) {
        const uint4 ka = lds128(at_k + st + g * kPage4);
        const uint4 kb = lds128(at_k + st + g * kPage4 + 8 * kRow4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mk[g][i] = lds32(at_m + st + g * kPage4 + 32 * i);
          mv[g][i] = lds32(at_m + st + g * kPage4 + 64 + 32 * i);
        }
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[g][t][e] = 0.f;
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t ca = wa[i >> 1] >> (8 * (i & 1)), cb = wb[i >> 1] >> (8 * (i & 1));
#pragma unroll
          for (int t = 0; t < kT; ++t)
            mma_f16(acc[g][t], ca & kNib0, cb & kNib0, ca & kNib1, cb & kNib1, qb[t][i][0],
                    qb[t][i][1]);
        }
      }

      // logits less the reference: acc[g][t][0], [1] of the thread's first key of page g,
      // [2], [3] of its second
#pragma unroll
      for (int g = 0; g < kPg; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float ks = lo16(mk[g][i]), kz = hi16(mk[g][i]);
#pragma unroll
          for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              acc[g][t][2 * i + c] =
                  fmaf(acc[g][t][2 * i + c] * ks, fac[t][c], fmaf(kz, off[t][c], nref[t][c]));
        }
      const int pos = k0 + (kSp * j + half) * kBlockSize;
      if (pos + kPg * kBlockSize > all_see) {
#pragma unroll
        for (int g = 0; g < kPg; ++g)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = pos + kBlockSize * g + key + 8 * i;
            if (at >= k1) mv[g][i] = 0u;
#pragma unroll
            for (int t = 0; t < kT; ++t)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (at >= vis[t][c]) acc[g][t][2 * i + c] = -INFINITY;
          }
      }
      float vs[kPg][2], e[kPg][kT][4], w[kPg][kT][4];
#pragma unroll
      for (int g = 0; g < kPg; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) vs[g][i] = fmaxf(lo16(mv[g][i]), kMinScale);
      auto weights = [&]() {
        float most = 0.f;
#pragma unroll
        for (int g = 0; g < kPg; ++g)
#pragma unroll
          for (int t = 0; t < kT; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[g][t][i] = fast_exp2(acc[g][t][i]);
              w[g][t][i] = e[g][t][i] * vs[g][i >> 1];
            }
            most = max3f(most, max3f(w[g][t][0], w[g][t][1], w[g][t][2]), w[g][t][3]);
          }
        return most > kMaxWeight;
      };
      const bool over = weights();
      if (__any_sync(0xffffffffu, over || unset != 0)) {
        // references moved up: to the largest logit + log2 of the value row's scale
        // (weights up to 1)
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = -INFINITY;
#pragma unroll
            for (int g = 0; g < kPg; ++g)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                m = fmaxf(m, acc[g][t][2 * i + c] + __log2f(vs[g][i]));
#pragma unroll
            for (int b = 4; b < 32; b <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, b));
            const uint32_t bit = 1u << (2 * t + c);
            const bool none = (unset & bit) != 0;
            // (m is relative to the reference, 0 if there is none; a row without one takes
            // whatever it sees first, another moves up only)
            const float up = none ? (m == -INFINITY ? 0.f : m) : fmaxf(m, 0.f);
            const float al = fast_exp2(-up);
            if (m != -INFINITY) unset &= ~bit;
            nref[t][c] -= up;
            if (!none) {  // (nothing is summed yet of a row without a reference)
              l[t][c] *= al;
              z[t][c] *= al;
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                o[t][d][c] *= al;
                o[t][d][2 + c] *= al;
              }
            }
#pragma unroll
            for (int g = 0; g < kPg; ++g)
#pragma unroll
              for (int i = 0; i < 2; ++i) acc[g][t][2 * i + c] -= up;
          }
        weights();
      }
      uint32_t pb[kPg][kT][2];
#pragma unroll
      for (int g = 0; g < kPg; ++g)
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            l[t][c] += e[g][t][c] + e[g][t][2 + c];
            z[t][c] = fmaf(e[g][t][c], hi16(mv[g][0]), fmaf(e[g][t][2 + c], hi16(mv[g][1]), z[t][c]));
            pb[g][t][c] = transpose8x8(pack_f16(w[g][t][2 * c], w[g][t][2 * c + 1]));
          }

      // O^T += V^T P^T: a register of a transposed load has a byte, two dimensions, of four
      // keys; the first and third are one operand register, the others the next, MMA rows
      // gid and gid + 8 the two nibbles.
#pragma unroll
      for (int g = 0; g < kPg; ++g) {
        const uint4 va = load_transposed(at_v + st + g * kPage4);
        const uint4 vb = load_transposed(at_v + st + g * kPage4 + 32);
        if (half + g == kSp - 1) {  // the stage is in registers: it can take another step
          __syncwarp();
          if (j + kStages < nstages) issue(j + kStages, ring.stage);
        }
        const uint32_t v[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const uint32_t lo = v[d], hi = v[d] >> 8;
#pragma unroll
          for (int t = 0; t < kT; ++t)
            mma_f16(o[t][d], lo & kNib0, lo & kNib1, hi & kNib0, hi & kNib1, pb[g][t][0],
                    pb[g][t][1]);
        }
      }
    }
    if (++ring.stage == kStages) {
      ring.stage = 0;
      ring.parity ^= 1;
    }
  }

  // The thread's columns 2 tig, 2 tig + 1 are query rows, o[d] the two dimensions of byte 8 d +
  // gid of a row's codes: 16 d + at and two on, at = 8 (gid / 4) + 4 (gid % 2) + (gid / 2) % 2.
  // Lanes gid and gid ^ 2 exchange one, so that each has two neighbours.
  const bool odd = gid & 2;
  const int at = 8 * (gid >> 2) + 4 * (gid & 1) + (gid & 2);
#pragma unroll
  for (int t = 0; t < kT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float ls = l[t][c], zs = z[t][c];
#pragma unroll
      for (int b = 4; b < 32; b <<= 1) {
        ls += __shfl_xor_sync(0xffffffffu, ls, b);
        zs += __shfl_xor_sync(0xffffffffu, zs, b);
      }
      float2 v[8];
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const float x = fmaf(o[t][d][c], 0x1p24f, zs), y = fmaf(o[t][d][2 + c], 0x1p20f, zs);
        const float other = __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
        v[d] = odd ? make_float2(other, y) : make_float2(x, other);
      }
      const int row = row0 + 8 * t + 2 * tig + c;
      if (row >= nrows) continue;
      if (un.nsplit == 1) {
        const float inv = 1.f / ls;
        uint16_t* dst = a.out + (int64_t)(un.q0 + row / G) * a.out_stride +
                        (int64_t)(ug * G + row % G) * kHeadSize + at;
#pragma unroll
        for (int d = 0; d < 8; ++d)
          *reinterpret_cast<uint32_t*>(dst + 16 * d) = pack_bf16(v[d].x * inv, v[d].y * inv);
      } else {
        float* dst = ws.part_o + ((int64_t)un.part + row) * kHeadSize + at;
#pragma unroll
        for (int d = 0; d < 8; ++d) *reinterpret_cast<float2*>(dst + 16 * d) = v[d];
        if (gid == 0)  // (no key seen: the merge skips a split with reference -inf)
          *reinterpret_cast<float2*>(ws.part_ml + ((int64_t)un.part + row) * 2) =
              make_float2((unset >> (2 * t + c)) & 1 ? -INFINITY : -nref[t][c], ls);
      }
    }
  return true;
}

// Groups of up to 8 heads: a unit's rows 8 at a time, its pages read again each time
// (single tokens: one time.  64 decodes of 8192 keys, 32 heads on 8, of 1 | 2 | 4 tokens:
// 120 | 124 | 220 us, pkv_attention 190 | 194 | 203; 64 of 2048 keys, 32 on 32, of 1 | 8 |
// 16: 120 | 128 | 231).  Larger groups: two tiles, and above 16 heads a unit is two items, of its first 16 query rows
// and of the rest, for two warps that each read its pages (the second out of the L2).
template <int kTiles>
__global__ void __launch_bounds__(Cfg4<kTiles>::kThreads, 1)
    decode_i4_kernel(AttnArgs a, Workspace ws) {
  using C = Cfg4<kTiles>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~(uintptr_t)127);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  Ring ring{sbase + warp * C::kWarpBytes, sbase + C::kOffBar + warp * C::kStages * 8, 0, 0};
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffCtl);
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(ring.bars + 8u * s, 1);
    if (warp == 0) *abort = 0;
    fence_barrier_init();
  }
  const int G = a.hq / a.hkv, shift = kTiles == 2 && G > 16 ? 1 : 0;
  // the set-up above overlaps the plan kernel; the work list is read after it
  grid_dep_wait();
  grid_dep_launch();
  const int left = sms_to_prefill<false, true>(a, ws, C::kWarps >> shift);
  if ((int)blockIdx.x < left || ws.hdr->n_dec_units == 0) return;
  // The first item of each warp by its index, spread over the CTAs; the cursor counts on
  // from there.  (With a cursor that every warp asks first, a step of two decodes and a
  // 298-token prompt took 29.5 us for 23.7.  The loop over a unit's pages takes all
  // registers: what is needed between units waits in shared memory.)
  volatile int* ctl = abort;
  if (lane == 0) ctl[2 + warp] = warp * (gridDim.x - left) + blockIdx.x - left;
  if (threadIdx.x == 0) ctl[1] = (gridDim.x - left) * C::kWarps;
  __syncthreads();
  const int n_items = ws.hdr->n_dec_units << shift;
  const uint64_t pol = l2_evict_first();  // pages are read once (or twice at a time)
  for (;;) {
    int u = 0;
    if (lane == 0) {
      u = ctl[2 + warp];
      ctl[2 + warp] = -1;
      if (u < 0) u = ctl[1] + atomicAdd(&ws.hdr->dec_counter, 1);
    }
    u = __shfl_sync(0xffffffffu, u, 0);
    if (u >= n_items || *abort) break;
    const DecUnit un = load_unit(ws.units + (u >> shift));
    bool ok = true;
    if (kTiles == 1) {
      const int rows = (un.gq >> 16) * G;
      for (int row0 = 0; ok && row0 < rows; row0 += 8)
        ok = run_unit<kTiles>(a, ws, un, row0, ring, pol, abort);
    } else {
      ok = run_unit<kTiles>(a, ws, un, 16 * (u & shift), ring, pol, abort);
    }
    if (!ok) break;
  }
}

template <int kTiles>
cudaError_t launch_i4(const AttnArgs& a, const Workspace& ws, int sms, cudaStream_t st) {
  using C = Cfg4<kTiles>;
  static std::atomic<bool> attr[kMaxAttrDevices];
  if (cudaError_t e = smem_attr_once(decode_i4_kernel<kTiles>, C::kSmem, attr)) return e;
  return launch_dependent(decode_i4_kernel<kTiles>, dim3(sms), dim3(C::kThreads), C::kSmem, st, a,
                          ws);
}

}  // namespace

// units at a time of a CTA
int decode_i4_warps(int group) {
  return group <= 8 ? Cfg4<1>::kWarps : group <= 16 ? Cfg4<2>::kWarps : Cfg4<2>::kWarps / 2;
}

cudaError_t launch_decode_i4(const AttnArgs& a, const Workspace& ws, int sms, cudaStream_t st) {
  return a.hq / a.hkv <= 8 ? launch_i4<1>(a, ws, sms, st) : launch_i4<2>(a, ws, sms, st);
}

}  // namespace pkv
