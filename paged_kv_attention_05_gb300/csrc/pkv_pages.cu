// Attention over the pages that a cheap score selects for each query row
// (block-sparse decode): the bounds of each page's keys, and the selection.  The
// attention over the selected pages is the split-KV decode kernel with a list of
// pages for each row and KV head (pkv_decode.cu).
//
// Mathematics.  Page j of KV head g holds keys K; lo_d and hi_d are their
// smallest and largest values in dimension d (bounds, exact in bf16).  No key of
// the page has a larger product with a query q than sum_d max(q_d lo_d, q_d hi_d);
// the page's score for a row is that bound summed over the query heads of g:
//   score_j = sum_h sum_d max(q_hd lo_jd, q_hd hi_jd) = sum_d U_d hi_jd + D_d lo_jd,
//   U_d = sum_h max(q_hd, 0),  D_d = sum_h min(q_hd, 0).
// A row at position p has n = p / 16 + 1 pages.  It takes all of them when n is
// at most the budget; else its first `first` and last `last` pages and the
// budget - first - last of the others with the largest scores, the lower page of
// two equal ones.
//
// The selection is exact, as if the scores had been formed in 64 bits.  Scores
// formed in fp32 are off by at most eps = (G + 16) 2^-24 S M, with S = sum_d U_d +
// |D_d| and M the largest bound of the row's pages: a sum of products over a tree of
// depth n is off by n 2^-24 of the sum of their sizes, here 8 products in a lane's
// chain, a join, 4 exchanges, G - 1 additions in U and D, and one in reserve for
// each product's second order.  With T the k-th largest fp32 score, a page above
// T + 2 eps is among the k largest and one below T - 2 eps is not; where those between
// are more than the places left, they are scored again in 64 bits.  (Where S M is 2^126
// or more, fp32 sums may overflow: all are.)
#include <algorithm>

#include "pkv_internal.cuh"
#include "pkv_device.cuh"

namespace pkv {
namespace {

using namespace dev;

// ---------------------------------------------------------------- page bounds

// Smallest and largest keys of the pages that the step's tokens wrote.  A token
// whose successor in the call lies in another page has the last slot of its page:
// it forms the bounds of slots 0 .. its own.  A warp takes kTok tokens and one KV
// head, a half-warp eight of a page's rows, eight dimensions a lane, all 16 rows in
// flight; the packed bf16 minimum and maximum are exact.  HBM-bound: 256 bytes a key.
// One token a warp while there are few (their pages are read side by side), sixteen
// when warps abound: nearly every warp of a prompt has a page then.  8 chunks of 2047
// tokens, 8 KV heads, floor 5.5 us: 8.6 (eight tokens a warp 9.0; and 8 bytes a lane, which
// the compiler did not keep in flight, 12.6); a step of 128 decodes 5.0, a launch's time.
// (asked for in program order: the compiler would rather wait than hold 16 rows)
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int kTok>
__global__ void __launch_bounds__(256)
    page_bounds_kernel(const uint16_t* __restrict__ kc, int64_t num_slots, int hkv,
                       uint16_t* __restrict__ bounds, const int64_t* __restrict__ slots,
                       int64_t n_tokens, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t groups = (n_tokens + kTok - 1) / kTok, units = groups * hkv;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t u = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; u < units; u += nwarps) {
    const int64_t t0 = u / hkv * kTok;
    const int h = (int)(u % hkv);
    const int64_t mine = lane <= kTok && t0 + lane < n_tokens ? __ldg(slots + t0 + lane) : -1;
    const int64_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    bool owner = lane < kTok && mine >= 0 && (next < 0 || next / kBlockSize != mine / kBlockSize);
    if (lane < kTok && mine >= num_slots) {
      if (h == 0) atomicOr(err, PKV_DEV_ERR_SLOT_RANGE);
      owner = false;
    }
    uint32_t todo = __ballot_sync(0xffffffffu, owner);
    while (todo) {
      const int64_t slot = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
      todo &= todo - 1;
      const int64_t block = slot / kBlockSize;
      const int last = (int)(slot % kBlockSize);
      // (rows past the last are it again)
      const uint16_t* src = kc + (block * kBlockSize * hkv + h) * kHeadSize + (lane & 15) * 8;
      uint4 r[kBlockSize / 2];
#pragma unroll
      for (int i = 0; i < kBlockSize / 2; ++i)
        r[i] = load16(src + (int64_t)min(2 * i + (lane >> 4), last) * hkv * kHeadSize);
      auto as2 = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
      auto bits = [](__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); };
      uint32_t lo[4] = {r[0].x, r[0].y, r[0].z, r[0].w}, hi[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
      for (int i = 1; i < kBlockSize / 2; ++i) {
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          lo[k] = bits(__hmin2(as2(lo[k]), as2(w[k])));
          hi[k] = bits(__hmax2(as2(hi[k]), as2(w[k])));
        }
      }
      // the other half-warp has the other eight rows: it keeps the maxima, this one the minima
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool upper = lane >= 16;
        const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? lo[k] : hi[k], 16);
        o[k] = bits(upper ? __hmax2(as2(hi[k]), as2(other)) : __hmin2(as2(lo[k]), as2(other)));
      }
      *reinterpret_cast<uint4*>(bounds + (block * hkv + h) * 2 * kHeadSize + lane * 8) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ------------------------------------------------------------------ selection

constexpr int kSelKeys = 8192;  // scores of a (row, KV head) kept in shared memory

constexpr int kNone = -1, kUnknown = -2;
struct Row {
  int r, pos;  // request (kNone: the row belongs to no valid one), position
  int n;       // pages
};

__device__ __forceinline__ int meta_errors(const SelectArgs& a, int q0, int q1, int L) {
  if (q0 < 0 || q1 < q0 || (int64_t)q1 > a.q_rows) return PKV_DEV_ERR_QSL;
  if (L < 0 || L < q1 - q0) return PKV_DEV_ERR_SEQ_LEN;
  if (((int64_t)L + kBlockSize - 1) / kBlockSize > a.bt_width) return PKV_DEV_ERR_BT_WIDTH;
  return 0;
}

__device__ __forceinline__ Row row_of(int64_t row, int r, int q0, int q1, int L) {
  const int pos = L - (q1 - q0) + (int)(row - q0);
  return Row{r, pos, pos / kBlockSize + 1};
}
// The request and position of a query row.  (Decode batches have a row per
// request: the guess r = row saves the search's chain of reads.)  kUnknown: an entry out
// of order misled the search, or the request that owns the row is bad (see scan_row).
__device__ __forceinline__ Row find_row(const SelectArgs& a, int64_t row) {
  int lo = (int)min(row, (int64_t)a.num_reqs - 1);
  int q0 = __ldcg(a.qsl + lo), q1 = __ldcg(a.qsl + lo + 1), L = __ldcg(a.seq_lens + lo);
  if (!(q0 <= row && row < q1)) {
    lo = 0;
    for (int hi = a.num_reqs - 1; lo < hi;) {  // the last request that starts at or before it
      const int mid = (lo + hi + 1) >> 1;
      if (__ldcg(a.qsl + mid) <= row) lo = mid; else hi = mid - 1;
    }
    q0 = __ldcg(a.qsl + lo), q1 = __ldcg(a.qsl + lo + 1), L = __ldcg(a.seq_lens + lo);
  }
  const bool past = lo == a.num_reqs - 1 && q0 <= q1 && q1 <= row;  // of the last request
  if (q0 <= row && row < q1 && !meta_errors(a, q0, q1, L)) return row_of(row, lo, q0, q1, L);
  return Row{past ? kNone : kUnknown, 0, 0};
}
// The first request that has the row and passes the checks, if there is one (by the whole
// warp, 32 at a time).
__device__ __forceinline__ Row scan_row(const SelectArgs& a, int64_t row) {
  int found = a.num_reqs;
  for (int r = threadIdx.x & 31; r < a.num_reqs && found == a.num_reqs; r += 32) {
    const int q0 = __ldcg(a.qsl + r), q1 = __ldcg(a.qsl + r + 1);
    if (q0 <= row && row < q1 && !meta_errors(a, q0, q1, __ldcg(a.seq_lens + r))) found = r;
  }
  const int r = (int)__reduce_min_sync(0xffffffffu, (unsigned)found);
  if (r == a.num_reqs) return Row{kNone, 0, 0};
  return row_of(row, r, __ldcg(a.qsl + r), __ldcg(a.qsl + r + 1), __ldcg(a.seq_lens + r));
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// fp32 and fp64 values as whole numbers of the same order
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ unsigned long long ordered64(double f) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(f);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// total over the block of one int per thread
template <int kSelWarps>
__device__ __forceinline__ int block_sum(int v, int* part) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();  // (part may still be read)
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) s += part[w];
  return s;
}

// The fp32 scores of pages from .. from + count - 1 of a row for one KV head, by the
// calling warp: put(page, score) for each; returns the largest bound met (in every
// lane).  A half-warp reads one page's bounds (512 consecutive bytes), eight dimensions
// a lane.  kStream: the bounds, none read twice, are not to push others out of the L2.
template <bool kStream, typename Put>
__device__ __forceinline__ float score_pages(const SelectArgs& a, const int32_t* bt, int g,
                                             int from, int count, const float (&up)[8],
                                             const float (&dn)[8], Put put) {
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
  for (int b = 0; b < count; b += 32) {
    const int page = b + lane;
    // (past the last page it is the last one again: no other page's bounds count)
    int id = __ldg(bt + from + min(page, count - 1));
    if (id < 0 || (int64_t)id >= a.num_blocks) {
      atomicOr(a.err, PKV_DEV_ERR_BLOCK_ID);
      id = 0;
    }
    float mine = 0.f;  // the score of page b + lane
    const int steps = min(16, (count - b + 1) / 2);
#pragma unroll kStream ? 4 : 8
    for (int i = 0; i < steps; ++i) {
      const int blk = __shfl_sync(0xffffffffu, id, 2 * i + half);
      const uint16_t* p = a.bounds + ((int64_t)blk * a.hkv + g) * 2 * kHeadSize + l * 8;
      const uint4* at = reinterpret_cast<const uint4*>(p);
      const uint4 lo4 = kStream ? __ldcs(at) : __ldg(at);
      const uint4 hi4 = kStream ? __ldcs(at + kHeadSize / 8) : __ldg(at + kHeadSize / 8);
      const uint32_t lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s0 = fmaf(up[2 * k], lo16(hi[k]), s0);
        s1 = fmaf(dn[2 * k], lo16(lo[k]), s1);
        s0 = fmaf(up[2 * k + 1], hi16(hi[k]), s0);
        s1 = fmaf(dn[2 * k + 1], hi16(lo[k]), s1);
        m2 = __hmax2(m2, __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&lo[k])),
                                 __habs2(*reinterpret_cast<const __nv_bfloat162*>(&hi[k]))));
      }
      float s = s0 + s1;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float other = __shfl_xor_sync(0xffffffffu, s, 16);
      // lanes 2 i and 2 i + 1 keep the two halves' scores
      if (lane >> 1 == i) mine = ((lane & 1) == half) ? s : other;
    }
    if (page < count) put(from + page, mine);
  }
  float m = fmaxf(__low2float(m2), __high2float(m2));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Scores and selection.  A CTA scores kPages pages of a (row, KV head), its warps equal
// shares; the last CTA of the (row, KV head) to finish selects.  Where one CTA has
// all of its pages the scores never leave it.
// Bound by HBM while it scores (512 bytes a page, a sixteenth of the page's own keys
// and values), by a chain of block-wide counts while it selects.  64 of 2050 pages for one
// row | 64 of 513 for 128 rows, 8 KV heads, us (floors 1.2 and 39.7): scores and selection
// in two launches, the border found bit by bit 32 | 112; in one 43 | 100; the border by
// histograms of eight bits 15 | 80; 256 pages a CTA 16 | 72; and all of a row's by four
// warps 14 | 60; with U and D formed again where a row's request has to be looked for, and
// so in other registers, 14 | 57.  Of these the scores alone take 47; the border by one
// warp, without barriers, and block ids kept in shared memory were slower (80, 73).  64
// registers a thread, of which 8 to 24 bytes are spilled; more would cost CTAs.
// The grid follows the block table's width, not the rows' pages: a CTA past its row's pages
// reads the queries and the metadata before it returns (the 128 rows in tables of 513 |
// 1024 | 8192 | 32,768 pages, one call at a time: 67 | 79 | 159 | 487).
template <int kPages, int kSelThreads, bool kStream>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads)
    select_kernel(SelectArgs a, int64_t row0) {
  constexpr int kSelWarps = kSelThreads / 32, kBins = kSelThreads < 256 ? 256 / kSelThreads : 1;
  extern __shared__ uint32_t keys[];  // [min(bt_width, kSelKeys)] in calls that score
  __shared__ int part[kSelWarps], part2[kSelWarps];
  __shared__ int hist[256];
  __shared__ float s_max[kSelWarps], s_sum[kSelWarps];
  constexpr int kFew = 64;
  __shared__ int s_last, s_idx[kFew];
  __shared__ double s_exact[kFew];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rh = blockIdx.y, chunk = blockIdx.x;
  const int64_t row = row0 + rh / a.hkv;
  const int g = rh % a.hkv, G = a.hq / a.hkv;
  grid_dep_wait();
  // U and D, eight dimensions a lane (asked for beside the metadata; once more where the
  // request has to be looked for, as they would cost registers meanwhile)
  const uint16_t* q = a.q + row * a.q_stride + (int64_t)g * G * kHeadSize;
  float up[8], dn[8];
  Row x{kUnknown, 0, 0};
  for (;;) {
#pragma unroll
    for (int i = 0; i < 8; ++i) up[i] = dn[i] = 0.f;
#pragma unroll 4
    for (int h = 0; h < G; ++h) {
      const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(q + h * kHeadSize + (lane & 15) * 8));
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = i & 1 ? hi16(w[i >> 1]) : lo16(w[i >> 1]);
        up[i] += fmaxf(v, 0.f);
        dn[i] += fminf(v, 0.f);
      }
    }
    if (x.r != kUnknown) break;
    x = find_row(a, row);
    if (x.r != kUnknown) break;
    x = scan_row(a, row);
  }
  if (chunk == 0 && rh == 0 && row0 == 0)
    for (int r = tid; r < a.num_reqs; r += kSelThreads) {
      const int bad = meta_errors(a, __ldcg(a.qsl + r), __ldcg(a.qsl + r + 1), __ldcg(a.seq_lens + r));
      if (bad) atomicOr(a.err, bad);
    }
  const int n = x.n;
  if (x.r < 0 || n <= a.budget || a.budget == a.first + a.last) {
    // nothing to score: no list, or all pages, or the first and last ones
    if (chunk > 0) return;
    const int taken = min(n, a.budget);
    if (tid == 0 && g == 0)
      a.sel_lens[row] = x.r < 0 ? 0 : (taken - 1) * kBlockSize + x.pos % kBlockSize + 1;
    if (x.r < 0) return;
    int32_t* out = a.sel_table + (row * a.hkv + g) * (int64_t)a.budget;
    const int32_t* bt = a.bt + (int64_t)x.r * a.bt_width;
    for (int i = tid; i < a.budget; i += kSelThreads)
      out[i] = i >= taken ? -1 : __ldg(bt + (n <= a.budget || i < a.first ? i : n - taken + i));
    return;
  }
  const int end = n - a.last;  // (the last pages are taken unseen)
  const int needed = (end + kPages - 1) / kPages;
  if (chunk >= needed) return;
  const int32_t* bt = a.bt + (int64_t)x.r * a.bt_width;
  float* scores = a.scores + (int64_t)rh * a.bt_width;
  const int first = a.first, mid = end - first, k = a.budget - first - a.last;
  const bool in_smem = mid <= kSelKeys;

  float m = 0.f, size = 0.f;  // largest bound of the row's pages; sum of |q|
  {
#pragma unroll
    for (int i = 0; i < 8; ++i) size += up[i] - dn[i];
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) size += __shfl_xor_sync(0xffffffffu, size, o);
    const int n_here = min(kPages, end - chunk * kPages);  // a warp's share: a multiple of 4
    const int share = (n_here + 4 * kSelWarps - 1) / (4 * kSelWarps) * 4;
    const int from = chunk * kPages + warp * share;
    const int count = min(share, n_here - warp * share);
    if (count > 0)
      m = score_pages<kStream>(a, bt, g, from, count, up, dn, [&](int page, float s) {
        if (needed > 1)
          scores[page] = s;
        else if (page >= first)
          keys[page - first] = ordered(s);
      });
    if (lane == 0) s_max[warp] = m;
  }
  __syncthreads();
  m = 0.f;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) m = fmaxf(m, s_max[w]);
  if (needed > 1) {
    // (counted by atomics in no order that matters: whoever comes last selects)
    if (tid == 0) {
      a.largest[(int64_t)rh * a.largest_stride + chunk] = m;
      __threadfence();
      s_last = atomicAdd(a.done + rh, 1) == needed - 1;
      if (s_last) a.done[rh] = 0;  // for the next call
      __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    m = 0.f;
    for (int i = tid; i < needed; i += kSelThreads)
      m = fmaxf(m, __ldcg(a.largest + (int64_t)rh * a.largest_stride + i));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_sum[warp] = m;
    if (in_smem)
      for (int i = tid; i < mid; i += kSelThreads) keys[i] = ordered(__ldcg(scores + first + i));
    __syncthreads();
    m = 0.f;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) m = fmaxf(m, s_sum[w]);
  }
  // Each thread has `own` consecutive pages (an odd number: neighbouring threads meet
  // different banks).
  const int own = ((mid + kSelThreads - 1) / kSelThreads) | 1;
  const int i0 = min(tid * own, mid), i1 = min(i0 + own, mid);
  auto key_of = [&](int i) { return in_smem ? keys[i] : ordered(__ldcg(scores + first + i)); };
  // (a little more than (G + 16) 2^-24, for the roundings of S itself, and what
  // products below fp32's range lose; sums that may have passed its largest number, 2^128,
  // say nothing: every page is scored again then)
  const float eps =
      size * m < 0x1p126f ? (float)(G + 18) * 0x1p-24f * (size * m) + 0x1p-140f : INFINITY;

  // The k-th largest key, eight bits a step from the highest that differs, until what is
  // left of it is below eps: it lies in t .. t + 2^bits - 1.
  uint32_t t;
  int bits, left = k;  // keys still to be counted from above within the prefix
  {
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const uint32_t v = key_of(i);
      lo = min(lo, v);
      hi = max(hi, v);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      part[warp] = (int)lo;
      part2[warp] = (int)hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      lo = min(lo, (uint32_t)part[w]);
      hi = max(hi, (uint32_t)part2[w]);
    }
    bits = 32 - __clz(lo ^ hi);
    t = bits >= 32 ? 0 : hi & ~((1u << bits) - 1);
  }
  while (bits > 0 && !(unordered(t + (uint32_t)((1ull << bits) - 1)) - unordered(t) <= eps)) {
    const int shift = max(bits - 8, 0);
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const uint32_t d = key_of(i) - t;  // (keys below t wrap far up)
      if (bits >= 32 || d >> bits == 0) atomicAdd(hist + (d >> shift), 1);
    }
    __syncthreads();
    // a thread's kBins bins, the highest first, and those above them
    int c[kBins], mine = 0;
#pragma unroll
    for (int i = 0; i < kBins; ++i) {
      c[i] = tid * kBins < 256 ? hist[255 - tid * kBins - i] : 0;
      mine += c[i];
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) sum += w < warp ? part[w] : 0;
    if (sum >= left && sum - mine < left) {
      int bin = 255 - tid * kBins, rest = left - (sum - mine);
#pragma unroll
      for (int i = 0; i + 1 < kBins; ++i)
        if (rest > c[i] && bin == 255 - tid * kBins - i) {
          rest -= c[i];
          --bin;
        }
      part2[0] = bin;
      part2[1] = rest;
    }
    __syncthreads();
    t += (uint32_t)part2[0] << shift;
    left = part2[1];
    bits = shift;
  }
  const float above = unordered(t + (uint32_t)((1ull << bits) - 1)) + 2.f * eps;
  const float below = unordered(t) - 2.f * eps;
  // kIn and kOut for certain, kTie: between
  enum { kOut, kTie, kIn };
  auto state_of = [&](int i) {
    const float e = unordered(key_of(i));
    return e > above ? kIn : e < below ? kOut : kTie;
  };
  // exclusive sums over the block of a thread's count, two in a word; *total for all
  auto scan = [&](unsigned v, unsigned* total) {
    unsigned s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    __syncthreads();  // (part may still be read)
    if (lane == 31) part[warp] = (int)s;
    __syncthreads();
    unsigned before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) before += (unsigned)part[w];
      all += (unsigned)part[w];
    }
    *total = all;
    return before + s - v;
  };
  unsigned total;
  unsigned mine = 0;  // of this thread's pages: certain ones << 16 | those between
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const int st = state_of(i);
    mine += st == kIn ? 0x10000u : st == kTie ? 1u : 0u;
  }
  const unsigned before = scan(mine, &total);
  int ties = k - (int)(total >> 16);  // of the pages between, how many are taken
  const int cand = (int)(total & 0xFFFF);
  if (tid == 0 && g == 0) a.sel_lens[row] = (a.budget - 1) * kBlockSize + x.pos % kBlockSize + 1;
  int32_t* out = a.sel_table + (row * a.hkv + g) * (int64_t)a.budget;
  for (int i = tid; i < first; i += kSelThreads) out[i] = __ldg(bt + i);
  for (int i = tid; i < a.last; i += kSelThreads) out[a.budget - a.last + i] = __ldg(bt + end + i);
  out += first;
  if (cand <= ties || size == 0.f || m == 0.f) {
    // all of those between, or (every score zero, exactly) the first of them
    int in = (int)(before >> 16), tie = (int)(before & 0xFFFF);
    for (int i = i0; i < i1; ++i) {
      const int st = state_of(i);
      if (st == kIn || (st == kTie && tie < ties)) out[in + min(tie, ties)] = __ldg(bt + first + i);
      in += st == kIn;
      tie += st == kTie;
    }
    return;
  }

  // More pages between than places: their scores in 64 bits, in the order of the pages.
  // (a few, usually: kept in shared memory then.  Of 1024 selections in one wave one is
  // among the last, and this is its path: 64 of 513 pages for 128 rows 65 -> 63 us)
  const bool few = cand <= kFew;
  double* s64 = few ? s_exact : a.exact + (int64_t)rh * a.bt_width;
  {
    int32_t* idx = few ? s_idx : a.index + (int64_t)rh * a.bt_width;
    int at = (int)(before & 0xFFFF);
    for (int i = i0; i < i1; ++i)
      if (state_of(i) == kTie) idx[at++] = i;
    __syncthreads();
    if (warp < cand) {
      double du[4] = {}, dd[4] = {};
      for (int h = 0; h < G; ++h) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(q + h * kHeadSize + lane * 4));
        const float v[4] = {lo16(w.x), hi16(w.x), lo16(w.y), hi16(w.y)};
#pragma unroll
        for (int i = 0; i < 4; ++i) (v[i] > 0.f ? du[i] : dd[i]) += v[i];
      }
      for (int c = warp; c < cand; c += kSelWarps) {
        const int id = __ldg(bt + first + idx[c]);
        const int64_t blk = id < 0 || (int64_t)id >= a.num_blocks ? 0 : id;
        const uint16_t* p = a.bounds + (blk * a.hkv + g) * 2 * kHeadSize + lane * 4;
        const uint2 lo = __ldg(reinterpret_cast<const uint2*>(p));
        const uint2 hi = __ldg(reinterpret_cast<const uint2*>(p + kHeadSize));
        double s = du[0] * lo16(hi.x) + du[1] * hi16(hi.x) + du[2] * lo16(hi.y) + du[3] * hi16(hi.y);
        s += dd[0] * lo16(lo.x) + dd[1] * hi16(lo.x) + dd[2] * lo16(lo.y) + dd[3] * hi16(lo.y);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) s64[c] = s + 0.0;  // (-0 as 0)
      }
    }
    __syncthreads();
  }
  // A candidate's rank: those with a larger score, or an equal one and before it.  Up to
  // 256 of them by comparing each with all; more by the ties-th largest, bit by bit.
  constexpr int kRanked = 256;
  unsigned long long t64 = 0;
  if (cand > kRanked) {
#pragma unroll 1
    for (int bit = 63; bit >= 0; --bit) {
      const unsigned long long c = t64 | 1ull << bit;
      int more = 0;
      for (int i = tid; i < cand; i += kSelThreads) more += ordered64(s64[i]) >= c;
      if (block_sum<kSelWarps>(more, part) >= ties) t64 = c;
    }
    int more = 0;
    for (int i = tid; i < cand; i += kSelThreads) more += ordered64(s64[i]) > t64;
    ties -= block_sum<kSelWarps>(more, part);  // of the equal ones, the first
  }
  auto taken = [&](int c, int equal) {  // candidate c; equal: candidates at t64 before it
    const unsigned long long v = ordered64(s64[c]);
    if (cand > kRanked) return v > t64 || (v == t64 && equal < ties);
    int rank = 0;
    for (int i = 0; i < cand; ++i) {
      const unsigned long long u = ordered64(s64[i]);
      rank += u > v || (u == v && i < c);
    }
    return rank < ties;
  };
  // equal ones before this thread's pages, then taken ones
  unsigned equal = 0;
  int c = (int)(before & 0xFFFF);
  if (cand > kRanked) {
    for (int i = i0; i < i1; ++i)
      if (state_of(i) == kTie) equal += ordered64(s64[c++]) == t64;
    equal = scan(equal, &total);
  }
  unsigned count = 0, e = equal;
  c = (int)(before & 0xFFFF);
  for (int i = i0; i < i1; ++i) {
    const int st = state_of(i);
    if (st == kTie) {
      count += taken(c, (int)e);
      e += cand > kRanked && ordered64(s64[c]) == t64;
      ++c;
    } else {
      count += st == kIn;
    }
  }
  int at = (int)scan(count, &total);
  c = (int)(before & 0xFFFF);
  e = equal;
  for (int i = i0; i < i1; ++i) {
    const int st = state_of(i);
    bool in = st == kIn;
    if (st == kTie) {
      in = taken(c, (int)e);
      e += cand > kRanked && ordered64(s64[c]) == t64;
      ++c;
    }
    if (in) out[at++] = __ldg(bt + first + i);
  }
}

}  // namespace

cudaError_t launch_page_bounds(const uint16_t* kc, int64_t num_blocks, int hkv, uint16_t* bounds,
                               const int64_t* slots, int64_t n_tokens, int* err, int sms,
                               cudaStream_t st) {
  const bool many = n_tokens * hkv > (int64_t)sms * 64;  // more than the warps an SM holds
  const int64_t warps = (many ? (n_tokens + 15) / 16 : n_tokens) * hkv;
  const unsigned blocks = (unsigned)std::min<int64_t>((warps + 7) / 8, (int64_t)sms * 8);
  return launch_dependent(many ? page_bounds_kernel<16> : page_bounds_kernel<1>, dim3(blocks),
                          dim3(256), 0, st, kc, num_blocks * kBlockSize, hkv, bounds, slots,
                          n_tokens, err);
}

// Pages a CTA scores.  512, by four warps, where one CTA then has all of a row's pages (the
// last is not scored) and the CTAs fill five of the eight places of each SM: no scores pass
// through memory, and eight CTAs an SM select and score at different times.  Else 256 by
// eight warps, or 128 where that leaves SMs without one.  us with 128 | 256 | 512, 8 KV heads:
//   4 rows of 513 pages    12 | 12 | 18      100 of 513    68 |  58 |  51
//   1 of 2050              16 | 16 | 26      128 of 513    82 |  67 |  56
//   1 of 8000              42 | 42 | 80      256 of 260   100 |  85 |  62
//   64 of 513              44 | 39 | 45      512 of 70     79 |  68 |  48
//   32 of 2050             80 | 68 | 69      256 of 513   148 | 119 | 103
// (512 by eight warps, four CTAs an SM: 128 of 513 in 75, by sixteen 82, before the last step
// at the kernel; 32 a CTA: 1 of 8000 in 55.)  Half of the L2 or more of bounds are streamed: 128 of 513 pages 63 -> 61, 32
// of 2050 77 -> 72, 30 of 1000 43 -> 40, 8 of 8000 94 -> 89.
int select_chunk_pages(int64_t rows, int hkv, int64_t bt_width, int sms) {
  if (bt_width - 1 <= 512 && rows * hkv >= 5 * (int64_t)sms) return 512;
  return rows * hkv * bt_width >= (int64_t)sms * 256 ? 256 : 128;
}

cudaError_t launch_select(const SelectArgs& a, int64_t row0, int rows, bool score,
                          cudaStream_t st) {
  const int64_t chunks = score ? (a.bt_width + a.chunk_pages - 1) / a.chunk_pages : 1;
  const size_t smem = score ? (size_t)std::min<int64_t>(a.bt_width, kSelKeys) * 4 : 0;
  const bool stream = rows * a.hkv * a.bt_width >= 131072;  // (pages' bounds of 512 bytes)
  return launch_dependent(a.chunk_pages == 512 ? select_kernel<512, 128, true>
                          : a.chunk_pages == 128 ? select_kernel<128, 256, false>
                          : stream               ? select_kernel<256, 256, true>
                                                 : select_kernel<256, 256, false>,
                          dim3((unsigned)chunks, (unsigned)(rows * a.hkv)),
                          dim3(a.chunk_pages == 512 ? 128 : 256), smem, st, a, row0);
}

}  // namespace pkv
