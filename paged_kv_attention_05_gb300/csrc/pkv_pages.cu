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
// are more than the places left, they are scored again in 64 bits.
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
// head, four dimensions a lane, the page's 16 rows all in flight; the packed bf16
// minimum and maximum are exact.  HBM-bound: 256 bytes a key.
// One token a warp while there are few (their pages are read side by side), eight
// when warps abound: a prompt's warps then look at eight slots at once instead of
// one, and half of them have a page.
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
      const uint16_t* src = kc + (block * kBlockSize * hkv + h) * kHeadSize + lane * 4;
      uint2 r[kBlockSize];
#pragma unroll
      for (int i = 0; i < kBlockSize; ++i)  // (rows past the last are it again)
        r[i] = __ldcg(reinterpret_cast<const uint2*>(src + (int64_t)min(i, last) * hkv * kHeadSize));
      auto as2 = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
      auto bits = [](__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); };
      __nv_bfloat162 lo0 = as2(r[0].x), lo1 = as2(r[0].y), hi0 = lo0, hi1 = lo1;
#pragma unroll
      for (int i = 1; i < kBlockSize; ++i) {
        lo0 = __hmin2(lo0, as2(r[i].x));
        lo1 = __hmin2(lo1, as2(r[i].y));
        hi0 = __hmax2(hi0, as2(r[i].x));
        hi1 = __hmax2(hi1, as2(r[i].y));
      }
      uint16_t* dst = bounds + (block * hkv + h) * 2 * kHeadSize + lane * 4;
      *reinterpret_cast<uint2*>(dst) = make_uint2(bits(lo0), bits(lo1));
      *reinterpret_cast<uint2*>(dst + kHeadSize) = make_uint2(bits(hi0), bits(hi1));
    }
  }
}

// ------------------------------------------------------------------ selection

struct Row {
  int r, pos;  // request (-1: the row belongs to no valid one), position
  int n;       // pages
};

// The PKV_DEV_ERR_* bits of request r.
__device__ __forceinline__ int request_errors(const SelectArgs& a, int r) {
  const int q0 = __ldcg(a.qsl + r), q1 = __ldcg(a.qsl + r + 1), L = __ldcg(a.seq_lens + r);
  if (q0 < 0 || q1 < q0 || (int64_t)q1 > a.q_rows) return PKV_DEV_ERR_QSL;
  if (L < 0 || L < q1 - q0) return PKV_DEV_ERR_SEQ_LEN;
  if (((int64_t)L + kBlockSize - 1) / kBlockSize > a.bt_width) return PKV_DEV_ERR_BT_WIDTH;
  return 0;
}

// The request and position of a query row.  (Decode batches have a row per
// request: the guess r = row saves the search's chain of reads.)
__device__ __forceinline__ Row find_row(const SelectArgs& a, int64_t row) {
  Row x{-1, 0, 0};
  int lo = 0, hi = a.num_reqs - 1;
  if (row < a.num_reqs) {
    const int q0 = __ldcg(a.qsl + row), q1 = __ldcg(a.qsl + row + 1);
    if (q0 <= row && row < q1) lo = hi = (int)row;
  }
  while (lo < hi) {  // the last request that starts at or before the row
    const int mid = (lo + hi + 1) >> 1;
    if (__ldcg(a.qsl + mid) <= row) lo = mid; else hi = mid - 1;
  }
  const int q0 = __ldcg(a.qsl + lo), q1 = __ldcg(a.qsl + lo + 1), L = __ldcg(a.seq_lens + lo);
  if (row < q0 || row >= q1 || request_errors(a, lo)) return x;  // (or past the last request)
  x.r = lo;
  x.pos = L - (q1 - q0) + (int)(row - q0);
  x.n = x.pos / kBlockSize + 1;
  return x;
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The fp32 scores of a row's pages for one KV head.  A warp takes kPages pages of a
// (row, head); a half-warp reads one page's bounds (512 consecutive bytes), eight
// dimensions a lane.  Bound by HBM: 512 bytes a page, a sixteenth of the page's
// own keys and values.  Beside the scores each warp leaves the largest bound it
// met, for eps.
template <int kPages>
__global__ void __launch_bounds__(256) page_scores_kernel(SelectArgs a, int64_t row0, int rows) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int G = a.hq / a.hkv;
  const int64_t chunks = (a.bt_width + kPages - 1) / kPages;
  const int64_t units = (int64_t)rows * a.hkv * chunks;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t u = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; u < units; u += nwarps) {
    // (chunk by chunk of all rows: the chunks that hold pages come first)
    const int chunk = (int)(u / (rows * a.hkv));
    const int rh = (int)(u - (int64_t)chunk * rows * a.hkv);
    const int64_t row = row0 + rh / a.hkv;
    const int g = rh % a.hkv;
    const Row x = find_row(a, row);
    const int from = chunk * kPages;
    const int end = x.n - a.last;  // (the last pages are taken unseen)
    if (x.r < 0 || x.n <= a.budget || from >= end) continue;
    const int count = min(kPages, end - from);
    float up[8], dn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) up[i] = dn[i] = 0.f;
    const uint16_t* q = a.q + row * a.q_stride + (int64_t)g * G * kHeadSize + l * 8;
#pragma unroll 4
    for (int h = 0; h < G; ++h) {
      const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(q + h * kHeadSize));
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = i & 1 ? hi16(w[i >> 1]) : lo16(w[i >> 1]);
        up[i] += fmaxf(v, 0.f);
        dn[i] += fminf(v, 0.f);
      }
    }
    const int32_t* bt = a.bt + (int64_t)x.r * a.bt_width + from;
    float* out = a.scores + ((int64_t)rh * a.bt_width + from);
    __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
    for (int b = 0; b < count; b += 32) {
      const int page = b + lane;
      int id = page < count ? __ldg(bt + page) : 0;
      if (id < 0 || (int64_t)id >= a.num_blocks) {
        atomicOr(a.err, PKV_DEV_ERR_BLOCK_ID);
        id = 0;
      }
      float mine = 0.f;  // the score of page b + lane
      const int steps = min(16, (count - b + 1) / 2);
#pragma unroll 4
      for (int i = 0; i < steps; ++i) {
        const int blk = __shfl_sync(0xffffffffu, id, 2 * i + half);
        const uint16_t* p = a.bounds + ((int64_t)blk * a.hkv + g) * 2 * kHeadSize + l * 8;
        const uint4 lo4 = __ldg(reinterpret_cast<const uint4*>(p));
        const uint4 hi4 = __ldg(reinterpret_cast<const uint4*>(p + kHeadSize));
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
      if (page < count) out[page] = mine;
    }
    float m = fmaxf(__low2float(m2), __high2float(m2));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) a.largest[(int64_t)rh * a.largest_stride + chunk] = m;
  }
}

constexpr int kSelThreads = 256;

// total over the block of one int per thread
__device__ __forceinline__ int block_sum(int v, int* part) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();  // (part may still be read)
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) s += part[w];
  return s;
}
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
// The k-th largest of n keys (1 <= k <= n), by its bits from the highest.
template <typename Key, typename Get>
__device__ Key kth_largest(int n, int k, int* part, Get get) {
  Key t = 0;
#pragma unroll 1
  for (int bit = 8 * (int)sizeof(Key) - 1; bit >= 0; --bit) {
    const Key c = t | (Key)1 << bit;
    int more = 0;
    for (int i = threadIdx.x; i < n; i += kSelThreads) more += get(i) >= c;
    if (block_sum(more, part) >= k) t = c;
  }
  return t;
}

// A page's state in the selection (in place of its key).
enum : uint32_t { kOut = 0, kTie = 1, kIn = 2 };

// The pages of one (row, KV head): a CTA each.  The keys sit in shared memory; the
// k-th largest is found bit by bit (a count of the block for each).
__global__ void __launch_bounds__(kSelThreads) select_pages_kernel(SelectArgs a, int64_t row0) {
  extern __shared__ uint32_t keys[];  // [bt_width] in calls that score
  __shared__ int part[kSelThreads / 32];
  __shared__ float s_max[kSelThreads / 32];
  grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rh = blockIdx.x;
  const int64_t row = row0 + rh / a.hkv;
  const int g = rh % a.hkv, G = a.hq / a.hkv;
  if (blockIdx.x == 0 && row0 == 0)
    for (int r = tid; r < a.num_reqs; r += kSelThreads)
      if (const int bad = request_errors(a, r)) atomicOr(a.err, bad);
  const Row x = find_row(a, row);
  if (x.r < 0) {
    if (tid == 0 && g == 0) a.sel_lens[row] = 0;
    return;
  }
  const int n = x.n, taken = min(n, a.budget);
  int32_t* out = a.sel_table + (row * a.hkv + g) * (int64_t)a.budget;
  const int32_t* bt = a.bt + (int64_t)x.r * a.bt_width;
  if (tid == 0 && g == 0) a.sel_lens[row] = (taken - 1) * kBlockSize + x.pos % kBlockSize + 1;
  for (int i = taken + tid; i < a.budget; i += kSelThreads) out[i] = -1;
  if (n <= a.budget) {
    for (int i = tid; i < n; i += kSelThreads) out[i] = __ldg(bt + i);
    return;
  }
  const int first = a.first, mid = n - a.first - a.last, k = a.budget - a.first - a.last;
  int ties = 0;  // of the pages in state kTie, the first `ties` are taken
  if (k > 0) {
    const float* sc = a.scores + (int64_t)rh * a.bt_width + first;
    for (int i = tid; i < mid; i += kSelThreads) keys[i] = ordered(__ldcg(sc + i));
    // eps
    const uint16_t* q = a.q + row * a.q_stride + (int64_t)g * G * kHeadSize;
    float m = 0.f, s = 0.f;
    const int chunks = (n - a.last + a.chunk_pages - 1) / a.chunk_pages;
    for (int i = tid; i < chunks; i += kSelThreads)
      m = fmaxf(m, __ldcg(a.largest + (int64_t)rh * a.largest_stride + i));
    for (int i = tid; i < G * kHeadSize / 2; i += kSelThreads) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q) + i);
      s += fabsf(lo16(w)) + fabsf(hi16(w));
    }
    for (int o = 16; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    __shared__ float s_sum[kSelThreads / 32];
    if (lane == 0) {
      s_max[warp] = m;
      s_sum[warp] = s;
    }
    __syncthreads();
    m = s = 0.f;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      m = fmaxf(m, s_max[w]);
      s += s_sum[w];
    }
    // (a little more than (G + 16) 2^-24, for the roundings of S itself, and what
    // products below fp32's range lose)
    const float eps = (float)(G + 18) * 0x1p-24f * s * m + 0x1p-140f;
    const uint32_t t = kth_largest<uint32_t>(mid, k, part, [&](int i) { return keys[i]; });
    const float tf = unordered(t);
    const float above = tf + 2.f * eps, below = tf - 2.f * eps;
    int in = 0, cand = 0;
    __syncthreads();
    for (int i = tid; i < mid; i += kSelThreads) {
      const float e = unordered(keys[i]);
      const uint32_t st = e > above ? kIn : e < below ? kOut : kTie;
      in += st == kIn;
      cand += st == kTie;
      keys[i] = st;
    }
    in = block_sum(in, part);
    cand = block_sum(cand, part);
    ties = k - in;
    if (cand > ties && s != 0.f && m != 0.f) {  // (else every score is zero, exactly)
      // more pages about the border than places: their scores in 64 bits
      double* s64 = a.exact + (int64_t)rh * a.bt_width;
      int32_t* idx = a.index + (int64_t)rh * a.bt_width;
      int at = 0;
      for (int b = 0; b < mid; b += kSelThreads) {  // their indices, in order
        const int i = b + tid;
        const bool c = i < mid && keys[i] == kTie;
        const uint32_t bal = __ballot_sync(0xffffffffu, c);
        __syncthreads();
        if (lane == 0) part[warp] = __popc(bal);
        __syncthreads();
        int before = at, all = at;
        for (int w = 0; w < kSelThreads / 32; ++w) {
          if (w < warp) before += part[w];
          all += part[w];
        }
        if (c) idx[before + __popc(bal & ((1u << lane) - 1))] = i;
        at = all;
      }
      __syncthreads();
      double up[4] = {}, dn[4] = {};
      for (int h = 0; h < G; ++h) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(q + h * kHeadSize + lane * 4));
        const float v[4] = {lo16(w.x), hi16(w.x), lo16(w.y), hi16(w.y)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          up[i] += fmaxf(v[i], 0.f);
          dn[i] += fminf(v[i], 0.f);
        }
      }
      for (int c = warp; c < cand; c += kSelThreads / 32) {
        const int id = __ldg(bt + first + idx[c]);
        const int64_t blk = id < 0 || (int64_t)id >= a.num_blocks ? 0 : id;
        const uint16_t* p = a.bounds + (blk * a.hkv + g) * 2 * kHeadSize + lane * 4;
        const uint2 lo = __ldg(reinterpret_cast<const uint2*>(p));
        const uint2 hi = __ldg(reinterpret_cast<const uint2*>(p + kHeadSize));
        double s = up[0] * lo16(hi.x) + up[1] * hi16(hi.x) + up[2] * lo16(hi.y) + up[3] * hi16(hi.y);
        s += dn[0] * lo16(lo.x) + dn[1] * hi16(lo.x) + dn[2] * lo16(lo.y) + dn[3] * hi16(lo.y);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) s64[c] = s + 0.0;  // (-0 as 0)
      }
      __syncthreads();
      const unsigned long long t64 = kth_largest<unsigned long long>(
          cand, ties, part, [&](int i) { return ordered64(s64[i]); });
      int more = 0;
      __syncthreads();
      for (int c = tid; c < cand; c += kSelThreads) {
        const unsigned long long v = ordered64(s64[c]);
        keys[idx[c]] = v > t64 ? kIn : v == t64 ? kTie : kOut;
        more += v > t64;
      }
      ties -= block_sum(more, part);
    }
    __syncthreads();
  }
  // the taken pages in their order
  int at = 0, tied = 0;
  for (int b = 0; b < n; b += kSelThreads) {
    const int i = b + tid, j = i - first;
    uint32_t st = kOut;
    if (i < n) st = j < 0 || j >= mid ? kIn : k > 0 ? keys[j] : kOut;
    const uint32_t bt_ = __ballot_sync(0xffffffffu, st == kTie);
    const uint32_t bi = __ballot_sync(0xffffffffu, st == kIn);
    __syncthreads();
    if (lane == 0) part[warp] = __popc(bt_) << 16 | __popc(bi);
    __syncthreads();
    int tb = tied, ib = 0, ta = tied, ia = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) {
        tb += part[w] >> 16;
        ib += part[w] & 0xFFFF;
      }
      ta += part[w] >> 16;
      ia += part[w] & 0xFFFF;
    }
    // ties before this page, and so how many of them are taken
    const uint32_t below = (1u << lane) - 1;
    const int t = tb + __popc(bt_ & below);
    const int place = at + ib + __popc(bi & below) + min(t, ties) - min(tied, ties);
    if (st == kIn || (st == kTie && t < ties)) out[place] = __ldg(bt + i);
    at += ia + min(ta, ties) - min(tied, ties);
    tied = ta;
  }
}

}  // namespace

cudaError_t launch_page_bounds(const uint16_t* kc, int64_t num_blocks, int hkv, uint16_t* bounds,
                               const int64_t* slots, int64_t n_tokens, int* err, int sms,
                               cudaStream_t st) {
  const bool many = n_tokens * hkv > (int64_t)sms * 64;  // more than the warps an SM holds
  const int64_t warps = (many ? (n_tokens + 7) / 8 : n_tokens) * hkv;
  const unsigned blocks = (unsigned)std::min<int64_t>((warps + 7) / 8, (int64_t)sms * 8);
  return launch_dependent(many ? page_bounds_kernel<8> : page_bounds_kernel<1>, dim3(blocks),
                          dim3(256), 0, st, kc, num_blocks * kBlockSize, hkv, bounds, slots,
                          n_tokens, err);
}

int select_chunk_pages(int64_t rows, int hkv, int64_t bt_width, int sms) {
  return rows * hkv * bt_width >= (int64_t)sms * 32 * 128 ? 128 : 32;
}

cudaError_t launch_page_scores(const SelectArgs& a, int64_t row0, int rows, int sms,
                               cudaStream_t st) {
  const int64_t chunks = (a.bt_width + a.chunk_pages - 1) / a.chunk_pages;
  const int64_t warps = (int64_t)rows * a.hkv * chunks;
  const unsigned blocks = (unsigned)std::min<int64_t>((warps + 7) / 8, (int64_t)sms * 8);
  return launch_dependent(a.chunk_pages == 128 ? page_scores_kernel<128> : page_scores_kernel<32>,
                          dim3(blocks), dim3(256), 0, st, a, row0, rows);
}

cudaError_t launch_select(const SelectArgs& a, int64_t row0, int rows, bool score,
                          cudaStream_t st) {
  static std::atomic<bool> attr[kMaxAttrDevices];
  if (cudaError_t e = smem_attr_once(select_pages_kernel, kMaxBtWidth * 4, attr)) return e;
  return launch_dependent(select_pages_kernel, dim3((unsigned)(rows * a.hkv)), dim3(kSelThreads),
                          score ? (size_t)a.bt_width * 4 : 0, st, a, row0);
}

}  // namespace pkv
