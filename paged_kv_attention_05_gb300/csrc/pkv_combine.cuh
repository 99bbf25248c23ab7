// The merge of split-KV decode results, run after the decode kernel: by every
// warp of the prefill kernel's launch at its end (bf16 calls), by the combine
// kernel (int8 calls).
#pragma once

#include "pkv_device.cuh"

namespace pkv {
namespace dev {

// What a warp reads of the plan for the merge: the header's counts and its
// first pair.  (The plan's lists are read through L2: the plan kernel ran two
// launches before this one.)
struct CombineStart {
  int max_rows, n_items;
  SplitPair first;
};
__device__ __forceinline__ SplitPair load_pair(const Workspace& ws, int i) {
  const int4 w0 = __ldcg(reinterpret_cast<const int4*>(ws.pairs + i));
  const int4 w1 = __ldcg(reinterpret_cast<const int4*>(ws.pairs + i) + 1);
  return SplitPair{w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
}
__device__ __forceinline__ CombineStart combine_start(const Workspace& ws, int warp_id) {
  CombineStart s{};
  s.max_rows = __ldcg(&ws.hdr->max_rows);
  s.n_items = __ldcg(&ws.hdr->n_pairs) * s.max_rows;
  if (warp_id < s.n_items) s.first = load_pair(ws, warp_id / s.max_rows);
  return s;
}
// Merge of split results: one (split pair, query row) per warp (warp_id of
// n_warps in the grid), four output columns per lane, the splits merged in
// one pass with the online-softmax identity the decode loop uses between
// pages (a running max M; the sum and the output so far are scaled by
// exp2(M_old - M_new) when it grows).  Any split of a request of several tokens
// may hold no key of a row, the first one too: a plain row's later splits lie past
// its position, and a scored call's units begin at the window of the request's
// first row, before the windows of the others.  Such a split has m = -inf (or, with
// the fixed reference, m = 0 and a sum of zero) and contributes nothing; M stays
// -inf, and its factor zero, until a split that has a key.  Rows are (query token,
// head in group); pairs with fewer rows than the largest skip the rest.
__device__ __forceinline__ void combine_splits(const AttnArgs& a, const Workspace& ws, int warp_id,
                                               int n_warps, const CombineStart& start) {
  const int G = a.hq / a.hkv;
  const int max_rows = start.max_rows, n_items = start.n_items;
  const int lane = threadIdx.x & 31;
  for (int item = warp_id; item < n_items; item += n_warps) {
    const SplitPair sp = item == warp_id ? start.first : load_pair(ws, item / max_rows);
    const int row = item % max_rows;
    const int q0 = sp.q0;
    const int rows = sp.qn * G;
    if (row >= rows) continue;
    const float* ml = ws.part_ml + ((int64_t)sp.first + row) * 2;
    const float* po = ws.part_o + ((int64_t)sp.first + row) * kHeadSize + 4 * lane;
    float M = -INFINITY, lsum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < sp.nsplit; ++s) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(ml + (int64_t)s * rows * 2));
      const float4 o = __ldcg(reinterpret_cast<const float4*>(po + (int64_t)s * rows * kHeadSize));
      const float Mn = fmaxf(M, v.x);
      const float fo = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
      const float fn = v.x == -INFINITY ? 0.f : fast_exp2(v.x - Mn);
      lsum = lsum * fo + v.y * fn;
      acc.x = acc.x * fo + o.x * fn;
      acc.y = acc.y * fo + o.y * fn;
      acc.z = acc.z * fo + o.z * fn;
      acc.w = acc.w * fo + o.w * fn;
      M = Mn;
    }
    const float inv = 1.f / lsum;
    uint16_t* orow = a.out + (int64_t)(q0 + row / G) * a.out_stride +
                     (int64_t)(sp.g * G + row % G) * kHeadSize + 4 * lane;
    *reinterpret_cast<uint2*>(orow) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
}
__device__ __forceinline__ void combine_splits(const AttnArgs& a, const Workspace& ws, int warp_id,
                                               int n_warps) {
  combine_splits(a, ws, warp_id, n_warps, combine_start(ws, warp_id));
}

}  // namespace dev
}  // namespace pkv
