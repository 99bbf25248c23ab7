// What the decode kernels of bf16 and 4-bit caches read of the plan: their units,
// and how many SMs they leave to the prefill kernel that runs beside them.
#pragma once

#include "pkv_device.cuh"
#include "pkv_score.cuh"

namespace pkv {
namespace dev {

// How many SMs are left to the prefill grid, launched after this one as its
// programmatic dependent: when the step has prefill items, the first P CTAs
// of the decode grid exit at once, so that the prefill items run on their SMs
// beside the decode units on the others (the prefill kernel does not wait for
// this grid before its items).  P is the number of SMs on
// which the prefill's key-tile steps (items x tiles) fit into the longest
// item's chain, at most one per item and half of the SMs: fewer would
// lengthen the prefill, more would take SMs the decode units need and sit
// idle once the items are done.  When the decode units fill fewer CTAs than
// the grid has (units_per_cta at a time each), the spare SMs would idle
// anyway: P then grows up to one per item (still at most half of the SMs; the
// single-head items of a scored call take an SM each, see single_head_items).
// A scored call leaves fewer where its decodes take so long that the prefill
// ends in their time all the same (kTilesPerStep: decode tiles of 128 keys, 64
// KB, that all SMs read in the 3 us of a prefill step; a step of scores past half
// of a cap takes 4.5).  128 decodes of up to 4096 keys beside a prompt of 1000
// tokens, 100 of up to 3000 beside two chunks of 700, and 256 of up to 2048
// beside one of 2000 (us; 213, 320 and 480 tiles a step):
//   cap 50, scores of rms 3  198 185 186 | 143 147 162 | 272 259 268
//   cap 50, scores of rms 8  210 190 187 | 161 147 164 | 299 259 269
//   bias                     199 186 188 | 146 150 173 | 272 262 277
//   window of 1024            93  97 108 |  92 104 103 | 194 185 205
// Every CTA computes the same from the plan header (read after the plan
// wait): P, 0 without prefill items.
constexpr int kTilesPerStep = 320;
template <bool kScored, bool kSingle = kScored>  // kSingle: items may be single heads
__device__ __forceinline__ int sms_to_prefill(const AttnArgs& a, const Workspace& ws,
                                              int units_per_cta) {
  const int G = a.hq / a.hkv;
  const bool single = kSingle && single_head_items(a, ws.hdr->n_pre_entries, gridDim.x);
  const int per_entry = G % 2 == 0 && !single ? a.hq / 2 : a.hq;  // items per entry
  const int items = ws.hdr->n_pre_entries * per_entry;
  if (items == 0) return 0;
  const long long steps = (long long)ws.hdr->pre_tiles * per_entry;
  const int longest = max(ws.hdr->pre_max_tiles, 1);
  const int cap = single ? items : min(items, (int)gridDim.x / 2);
  int p = (int)min((long long)cap, (steps + longest - 1) / longest);
  const int spare = (int)gridDim.x - (ws.hdr->n_dec_units + units_per_cta - 1) / units_per_cta;
  if (spare > p) {
    p = min(cap, spare);
  } else if (kScored) {
    const int room = ws.hdr->dec_tiles / kTilesPerStep - longest;
    if (room > 0) p = min(p, (int)((steps + room - 1) / room));
  }
  return max(p, 1);
}
__device__ __forceinline__ bool leaves_sm_to_prefill(const AttnArgs& a, const Workspace& ws,
                                                     int units_per_cta) {
  return (int)blockIdx.x < sms_to_prefill<false>(a, ws, units_per_cta);
}

// a work unit written by the plan kernel
__device__ __forceinline__ DecUnit load_unit(const DecUnit* p) {
  const int4 w0 = __ldcg(reinterpret_cast<const int4*>(p));
  const int4 w1 = __ldcg(reinterpret_cast<const int4*>(p) + 1);
  return DecUnit{w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
}

}  // namespace dev
}  // namespace pkv
