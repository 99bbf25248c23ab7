// The cache write with the position rotation on the way: a token's query and
// key head rows are (optionally) RMS-normalised and rotated by the angles of
// the token's position, the queries go to q_out, the keys and the unchanged
// values into the paged cache (bf16, or int8 codes).
//
// Mathematics, for a head row x of 128 values and a token at position p:
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset)        (with a weight w only)
//   pairs (a, b) = (i, i + half) or, interleaved, (2i, 2i + 1), i < half:
//     y_a' = y_a cos(p, i) - y_b sin(p, i)
//     y_b' = y_b cos(p, i) + y_a sin(p, i)
// half = rotary_dim / 2; dimensions >= rotary_dim pass unrotated.  Everything
// is fp32 from the bf16 input to the one rounding at the end (bf16, or the
// int8 code).  cos and sin come from a caller's fp32 table, whose angles it
// can form in 64 bits (a position of 10^5 times a frequency loses its
// fraction in fp32).
//
// GB300 layout of the work: pure HBM traffic (each row is read once and
// written once), so the layout keeps whole 16-byte vectors per thread and no
// exchange for the rotation.  Eight lanes share a head row, two vectors each,
// both members of every pair in one thread: lane t holds vectors t and t + 8
// (interleaved, whose pairs lie inside a vector), or the vectors with
// dimensions 8t .. 8t + 7 of both halves (halves style).  The only exchange is
// the three shuffles of the norm's sum of squares.
#include <cuda_bf16.h>

#include <algorithm>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;

// Four codes clamp(rne(x / scale), -127, 127) (0 for a NaN) as bytes.  The
// quotient is the IEEE one: q = x * r with r the rounded 1 / scale, then one
// correction by the exact remainder (Markstein's division).  Clamping x to
// +-127 scale first gives the same code and keeps q in range; adding 1.5 * 2^23
// rounds q to an integer whose code is the sum's lowest byte.  Nine operations
// a code, where division, rintf and conversion take twenty.  r = 0: a scale so
// small or large that r or the remainder could lose bits; divided.
__device__ __forceinline__ uint32_t codes4(const float* x, float scale, float r) {
  uint32_t b[4];
  if (r > 0.f) {
    const float lim = 127.f * scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float xc = fminf(fmaxf(x[i], -lim), lim);
      const float q = xc * r;
      const float c = fmaf(fmaf(-q, scale, xc), r, q) + 12582912.f;
      b[i] = x[i] == x[i] ? __float_as_uint(c) : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float q = rintf(__fdiv_rn(x[i], scale));
      b[i] = q == q ? (uint32_t)(int)fminf(fmaxf(q, -127.f), 127.f) : 0u;
    }
  }
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// A lane's two 8-element vectors of a row, whether each is rotated, and where
// the table has the four pairs of each (from cos; sin half a row further).
struct Lane {
  int va, vb, ta, tb;
  bool ra, rb;
};
template <bool kInterleaved>
__device__ __forceinline__ Lane lane_of(int t, int rotary_dim) {
  Lane l;
  if (kInterleaved) {
    l.va = t;
    l.vb = t + 8;
    l.ra = 8 * l.va < rotary_dim;
    l.rb = 8 * l.vb < rotary_dim;
    l.ta = 4 * l.va;
    l.tb = 4 * l.vb;
  } else {
    const int lanes_rot = rotary_dim >> 4;  // lanes that hold pairs; the others the rest
    l.ra = l.rb = t < lanes_rot;
    l.va = l.ra ? t : 2 * t;
    l.vb = l.ra ? t + lanes_rot : 2 * t + 1;
    l.ta = 8 * t;
    l.tb = 8 * t + 4;
  }
  return l;
}
// cos and sin of the lane's eight pairs from its token's table row
__device__ __forceinline__ void lane_angles(const float* row, int rotary_dim, const Lane& ln,
                                            float (&c)[8], float (&sn)[8]) {
  auto load4 = [&](int at, int i) {
    const float4 cv = *reinterpret_cast<const float4*>(row + at);
    const float4 sv = *reinterpret_cast<const float4*>(row + rotary_dim / 2 + at);
    c[i] = cv.x, c[i + 1] = cv.y, c[i + 2] = cv.z, c[i + 3] = cv.w;
    sn[i] = sv.x, sn[i + 1] = sv.y, sn[i + 2] = sv.z, sn[i + 3] = sv.w;
  };
  if (ln.ra) load4(ln.ta, 0);
  if (ln.rb) load4(ln.tb, 4);
}

// What a lane does to its two vectors (raw bf16: u) of head row `row` of a
// token: norm, rotation, rounding, store.  c, sn: its eight pairs' cos and sin;
// wt: its sixteen values of the two norm weights.
struct RowWeights {
  uint4 q[2], k[2];
};
template <bool kInt8, bool kNorm, bool kInterleaved>
__device__ __forceinline__ void rope_row(const RopeArgs& a, int64_t tok, int64_t slot, int row,
                                         uint32_t (&u)[8], const float (&c)[8],
                                         const float (&sn)[8], const Lane& ln,
                                         const RowWeights& wt) {
  const bool is_q = row < a.hq, is_v = row >= a.hq + a.hkv;
  const int head = is_q ? row : (is_v ? row - a.hq - a.hkv : row - a.hq);
  if (!is_v || kInt8) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    if (kNorm && !is_v && (is_q ? a.q_weight : a.k_weight) != nullptr) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s0 = fmaf(x[2 * i], x[2 * i], s0);
        s1 = fmaf(x[2 * i + 1], x[2 * i + 1], s1);
      }
      float ss = s0 + s1;
      const unsigned m = 0xFFu << (threadIdx.x & 24);  // the row's eight lanes
      ss += __shfl_xor_sync(m, ss, 1);
      ss += __shfl_xor_sync(m, ss, 2);
      ss += __shfl_xor_sync(m, ss, 4);
      const float r = rsqrtf(ss * (1.f / kHeadSize) + a.eps);
      const uint4 wa = is_q ? wt.q[0] : wt.k[0], wb = is_q ? wt.q[1] : wt.k[1];
      const uint32_t ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] *= r * (__uint_as_float(ww[i] << 16) + a.weight_offset);
        x[2 * i + 1] *= r * (__uint_as_float(ww[i] & 0xFFFF0000u) + a.weight_offset);
      }
    }
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : i + 8;
        const float xa = x[ia], xb = x[ib];
        if (i < 4 ? ln.ra : ln.rb) {
          x[ia] = xa * c[i] - xb * sn[i];
          x[ib] = xb * c[i] + xa * sn[i];
        }
      }
    }
    if (kInt8 && !is_q) {
      const float sc = is_v ? a.v_scale : a.k_scale, r = is_v ? a.v_rcp : a.k_rcp;
      int8_t* dst = (is_v ? static_cast<int8_t*>(a.vc) : static_cast<int8_t*>(a.kc)) +
                    (slot * a.hkv + head) * kHeadSize;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = codes4(x + 4 * i, sc, r);
      *reinterpret_cast<uint2*>(dst + ln.va * 8) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(dst + ln.vb * 8) = make_uint2(w[2], w[3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  // (bf16 values are copied bit for bit)
  uint16_t* dst = is_q ? a.q_out + tok * a.q_out_stride + head * kHeadSize
                       : (is_v ? static_cast<uint16_t*>(a.vc) : static_cast<uint16_t*>(a.kc)) +
                             (slot * a.hkv + head) * kHeadSize;
  *reinterpret_cast<uint4*>(dst + ln.va * 8) = make_uint4(u[0], u[1], u[2], u[3]);
  *reinterpret_cast<uint4*>(dst + ln.vb * 8) = make_uint4(u[4], u[5], u[6], u[7]);
}

__device__ __forceinline__ const uint16_t* row_source(const RopeArgs& a, int64_t tok, int row) {
  return row < a.hq          ? a.q + tok * a.q_stride + row * kHeadSize
         : row < a.hq + a.hkv ? a.k + tok * a.k_stride + (row - a.hq) * kHeadSize
                             : a.v + tok * a.v_stride + (row - a.hq - a.hkv) * kHeadSize;
}
template <bool kNorm>
__device__ __forceinline__ RowWeights row_weights(const RopeArgs& a, const Lane& ln) {
  RowWeights w{};
  if (kNorm && a.q_weight) {
    w.q[0] = __ldg(reinterpret_cast<const uint4*>(a.q_weight + ln.va * 8));
    w.q[1] = __ldg(reinterpret_cast<const uint4*>(a.q_weight + ln.vb * 8));
  }
  if (kNorm && a.k_weight) {
    w.k[0] = __ldg(reinterpret_cast<const uint4*>(a.k_weight + ln.va * 8));
    w.k[1] = __ldg(reinterpret_cast<const uint4*>(a.k_weight + ln.vb * 8));
  }
  return w;
}
// Whether the token at (slot, pos) is written; reports a bad one (once: the
// lane that says so).
__device__ __forceinline__ bool token_ok(const RopeArgs& a, int64_t slot, int64_t pos,
                                         bool reports) {
  if (slot < 0) return false;  // padding: nothing of it is read or written
  if (slot < a.num_slots && pos >= 0 && pos < a.max_positions) return true;
  if (reports)
    atomicOr(a.err, slot >= a.num_slots ? PKV_DEV_ERR_SLOT_RANGE : PKV_DEV_ERR_POSITION);
  return false;
}

// Steps of few tokens: four rows a warp, straight through (plain loads: q_out
// may be q).  Programmatic launch as in pkv_write.cu: wait for the kernel
// before this one before touching any memory, then let the next (the step
// plan) set up.
template <bool kInt8, bool kNorm, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, t = lane & 7;
  const int rows = a.hq + 2 * a.hkv;  // head rows of a token: q | k | v
  const int per_token = (rows + 3) >> 2;
  const Lane ln = lane_of<kInterleaved>(t, a.rotary_dim);
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const int64_t units = a.n_tokens * per_token;
  for (int64_t w = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; w < units;
       w += nwarps) {
    const int64_t tok = w / per_token;
    const int row = (int)(w - tok * per_token) * 4 + (lane >> 3);
    const int64_t slot = __ldg(a.slots + tok), pos = slot >= 0 ? __ldg(a.positions + tok) : 0;
    if (!token_ok(a, slot, pos, row == 0 && t == 0) || row >= rows) continue;
    const uint16_t* src = row_source(a, tok, row);
    const uint4 va = *reinterpret_cast<const uint4*>(src + ln.va * 8);
    const uint4 vb = *reinterpret_cast<const uint4*>(src + ln.vb * 8);
    const RowWeights wt = row_weights<kNorm>(a, ln);
    float c[8] = {}, sn[8] = {};
    if (row < a.hq + a.hkv)
      lane_angles(a.table + pos * a.rotary_dim, a.rotary_dim, ln, c, sn);
    uint32_t u[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
    rope_row<kInt8, kNorm, kInterleaved>(a, tok, slot, row, u, c, sn, ln, wt);
  }
}

// Larger steps: a warp takes a unit of 4 * kRopeGroups rows of a token at a
// time and copies the rows and the table entry of the units ahead into shared
// memory (cp.async, its own ring of kRopeStages) while it works on the present
// one, so that it keeps bytes in flight whatever its arithmetic takes; the slot
// of the unit after those, which says whether there is anything to copy and a
// position to load, is asked for a step earlier still.
constexpr int kRopeGroups = 4;   // of four rows
constexpr int kRopeStages = 3;
constexpr int kRopeCtas = 2;     // an SM
constexpr int kRopeTable = kRopeGroups * 1024;    // stage: rows | cos, sin | slot
constexpr int kRopeSlot = kRopeTable + 512;
constexpr int kRopeStage = kRopeSlot + 16;
constexpr int kRopeSmem = kRopeThreads / 32 * kRopeStages * kRopeStage;
static_assert(kRopeCtas * (kRopeSmem + 1024) <= 228 * 1024, "shared memory of an SM");

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

template <bool kInt8, bool kNorm, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_stream_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, t = lane & 7, sub = lane >> 3;
  const int rows = a.hq + 2 * a.hkv;
  const uint32_t per_token = (uint32_t)(rows + 4 * kRopeGroups - 1) / (4 * kRopeGroups);
  const Lane ln = lane_of<kInterleaved>(t, a.rotary_dim);
  const RowWeights wt = row_weights<kNorm>(a, ln);
  uint8_t* ring = smem + (threadIdx.x >> 5) * kRopeStages * kRopeStage;
  const uint32_t ring32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t nwarps = (gridDim.x * blockDim.x) >> 5;
  const uint32_t units = (uint32_t)a.n_tokens * per_token;  // (the launcher: below 2^30)

  int64_t slot_raw = -1;  // of unit `ahead`, used a step after it is asked for
  auto ask = [&](uint32_t w) { slot_raw = w < units ? __ldg(a.slots + w / per_token) : -1; };
  // copies unit w into a stage, by its raw slot; its position comes while the rows
  // are asked for
  auto fetch = [&](uint32_t w, int stage) {
    const uint32_t tok = w / per_token;
    const int row0 = (int)(w - tok * per_token) * 4 * kRopeGroups + sub;
    const int64_t pos = slot_raw >= 0 ? __ldg(a.positions + tok) : 0;
    const uint32_t dst = ring32 + stage * kRopeStage + lane * 16;
    if (slot_raw >= 0) {
#pragma unroll
      for (int g = 0; g < kRopeGroups; ++g) {
        const int row = row0 + 4 * g;
        if (row < rows) {
          const uint16_t* src = row_source(a, tok, row);
          copy16(dst + g * 1024, src + ln.va * 8);
          copy16(dst + g * 1024 + 512, src + ln.vb * 8);
        }
      }
    }
    const bool ok = token_ok(a, slot_raw, pos, row0 == 0 && t == 0);
    if (lane == 0)
      *reinterpret_cast<int64_t*>(ring + stage * kRopeStage + kRopeSlot) = ok ? slot_raw : -1;
    if (ok && lane * 4 < a.rotary_dim)
      copy16(dst + kRopeTable, a.table + pos * a.rotary_dim + lane * 4);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };

  uint32_t w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, ahead = w;
#pragma unroll
  for (int s = 0; s < kRopeStages - 1; ++s, ahead += nwarps) {
    ask(ahead);
    fetch(ahead, s);
  }
  ask(ahead);
  for (int stage = 0; w < units; w += nwarps) {
    int to = stage + kRopeStages - 1;
    if (to >= kRopeStages) to -= kRopeStages;
    fetch(ahead, to);
    ask(ahead += nwarps);
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kRopeStages - 1) : "memory");
    __syncwarp();  // (the table entry and the slot came from other lanes)
    const uint8_t* st = ring + stage * kRopeStage;
    const int64_t slot = *reinterpret_cast<const int64_t*>(st + kRopeSlot);
    if (slot >= 0) {
      const uint32_t tok = w / per_token;
      const int row0 = (int)(w - tok * per_token) * 4 * kRopeGroups + sub;
      float c[8] = {}, sn[8] = {};
      lane_angles(reinterpret_cast<const float*>(st + kRopeTable), a.rotary_dim, ln, c, sn);
#pragma unroll 1
      for (int g = 0; g < kRopeGroups; ++g) {
        const int row = row0 + 4 * g;
        if (row >= rows) break;  // (the row's eight lanes together)
        const uint4 va = *reinterpret_cast<const uint4*>(st + g * 1024 + lane * 16);
        const uint4 vb = *reinterpret_cast<const uint4*>(st + g * 1024 + 512 + lane * 16);
        uint32_t u[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
        rope_row<kInt8, kNorm, kInterleaved>(a, tok, slot, row, u, c, sn, ln, wt);
      }
    }
    __syncwarp();  // (the stage is refilled next)
    if (++stage == kRopeStages) stage = 0;
  }
}

template <bool kInt8, bool kNorm, bool kInterleaved>
cudaError_t launch_rope_as(const RopeArgs& a, int sms, cudaStream_t st) {
  constexpr int kWarps = kRopeThreads / 32;
  const int rows = a.hq + 2 * a.hkv;
  const int64_t streamed = a.n_tokens * ((rows + 4 * kRopeGroups - 1) / (4 * kRopeGroups));
  // The streaming form from ten units an SM (sixteen warps are resident); a
  // step of fewer tokens is spread over four times the warps instead.  Measured
  // at 6, 10, 14, 30 and 120 units an SM (straight, streamed; us a call by
  // events, with the rows out of the caches):
  //   64 / 8 heads, norms:  10.7 10.7 | 12.5 10.4 | 14.6 10.7 | 20.6 14.5 | 51.7 33.2
  //   32 / 8, no norms:      8.7  8.7 | 12.4 10.7 | 12.8 10.7 | 16.5 14.5 | 41.4 31.2
  //   32 / 32, int8:         8.7 10.8 | 12.4 12.4 | 12.8 12.8 | 16.6 16.5 | 41.8 33.3
  //   12 / 4, int8, norms:   8.7 10.8 | 12.8 10.8 | 12.5 11.1 | 16.5 14.8 | 38.9 31.9
  //   8 / 1, norms:          8.7 10.7 | 10.8 10.7 | 12.4 11.0 | 16.5 14.8 | 43.5 31.2
  //   2 / 1, norms:          8.7  8.7 |  9.0  8.7 | 10.7  9.0 | 12.4 12.7 | 25.1 25.0
  // With the rows in L2 either is up to a quarter ahead between 10 and 30 units
  // (streamed with norms, 10.7 8.4 at 30; straight with int8, 6.9 8.5 at 20), and
  // straight is ahead up to 120 for the few rows of a 2 / 1 token, which fill a
  // quarter of a unit (14.3 16.6).
  if (streamed >= (int64_t)sms * 10 && streamed < (1LL << 30)) {
    static std::atomic<bool> attr[kMaxAttrDevices];
    auto* kernel = rope_stream_kernel<kInt8, kNorm, kInterleaved>;
    if (cudaError_t e = smem_attr_once(kernel, kRopeSmem, attr)) return e;
    return launch_dependent(kernel, dim3((unsigned)(sms * kRopeCtas)), dim3(kRopeThreads),
                            kRopeSmem, st, a);
  }
  const int64_t units = a.n_tokens * ((rows + 3) / 4);
  const int64_t blocks = std::min<int64_t>((units + kWarps - 1) / kWarps, (int64_t)sms * 8);
  return launch_dependent(rope_write_kernel<kInt8, kNorm, kInterleaved>, dim3((unsigned)blocks),
                          dim3(kRopeThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_write_rope(const RopeArgs& args, bool int8, int sms, cudaStream_t st) {
  RopeArgs a = args;
  auto rcp = [](float s) { return s >= 0x1p-60f && s <= 0x1p60f ? 1.f / s : 0.f; };
  a.k_rcp = rcp(a.k_scale);
  a.v_rcp = rcp(a.v_scale);
  const bool norm = a.q_weight != nullptr || a.k_weight != nullptr;
  if (int8) {
    if (norm)
      return a.interleaved ? launch_rope_as<true, true, true>(a, sms, st)
                           : launch_rope_as<true, true, false>(a, sms, st);
    return a.interleaved ? launch_rope_as<true, false, true>(a, sms, st)
                         : launch_rope_as<true, false, false>(a, sms, st);
  }
  if (norm)
    return a.interleaved ? launch_rope_as<false, true, true>(a, sms, st)
                         : launch_rope_as<false, true, false>(a, sms, st);
  return a.interleaved ? launch_rope_as<false, false, true>(a, sms, st)
                       : launch_rope_as<false, false, false>(a, sms, st);
}

}  // namespace pkv
