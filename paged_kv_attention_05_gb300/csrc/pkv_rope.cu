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
// exchange for the rotation.  Eight lanes share a head row, two vectors each:
// lane t holds the vectors with dimensions 8t.. of both halves (halves style)
// or dimensions 16t .. 16t + 15 (interleaved), so both members of every pair
// sit in one thread, and in both styles its pairs are i = 8t .. 8t + 7, one
// 32-byte piece of the table's cos and of its sin.  The only exchange is the
// three shuffles of the norm's sum of squares.
#include "pkv_internal.cuh"

#include <cuda_bf16.h>

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;

// Programmatic launch as in pkv_write.cu: wait for the kernel before this one
// before touching any memory, then let the next (the step plan) set up.
template <bool kInt8, bool kNorm, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int t = lane & 7, sub = lane >> 3;
  const int rows = a.hq + 2 * a.hkv;      // head rows of a token: q | k | v
  const int groups = (rows + 3) >> 2;     // four rows per warp step
  const int lanes_rot = a.rotary_dim >> 4;  // lanes of a row that hold pairs
  const bool rot = t < lanes_rot;
  // this lane's two 8-element vectors of a row
  int va, vb;
  if (kInterleaved) {
    va = 2 * t;
    vb = 2 * t + 1;
  } else {
    va = rot ? t : 2 * t;
    vb = rot ? t + lanes_rot : 2 * t + 1;
  }
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const int64_t units = a.n_tokens * groups;
  for (int64_t w = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; w < units;
       w += nwarps) {
    const int64_t tok = w / groups;
    const int row = (int)(w - tok * groups) * 4 + sub;
    const int64_t slot = __ldg(a.slots + tok);
    if (slot < 0) continue;  // padding token: nothing of it is read or written
    const int64_t pos = __ldg(a.positions + tok);
    if (slot >= a.num_slots || pos < 0 || pos >= a.max_positions) {
      if (row == 0 && t == 0)
        atomicOr(a.err, slot >= a.num_slots ? PKV_DEV_ERR_SLOT_RANGE : PKV_DEV_ERR_POSITION);
      continue;
    }
    if (row >= rows) continue;
    const bool is_q = row < a.hq, is_v = row >= a.hq + a.hkv;
    const int head = is_q ? row : (is_v ? row - a.hq - a.hkv : row - a.hq);
    const uint16_t* src = (is_q ? a.q + tok * a.q_stride
                                : (is_v ? a.v + tok * a.v_stride : a.k + tok * a.k_stride)) +
                          head * kHeadSize;
    // (plain loads: q_out may be q)
    const uint4 ra = *reinterpret_cast<const uint4*>(src + va * 8);
    const uint4 rb = *reinterpret_cast<const uint4*>(src + vb * 8);
    float x[16];
    {
      const uint32_t u[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
    if (kNorm) {
      const uint16_t* wt = is_q ? a.q_weight : (is_v ? nullptr : a.k_weight);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
      const unsigned m = 0xFFu << (lane & 24);  // the row's eight lanes (the others may be gone)
      ss += __shfl_xor_sync(m, ss, 1);
      ss += __shfl_xor_sync(m, ss, 2);
      ss += __shfl_xor_sync(m, ss, 4);
      if (wt) {
        const float r = rsqrtf(ss * (1.f / kHeadSize) + a.eps);
        const uint4 wa = __ldg(reinterpret_cast<const uint4*>(wt + va * 8));
        const uint4 wb = __ldg(reinterpret_cast<const uint4*>(wt + vb * 8));
        const uint32_t u[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[2 * i] *= r * (__uint_as_float(u[i] << 16) + a.weight_offset);
          x[2 * i + 1] *= r * (__uint_as_float(u[i] & 0xFFFF0000u) + a.weight_offset);
        }
      }
    }
    if (rot && !is_v) {
      const float* tr = a.table + pos * a.rotary_dim + 8 * t;
      float c[8], s[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(tr) + i);
        const float4 sv = __ldg(reinterpret_cast<const float4*>(tr + a.rotary_dim / 2) + i);
        c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
        s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : i + 8;
        const float xa = x[ia], xb = x[ib];
        x[ia] = xa * c[i] - xb * s[i];
        x[ib] = xb * c[i] + xa * s[i];
      }
    }
    if (kInt8 && !is_q) {
      const float sc = is_v ? a.v_scale : a.k_scale;
      int8_t* dst = (is_v ? static_cast<int8_t*>(a.vc) : static_cast<int8_t*>(a.kc)) +
                    (slot * a.hkv + head) * kHeadSize;
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float r = rintf(__fdiv_rn(x[4 * i + j], sc));
          r = (r == r) ? fminf(fmaxf(r, -127.f), 127.f) : 0.f;
          c[i] |= ((uint32_t)(int)r & 0xFFu) << (8 * j);
        }
      }
      *reinterpret_cast<uint2*>(dst + va * 8) = make_uint2(c[0], c[1]);
      *reinterpret_cast<uint2*>(dst + vb * 8) = make_uint2(c[2], c[3]);
    } else {
      uint16_t* dst = is_q ? a.q_out + tok * a.q_out_stride + head * kHeadSize
                           : (is_v ? static_cast<uint16_t*>(a.vc) : static_cast<uint16_t*>(a.kc)) +
                                 (slot * a.hkv + head) * kHeadSize;
      uint32_t u[8];
      if (is_v) {  // copied bit for bit
        u[0] = ra.x, u[1] = ra.y, u[2] = ra.z, u[3] = ra.w;
        u[4] = rb.x, u[5] = rb.y, u[6] = rb.z, u[7] = rb.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          u[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
      *reinterpret_cast<uint4*>(dst + va * 8) = make_uint4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<uint4*>(dst + vb * 8) = make_uint4(u[4], u[5], u[6], u[7]);
    }
  }
}

}  // namespace

cudaError_t launch_write_rope(const RopeArgs& a, bool int8, int sms, cudaStream_t st) {
  const int rows = a.hq + 2 * a.hkv;
  const int64_t units = a.n_tokens * ((rows + 3) / 4);  // a warp per four head rows
  constexpr int kWarps = kRopeThreads / 32;
  int64_t blocks = (units + kWarps - 1) / kWarps;
  const int64_t cap = (int64_t)sms * 8;
  if (blocks > cap) blocks = cap;
  const bool norm = a.q_weight != nullptr || a.k_weight != nullptr;
  void (*kernel)(RopeArgs) = nullptr;
  if (int8)
    kernel = norm ? (a.interleaved ? rope_write_kernel<true, true, true>
                                   : rope_write_kernel<true, true, false>)
                  : (a.interleaved ? rope_write_kernel<true, false, true>
                                   : rope_write_kernel<true, false, false>);
  else
    kernel = norm ? (a.interleaved ? rope_write_kernel<false, true, true>
                                   : rope_write_kernel<false, true, false>)
                  : (a.interleaved ? rope_write_kernel<false, false, true>
                                   : rope_write_kernel<false, false, false>);
  return launch_dependent(kernel, dim3((unsigned)blocks), dim3(kRopeThreads), 0, st, a);
}

}  // namespace pkv
