// The cache of 4-bit codes: its write, and the read back into bf16 rows.
//
// A page of one KV head is one record of 2176 consecutive bytes (kPage4), so
// that the attention kernels fetch a page of keys, values and their scales in one
// bulk copy of whole 128-byte lines:
//   [0, 1024)     key codes: slot s at 64 s, 128 codes of 4 bits
//   [1024, 2048)  value codes
//   [2048, 2112)  keys: (scale, zero) of slot s, two bf16, at 4 s
//   [2112, 2176)  values: the same
// Word i (32 bits) of a row holds dimensions 8 i .. 8 i + 7, dimension 8 i + 2 a + b
// in bits 4 a + 16 b: one mask of a word (shifted by 0, 4, 8 or 12) gives two
// neighbouring dimensions in the two halves of a register, which is how every
// consumer takes them (fp16 pairs of an MMA operand, bf16 pairs of a row).
//
// Mathematics, for a head row x of 128 bf16 values (NaN counts as 0, |x| is
// clamped to 2^126): z = min x, w = max x - z, s = w / 15 rounded to bf16 (0
// for w < 2^-36), code = rne((x - z) / s), value = s * code + z.  z is one of the
// row's values, so that it is exact in bf16; the code is formed against the
// rounded s and z, so that their rounding adds nothing to a value's error of half
// a step (s is off by 2^-9 of itself at most: the largest code is 15.03 at most,
// which rounds to 15).  (x - z) / s is the IEEE quotient: halves of a step are
// exact there (x - z and s have few bits) and go to the even code.
//
// Pure HBM traffic: 512 bytes read and 136 written per token and KV head, or the
// reverse.  A half-warp takes a key row, the other the value row: 8 values, one
// code word a lane; the row's minimum and maximum are four shuffles.  kRows
// heads a warp, all loads before the first use.
#include "pkv_int4.cuh"

namespace pkv {
namespace {

constexpr int kThreads4 = 256;
constexpr int kRows = 4;  // heads of a token that a warp takes at once

// 8 bf16 values of a row (the other lanes of the half-warp hold the rest) to their
// code word; *pair = the row's (scale, zero).
__device__ __forceinline__ uint32_t quantise8(const uint4& raw, uint32_t* pair) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    big = max(big, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  }
  if (big > 0x7E80u) {  // some |x| > 2^126, or a NaN
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -0x1p126f), 0x1p126f) : 0.f;
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float spread = hi - lo;
  const float s = spread < 0x1p-36f ? 0.f : __bfloat162float(__float2bfloat16_rn(__fdiv_rn(spread, 15.f)));
  *pair = __float_as_uint(s) >> 16 | (__float_as_uint(lo) & 0xFFFF0000u);
  if (s == 0.f) return 0u;
  // the IEEE quotient by the rounded reciprocal and one exact remainder
  // (Markstein's division; s is between 2^-41 and 2^124); adding 2^23 rounds it
  // to an integer in the sum's low bits
  const float r = __frcp_rn(s);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = x[i] - lo, q = d * r;
    const uint32_t c = __float_as_uint(fmaf(fmaf(-q, s, d), r, q) + 8388608.f) & 15u;
    word |= c << (4 * (i >> 1) + 16 * (i & 1));
  }
  return word;
}

__global__ void __launch_bounds__(kThreads4)
    write_int4_kernel(const uint16_t* __restrict__ k, int64_t k_stride,
                      const uint16_t* __restrict__ v, int64_t v_stride, uint8_t* __restrict__ cache,
                      int64_t num_slots, int hkv, const int64_t* __restrict__ slots,
                      int64_t n_tokens, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, l = lane & 15, side = lane >> 4;
  const int groups = (hkv + kRows - 1) / kRows;
  const int64_t units = n_tokens * groups, nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t u = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; u < units; u += nwarps) {
    const int64_t t = u / groups;
    const int h0 = (int)(u - t * groups) * kRows;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) continue;  // padding token
    if (slot >= num_slots) {
      if (lane == 0 && h0 == 0) atomicOr(err, PKV_DEV_ERR_SLOT_RANGE);
      continue;
    }
    const uint16_t* src = (side ? v + t * v_stride : k + t * k_stride) + h0 * kHeadSize + l * 8;
    uint4 raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      raw[i] = h0 + i < hkv ? __ldg(reinterpret_cast<const uint4*>(src + i * kHeadSize))
                            : make_uint4(0, 0, 0, 0);
    const int off = (int)(slot % kBlockSize);
    uint8_t* page = cache + ((slot / kBlockSize) * hkv + h0) * (int64_t)kPage4;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      uint32_t pair;
      const uint32_t word = quantise8(raw[i], &pair);
      if (h0 + i >= hkv) continue;
      uint8_t* p = page + i * kPage4;
      *reinterpret_cast<uint32_t*>(p + side * kSide4 + off * kRow4 + l * 4) = word;
      if (l == 0) *reinterpret_cast<uint32_t*>(p + kMeta4 + side * 64 + off * 4) = pair;
    }
  }
}

__global__ void __launch_bounds__(kThreads4)
    read_int4_kernel(const uint8_t* __restrict__ cache, int64_t num_slots, int hkv,
                     const int64_t* __restrict__ slots, int64_t n_tokens,
                     uint16_t* __restrict__ k_out, int64_t k_stride, uint16_t* __restrict__ v_out,
                     int64_t v_stride, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, l = lane & 15, side = lane >> 4;
  const int groups = (hkv + kRows - 1) / kRows;
  const int64_t units = n_tokens * groups, nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t u = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; u < units; u += nwarps) {
    const int64_t t = u / groups;
    const int h0 = (int)(u - t * groups) * kRows;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (lane == 0 && h0 == 0) atomicOr(err, PKV_DEV_ERR_SLOT_RANGE);
      continue;
    }
    const int off = (int)(slot % kBlockSize);
    const uint8_t* page = cache + ((slot / kBlockSize) * hkv + h0) * (int64_t)kPage4;
    uint32_t word[kRows], pair[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint8_t* p = page + (h0 + i < hkv ? i : 0) * kPage4;
      word[i] = __ldcg(reinterpret_cast<const uint32_t*>(p + side * kSide4 + off * kRow4 + l * 4));
      pair[i] = __ldcg(reinterpret_cast<const uint32_t*>(p + kMeta4 + side * 64 + off * 4));
    }
    uint16_t* dst = (side ? v_out + t * v_stride : k_out + t * k_stride) + h0 * kHeadSize + l * 8;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (h0 + i >= hkv) break;
      const float s = __uint_as_float(pair[i] << 16), z = __uint_as_float(pair[i] & 0xFFFF0000u);
      uint32_t o[4];
#pragma unroll
      for (int a = 0; a < 4; ++a)
        o[a] = dev::pack_bf16(fmaf((float)((word[i] >> (4 * a)) & 15u), s, z),
                              fmaf((float)((word[i] >> (4 * a + 16)) & 15u), s, z));
      *reinterpret_cast<uint4*>(dst + i * kHeadSize) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// a warp per token and kRows heads, at most 8 CTAs an SM
unsigned grid4(int64_t n_tokens, int hkv, int sms) {
  const int64_t warps = n_tokens * ((hkv + kRows - 1) / kRows);
  const int64_t blocks = (warps + kThreads4 / 32 - 1) / (kThreads4 / 32);
  return (unsigned)(blocks < (int64_t)sms * 8 ? blocks : (int64_t)sms * 8);
}

}  // namespace

cudaError_t launch_write_int4(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, uint8_t* cache, int64_t num_blocks, int hkv,
                              const int64_t* slots, int64_t n_tokens, int* err, int sms,
                              cudaStream_t st) {
  return launch_dependent(write_int4_kernel, dim3(grid4(n_tokens, hkv, sms)), dim3(kThreads4), 0,
                          st, k, k_stride, v, v_stride, cache, num_blocks * kBlockSize, hkv, slots,
                          n_tokens, err);
}

cudaError_t launch_read_int4(const uint8_t* cache, int64_t num_blocks, int hkv,
                             const int64_t* slots, int64_t n_tokens, uint16_t* k_out,
                             int64_t k_stride, uint16_t* v_out, int64_t v_stride, int* err, int sms,
                             cudaStream_t st) {
  return launch_dependent(read_int4_kernel, dim3(grid4(n_tokens, hkv, sms)), dim3(kThreads4), 0, st,
                          cache, num_blocks * kBlockSize, hkv, slots, n_tokens, k_out, k_stride,
                          v_out, v_stride, err);
}

}  // namespace pkv
