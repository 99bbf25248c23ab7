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
// HBM traffic: 512 bytes read and 136 written per token and KV head, or the
// reverse.  A half-warp takes a key row, the other the value row: 8 values, one
// code word a lane; the row's minimum and maximum are four exchanges of both
// together.  kRows heads a warp, all loads before the first use.  What bounds the write
// beside HBM is the codes' arithmetic (issue slots 66%, alu pipe 51%).  8191 tokens
// of 32 KV heads written and read back, floor 50 us: 81.6 with IEEE divisions and one value
// an instruction; 73.7 with packed minima and maxima; 65.6 with as many CTAs as
// the GPU holds (no second wave); 61.5 with the quotients by reciprocals.  Asking for the
// next token's rows before this one's codes: 68.
#include <algorithm>

#include "pkv_int4.cuh"

namespace pkv {
namespace {

constexpr int kThreads4 = 256;
constexpr int kRows = 4;  // heads of a token that a warp takes at once
constexpr int kWriteCtas = 5, kReadCtas = 6;  // of an SM at a time, by their registers

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 8 bf16 values of a row (the other lanes of the half-warp hold the rest) to their
// code word; *pair = the row's (scale, zero).  Packed bf16 minima and maxima (exact),
// the row's largest value and negative smallest exchanged together; two values an
// instruction where fp32 is needed.
__device__ __forceinline__ uint32_t quantise8(uint4 raw, uint32_t* pair) {
  uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t m = 0;
  auto row_range = [&]() {  // (max, -min) of the row, a NaN in it kept
    const __nv_bfloat162 a = as_bf16x2(w[0]), b = as_bf16x2(w[1]), c = as_bf16x2(w[2]),
                         d = as_bf16x2(w[3]);
    const uint32_t hi = bits_of(__hmax2_nan(__hmax2_nan(a, b), __hmax2_nan(c, d)));
    const uint32_t lo = bits_of(__hmin2(__hmin2(a, b), __hmin2(c, d))) ^ 0x80008000u;
    m = bits_of(__hmax2_nan(as_bf16x2(__byte_perm(hi, lo, 0x5410)),
                            as_bf16x2(__byte_perm(hi, lo, 0x7632))));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
      m = bits_of(__hmax2_nan(as_bf16x2(m), as_bf16x2(__shfl_xor_sync(0xffffffffu, m, o))));
  };
  row_range();
  const bool odd = (m & 0x7FFFu) > 0x7E80u || ((m >> 16) & 0x7FFFu) > 0x7E80u;
  if (__any_sync(0xffffffffu, odd)) {  // some |x| > 2^126, or a NaN
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2] = {w[i] & 0xFFFFu, w[i] >> 16};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t size = h[k] & 0x7FFFu;
        if (size > 0x7F80u)
          h[k] = 0;
        else if (size > 0x7E80u)
          h[k] = (h[k] & 0x8000u) | 0x7E80u;
      }
      w[i] = h[0] | h[1] << 16;
    }
    row_range();
  }
  // The IEEE quotients w / 15 and (x - z) / s by a rounded reciprocal and one exact
  // remainder (Markstein's division; s is between 2^-41 and 2^124, or 0: then every
  // code is 0).  1 / s rounded: the approximation (2^-23) and one step of Newton's;
  // equal to the IEEE reciprocal for every bf16 in the range.  Adding 2^23 rounds a
  // quotient to an integer in the sum's low bits.
  const float hi = __uint_as_float(m << 16), lo = -__uint_as_float(m & 0xFFFF0000u);
  const float spread = hi - lo, q15 = spread * (1.f / 15.f);
  const float sf = fmaf(fmaf(-15.f, q15, spread), 1.f / 15.f, q15);
  const float s = spread < 0x1p-36f ? 0.f : __bfloat162float(__float2bfloat16_rn(sf));
  *pair = __float_as_uint(s) >> 16 | (__float_as_uint(lo) & 0xFFFF0000u);
  float r = dev::fast_rcp(s);
  r = s == 0.f ? 0.f : fmaf(fmaf(-r, s, 1.f), r, r);
  const dev::f32x2 r2 = dev::pair(r, r), s2 = dev::pair(-s, -s), lo2 = dev::pair(-lo, -lo);
  const dev::f32x2 big = dev::pair(8388608.f, 8388608.f);
  uint32_t word = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const dev::f32x2 d = dev::add2(
        dev::pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), lo2);
    const dev::f32x2 q = dev::mul2(d, r2);
    float c0, c1;
    dev::split(dev::add2(dev::fma2(dev::fma2(q, s2, d), r2, q), big), c0, c1);
    word = word * 16u + __byte_perm(__float_as_uint(c0), __float_as_uint(c1), 0x5410);
  }
  return word;
}

__global__ void __launch_bounds__(kThreads4, kWriteCtas)
    write_int4_kernel(const uint16_t* __restrict__ k, int64_t k_stride,
                      const uint16_t* __restrict__ v, int64_t v_stride, uint8_t* __restrict__ cache,
                      int64_t num_slots, int hkv, const int64_t* __restrict__ slots,
                      int64_t n_tokens, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, l = lane & 15, side = lane >> 4;
  const int h0 = blockIdx.y * kRows;
  const int64_t step = (int64_t)gridDim.x * (kThreads4 / 32);
  for (int64_t t = blockIdx.x * (int64_t)(kThreads4 / 32) + (threadIdx.x >> 5); t < n_tokens;
       t += step) {
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
      if (h0 + i >= hkv) break;
      uint32_t pair;
      const uint32_t word = quantise8(raw[i], &pair);
      uint8_t* p = page + i * kPage4;
      *reinterpret_cast<uint32_t*>(p + side * kSide4 + off * kRow4 + l * 4) = word;
      if (l == 0) *reinterpret_cast<uint32_t*>(p + kMeta4 + side * 64 + off * 4) = pair;
    }
  }
}

__global__ void __launch_bounds__(kThreads4, kReadCtas)
    read_int4_kernel(const uint8_t* __restrict__ cache, int64_t num_slots, int hkv,
                     const int64_t* __restrict__ slots, int64_t n_tokens,
                     uint16_t* __restrict__ k_out, int64_t k_stride, uint16_t* __restrict__ v_out,
                     int64_t v_stride, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, l = lane & 15, side = lane >> 4;
  const int h0 = blockIdx.y * kRows;
  const int64_t step = (int64_t)gridDim.x * (kThreads4 / 32);
  for (int64_t t = blockIdx.x * (int64_t)(kThreads4 / 32) + (threadIdx.x >> 5); t < n_tokens;
       t += step) {
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
      // (128 + code has its code in the last bits of a bf16, less 128 is exact; one
      // rounding in the multiply-add)
      const __nv_bfloat162 s = as_bf16x2(__byte_perm(pair[i], 0, 0x1010));
      const __nv_bfloat162 z = as_bf16x2(__byte_perm(pair[i], 0, 0x3232));
      uint32_t o[4];
#pragma unroll
      for (int a = 0; a < 4; ++a)
        o[a] = bits_of(__hfma2(__hsub2(as_bf16x2(((word[i] >> (4 * a)) & 0x000F000Fu) | 0x43004300u),
                                       __float2bfloat162_rn(128.f)),
                               s, z));
      *reinterpret_cast<uint4*>(dst + i * kHeadSize) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// A warp per token and kRows heads (a row of CTAs for each kRows heads: no division in the
// kernel), as many CTAs as the GPU holds at once.
dim3 grid4(int64_t n_tokens, int hkv, int ctas) {
  const int groups = (hkv + kRows - 1) / kRows;
  const int64_t blocks = (n_tokens + kThreads4 / 32 - 1) / (kThreads4 / 32);
  const int64_t most = std::max(1, ctas / groups);
  return dim3((unsigned)std::min(blocks, most), groups);
}

}  // namespace

cudaError_t launch_write_int4(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, uint8_t* cache, int64_t num_blocks, int hkv,
                              const int64_t* slots, int64_t n_tokens, int* err, int sms,
                              cudaStream_t st) {
  return launch_dependent(write_int4_kernel, grid4(n_tokens, hkv, sms * kWriteCtas),
                          dim3(kThreads4), 0, st, k, k_stride, v, v_stride, cache,
                          num_blocks * kBlockSize, hkv, slots, n_tokens, err);
}

cudaError_t launch_read_int4(const uint8_t* cache, int64_t num_blocks, int hkv,
                             const int64_t* slots, int64_t n_tokens, uint16_t* k_out,
                             int64_t k_stride, uint16_t* v_out, int64_t v_stride, int* err, int sms,
                             cudaStream_t st) {
  return launch_dependent(read_int4_kernel, grid4(n_tokens, hkv, sms * kReadCtas),
                          dim3(kThreads4), 0, st, cache, num_blocks * kBlockSize, hkv, slots,
                          n_tokens, k_out, k_stride, v_out, v_stride, err);
}

}  // namespace pkv
