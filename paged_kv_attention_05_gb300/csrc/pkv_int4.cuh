// The record of a page of 4-bit codes (pkv_write_i4.cu describes it).
#pragma once

#include "pkv_device.cuh"

namespace pkv {

constexpr int kRow4 = kHeadSize / 2;              // bytes of a row's codes
constexpr int kSide4 = kBlockSize * kRow4;        // key codes; then value codes
constexpr int kMeta4 = 2 * kSide4;                // (scale, zero) of keys, 64 bytes, and of values
constexpr int kPage4 = kMeta4 + 2 * kBlockSize * 4;
static_assert(kPage4 == PKV_INT4_PAGE_BYTES, "the page record of include/pkv.h");

}  // namespace pkv
