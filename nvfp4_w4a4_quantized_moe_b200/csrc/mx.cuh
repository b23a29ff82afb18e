// MXFP4 (OCP Microscaling Formats v1.0: E2M1 elements in blocks of 32 under
// one E8M0 scale): sizes, layouts and the device conversions shared by the
// quantisers and the products.
#pragma once

#include "common.cuh"
#include "host.cuh"
#include "../../include/mxfp4.h"

namespace nvfp4moe {

constexpr int kMxBlock = 32;                 // elements per E8M0 scale
constexpr int kMxGroup = 128;                // elements per scale atom (4 blocks)

__host__ __device__ inline int mx_blocks(int cols) { return (int)(((unsigned)cols + kMxBlock - 1) / kMxBlock); }
__host__ __device__ inline int mx_groups(int cols) { return (int)(((unsigned)cols + kMxGroup - 1) / kMxGroup); }
__host__ __device__ inline int mx_row_bytes(int cols) { return mx_blocks(cols) * (kMxBlock / 2); }

// Byte offset of the four scales of (row, block group) in the tiled layout.
NVDEV size_t mx_tiled_offset(int row, int group, int groups) {
  return ((size_t)(row >> 7) * groups + group) * kAtomBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Element types of unquantised matrices (MXFP4_DTYPE_*), as tags.
struct Bf16 {
  static constexpr int size = 2;
  NVDEV static float lo(uint32_t w) { return bf16_lo(w); }
  NVDEV static float hi(uint32_t w) { return bf16_hi(w); }
  NVDEV static uint32_t pack(float a, float b) { return pack_bf16x2(a, b); }
  NVDEV static uint16_t one(float a) { return (uint16_t)pack_bf16x2(a, 0.0f); }
  NVDEV static float from(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
};
struct F16 {
  static constexpr int size = 2;
  NVDEV static float lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu))); }
  NVDEV static float hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
  NVDEV static uint32_t pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
  NVDEV static uint16_t one(float a) { return __half_as_ushort(__float2half_rn(a)); }
  NVDEV static float from(uint16_t h) { return __half2float(__ushort_as_half(h)); }
};
struct F32 {
  static constexpr int size = 4;
};

// |v| as an integer that orders like the magnitude, with every infinity and
// NaN above every finite value.
NVDEV uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// E8M0 byte of a block from the mag_bits of its largest element: the exponent
// field less 2 (floor(log2 a) - 2 + 127), 0 where that would be below 2^-127
// (subnormal maxima included), 255 for a block with a NaN or an infinity.
NVDEV uint32_t mx_scale(uint32_t amax_bits) {
  const uint32_t f = amax_bits >> 23;
  return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}
// 1 / scale, exact (2^(127 - s)); a NaN block's codes become 0.
NVDEV float mx_inv_scale(uint32_t s) { return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23); }
// The scale itself: 2^(s - 127), a subnormal for s = 0.
NVDEV float mx_scale_value(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7FFFFFFFu : (s == 0u ? 0x00400000u : s << 23));
}
// Eight scaled values -> 4 bytes of codes.  A NaN block's values are
// inf * 0 or x * 0 here: its codes are forced to 0.
NVDEV uint32_t mx_codes8(const float* v, float inv, bool nan_block) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(v[i], inv);
  return nan_block ? 0u : e2m1x8_hw(y);
}

// Loads of V consecutive bytes.
template <int V> struct VecOf;
template <> struct VecOf<16> { using type = uint4; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<4> { using type = uint32_t; };

// The widest access (16, 8, 4 bytes, or one element) that every row of a
// matrix at `p` with rows `stride_bytes` apart allows.
inline int row_access_bytes(const void* p, long long stride_bytes, int elem) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes;
  return a % 16 == 0 ? 16 : a % 8 == 0 ? 8 : a % 4 == 0 ? 4 : elem;
}

inline int mx_elem_size(int dtype) { return dtype == MXFP4_DTYPE_F32 ? 4 : 2; }
inline bool mx_dtype_ok(int dtype) { return dtype >= MXFP4_DTYPE_BF16 && dtype <= MXFP4_DTYPE_F32; }

// Queues mxfp4_quantize on checked arguments (used by the product too).
nvfp4_status launch_mx_quantize(const void* x, int dtype, int rows, int cols, long long row_stride,
                                const int32_t* perm, int out_rows, int layout, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s);
nvfp4_status check_mx_source(const char* name, const void* x, int dtype, int rows, int cols, long long row_stride);

}  // namespace nvfp4moe
