// MXFP4 (OCP Microscaling Formats v1.0: E2M1 elements in blocks of 32 under
// one E8M0 scale): sizes, layouts and the device conversions shared by the
// quantisers and the products.
#pragma once

#include <algorithm>

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

// The rows that expert e's matrix meets in a product of M rows.  Offsets and
// counts come from the device and are not trusted: a segment is clamped to
// [0, M] and its rows to the segment, so one that starts at or past M is empty
// whatever M is.  Scale tiles hold 128 rows: a segment that starts inside one
// has no rows.
struct MxSegment {
  int row0, rows;
};
__host__ __device__ inline MxSegment mx_segment(const int32_t* offsets, const int32_t* counts, int M, int e) {
  const int lo = std::min(std::max(offsets[e], 0), M), hi = std::min(std::max(offsets[e + 1], lo), M);
  int n = lo % 128 ? 0 : hi - lo;
  if (counts) n = std::min(n, std::max(counts[e], 0));
  return {lo, n};
}

// Element types of unquantised matrices (MXFP4_DTYPE_*), as tags.
struct Bf16 {
  static constexpr int size = 2;
  NVDEV static float lo(uint32_t w) { return bf16_lo(w); }
  NVDEV static float hi(uint32_t w) { return bf16_hi(w); }
  NVDEV static uint32_t pack(float a, float b) { return pack_bf16x2(a, b); }
  NVDEV static uint16_t one(float a) { return (uint16_t)pack_bf16x2(a, 0.0f); }
  NVDEV static uint32_t mag(uint32_t h) { return h << 16; }          // |h| as fp32 bits
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
  NVDEV static uint32_t mag(uint32_t h) {
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h))) & 0x7FFFFFFFu;
  }
};
struct F32 {
  static constexpr int size = 4;
};

// E8M0 byte of a block from its largest magnitude, as the bits of fp32 without
// the sign (they order like the magnitudes, with every infinity and NaN above
// every finite value): the exponent
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
// Eight values times the reciprocal scale -> 4 bytes of codes.  A NaN block's
// values are inf * 0 or NaN here: its codes are forced to 0.
NVDEV uint32_t mx_codes8(const float* v, float inv, bool nan_block) {
  const uint64_t inv2 = pack_f32x2(inv, inv);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t r = mul_f32x2(pack_f32x2(v[i], v[i + 1]), inv2);
    y[i] = lo_f32(r);
    y[i + 1] = hi_f32(r);
  }
  return nan_block ? 0u : e2m1x8_hw(y);
}

// n / d for n < 2^31 by a precomputed multiplier (division by an invariant
// integer: m = floor(2^(31 + l) / d) + 1 with 2^(l - 1) < d <= 2^l gives
// floor(n m / 2^(31 + l)) = floor(n / d), since m d exceeds 2^(31 + l) by at
// most d <= 2^l).
struct FastDiv {
  uint32_t d, shift;
  uint64_t m;
  explicit FastDiv(uint32_t div) : d(div) {
    uint32_t l = 0;
    while ((1ull << l) < div) ++l;
    shift = 31 + l;
    m = (1ull << shift) / div + 1;
  }
  // m <= 2^32 + 1 and n < 2^31: the product fits 64 bits
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> shift); }
};

// The widest access (32, 16, 8, 4 bytes, or one element) that every row of a
// matrix at `p` with rows `stride_bytes` apart allows.
inline int row_access_bytes(const void* p, long long stride_bytes, int elem) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes;
  return a % 32 == 0 ? 32 : a % 16 == 0 ? 16 : a % 8 == 0 ? 8 : a % 4 == 0 ? 4 : elem;
}

// 32 consecutive bytes as eight words, in loads of VB bytes (32, 16 or 8) and
// stores of VB bytes (32 or 16); narrower rows are read shifted and written
// through shared memory.
template <int VB>
NVDEV void load_words8(const void* p, uint32_t* w) {
  if constexpr (VB == 32) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
  } else if constexpr (VB == 16) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = __ldg(static_cast<const uint4*>(p) + i);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else {
    static_assert(VB == 8, "width of a load");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 v = __ldg(static_cast<const uint2*>(p) + i);
      w[2 * i] = v.x; w[2 * i + 1] = v.y;
    }
  }
}
template <int VB>
NVDEV void store_words8(void* p, const uint32_t* w) {
  if constexpr (VB == 32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_assert(VB == 16, "width of a store");
#pragma unroll
    for (int i = 0; i < 2; ++i)
      static_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

// A lane's share of a 128-element unit is 32 bytes of the source, eight words:
// 16 elements of a 16-bit type (8 lanes a unit, 2 a block) or 8 of fp32 (16
// lanes, 4 a block).  One 256-bit access a lane where the rows allow it.
template <typename T> __host__ __device__ constexpr int lane_elems() { return 32 / T::size; }
template <typename T> __host__ __device__ constexpr int unit_lanes() { return kMxGroup / lane_elems<T>(); }

// Elements at or past `n` read as 0.  `lo` and `hi` bound the matrix's bytes:
// the aligned pieces of a narrow row may reach into its neighbours, not past
// the matrix.
template <typename T, int VB>
NVDEV void load_share(const uint8_t* row, int c, int n, const uint8_t* lo, const uint8_t* hi, uint32_t* w) {
  constexpr int EPL = lane_elems<T>();
  if (c + EPL <= n) {
    const uint8_t* at = row + (size_t)c * T::size;
    if constexpr (VB >= 8) {
      load_words8<VB>(at, w);
      return;
    } else {
      const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(at) & 15u);
      const uint8_t* base = at - off;
      if (base >= lo && base + 48 <= hi) {
        uint32_t r[12];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(base) + i);
          r[4 * i] = v.x; r[4 * i + 1] = v.y; r[4 * i + 2] = v.z; r[4 * i + 3] = v.w;
        }
        // whole words by two conditional moves, the rest by funnel shifts
#pragma unroll
        for (int i = 0; i < 10; ++i) r[i] = (off & 8u) ? r[i + 2] : r[i];
#pragma unroll
        for (int i = 0; i < 9; ++i) r[i] = (off & 4u) ? r[i + 1] : r[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = T::size == 4 ? r[i] : __funnelshift_r(r[i], r[i + 1], (off & 3u) * 8u);
        return;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0u;
  if constexpr (T::size == 2) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + c;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (c + i < n) w[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + c;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (c + i < n) w[i] = __ldg(p + i);
  }
}

// fp32 bits of the largest magnitude of the block that these lanes share
// (magnitudes compare as integers; packed pairs for 16-bit types).
template <typename T>
NVDEV uint32_t share_amax(const uint32_t* w) {
  if constexpr (T::size == 2) {
    uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return T::mag(max(m & 0xFFFFu, m >> 16));
  } else {
    uint32_t m = w[0] & 0x7FFFFFFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  }
}
template <typename T>
NVDEV float share_value(const uint32_t* w, int i) {
  if constexpr (T::size == 2) return (i & 1) ? T::hi(w[i >> 1]) : T::lo(w[i >> 1]);
  else return __uint_as_float(w[i]);
}

// A lane's share of a unit -> its codes, and the scale bytes of the lane's
// block and (in the unit's first lane) the three behind it.  Whole warps.
template <typename T>
NVDEV void mx_unit(const uint32_t* w, uint32_t* q, uint32_t& sf) {
  constexpr int EPL = lane_elems<T>(), LPU = unit_lanes<T>();
  const uint32_t s = mx_scale(share_amax<T>(w));
  const float inv = mx_inv_scale(s);
#pragma unroll
  for (int h = 0; h < EPL / 8; ++h) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = share_value<T>(w, h * 8 + j);
    q[h] = mx_codes8(v, inv, s == 255u);
  }
  const uint32_t s1 = __shfl_down_sync(0xffffffffu, s, LPU / 4, LPU);
  const uint32_t s2 = __shfl_down_sync(0xffffffffu, s, LPU / 2, LPU);
  const uint32_t s3 = __shfl_down_sync(0xffffffffu, s, LPU / 4 * 3, LPU);
  sf = s | (s1 << 8) | (s2 << 16) | (s3 << 24);
}

inline int mx_elem_size(int dtype) { return dtype == MXFP4_DTYPE_F32 ? 4 : 2; }
inline bool mx_dtype_ok(int dtype) { return dtype >= MXFP4_DTYPE_BF16 && dtype <= MXFP4_DTYPE_F32; }

// Queues mxfp4_quantize on checked arguments (used by the product too, which
// with expert_counts needs no codes of rows outside the experts' tokens: those
// of them that have no source are left unwritten).
nvfp4_status launch_mx_quantize(const void* x, int dtype, int rows, int cols, long long row_stride,
                                const int32_t* perm, int out_rows, int layout, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s, const int32_t* expert_offsets = nullptr,
                                const int32_t* expert_counts = nullptr, int E = 0);
nvfp4_status check_mx_source(const char* name, const void* x, int dtype, int rows, int cols, long long row_stride);

}  // namespace nvfp4moe
