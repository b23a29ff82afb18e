// MXFP4 quantisers (row-wise, gathered, transposed) and the read-back.
//
// All three stream: each element is read once and written once, so HBM bounds
// them (b + 17/32 bytes an element for b-byte inputs), and for few rows the
// launch.  The arithmetic is exact: a block's scale is a power of two taken
// from the exponent field of its largest magnitude, x * (1 / scale) is exact,
// and the one rounding is the hardware's E2M1 conversion.
#include "mx.cuh"

namespace nvfp4moe {

constexpr int kMxThreads = 256;
constexpr int kMxSubs = kMxThreads / 16;     // 16-lane subgroups per block

// Eight consecutive elements (one lane's share of a 128-element unit) as raw
// words: 4 words of 16-bit elements or 8 of fp32.  VB is the access width the
// rows allow; elements at or past `n` read as 0.
template <typename T, int VB>
NVDEV void load8(const uint8_t* row, int c, int n, uint32_t* w) {
  constexpr int NW = T::size * 2;
  if (VB >= 4 && c + 8 <= n) {
    using V = typename VecOf<VB >= 4 ? VB : 4>::type;
    const V* p = reinterpret_cast<const V*>(row + (size_t)c * T::size);
    constexpr int per = sizeof(V) / 4;
#pragma unroll
    for (int i = 0; i < NW / per; ++i) {
      const V v = __ldg(p + i);
      if constexpr (per == 4) {
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      } else if constexpr (per == 2) {
        w[2 * i] = v.x; w[2 * i + 1] = v.y;
      } else {
        w[i] = v;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NW; ++i) w[i] = 0u;
  if constexpr (T::size == 2) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + c;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) w[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + c;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) w[i] = __ldg(p + i);
  }
}

template <typename T>
NVDEV void unpack8(const uint32_t* w, float* v) {
  if constexpr (T::size == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = T::lo(w[i]);
      v[2 * i + 1] = T::hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
}

// A unit is 128 consecutive elements of a row: one lane of a 16-lane subgroup
// holds 8 of them, 4 lanes a block (two shuffles for its maximum), and the
// unit's four scale bytes leave as one word.  A warp's loads then cover two
// contiguous runs of 256 (16-bit) or 512 bytes.  Each subgroup takes U units
// 16 apart, all their loads issued before the first is used.
template <typename T, int VB, int U>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(const uint8_t* __restrict__ x, int rows, int cols,
                                                                 long long stride_bytes,
                                                                 const int32_t* __restrict__ perm, uint32_t units,
                                                                 int groups, int tiled, uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  griddep_wait();
  griddep_launch();
  constexpr int NW = T::size * 2;
  const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
  const uint32_t u0 = blockIdx.x * (uint32_t)(kMxSubs * U) + sub;
  const int blocks = mx_blocks(cols);
  uint32_t w[U][NW];
  int row[U], grp[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = u0 + (uint32_t)i * kMxSubs;
    row[i] = (int)(u / (uint32_t)groups);
    grp[i] = (int)(u % (uint32_t)groups);
    int src = -1;
    if (u < units) src = perm ? __ldg(perm + row[i]) : row[i];
    const int n = (src >= 0 && src < rows) ? cols : 0;       // a row without a source reads as zeros
    load8<T, VB>(x + (n ? (size_t)src * (size_t)stride_bytes : 0), grp[i] * kMxGroup + l * 8, n, w[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = u0 + (uint32_t)i * kMxSubs;
    float v[8];
    unpack8<T>(w[i], v);
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, mag_bits(v[j]));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t s = mx_scale(m);
    const uint32_t q = mx_codes8(v, mx_inv_scale(s), s == 255u);
    const uint32_t s1 = __shfl_down_sync(0xffffffffu, s, 4, 16);
    const uint32_t s2 = __shfl_down_sync(0xffffffffu, s, 8, 16);
    const uint32_t s3 = __shfl_down_sync(0xffffffffu, s, 12, 16);
    if (u < units) {
      const int blk = grp[i] * 4 + (l >> 2);
      if (blk < blocks)
        *reinterpret_cast<uint32_t*>(codes + (size_t)row[i] * (size_t)blocks * 16 + grp[i] * 64 + l * 4) = q;
      if (tiled) {
        if (l == 0)
          *reinterpret_cast<uint32_t*>(scales + mx_tiled_offset(row[i], grp[i], groups)) =
              s | (s1 << 8) | (s2 << 16) | (s3 << 24);
      } else if ((l & 3) == 0 && blk < blocks) {
        scales[(size_t)row[i] * blocks + blk] = (uint8_t)s;
      }
    }
  }
}

// The transpose: a thread owns C neighbouring columns (two 16-bit ones where
// rows are 4-byte aligned, else one) over 64 rows of x, so its two blocks of
// a column are 32 contiguous bytes of codes, a whole sector, without a trip
// through shared memory.  A warp reads 64 (or 32) columns of a row at once;
// the eight warps of a block cover 512 rows, whose codes are contiguous.
constexpr int kMxTRows = 64;
template <typename T, int C>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_t_kernel(const uint8_t* __restrict__ x, int rows, int cols,
                                                                   long long stride_bytes, int groups, int tiled,
                                                                   uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * C;
  const long long r0 = ((long long)blockIdx.y * (kMxThreads / 32) + warp) * kMxTRows;
  const int blocks = mx_blocks(rows);
  const long long r_end = tiled ? (long long)groups * kMxGroup : (long long)blocks * kMxBlock;
  if (c >= cols || r0 >= r_end) return;
  const uint8_t* p = x + (size_t)r0 * (size_t)stride_bytes + (size_t)c * T::size;
  uint32_t w[kMxTRows];
#pragma unroll
  for (int i = 0; i < kMxTRows; ++i) {
    w[i] = 0u;
    if (r0 + i < rows) {
      const uint8_t* q = p + (size_t)i * (size_t)stride_bytes;
      if constexpr (T::size == 4 || C == 2) w[i] = __ldg(reinterpret_cast<const uint32_t*>(q));
      else w[i] = __ldg(reinterpret_cast<const uint16_t*>(q));
    }
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    uint32_t sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      auto val = [&](int i) -> float {
        const uint32_t b = w[h * 32 + i];
        if constexpr (T::size == 4) return __uint_as_float(b);
        else return j ? T::hi(b) : T::lo(b);
      };
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = max(m, mag_bits(val(i)));
      const uint32_t s = sc[h] = mx_scale(m);
      const float inv = mx_inv_scale(s);
      uint32_t q[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = val(g * 8 + i);
        q[g] = mx_codes8(v, inv, s == 255u);
      }
      const int blk = (int)(r0 / kMxBlock) + h;
      if (c + j < cols && blk < blocks)
        *reinterpret_cast<uint4*>(codes + ((size_t)(c + j) * blocks + blk) * 16) = make_uint4(q[0], q[1], q[2], q[3]);
    }
    if (c + j < cols) {
      const int blk = (int)(r0 / kMxBlock);                  // even: the pair stays inside a group
      if (tiled) {
        *reinterpret_cast<uint16_t*>(scales + mx_tiled_offset(c + j, blk >> 2, groups) + (blk & 3)) =
            (uint16_t)(sc[0] | (sc[1] << 8));
      } else {
        uint8_t* d = scales + (size_t)(c + j) * blocks + blk;
        d[0] = (uint8_t)sc[0];
        if (blk + 1 < blocks) d[1] = (uint8_t)sc[1];
      }
    }
  }
}

// Four bytes of codes -> eight values (hardware conversion to fp16 pairs).
NVDEV void mx_values8(uint32_t q, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h2;
    const uint16_t in = (uint16_t)((q >> (8 * i)) & 0xFFu);
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u16 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h2) : "h"(in));
    v[2 * i] = F16::lo(h2);
    v[2 * i + 1] = F16::hi(h2);
  }
}

// Read-back: the same units and lanes as the quantiser.
template <typename T, int VB, int U>
__global__ void __launch_bounds__(kMxThreads) mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales, int cols,
                                                                   uint32_t units, int groups, int tiled,
                                                                   uint8_t* __restrict__ out, long long stride_bytes) {
  griddep_wait();
  griddep_launch();
  const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
  const uint32_t u0 = blockIdx.x * (uint32_t)(kMxSubs * U) + sub;
  const int blocks = mx_blocks(cols);
  uint32_t q[U], s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = u0 + (uint32_t)i * kMxSubs;
    const int row = (int)(u / (uint32_t)groups), grp = (int)(u % (uint32_t)groups);
    const int blk = grp * 4 + (l >> 2);
    q[i] = s[i] = 0u;
    if (u < units && blk < blocks) {
      q[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + (size_t)row * (size_t)blocks * 16 + grp * 64 + l * 4));
      s[i] = __ldg(scales + (tiled ? mx_tiled_offset(row, grp, groups) + (l >> 2) : (size_t)row * blocks + blk));
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = u0 + (uint32_t)i * kMxSubs;
    const int row = (int)(u / (uint32_t)groups), grp = (int)(u % (uint32_t)groups);
    const int c = grp * kMxGroup + l * 8;
    if (u >= units || c >= cols) continue;
    float v[8];
    mx_values8(q[i], v);
    const float S = mx_scale_value(s[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], S);
    uint8_t* dst = out + (size_t)row * (size_t)stride_bytes + (size_t)c * T::size;
    if (VB >= 4 && c + 8 <= cols) {
      constexpr int NW = T::size * 2;
      uint32_t w[NW];
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        if constexpr (T::size == 2) w[j] = T::pack(v[2 * j], v[2 * j + 1]);
        else w[j] = __float_as_uint(v[j]);
      }
      using V = typename VecOf<VB >= 4 ? VB : 4>::type;
      V* d = reinterpret_cast<V*>(dst);
      constexpr int per = sizeof(V) / 4;
#pragma unroll
      for (int j = 0; j < NW / per; ++j) {
        if constexpr (per == 4) d[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        else if constexpr (per == 2) d[j] = make_uint2(w[2 * j], w[2 * j + 1]);
        else d[j] = w[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) {
          if constexpr (T::size == 2) reinterpret_cast<uint16_t*>(dst)[j] = T::one(v[j]);
          else reinterpret_cast<float*>(dst)[j] = v[j];
        }
    }
  }
}

// Units per subgroup: four where that still leaves every SM several blocks,
// else one, so that a few rows spread over the whole GPU.
static inline int units_per_sub(uint32_t units, int sms) { return units >= (uint32_t)(sms * kMxSubs * 16) ? 4 : 1; }

template <typename F>
static nvfp4_status with_type(int dtype, F&& f) {
  switch (dtype) {
    case MXFP4_DTYPE_BF16: return f(Bf16{});
    case MXFP4_DTYPE_F16: return f(F16{});
    default: return f(F32{});
  }
}

template <typename T, int VB>
static nvfp4_status run_quantize(int per, uint32_t units, const uint8_t* x, int rows, int cols, long long stride_bytes,
                                 const int32_t* perm, int groups, int tiled, uint8_t* codes, uint8_t* scales,
                                 cudaStream_t s) {
  const dim3 grid((units + kMxSubs * per - 1) / (kMxSubs * per));
  if (per == 4)
    return launch_dependent("mx_quantize_kernel", mx_quantize_kernel<T, VB, 4>, grid, dim3(kMxThreads), 0, s, x, rows,
                            cols, stride_bytes, perm, units, groups, tiled, codes, scales);
  return launch_dependent("mx_quantize_kernel", mx_quantize_kernel<T, VB, 1>, grid, dim3(kMxThreads), 0, s, x, rows,
                          cols, stride_bytes, perm, units, groups, tiled, codes, scales);
}

template <typename T, int VB>
static nvfp4_status run_dequantize(int per, uint32_t units, const uint8_t* codes, const uint8_t* scales, int cols,
                                   int groups, int tiled, uint8_t* out, long long stride_bytes, cudaStream_t s) {
  const dim3 grid((units + kMxSubs * per - 1) / (kMxSubs * per));
  if (per == 4)
    return launch_dependent("mx_dequantize_kernel", mx_dequantize_kernel<T, VB, 4>, grid, dim3(kMxThreads), 0, s,
                            codes, scales, cols, units, groups, tiled, out, stride_bytes);
  return launch_dependent("mx_dequantize_kernel", mx_dequantize_kernel<T, VB, 1>, grid, dim3(kMxThreads), 0, s, codes,
                          scales, cols, units, groups, tiled, out, stride_bytes);
}

nvfp4_status check_mx_source(const char* name, const void* x, int dtype, int rows, int cols, long long row_stride) {
  NV_REQUIRE(mx_dtype_ok(dtype), NVFP4_ERR_INVALID_ARG, "%s: unknown dtype %d", name, dtype);
  NV_REQUIRE(rows >= 0 && cols >= 1, NVFP4_ERR_INVALID_ARG, "%s: rows=%d cols=%d", name, rows, cols);
  NV_REQUIRE(cols <= (1 << 30), NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: cols=%d is above 2^30", name, cols);
  NV_REQUIRE(rows <= 1 || row_stride >= cols, NVFP4_ERR_INVALID_ARG, "%s: row stride %lld is below cols=%d", name,
             row_stride, cols);
  NV_REQUIRE(rows == 0 || x, NVFP4_ERR_INVALID_ARG, "%s: the matrix is NULL", name);
  NV_REQUIRE(aligned(x, mx_elem_size(dtype)), NVFP4_ERR_INVALID_ARG, "%s: the matrix is not aligned to its elements",
             name);
  return NVFP4_OK;
}

static nvfp4_status check_mx_quantized(const char* name, const uint8_t* codes, const uint8_t* scales, int layout) {
  NV_REQUIRE(layout == NVFP4_LAYOUT_CANONICAL || layout == NVFP4_LAYOUT_TILED, NVFP4_ERR_INVALID_ARG,
             "%s: layout %d (MXFP4 scales are canonical or tiled)", name, layout);
  NV_REQUIRE(codes && scales, NVFP4_ERR_INVALID_ARG, "%s: codes or scales is NULL", name);
  NV_REQUIRE(aligned(codes, 16) && aligned(scales, 4), NVFP4_ERR_INVALID_ARG,
             "%s: codes need 16-byte and scales 4-byte alignment", name);
  return NVFP4_OK;
}

static nvfp4_status count_units(const char* name, int rows, int cols, uint32_t* units) {
  const long long n = (long long)rows * mx_groups(cols);
  NV_REQUIRE(n < (1ll << 31), NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: %d x %d has 2^38 elements or more", name, rows, cols);
  *units = (uint32_t)n;
  return NVFP4_OK;
}

nvfp4_status launch_mx_quantize(const void* x, int dtype, int rows, int cols, long long row_stride,
                                const int32_t* perm, int out_rows, int layout, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s) {
  uint32_t units = 0;
  NV_CHECK(count_units("mxfp4_quantize", out_rows, cols, &units));
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  const int groups = mx_groups(cols), tiled = layout == NVFP4_LAYOUT_TILED;
  const int per = units_per_sub(units, sms);
  const uint8_t* xb = static_cast<const uint8_t*>(x);
  return with_type(dtype, [&](auto tag) -> nvfp4_status {
    using T = decltype(tag);
    const long long sb = row_stride * T::size;
    const int vb = row_access_bytes(x, rows > 1 ? sb : 0, T::size);
    if (vb == 16) return run_quantize<T, 16>(per, units, xb, rows, cols, sb, perm, groups, tiled, codes, scales, s);
    if (vb == 8) return run_quantize<T, 8>(per, units, xb, rows, cols, sb, perm, groups, tiled, codes, scales, s);
    if (vb == 4) return run_quantize<T, 4>(per, units, xb, rows, cols, sb, perm, groups, tiled, codes, scales, s);
    if constexpr (T::size == 2)
      return run_quantize<T, 2>(per, units, xb, rows, cols, sb, perm, groups, tiled, codes, scales, s);
    return NVFP4_ERR_INVALID_ARG;
  });
}

}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" size_t mxfp4_scale_bytes(int rows, int cols, int layout) {
  if (rows < 0 || cols < 0) return 0;
  if (layout == NVFP4_LAYOUT_CANONICAL) return (size_t)rows * mx_blocks(cols);
  if (layout == NVFP4_LAYOUT_TILED) return ((size_t)rows + 127) / 128 * mx_groups(cols) * kAtomBytes;
  return 0;
}

extern "C" nvfp4_status mxfp4_quantize(const void* x, int dtype, int rows, int cols, long long row_stride,
                                       const int32_t* perm, int perm_rows, int layout, uint8_t* codes,
                                       uint8_t* scales, void* stream) {
  NV_CHECK(check_mx_source("mxfp4_quantize", x, dtype, rows, cols, row_stride));
  NV_REQUIRE(!perm || perm_rows >= 0, NVFP4_ERR_INVALID_ARG, "mxfp4_quantize: perm_rows=%d", perm_rows);
  NV_REQUIRE(aligned(perm, 4), NVFP4_ERR_INVALID_ARG, "mxfp4_quantize: perm is not aligned to its elements");
  const int out_rows = perm ? perm_rows : rows;
  if (out_rows == 0) return NVFP4_OK;
  NV_CHECK(check_mx_quantized("mxfp4_quantize", codes, scales, layout));
  return launch_mx_quantize(x, dtype, rows, cols, row_stride, perm, out_rows, layout, codes, scales,
                            as_stream(stream));
}

extern "C" nvfp4_status mxfp4_quantize_transposed(const void* x, int dtype, int rows, int cols, long long row_stride,
                                                  int layout, uint8_t* codes, uint8_t* scales, void* stream) {
  NV_CHECK(check_mx_source("mxfp4_quantize_transposed", x, dtype, rows, cols, row_stride));
  NV_REQUIRE(rows >= 1, NVFP4_ERR_INVALID_ARG, "mxfp4_quantize_transposed: rows=%d (the result's columns)", rows);
  NV_CHECK(check_mx_quantized("mxfp4_quantize_transposed", codes, scales, layout));
  constexpr int per_block = kMxThreads / 32 * kMxTRows;
  NV_REQUIRE(rows <= 65535 * per_block, NVFP4_ERR_UNSUPPORTED_SHAPE, "mxfp4_quantize_transposed: rows=%d is above %d",
             rows, 65535 * per_block);
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  const int groups = mx_groups(rows), tiled = layout == NVFP4_LAYOUT_TILED;
  const int gy = (groups * kMxGroup + per_block - 1) / per_block;
  const uint8_t* xb = static_cast<const uint8_t*>(x);
  cudaStream_t s = as_stream(stream);
  return with_type(dtype, [&](auto tag) -> nvfp4_status {
    using T = decltype(tag);
    const long long sb = row_stride * T::size;
    if constexpr (T::size == 2) {
      // pairs of columns need 4-byte aligned rows and a second column in the last pair
      if (row_access_bytes(x, rows > 1 ? sb : 0, 2) >= 4 && cols % 2 == 0)
        return launch_dependent("mx_quantize_t_kernel", mx_quantize_t_kernel<T, 2>, dim3((cols + 63) / 64, gy),
                                dim3(kMxThreads), 0, s, xb, rows, cols, sb, groups, tiled, codes, scales);
    }
    return launch_dependent("mx_quantize_t_kernel", mx_quantize_t_kernel<T, 1>, dim3((cols + 31) / 32, gy),
                            dim3(kMxThreads), 0, s, xb, rows, cols, sb, groups, tiled, codes, scales);
  });
}

extern "C" nvfp4_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int layout, int rows, int cols,
                                         int dtype, void* out, long long row_stride, void* stream) {
  NV_CHECK(check_mx_source("mxfp4_dequantize", out, dtype, rows, cols, row_stride));
  if (rows == 0) return NVFP4_OK;
  NV_CHECK(check_mx_quantized("mxfp4_dequantize", codes, scales, layout));
  uint32_t units = 0;
  NV_CHECK(count_units("mxfp4_dequantize", rows, cols, &units));
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  const int groups = mx_groups(cols), tiled = layout == NVFP4_LAYOUT_TILED;
  const int per = units_per_sub(units, sms);
  uint8_t* ob = static_cast<uint8_t*>(out);
  cudaStream_t s = as_stream(stream);
  return with_type(dtype, [&](auto tag) -> nvfp4_status {
    using T = decltype(tag);
    const long long sb = row_stride * T::size;
    const int vb = row_access_bytes(out, rows > 1 ? sb : 0, T::size);
    if (vb == 16) return run_dequantize<T, 16>(per, units, codes, scales, cols, groups, tiled, ob, sb, s);
    if (vb == 8) return run_dequantize<T, 8>(per, units, codes, scales, cols, groups, tiled, ob, sb, s);
    if (vb == 4) return run_dequantize<T, 4>(per, units, codes, scales, cols, groups, tiled, ob, sb, s);
    if constexpr (T::size == 2)
      return run_dequantize<T, 2>(per, units, codes, scales, cols, groups, tiled, ob, sb, s);
    return NVFP4_ERR_INVALID_ARG;
  });
}
