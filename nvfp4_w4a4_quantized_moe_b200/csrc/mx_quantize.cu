// MXFP4 quantisers (row-wise, gathered, transposed) and the read-back.
//
// All three stream: each element is read once and written once, so HBM bounds
// them (b + 17/32 bytes an element for b-byte inputs), and for few rows the
// launch.  The arithmetic is exact: a block's scale is a power of two taken
// from the exponent field of its largest magnitude, x * (1 / scale) is exact,
// and the one rounding is the hardware's E2M1 conversion.
//
// Measured on one B200 as a share of its copy rate (6,449 GB/s):
//   65536 x 6144 bf16: quantise 158 us (100 %), transposed 199 us (80 %),
//   read-back 154 us (103 %); 32768 x 6144 fp32: 139 us (102 %), 149 us
//   (95 %), 139 us (102 %); 8192 x 6144 bf16: 22 us (91 %), 24 us (81 %),
//   21 us (95 %).
// The first form, with 16-byte loads, two packed maxima less and a 32-bit
// division a unit, took 259 and 202 us at 65536 x 6144.
#include <type_traits>

#include "mx.cuh"

namespace nvfp4moe {

constexpr int kMxThreads = 256;

// Units a block takes at once.
template <typename T> __host__ __device__ constexpr int block_subs() { return kMxThreads / unit_lanes<T>(); }

// Rows that allow only narrow accesses (8 bytes or less).
//   Reading rows that are 2- or 4-byte aligned: a lane's 32 bytes lie inside
//   three aligned 16-byte pieces; it reads those and shifts them into place.
//   8-byte accesses are left as they are (L1 serves the neighbours' share of a
//   line).
//   Writing: the warp's consecutive units (1 KiB in all) go through shared
//   memory, so that neighbouring lanes write neighbouring words instead of 4
//   to 16 accesses 32 bytes apart each.
// Measured (one B200, us; quantise reads x, read-back writes it):
//                                   one by one   through shared   shifted
//   read  16384 x 6145 bf16 (2 B)      107            127           59
//   read  16384 x 6146 bf16 (4 B)       61             72           59
//   read  8192 x 6145 fp32 (4 B)        58             58           50
//   read  8191 x 6100 fp16 (8 B)        23             31           35
//   write 16384 x 6145 bf16 (2 B)      544             71
//   write 16384 x 6146 bf16 (4 B)        -             52
//   write 8191 x 6100 fp16 (8 B)        53             25
constexpr bool is_narrow(int vb) { return vb < 16; }
constexpr int kMxWarpBytes = 1024;

template <int VB> struct Narrow;
template <> struct Narrow<8> { using type = uint2; };
template <> struct Narrow<4> { using type = uint32_t; };

// Writes the warp's units, a lane's share of which is `w`: unit by unit, with
// neighbouring lanes on neighbouring words.  row, grp: the lane's own unit.
template <typename T, int VB>
NVDEV void store_staged(uint8_t* out, int cols, long long stride_bytes, int row, int grp, bool real, uint8_t* buf,
                        const uint32_t* w) {
  constexpr int LPU = unit_lanes<T>(), unit_bytes = kMxGroup * T::size;
  const int lane = threadIdx.x & 31;
  __syncwarp();                                              // the previous units have left buf
  uint4* mine = reinterpret_cast<uint4*>(buf + lane * 32);
  mine[0] = make_uint4(w[0], w[1], w[2], w[3]);
  mine[1] = make_uint4(w[4], w[5], w[6], w[7]);
  __syncwarp();
  if constexpr (VB >= 4) {
    // the usual case, every unit whole: no checks
    if (__all_sync(0xffffffffu, real && grp * kMxGroup + kMxGroup <= cols)) {
      using V = typename Narrow<VB>::type;
      uint8_t* own = out + (size_t)row * (size_t)stride_bytes + (size_t)grp * unit_bytes;
#pragma unroll
      for (int unit = 0; unit < 32 / LPU; ++unit) {
        V* to = reinterpret_cast<V*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(own), unit * LPU)) + lane;
        const V* from = reinterpret_cast<const V*>(buf + unit * unit_bytes) + lane;
#pragma unroll
        for (int it = 0; it < unit_bytes / (32 * VB); ++it) to[it * 32] = from[it * 32];
      }
      return;
    }
  }
#pragma unroll
  for (int unit = 0; unit < 32 / LPU; ++unit) {
    const int r = __shfl_sync(0xffffffffu, row, unit * LPU), g = __shfl_sync(0xffffffffu, grp, unit * LPU);
    if (!__shfl_sync(0xffffffffu, (int)real, unit * LPU)) continue;
    const uint8_t* from = buf + unit * unit_bytes;
    uint8_t* to = out + (size_t)r * (size_t)stride_bytes + (size_t)g * unit_bytes;
    const int n = min(kMxGroup, cols - g * kMxGroup);        // elements of the unit
    if constexpr (VB == 2) {
      // rows of 2-byte elements at any of them: words from the first aligned
      // one on, the ends by themselves
      const int mis = (int)(reinterpret_cast<uintptr_t>(to) >> 1) & 1;
      const uint16_t* f = reinterpret_cast<const uint16_t*>(from);
      uint16_t* t = reinterpret_cast<uint16_t*>(to);
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int e = 2 * (it * 32 + lane) + mis;
        if (e + 1 < n) {
          *reinterpret_cast<uint32_t*>(t + e) = (uint32_t)f[e] | ((uint32_t)f[e + 1] << 16);
        } else if (e < n) {
          t[e] = f[e];
        }
      }
      if (mis && lane == 0) t[0] = f[0];
    } else {
      using V = typename Narrow<VB>::type;
      constexpr int per = VB / T::size;                      // elements per access
#pragma unroll
      for (int it = 0; it < unit_bytes / (32 * VB); ++it) {
        const int i = it * 32 + lane, e = i * per;
        if (e + per <= n) {
          reinterpret_cast<V*>(to)[i] = reinterpret_cast<const V*>(from)[i];
        } else {
#pragma unroll
          for (int j = 0; j < per; ++j)
            if (e + j < n) {
              if constexpr (T::size == 2) reinterpret_cast<uint16_t*>(to)[e + j] = reinterpret_cast<const uint16_t*>(from)[e + j];
              else reinterpret_cast<uint32_t*>(to)[e + j] = reinterpret_cast<const uint32_t*>(from)[e + j];
            }
        }
      }
    }
  }
}

// Quantises the unit (row, group) from its lanes' shares; every lane of the
// warp takes part, `real` units are written.  The unit's four scale bytes
// leave as one word.
template <typename T>
NVDEV void quantize_unit(const uint32_t* w, int row, int grp, bool real, int cols, int groups, int tiled,
                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int EPL = lane_elems<T>(), LPU = unit_lanes<T>();
  const int l = threadIdx.x & (LPU - 1), blocks = mx_blocks(cols);
  uint32_t q[EPL / 8], sf;
  mx_unit<T>(w, q, sf);
  if (!real) return;
  const int blk = grp * 4 + l / (LPU / 4);
  if (blk < blocks) {
    uint8_t* dst = codes + (size_t)row * (size_t)blocks * 16 + grp * 64 + l * (EPL / 2);
    if constexpr (EPL == 16) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(dst) = q[0];
  }
  if (tiled) {
    if (l == 0)
      *reinterpret_cast<uint32_t*>(scales + mx_tiled_offset(row, grp, groups)) = sf;
  } else if (l % (LPU / 4) == 0 && blk < blocks) {
    scales[(size_t)row * blocks + blk] = (uint8_t)sf;
  }
}

// Each group of lanes takes U units, all their loads issued before the first
// is used.
template <typename T, int VB, int U>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(const uint8_t* __restrict__ x, int rows, int cols,
                                                                 long long stride_bytes,
                                                                 const int32_t* __restrict__ perm, uint32_t units,
                                                                 const FastDiv groups, int tiled,
                                                                 uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  griddep_wait();
  griddep_launch();
  constexpr int EPL = lane_elems<T>(), LPU = unit_lanes<T>(), SUBS = block_subs<T>();
  const int sub = threadIdx.x / LPU, l = threadIdx.x & (LPU - 1);
  const uint32_t u0 = blockIdx.x * (uint32_t)(SUBS * U) + sub;
  const int blocks = mx_blocks(cols);
  const uint8_t* x_end = x + (rows > 0 ? (size_t)(rows - 1) * (size_t)stride_bytes + (size_t)cols * T::size : 0);
  uint32_t w[U][8];
  int row[U], grp[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = min(u0 + (uint32_t)i * SUBS, units - 1);
    row[i] = (int)groups.quotient(u);
    grp[i] = (int)(u - (uint32_t)row[i] * groups.d);
    const int src = perm ? __ldg(perm + row[i]) : row[i];
    const int n = (src >= 0 && src < rows) ? cols : 0;       // a row without a source reads as zeros
    load_share<T, VB>(x + (n ? (size_t)src * (size_t)stride_bytes : 0), grp[i] * kMxGroup + l * EPL, n, x, x_end, w[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i)
    quantize_unit<T>(w[i], row[i], grp[i], u0 + (uint32_t)i * SUBS < units, cols, (int)groups.d, tiled, codes, scales);
}

// The gathered rows of a grouped product, one block a row.  Rows without a
// source are zeros where a product reads them, inside an expert's tokens (the
// product's own mx_segment of the last expert that starts at or before the
// row); outside, where most of a decoding step's rows lie (127 of padding an
// expert), nothing is written.
constexpr int kMxRowThreads = 128;
constexpr int kMxRowUnits = 3;
template <typename T, int VB>
__global__ void __launch_bounds__(kMxRowThreads) mx_quantize_rows_kernel(
    const uint8_t* __restrict__ x, int rows, int cols, long long stride_bytes, const int32_t* __restrict__ perm,
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ counts, int E, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
  griddep_wait();
  griddep_launch();
  constexpr int EPL = lane_elems<T>(), LPU = unit_lanes<T>(), SUBS = kMxRowThreads / LPU;
  const int row = blockIdx.x, src = __ldg(perm + row);
  const bool live = src >= 0 && src < rows;
  if (!live) {                                               // the same for the whole block
    int before = 0;                                          // experts that start at or before the row
    for (int e0 = 0; e0 < E; e0 += kMxRowThreads) {
      const int e = e0 + (int)threadIdx.x;
      before += __syncthreads_count(e < E && __ldg(offsets + e) <= row);
    }
    if (before == 0) return;
    const MxSegment seg = mx_segment(offsets, counts, (int)gridDim.x, before - 1);
    if (row - seg.row0 >= seg.rows) return;
  }
  const int n = live ? cols : 0, groups = mx_groups(cols);
  const int sub = threadIdx.x / LPU, l = threadIdx.x & (LPU - 1);
  const uint8_t* x_end = x + (rows > 0 ? (size_t)(rows - 1) * (size_t)stride_bytes + (size_t)cols * T::size : 0);
  const uint8_t* from = x + (live ? (size_t)src * (size_t)stride_bytes : 0);
  for (int g0 = 0; g0 < groups; g0 += SUBS * kMxRowUnits) {
    uint32_t w[kMxRowUnits][8];
#pragma unroll
    for (int i = 0; i < kMxRowUnits; ++i)
      load_share<T, VB>(from, (g0 + i * SUBS + sub) * kMxGroup + l * EPL, n, x, x_end, w[i]);
#pragma unroll
    for (int i = 0; i < kMxRowUnits; ++i) {
      const int grp = g0 + i * SUBS + sub;
      quantize_unit<T>(w[i], row, grp, grp < groups, cols, groups, 1, codes, scales);
    }
  }
}

// The transpose: a thread owns C neighbouring columns (one word of a row) over
// 32 rows of x, one block of each column, without a trip through shared
// memory.  A warp reads 32 C columns of a row at once; the warps of a block
// cover consecutive rows, whose codes are contiguous, so that the 16 bytes a
// lane writes join their sector in L2.  64 rows a thread (whole sectors, twice
// the registers) measured slower but at the largest size: 8192 x 6144 bf16
// 29.0 us against 24.5, 4096 x 6144 16.3 against 12.7, 32768 x 6144 fp32 160
// against 149, 65536 x 6144 bf16 191 against 199.
constexpr int kMxTThreads = 128;
constexpr int kMxTRows = kMxTThreads / 32 * kMxBlock;      // rows of x per block
template <typename T, int C, bool WIDE>
__global__ void __launch_bounds__(kMxTThreads) mx_quantize_t_kernel(const uint8_t* __restrict__ x, int rows, int cols,
                                                                    long long stride_bytes, int groups, int tiled,
                                                                    uint8_t* __restrict__ codes,
                                                                    uint8_t* __restrict__ scales) {
  static_assert(C * T::size == 4, "a thread's columns of a row are one word");
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * C;
  const long long r0 = ((long long)blockIdx.y * (kMxTThreads / 32) + warp) * kMxBlock;
  const int blocks = mx_blocks(rows);
  const long long r_end = tiled ? (long long)groups * kMxGroup : (long long)blocks * kMxBlock;
  if (r0 >= r_end) return;                                   // whole warps
  const uint8_t* p = x + (size_t)r0 * (size_t)stride_bytes + (size_t)c * T::size;
  uint32_t w[kMxBlock];
  if constexpr (WIDE) {
    if (c >= cols) return;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i)
      w[i] = r0 + i < rows ? __ldg(reinterpret_cast<const uint32_t*>(p + (size_t)i * (size_t)stride_bytes)) : 0u;
  } else {
    // Rows that are only 2-byte aligned: each lane reads the aligned word that
    // holds its first column, takes the word behind it from the next lane and
    // shifts the pair into place.  The word behind the last lane's is read by
    // lane i for row i, so that no load sits in a branch.  Warps
    // whose words would reach past the matrix read element by element.
    const uint8_t* x_end = x + (size_t)(rows - 1) * (size_t)stride_bytes + (size_t)cols * 2;
    const long long rl = min(r0 + kMxBlock, (long long)rows) - 1;
    const uint8_t* first = p - (size_t)lane * 4;
    const uint8_t* last = x + (size_t)max(rl, 0ll) * (size_t)stride_bytes + (size_t)(c - lane * C) * 2 + 32 * 4;
    if (r0 < rows && first - 2 >= x && last + 4 <= x_end) {
      const int n = (int)(rl + 1 - r0);                      // rows that exist: 32 but at the end
      auto behind = [&](int i) -> uint32_t {
        const uint8_t* q = first + (size_t)min(i, n - 1) * (size_t)stride_bytes;
        return __ldg(reinterpret_cast<const uint32_t*>(q - (reinterpret_cast<uintptr_t>(q) & 2u)) + 32);
      };
      const uint32_t behind_last = behind(lane);
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) {
        const uint8_t* q = p + (size_t)i * (size_t)stride_bytes;
        w[i] = i < n ? __ldg(reinterpret_cast<const uint32_t*>(q - (reinterpret_cast<uintptr_t>(q) & 2u))) : 0u;
      }
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) {
        const uint8_t* q = p + (size_t)i * (size_t)stride_bytes;
        const uint32_t other = __shfl_down_sync(0xffffffffu, w[i], 1);
        const uint32_t next = __shfl_sync(0xffffffffu, behind_last, i);
        const uint32_t pair = __funnelshift_r(w[i], lane == 31 ? next : other, (uint32_t)(reinterpret_cast<uintptr_t>(q) & 2u) * 8u);
        w[i] = i < n ? pair : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p + (size_t)i * (size_t)stride_bytes);
        const bool in = r0 + i < rows;
        const uint32_t a = in && c < cols ? __ldg(q) : 0u, b = in && c + 1 < cols ? __ldg(q + 1) : 0u;
        w[i] = a | (b << 16);
      }
    }
    if (c >= cols) return;
  }
  const int blk = (int)(r0 / kMxBlock);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    uint32_t m = 0u;
    if constexpr (T::size == 2) {
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      m = T::mag(j ? m >> 16 : m & 0xFFFFu);
    } else {
#pragma unroll
      for (int i = 0; i < kMxBlock; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    }
    const uint32_t s = mx_scale(m);
    const float inv = mx_inv_scale(s);
    uint32_t q[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = w[g * 8 + i];
        if constexpr (T::size == 4) v[i] = __uint_as_float(b);
        else v[i] = j ? T::hi(b) : T::lo(b);
      }
      q[g] = mx_codes8(v, inv, s == 255u);
    }
    if (c + j >= cols) continue;
    if (blk < blocks)
      *reinterpret_cast<uint4*>(codes + ((size_t)(c + j) * blocks + blk) * 16) = make_uint4(q[0], q[1], q[2], q[3]);
    // (tiled: the padding blocks of the last group get scale 0, as no row exists)
    if (tiled) scales[mx_tiled_offset(c + j, blk >> 2, groups) + (blk & 3)] = (uint8_t)s;
    else if (blk < blocks) scales[(size_t)(c + j) * blocks + blk] = (uint8_t)s;
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
                                                                   uint32_t units, const FastDiv groups, int tiled,
                                                                   uint8_t* __restrict__ out, long long stride_bytes) {
  griddep_wait();
  griddep_launch();
  constexpr int EPL = lane_elems<T>(), LPU = unit_lanes<T>(), SUBS = block_subs<T>();
  const int sub = threadIdx.x / LPU, l = threadIdx.x & (LPU - 1);
  const uint32_t u0 = blockIdx.x * (uint32_t)(SUBS * U) + sub;
  const int blocks = mx_blocks(cols), bl = l / (LPU / 4);      // the lane's block of the unit
  __shared__ __align__(16) uint8_t warp_buf[is_narrow(VB) ? kMxThreads / 32 : 1][is_narrow(VB) ? kMxWarpBytes : 16];
  uint32_t q[U][2], s[U];
  int row[U], grp[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = min(u0 + (uint32_t)i * SUBS, units - 1);
    row[i] = (int)groups.quotient(u);
    grp[i] = (int)(u - (uint32_t)row[i] * groups.d);
    const int blk = grp[i] * 4 + bl;
    q[i][0] = q[i][1] = s[i] = 0u;
    if (blk < blocks) {
      const uint8_t* src = codes + (size_t)row[i] * (size_t)blocks * 16 + grp[i] * 64 + l * (EPL / 2);
      if constexpr (EPL == 16) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
        q[i][0] = v.x;
        q[i][1] = v.y;
      } else {
        q[i][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
      }
      s[i] = __ldg(scales + (tiled ? mx_tiled_offset(row[i], grp[i], (int)groups.d) + bl
                                   : (size_t)row[i] * blocks + blk));
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const float S = mx_scale_value(s[i]);
    float v[EPL];
#pragma unroll
    for (int h = 0; h < EPL / 8; ++h) mx_values8(q[i][h], v + 8 * h);
    const uint64_t S2 = pack_f32x2(S, S);
#pragma unroll
    for (int j = 0; j < EPL; j += 2) {
      const uint64_t r = mul_f32x2(pack_f32x2(v[j], v[j + 1]), S2);
      v[j] = lo_f32(r);
      v[j + 1] = hi_f32(r);
    }
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (T::size == 2) w[j] = T::pack(v[2 * j], v[2 * j + 1]);
      else w[j] = __float_as_uint(v[j]);
    }
    if constexpr (is_narrow(VB)) {
      store_staged<T, VB>(out, cols, stride_bytes, row[i], grp[i], u0 + (uint32_t)i * SUBS < units,
                          warp_buf[threadIdx.x >> 5], w);
    } else {
      const int c = grp[i] * kMxGroup + l * EPL;
      if (u0 + (uint32_t)i * SUBS >= units || c >= cols) continue;
      uint8_t* dst = out + (size_t)row[i] * (size_t)stride_bytes + (size_t)c * T::size;
      if (c + EPL <= cols) {
        store_words8<VB>(dst, w);
      } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          if (c + j < cols) {
            if constexpr (T::size == 2) reinterpret_cast<uint16_t*>(dst)[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
            else reinterpret_cast<uint32_t*>(dst)[j] = w[j];
          }
      }
    }
  }
}

// Units per group of lanes: two where that still leaves every SM eight blocks,
// else one, so that a few rows spread over the whole GPU.  Measured, one
// against two, 6144 columns of bf16 (us): 256 rows 1.75 and 1.83, 1600 rows
// 4.9 and 4.7, 8192 rows 21.8 and 21.0, 65536 rows 170 and 157.
constexpr int kMxUnits = 2;
template <typename T>
static inline bool many_units(uint32_t units, int sms) {
  return units >= (uint32_t)(sms * block_subs<T>() * kMxUnits * 8);
}

template <typename F>
static nvfp4_status with_type(int dtype, F&& f) {
  switch (dtype) {
    case MXFP4_DTYPE_BF16: return f(Bf16{});
    case MXFP4_DTYPE_F16: return f(F16{});
    default: return f(F32{});
  }
}
// Calls f(access width) with the width as a compile-time constant.
template <typename T, typename F>
static nvfp4_status with_width(int vb, F&& f) {
  if (vb == 32) return f(std::integral_constant<int, 32>{});
  if (vb == 16) return f(std::integral_constant<int, 16>{});
  if (vb == 8) return f(std::integral_constant<int, 8>{});
  if (vb == 4 || T::size == 4) return f(std::integral_constant<int, 4>{});
  if constexpr (T::size == 2) return f(std::integral_constant<int, 2>{});
  return NVFP4_ERR_INVALID_ARG;
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
                                cudaStream_t s, const int32_t* expert_offsets, const int32_t* expert_counts, int E) {
  uint32_t units = 0;
  NV_CHECK(count_units("mxfp4_quantize", out_rows, cols, &units));
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  const FastDiv groups((uint32_t)mx_groups(cols));
  const int tiled = layout == NVFP4_LAYOUT_TILED;
  const uint8_t* xb = static_cast<const uint8_t*>(x);
  return with_type(dtype, [&](auto tag) -> nvfp4_status {
    using T = decltype(tag);
    const long long sb = row_stride * T::size;
    const bool many = many_units<T>(units, sms);
    const uint32_t per_block = block_subs<T>() * (many ? kMxUnits : 1);
    const dim3 grid((units + per_block - 1) / per_block);
    return with_width<T>(row_access_bytes(x, rows > 1 ? sb : 0, T::size), [&](auto vb) -> nvfp4_status {
      constexpr int VB = decltype(vb)::value;
      if (perm && expert_counts && out_rows < 2ll * 127 * E)
        return launch_dependent("mx_quantize_rows_kernel", mx_quantize_rows_kernel<T, VB>, dim3((unsigned)out_rows),
                                dim3(kMxRowThreads), 0, s, xb, rows, cols, sb, perm, expert_offsets, expert_counts, E,
                                codes, scales);
      return launch_dependent("mx_quantize_kernel",
                              many ? mx_quantize_kernel<T, VB, kMxUnits> : mx_quantize_kernel<T, VB, 1>, grid,
                              dim3(kMxThreads), 0, s, xb, rows, cols, sb, perm, units, groups, tiled, codes, scales);
    });
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
  NV_REQUIRE(rows <= 65535 * kMxTRows, NVFP4_ERR_UNSUPPORTED_SHAPE, "mxfp4_quantize_transposed: rows=%d is above %d",
             rows, 65535 * kMxTRows);
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  const int groups = mx_groups(rows), tiled = layout == NVFP4_LAYOUT_TILED;
  const uint8_t* xb = static_cast<const uint8_t*>(x);
  cudaStream_t s = as_stream(stream);
  return with_type(dtype, [&](auto tag) -> nvfp4_status {
    using T = decltype(tag);
    constexpr int C = 4 / T::size;
    const long long sb = row_stride * T::size;
    // one word a thread and row: needs 4-byte aligned rows and, for pairs, a
    // second column in the last pair
    const bool wide = row_access_bytes(x, rows > 1 ? sb : 0, T::size) >= 4 && cols % C == 0;
    const dim3 grid((unsigned)((cols + 32ll * C - 1) / (32 * C)),
                    (unsigned)((groups * kMxGroup + kMxTRows - 1) / kMxTRows));
    if constexpr (C == 2) {
      if (!wide)
        return launch_dependent("mx_quantize_t_kernel", mx_quantize_t_kernel<T, C, false>, grid, dim3(kMxTThreads), 0,
                                s, xb, rows, cols, sb, groups, tiled, codes, scales);
    }
    return launch_dependent("mx_quantize_t_kernel", mx_quantize_t_kernel<T, C, true>, grid, dim3(kMxTThreads), 0, s,
                            xb, rows, cols, sb, groups, tiled, codes, scales);
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
  const FastDiv groups((uint32_t)mx_groups(cols));
  const int tiled = layout == NVFP4_LAYOUT_TILED;
  uint8_t* ob = static_cast<uint8_t*>(out);
  return with_type(dtype, [&](auto tag) -> nvfp4_status {
    using T = decltype(tag);
    const long long sb = row_stride * T::size;
    const bool many = many_units<T>(units, sms);
    const uint32_t per_block = block_subs<T>() * (many ? kMxUnits : 1);
    const dim3 grid((units + per_block - 1) / per_block);
    return with_width<T>(row_access_bytes(out, rows > 1 ? sb : 0, T::size), [&](auto vb) -> nvfp4_status {
      constexpr int VB = decltype(vb)::value;
      return launch_dependent("mx_dequantize_kernel",
                              many ? mx_dequantize_kernel<T, VB, kMxUnits> : mx_dequantize_kernel<T, VB, 1>, grid,
                              dim3(kMxThreads), 0, as_stream(stream), codes, scales, cols, units, groups, tiled, ob,
                              sb);
    });
  });
}
