// MXFP4 products on the 5th-generation tensor cores (tcgen05, sm_100a):
// y[m][n] = row_weight[m] * (sum_k a[m][k] b[n][k] + bias[n]), dense or
// grouped by expert.
//
// The block scales are applied inside the MMA (kind::mxf4, scale_vec::2X: two
// E8M0 bytes per row and 64-element step): products of E2M1 values under powers
// of two are exact, their sums fp32 (operands with a common scale sum exactly
// up to 2^24 units), bias and row weight one fp32 operation each, and the
// store rounds to the output type.
//
// Orientation: the 128 rows of an MMA tile (the tensor-memory lanes) are rows
// of b, its N columns are rows of a ("tokens").  A decoding step's few tokens
// are then a narrow N (16 columns) instead of a 128-row tile that is nearly
// empty, and a warp's 32 lanes hold 32 neighbouring outputs of one token, so
// y leaves straight from registers, coalesced for any N.
//
// One CTA per tile of 128 b rows x up to 128 tokens; warp 0 issues the loads
// (TMA for codes, bulk copies for scale atoms), warp 1 the MMAs, warps 2..9
// drain the accumulator.  A K stage is 256 elements: 128-byte code rows in the
// 128-byte swizzle, two scale atoms per 128 rows.
//
// Few tiles (a decoding step) split K over a cluster of CTAs: each leaves its
// fp32 partial sums in its own shared memory and, behind a cluster barrier,
// rank r adds the columns r, r + S, ... of all of them in rank order and
// stores them, so the result does not depend on scheduling and takes no
// second kernel and no workspace.
//
// Bound: many tokens by the tensor pipe (the power-capped clock included) and
// by how fast L2 feeds the SMs, few tokens by HBM reading b, a single small
// product by the chain launch, TMA, MMA, join, store.  Measured on one B200,
// bf16 outputs, in a stream of calls:
//   8192 x 4096 x 6144   72 us, 5.7 PFLOP/s (0.86 of four times the measured
//                        bf16 rate)
//   1024 x 4096 x 6144   16 us; 256 x 6144 x 6144 13 us; 64 x 6144 x 6144 9.7
//   16 x 6144 x 6144     8.1 us, 2.4 TB/s; 1 x 6144 x 6144 7.5 us (b in L2: 6.8, 6.5)
//   1 x 6144 x 6144 with x quantised in the same kernel 7.9 us (two kernels 9.5)
//   16 tokens, top-8 of 80 experts, 4096 x 6144: 140 us, 97 % of the copy rate
// What brought it there, at 8192 x 4096 x 6144: one CTA a tile, the accumulator
// held while it was stored, 125 us; CTA pairs 111; outputs packed before the
// hand-over by straight-line code that fits the instruction cache 74 (the
// epilogue took longer than the K loop); at 256 x 6144 x 6144, all ranks' sums
// loaded before the first is added and splits that fit the GPU at once, 48 us
// to 13; two CTAs on an SM where there are more tiles than SMs, the 80 experts
// 146 us to 140.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "mx.cuh"
#include "../../include/nvfp4_moe_testing.h"

namespace nvfp4moe {

constexpr int kXBM = 128;                        // b rows per tile
constexpr int kXNT = 128;                        // tokens per tile, at most
constexpr int kXBK = 256;                        // K elements per stage
constexpr int kXRowBytes = kXBK / 2;             // 128 bytes of codes per row and stage
constexpr int kXWBytes = kXBM * kXRowBytes;      // 16 KiB
constexpr int kXAtoms = kXBK / kMxGroup;         // 2 scale atoms per 128 rows and stage
constexpr int kXSfBytes = kXAtoms * kAtomBytes;  // 1 KiB
constexpr int kXThreads = 320;
constexpr int kXEpiWarps = 8;
constexpr int kXMaxStages = 8;
constexpr int kXMaxE = 1024;
constexpr int kXMaxSplits = 4;                   // CTAs of a cluster that share K, at most (plan_mx_gemm)
// Dynamic shared memory of a CTA that has an SM to itself, and of one of two
// on an SM (228 KiB less 1 KiB a CTA; the static part is below 256 bytes).
constexpr int kXMaxSmem = 227 * 1024 - 256;
constexpr int kXSmemPair = 228 * 1024 / 2 - 1024 - 256;
constexpr int kXFuseSmem = 256;                  // further barriers of a fused product

struct MxGemmParams {
  int M, N, E;               // E = 0: dense
  int groups;                // scale atoms along K
  int kt_total;              // K stages
  int n_wt, n_tt;            // b tiles (per expert), token tiles (dense)
  int nt;                    // tokens per tile
  int stages;
  int n_acc;                 // accumulators that tiles alternate between
  int splits;                // K splits (CTAs per cluster)
  int pairs;                 // 16-bit y whose rows are 4-byte aligned (pair kernel)
  int quads;                 // y whose rows are aligned to four elements
  int early_b;               // b is not written by the previous kernel of this call: load before the wait
  const int32_t* expert_offsets;
  const int32_t* expert_counts;
  const uint8_t* a_sf;
  const uint8_t* b_sf;
  const float* row_weight;
  const float* bias;
  void* y;
  long long y_stride;
  uint32_t* status;
  // FUSED: the unquantised rows
  const uint8_t* x;
  const int32_t* perm;
  long long x_stride;        // bytes
  int x_rows, x_dtype, x_wide, K;
};

// One stage: b codes, token codes, b scales, token scales.
__host__ __device__ constexpr int mx_stage_bytes(int nt) { return kXWBytes + nt * kXRowBytes + 2 * kXSfBytes; }

// Fused: a stage holds b only; behind the stages, a's codes and scales of every K stage.
constexpr int kXFuseStageBytes = kXWBytes + kXSfBytes;
__host__ __device__ constexpr int mx_fused_a_bytes(int nt) { return nt * kXRowBytes + kXSfBytes; }
// Columns of an accumulator, and tensor memory that a CTA allocates: its
// accumulators and the scales of b and of the tokens behind them.
__host__ __device__ constexpr int mx_acc_columns(int nt) { return nt > 32 ? nt : 32; }
__host__ __device__ constexpr uint32_t mx_tmem_columns(int nt, int n_acc) {
  const uint32_t need = (uint32_t)(n_acc * mx_acc_columns(nt)) + 4 * kXAtoms * 2;
  return need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
}
// Instruction descriptor: kind::mxf4, E2M1 x E2M1, UE8M0 scales, K-major
// operands, M x N tile, the scales of byte pair `id` (0 or 2) of each word.
NVDEV uint32_t idesc_mxf4(int M, int N, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) |
         (id << 29);
}
NVDEV void mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa_tmem,
                    uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem));
}
NVDEV float4 ld_shared_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A tile of the work list: its expert, its first token row, its tokens and
// its b tile.
struct MxTile {
  int e, row0, tokens, wt;
};

// Grouped products: every expert's first tile group (`nt` tokens of one
// expert), first row and tokens, in shared memory behind the stages.
struct MxSegments {
  int *start, *row0, *tokens;      // [E + 1], [E], [E]
};
__host__ __device__ constexpr int mx_segment_bytes(int E) { return E ? (3 * E + 1) * 4 : 0; }
NVDEV MxSegments mx_scan_segments(const MxGemmParams& p, uint8_t* at) {
  MxSegments g;
  g.start = reinterpret_cast<int*>(at);
  g.row0 = g.start + p.E + 1;
  g.tokens = g.row0 + p.E;
  if (p.E == 0) return g;
  if ((threadIdx.x >> 5) == 0) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int v = 0;
      if (e < p.E) {
        const MxSegment s = mx_segment(p.expert_offsets, p.expert_counts, p.M, e);
        g.row0[e] = s.row0;
        g.tokens[e] = s.rows;
        v = (s.rows + p.nt - 1) / p.nt;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (e < p.E) g.start[e + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) g.start[0] = 0;
  }
  __syncthreads();
  return g;
}
NVDEV int mx_num_tiles(const MxGemmParams& p, const MxSegments& g) {
  return (p.E == 0 ? p.n_tt : g.start[p.E]) * p.n_wt;
}
NVDEV MxTile mx_tile(const MxGemmParams& p, const MxSegments& s, int t) {
  MxTile c;
  c.wt = t % p.n_wt;
  const int g = t / p.n_wt;
  if (p.E == 0) {
    c.e = 0;
    c.row0 = g * p.nt;
    c.tokens = min(p.nt, p.M - c.row0);
    return c;
  }
  int lo = 0, hi = p.E - 1;                      // the last expert whose tiles start at or before g
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.start[mid] <= g) lo = mid; else hi = mid - 1;
  }
  const int j = g - s.start[lo];
  c.e = lo;
  c.row0 = s.row0[lo] + j * p.nt;
  c.tokens = min(p.nt, s.tokens[lo] - j * p.nt);
  return c;
}

template <typename T>
NVDEV void mx_store(void* y, size_t i, float v) {
  if constexpr (T::size == 2) static_cast<uint16_t*>(y)[i] = T::one(v);
  else static_cast<float*>(y)[i] = v;
}

// Bias and row weight of one accumulator value.  PLAIN: neither.
template <bool PLAIN>
NVDEV float mx_value(uint32_t acc, float weight, float bias) {
  const float v = __uint_as_float(acc);
  return PLAIN ? v : __fmul_rn(__fadd_rn(v, bias), weight);
}
// The row weights of 32 tokens from m0 on, one a lane (1 where there are
// none); mx_weight broadcasts token i's.
template <bool PLAIN>
NVDEV float mx_load_weight(const MxGemmParams& p, int m0, int cnt) {
  const int lane = threadIdx.x & 31;
  return !PLAIN && p.row_weight && lane < cnt ? __ldg(p.row_weight + m0 + lane) : 1.0f;
}
template <bool PLAIN>
NVDEV float mx_weight(float held, int i) {
  return PLAIN ? 1.0f : __shfl_sync(0xffffffffu, held, i);
}

// 16-bit outputs of two neighbouring tokens m, m + 1 of the thread's column n,
// packed in one word (m in the low half).  The lanes of the warp hold 32
// neighbouring n: lanes trade halves with their neighbour, so that each stores
// two neighbouring outputs of one token (even lanes m, odd lanes m + 1) where
// rows of y are 4-byte aligned.  `left`: real tokens from m on.
NVDEV void mx_store_pair(const MxGemmParams& p, uint32_t word, uint16_t* at, int left, int n) {
  const uint32_t got = __shfl_xor_sync(0xffffffffu, word, 1);
  const bool odd = n & 1;
  const uint32_t v = __byte_perm(word, got, odd ? 0x3276 : 0x5410);
  if (left > (odd ? 1 : 0)) {
    if ((n | 1) < p.N) *reinterpret_cast<uint32_t*>(at) = v;
    else if ((n & ~1) < p.N) *at = (uint16_t)v;              // y's last column is an even one
  }
}

// A thread's 32 accumulator columns (tokens m0 ..., the first `cnt` real) of
// output column n; `held` from mx_load_weight.  (Storing pairs here, as the
// pair kernel does, measured slower: 12.1 us against 11.3 at 1000 x 2500 x
// 2000 bf16.)
template <typename T, bool PLAIN>
NVDEV void mx_store32(const MxGemmParams& p, const uint32_t* r, int m0, int cnt, int n, float bias, float held) {
  size_t at = (size_t)m0 * (size_t)p.y_stride + n;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float w = mx_weight<PLAIN>(held, i);               // every lane takes part in the shuffle
    if (i < cnt && n < p.N) mx_store<T>(p.y, at, mx_value<PLAIN>(r[i], w, bias));
    at += (size_t)p.y_stride;
  }
}

// FUSED: the epilogue's warps, idle until the accumulator is full, quantise
// this CTA's share of K of every token into shared memory behind the stages:
// for each K stage the codes as the TMA would put them (128-byte rows, 16-byte
// chunk c of row r at c ^ (r & 7)), then for each K stage the scale atoms.
// Units (stage, token, atom) go over the warps in that order; a stage's barrier
// counts the warps.  A rolled loop without loads ahead: the passes are few, and
// fetching straight-line code costs more than it saves (four passes at a time
// with their loads first: 6.0 us for 1 x 1024 x 6144, one by one 5.4).
constexpr int kXFuseTokens = 16;                 // rows of x that a product quantises itself, at most
constexpr int kXFuseStages = 32;                 // and K stages of a CTA
template <typename T> __host__ __device__ constexpr int fuse_pass() { return kXEpiWarps * 32 / unit_lanes<T>(); }
template <typename T, bool WIDE>
NVDEV void mx_quantize_tokens(const MxGemmParams& p, uint8_t* at_codes, uint8_t* at_scales, int kt0, int nkt,
                              uint64_t* a_bar) {
  constexpr int EPL = lane_elems<T>(), LPU = unit_lanes<T>(), kPass = fuse_pass<T>();
  const int lane = threadIdx.x & 31, l = lane & (LPU - 1);
  const int mine = ((threadIdx.x >> 5) - 2) * (32 / LPU) + lane / LPU;
  const int per = 2 * p.M, units = nkt * per;                // units of a stage, of all
  // u / per = u m >> 16, exact for u < 2^16 / per (here u < units + kPass)
  static_assert((kXFuseStages * 2 * kXFuseTokens + fuse_pass<Bf16>()) * 2 * kXFuseTokens <= 65536, "unit division");
  const uint32_t m = 65536u / (uint32_t)per + 1u;
  const uint8_t* x_end = p.x + (size_t)(p.x_rows - 1) * (size_t)p.x_stride + (size_t)p.K * T::size;
  int done = 0;                                              // stages handed over
#pragma unroll 1
  for (int first = 0; first < units; first += kPass) {
    const int u = first + mine, i = (int)(((uint32_t)u * m) >> 16), r = u - i * per, row = r >> 1, atom = r & 1;
    const int src = u >= units ? -1 : p.perm ? __ldg(p.perm + row) : row;
    const int n = src >= 0 && src < p.x_rows ? p.K : 0;      // a row without a source reads as zeros
    uint32_t w[8];
    load_share<T, WIDE ? 16 : T::size>(p.x + (n ? (size_t)src * (size_t)p.x_stride : 0),
                                       ((kt0 + i) * kXAtoms + atom) * kMxGroup + l * EPL, n, p.x, x_end, w);
    uint32_t q[EPL / 8], sf;
    mx_unit<T>(w, q, sf);
    if (u < units) {
      const int byte = atom * 64 + l * (EPL / 2);
      uint8_t* dst = at_codes + (i * p.nt + row) * kXRowBytes + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
      if constexpr (EPL == 16) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
      else *reinterpret_cast<uint32_t*>(dst) = q[0];
      if (l == 0) *reinterpret_cast<uint32_t*>(at_scales + i * kXSfBytes + atom * kAtomBytes + row * 16) = sf;
    }
    const int all = min(first + kPass, units);               // units that the warps have now
    if ((done + 1) * per <= all) {
      fence_proxy_async();                                   // the MMA reads through the async proxy
      __syncwarp();
      for (; (done + 1) * per <= all; ++done)
        if (lane == 0) mbar_arrive(&a_bar[done]);
    }
  }
}

// PLAIN: neither bias nor row weight.  FUSED: a single tile a CTA, dense, its
// tokens quantised here.
template <typename T, bool PLAIN, bool FUSED>
__global__ void __launch_bounds__(kXThreads, 2)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ CUtensorMap tmX32, const MxGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kXMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[kXMaxStages];
  __shared__ __align__(8) uint64_t acc_full_bar[2];
  __shared__ __align__(8) uint64_t acc_empty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ __align__(8) uint64_t a_bar[FUSED ? kXFuseStages : 1];
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // A CTA that has its SM to itself alternates between two accumulators, so
  // that the next tile's MMAs run while one is drained; of two CTAs on an SM
  // one works while the other drains, and wide ones have half of tensor memory
  // each, room for one.
  const int nt_pad = mx_acc_columns(p.nt), n_acc = p.n_acc;
  const uint32_t tcols = mx_tmem_columns(p.nt, n_acc);
  // (FUSED: a's codes and scales lie behind the stages, for all of K)
  const int stage_bytes = FUSED ? kXFuseStageBytes : mx_stage_bytes(p.nt);
  const int x_bytes = FUSED ? 0 : p.nt * kXRowBytes;         // nt is a multiple of 16: whole 8-row swizzle groups
  // this CTA's share of K
  const int rank = p.splits > 1 ? (int)cluster_ctarank() : 0;
  const int kt0 = (int)((long long)p.kt_total * rank / p.splits);
  const int nkt = (int)((long long)p.kt_total * (rank + 1) / p.splits) - kt0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full_bar[i], 1);
      mbar_init(&acc_empty_bar[i], kXEpiWarps);
    }
    mbar_init(&drain_bar, 1);
    if constexpr (FUSED) {
      for (int i = 0; i < nkt; ++i) mbar_init(&a_bar[i], kXEpiWarps);
    }
    abort_s = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    if constexpr (!FUSED) {
      prefetch_tmap(&tmX);
      prefetch_tmap(&tmX32);
    }
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_s, tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  const int t_first = p.splits > 1 ? (int)blockIdx.x / p.splits : (int)blockIdx.x;
  const int t_step = p.splits > 1 ? (int)gridDim.x / p.splits : (int)gridDim.x;
  const size_t sf_tile = (size_t)p.groups * kAtomBytes;      // one 128-row tile's scales

  auto load_b = [&](int wt, int e, int kt, int stage) {
    uint8_t* sW = smem + stage * stage_bytes;
    const int brow = e * p.N + wt * kXBM;
    const uint32_t sf_bytes = (uint32_t)min(kXAtoms, p.groups - kt * kXAtoms) * kAtomBytes;
    tma_load_2d(sW, &tmW, kt * kXRowBytes, brow, &full_bar[stage]);
    bulk_load(sW + kXWBytes + x_bytes, p.b_sf + (size_t)(brow / kRowTile) * sf_tile + (size_t)kt * kXSfBytes, sf_bytes,
              &full_bar[stage]);
  };

  // A call that quantised its own a (early_b) has nothing but a to wait for:
  // the quantiser ran behind everything older.  The tile list is made and the
  // pipeline filled with b while the quantiser still runs.
  MxSegments segs;
  int early = 0;
  if (p.early_b) {
    segs = mx_scan_segments(p, smem + p.stages * stage_bytes);
    if (t_first < mx_num_tiles(p, segs)) early = min(p.stages, nkt);
    if (warp == 0 && early && elect_one()) {
      const MxTile c = mx_tile(p, segs, t_first);
      for (int i = 0; i < early; ++i) load_b(c.wt, c.e, kt0 + i, i);
    }
    __syncwarp();
  }
  griddep_wait();
  griddep_launch();
  // first kernel of a call: the status word is cleared here, before any wait
  // of this call can give up
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  if (!p.early_b) segs = mx_scan_segments(p, smem + p.stages * stage_bytes);
  const int num_tiles = mx_num_tiles(p, segs);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t elected = elect_one();
    int stage = 0, issued = 0;
    uint32_t phase = 0, filled = 0, fill_parity = 0;
    bool ok = true;
    for (int t = t_first; ok && t < num_tiles; t += t_step) {
      const MxTile c = mx_tile(p, segs, t);
      // token rows in 32-row boxes where a tile is not full (dense tiles:
      // rows past M read as zeros and move no bytes)
      const bool whole = p.E == 0 || c.tokens > p.nt - 32;
      const int boxes = (c.tokens + 31) / 32;
      const uint32_t xb = (uint32_t)(whole ? p.nt : boxes * 32) * kXRowBytes;
      for (int i = 0; i < nkt; ++i, ++issued) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag));
        if (!ok) {
          if (elected) {
            *abort_flag = 1;
            atomicExch(p.status, kDevTimeout);
          }
          break;
        }
        if (elected) {
          const int kt = kt0 + i;
          uint8_t* sX = smem + stage * stage_bytes + kXWBytes;
          uint8_t* sSFX = sX + x_bytes + kXSfBytes;
          const uint32_t sf_bytes = (uint32_t)min(kXAtoms, p.groups - kt * kXAtoms) * kAtomBytes;
          mbar_arrive_expect_tx(&full_bar[stage], kXWBytes + (FUSED ? sf_bytes : xb + 2 * sf_bytes));
          if (issued >= early) load_b(c.wt, c.e, kt, stage);
          if constexpr (FUSED) {
          } else if (whole) {
            tma_load_2d(sX, &tmX, kt * kXRowBytes, c.row0, &full_bar[stage]);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(sX + b * 32 * kXRowBytes, &tmX32, kt * kXRowBytes, c.row0 + 32 * b, &full_bar[stage]);
          }
          if constexpr (!FUSED)
            bulk_load(sSFX, p.a_sf + (size_t)(c.row0 / kRowTile) * sf_tile + (size_t)kt * kXSfBytes, sf_bytes,
                    &full_bar[stage]);
        }
        __syncwarp();
        filled |= 1u << stage;
        fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && elected) {
      // every copy already issued lands before the CTA's shared memory goes away
      volatile int never = 0;
      for (int s = 0; s < p.stages; ++s)
        if ((filled >> s) & 1u) mbar_wait(&full_bar[s], (fill_parity >> s) & 1u, &never);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // the whole warp runs the loop and one elected lane issues (a loop run by
    // a single divergent lane issues too slowly to keep the tensor pipe busy)
    const uint32_t elected = elect_one();
    const uint32_t s0 = smem_u32(smem);
    const uint32_t a_at = s0 + p.stages * stage_bytes;
    const uint64_t w0 = sdesc_sw128(s0), x0 = sdesc_sw128(FUSED ? a_at : s0 + kXWBytes);
    const uint64_t sfw0 = sdesc_scale_atom(s0 + kXWBytes + x_bytes);
    const uint64_t sfx0 = sdesc_scale_atom(FUSED ? a_at + nkt * p.nt * kXRowBytes : s0 + kXWBytes + x_bytes + kXSfBytes);
    const uint64_t stage_step = (uint64_t)stage_bytes >> 4;
    constexpr uint64_t kAtomStep = kAtomBytes >> 4;
    const uint32_t sfw_t = tmem + (uint32_t)(n_acc * nt_pad), sfx_t = sfw_t + 4 * kXAtoms;
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = t_first; ok && t < num_tiles; t += t_step) {
      const MxTile c = mx_tile(p, segs, t);
      const int n_mma = (c.tokens + 15) & ~15;
      const uint32_t id0 = idesc_mxf4(kXBM, n_mma, 0), id2 = idesc_mxf4(kXBM, n_mma, 2);
      ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty_bar[buf], acc_phase ^ 1u, abort_flag));
      if (!ok) {
        if (elected) {
          *abort_flag = 1;
          atomicExch(p.status, kDevTimeout);
        }
        break;
      }
      tc_fence_after();
      const uint32_t acc_t = tmem + (uint32_t)(buf * nt_pad);
      uint32_t accumulate = 0;
      for (int i = 0; i < nkt; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort_flag) &&
                                         (!FUSED || mbar_wait(&a_bar[FUSED ? i : 0], 0, abort_flag)));
        if (!ok) {
          if (elected) {
            *abort_flag = 1;
            atomicExch(p.status, kDevTimeout);
          }
          break;
        }
        const bool whole = p.groups - (kt0 + i) * kXAtoms >= kXAtoms;     // else K ends with one atom
        if (elected) {
          const uint64_t d = (uint64_t)stage * stage_step;
          const uint64_t dx = FUSED ? (uint64_t)(i * p.nt * kXRowBytes >> 4) : d;
          const uint64_t dsx = FUSED ? (uint64_t)(i * kXSfBytes >> 4) : d;
          // straight-line code for either length of a stage: a branch per
          // instruction would starve the tensor pipe
          auto issue = [&](auto n_atoms) {
            constexpr int A = decltype(n_atoms)::value;
#pragma unroll
            for (int j = 0; j < A; ++j) {
              tc_cp_scale_atom(sfw_t + 4 * j, sfw0 + d + j * kAtomStep);
              tc_cp_scale_atom(sfx_t + 4 * j, sfx0 + dsx + j * kAtomStep);
            }
#pragma unroll
            for (int j = 0; j < 2 * A; ++j)          // 64 elements = 32 bytes of K per MMA, two per atom
              mma_mxf4(acc_t, w0 + d + 2 * j, x0 + dx + 2 * j, (j & 1) ? id2 : id0, sfw_t + 4 * (j >> 1),
                       sfx_t + 4 * (j >> 1), accumulate | j);
          };
          if (whole) issue(std::integral_constant<int, kXAtoms>{});
          else issue(std::integral_constant<int, 1>{});
          tc_commit(&empty_bar[stage]);
        }
        __syncwarp();
        accumulate = 1;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elected) tc_commit(&acc_full_bar[buf]);
      __syncwarp();
      if (++buf == n_acc) {
        buf = 0;
        acc_phase ^= 1u;
      }
    }
    // every MMA completes before tensor memory is freed
    if (elected) {
      tc_commit(&drain_bar);
      volatile int never = 0;
      mbar_wait(&drain_bar, 0, &never);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int n_in = quad * 32 + lane;
    const uint32_t tacc = tmem + ((uint32_t)(quad * 32) << 16);
    float* red = reinterpret_cast<float*>(smem);             // split K: [token][128], the idle stages
    int buf = 0;
    uint32_t acc_phase = 0;
    if constexpr (FUSED) {
      uint8_t* codes = smem + p.stages * stage_bytes;
      uint8_t* scales = codes + nkt * p.nt * kXRowBytes;
      auto quantize = [&](auto tag) {
        if (p.x_wide) mx_quantize_tokens<decltype(tag), true>(p, codes, scales, kt0, nkt, a_bar);
        else mx_quantize_tokens<decltype(tag), false>(p, codes, scales, kt0, nkt, a_bar);
      };
      if (p.x_dtype == MXFP4_DTYPE_BF16) quantize(Bf16{});
      else if (p.x_dtype == MXFP4_DTYPE_F16) quantize(F16{});
      else quantize(F32{});
    }
    for (int t = t_first; t < num_tiles; t += t_step) {
      const MxTile c = mx_tile(p, segs, t);
      const int n = c.wt * kXBM + n_in;
      const float bias = !PLAIN && p.bias && n < p.N && p.splits == 1 ? p.bias[(size_t)c.e * p.N + n] : 0.0f;
      if (!mbar_wait(&acc_full_bar[buf], acc_phase, abort_flag)) {
        *abort_flag = 1;
        atomicExch(p.status, kDevTimeout);
        break;
      }
      tc_fence_after();
      // handed back as soon as the warp has read its last columns
      bool held = true;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty_bar[buf]);
        held = false;
      };
#pragma unroll 1
      for (int col = half * 32; col < c.tokens; col += 64) {
        uint32_t r[32];
        tmem_ld32(tacc + buf * nt_pad + col, r);
        const int cnt = min(32, c.tokens - col);
        const float weights = mx_load_weight<PLAIN>(p, c.row0 + col, cnt);
        tmem_ld_wait();
        if (col + 64 >= c.tokens) release();
        if (p.splits > 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < cnt) red[(col + i) * kXBM + n_in] = __uint_as_float(r[i]);
        } else {
          mx_store32<T, PLAIN>(p, r, c.row0 + col, cnt, n, bias, weights);
        }
      }
      if (held) release();
      if (++buf == n_acc) {
        buf = 0;
        acc_phase ^= 1u;
      }
    }
    __syncwarp();
  }
  if (p.splits > 1) {
    // one tile per cluster (the grid has splits CTAs per tile)
    cluster_sync_all();                                      // every rank's partial sums are in place
    if (warp >= 2 && t_first < num_tiles) {
      // A warp adds one token's 128 sums, four neighbouring outputs a lane;
      // tokens rank, rank + S, ... are this CTA's.  All ranks' loads are
      // issued before the first is added: one trip to the neighbours a token.
      const MxTile c = mx_tile(p, segs, t_first);
      const int n = c.wt * kXBM + lane * 4;
      const uint32_t red = smem_u32(smem) + lane * 16;
      float bias[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        bias[j] = !PLAIN && p.bias && n + j < p.N ? p.bias[(size_t)c.e * p.N + n + j] : 0.0f;
      for (int m = rank + p.splits * (warp - 2); m < c.tokens; m += p.splits * kXEpiWarps) {
        float4 v[kXMaxSplits];
#pragma unroll
        for (int q = 0; q < kXMaxSplits; ++q)
          if (q < p.splits) v[q] = ld_shared_cluster_f32x4(mapa_shared(red + (uint32_t)m * (kXBM * 4), (uint32_t)q));
        float4 z = v[0];
#pragma unroll
        for (int q = 1; q < kXMaxSplits; ++q)
          if (q < p.splits) {
            z.x = __fadd_rn(z.x, v[q].x);
            z.y = __fadd_rn(z.y, v[q].y);
            z.z = __fadd_rn(z.z, v[q].z);
            z.w = __fadd_rn(z.w, v[q].w);
          }
        const float w = !PLAIN && p.row_weight ? __ldg(p.row_weight + c.row0 + m) : 1.0f;
        const float o[4] = {mx_value<PLAIN>(__float_as_uint(z.x), w, bias[0]),
                            mx_value<PLAIN>(__float_as_uint(z.y), w, bias[1]),
                            mx_value<PLAIN>(__float_as_uint(z.z), w, bias[2]),
                            mx_value<PLAIN>(__float_as_uint(z.w), w, bias[3])};
        const size_t at = (size_t)(c.row0 + m) * (size_t)p.y_stride + n;
        if (p.quads && n + 3 < p.N) {
          if constexpr (T::size == 2)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) = make_uint2(T::pack(o[0], o[1]), T::pack(o[2], o[3]));
          else
            *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < p.N) mx_store<T>(p.y, at + j, o[j]);
        }
      }
    }
    __syncwarp();
    cluster_sync_all();                                      // no rank leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

// ---------------------------------------------------------------------------
// CTA pairs, for products with many tiles: clusters of two CTAs share one
// .cta_group::2 MMA of 256 b rows x kPNT tokens (each CTA 128 of the b rows
// and half of the tokens).  Per 256-element K stage a CTA then loads 16 KiB of
// b, 24 KiB of tokens and 4 KiB of scales for 768 MMA cycles, 58 bytes a cycle
// where a CTA by itself needs 102: L2 feeds an SM at 60-odd.  384 tokens (an
// MMA of 256 and one of 128 columns) instead of 256 is what tensor memory
// holds beside the scales, and takes 1.5 times fewer accumulator hand-overs.
// No load is multicast: each CTA reads its own share.
// ---------------------------------------------------------------------------
constexpr int kPNT = 384;
constexpr int kPQ = kPNT / 128;                   // 128-token scale tiles
constexpr int kPXBytes = kPNT / 2 * kXRowBytes;   // 24 KiB of tokens per CTA
constexpr int kPSfBytes = kXSfBytes * (1 + kPQ);  // 4 KiB
constexpr int kPStageBytes = kXWBytes + kPXBytes + kPSfBytes;
constexpr int kPStages = 5;
constexpr int kPEpiWarps = 4 * kPQ;               // 128 accumulator columns a thread
constexpr int kPThreads = 64 + 32 * kPEpiWarps;
constexpr int kPMaxE = 480;                       // experts whose segment table fits behind the stages
static_assert(kPStages * kPStageBytes + mx_segment_bytes(kPMaxE) + 1024 <= kXMaxSmem, "pair kernel shared memory");
constexpr uint32_t kPSfCol = kPNT;                // scales behind the accumulator
static_assert(kPNT + 4 * kXAtoms * (1 + kPQ) <= 512, "tensor memory");

NVDEV void mma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa_tmem,
                         uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem));
}
// A CTA that gives up also ends the other CTA's waits.
NVDEV void mx_give_up_pair(uint32_t* status, volatile int* abort_flag, uint32_t peer_abort) {
  *abort_flag = 1;
  atomicExch(status, kDevTimeout);
  asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(peer_abort) : "memory");
}

struct MxPairMaps {
  CUtensorMap w, x, x64;      // codes: boxes of 128, 128 and 64 rows
  CUtensorMap sfw, sfx;       // scale atoms as rows of 128 words, two per stage
};

template <typename T, bool PLAIN>
__global__ void __launch_bounds__(kPThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ MxPairMaps tm, const MxGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kPStages];
  __shared__ __align__(8) uint64_t empty_bar[kPStages];
  __shared__ __align__(8) uint64_t acc_full_bar;
  __shared__ __align__(8) uint64_t acc_empty_bar;
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPStages; ++s) {
      // only the leader's producer arrives on the leader's stage barrier,
      // expecting the bytes of both CTAs
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&acc_full_bar, 1);
    mbar_init(&acc_empty_bar, 2 * kPEpiWarps);               // drained by both CTAs
    mbar_init(&drain_bar, 1);
    abort_s = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm.w);
    prefetch_tmap(&tm.x);
    prefetch_tmap(&tm.x64);
    prefetch_tmap(&tm.sfw);
    prefetch_tmap(&tm.sfx);
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_s, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();            // both CTAs' barriers exist before either touches the other's
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  const uint32_t peer_abort = mapa_shared(smem_u32(&abort_s), rank ^ 1u);
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;

  const MxSegments segs = mx_scan_segments(p, smem + kPStages * kPStageBytes);
  const int num_tiles = mx_num_tiles(p, segs);
  const int t_first = (int)(blockIdx.x >> 1), t_step = (int)(gridDim.x >> 1);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t elected = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = t_first; ok && t < num_tiles; t += t_step) {
      const MxTile c = mx_tile(p, segs, t);
      const int brow = c.e * p.N + (c.wt * 2 + (int)rank) * kXBM;
      const int sfw_row = brow / kRowTile * p.groups, sfx_row = c.row0 / kRowTile * p.groups;
      for (int kt = 0; kt < p.kt_total; ++kt) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag));
        if (!ok) {
          if (elected) mx_give_up_pair(p.status, abort_flag, peer_abort);
          break;
        }
        if (elected) {
          uint8_t* sW = smem + stage * kPStageBytes;
          uint8_t* sX = sW + kXWBytes;
          uint8_t* sSF = sX + kPXBytes;
          // every load of both CTAs counts on the leader's stage barrier; the
          // other CTA's bytes may land first (the phase cannot complete
          // before the leader's arrival)
          const uint32_t fb = mapa_shared(smem_u32(&full_bar[stage]), 0);
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2u * (uint32_t)kPStageBytes);
          const int x = kt * kXRowBytes, ka = kt * kXAtoms;
          tma_load_2d_pair(sSF, &tm.sfw, 0, sfw_row + ka, fb);
#pragma unroll
          for (int h = 0; h < kPQ; ++h)
            tma_load_2d_pair(sSF + kXSfBytes * (1 + h), &tm.sfx, 0, sfx_row + h * p.groups + ka, fb);
          tma_load_2d_pair(sW, &tm.w, x, brow, fb);
          // the CTA's half of each MMA's tokens
          tma_load_2d_pair(sX, &tm.x, x, c.row0 + (int)rank * 128, fb);
          tma_load_2d_pair(sX + 128 * kXRowBytes, &tm.x64, x, c.row0 + 256 + (int)rank * 64, fb);
        }
        __syncwarp();
        if (++stage == kPStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------ MMA issuer (the leader's, for both)
    const uint32_t elected = elect_one();
    const uint32_t s0 = smem_u32(smem);
    const uint64_t w0 = sdesc_sw128(s0), x0 = sdesc_sw128(s0 + kXWBytes);
    const uint64_t sf0 = sdesc_scale_atom(s0 + kXWBytes + kPXBytes);
    constexpr uint64_t kStageStep = kPStageBytes >> 4, kAtomStep = kAtomBytes >> 4, kSfStep = kXSfBytes >> 4;
    constexpr uint64_t kXHalf = (128 * kXRowBytes) >> 4;
    const uint32_t sfw_t = tmem + kPSfCol, sfx_t = sfw_t + 4 * kXAtoms;
    const uint32_t empty_own = mapa_shared(smem_u32(&empty_bar[0]), 0);
    const uint32_t empty_peer = mapa_shared(smem_u32(&empty_bar[0]), 1);
    const uint32_t accf_own = mapa_shared(smem_u32(&acc_full_bar), 0);
    const uint32_t accf_peer = mapa_shared(smem_u32(&acc_full_bar), 1);
    const uint32_t a0 = idesc_mxf4(256, 256, 0), a2 = idesc_mxf4(256, 256, 2);
    const uint32_t b0 = idesc_mxf4(256, 128, 0), b2 = idesc_mxf4(256, 128, 2);
    int stage = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = t_first; ok && t < num_tiles; t += t_step) {
      const bool third = mx_tile(p, segs, t).tokens > 256;   // the 128-column MMA has real tokens
      ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty_bar, acc_phase ^ 1u, abort_flag));
      if (!ok) {
        if (elected) mx_give_up_pair(p.status, abort_flag, peer_abort);
        break;
      }
      tc_fence_after();
      uint32_t accumulate = 0;
      for (int kt = 0; kt < p.kt_total; ++kt) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort_flag));
        if (!ok) {
          if (elected) mx_give_up_pair(p.status, abort_flag, peer_abort);
          break;
        }
        const bool whole = p.groups - kt * kXAtoms >= kXAtoms;     // else K ends with one atom
        if (elected) {
          const uint64_t d = (uint64_t)stage * kStageStep;
          // straight-line code for each of the four shapes of a stage: a
          // branch per instruction would starve the tensor pipe
          auto issue = [&](auto n_atoms, auto with_third) {
            constexpr int A = decltype(n_atoms)::value;
            constexpr bool Third = decltype(with_third)::value;
#pragma unroll
            for (int j = 0; j < A; ++j) {
              tc_cp_scale_atom_pair(sfw_t + 4 * j, sf0 + d + j * kAtomStep);
#pragma unroll
              for (int h = 0; h < (Third ? kPQ : 2); ++h)
                tc_cp_scale_atom_pair(sfx_t + 4 * kPQ * j + 4 * h, sf0 + d + (1 + h) * kSfStep + j * kAtomStep);
            }
#pragma unroll
            for (int j = 0; j < 2 * A; ++j) {
              const uint32_t sw = sfw_t + 4 * (j >> 1), sx = sfx_t + 4 * kPQ * (j >> 1);
              mma_mxf4_pair(tmem, w0 + d + 2 * j, x0 + d + 2 * j, (j & 1) ? a2 : a0, sw, sx, accumulate | j);
              if constexpr (Third)
                mma_mxf4_pair(tmem + 256, w0 + d + 2 * j, x0 + d + kXHalf + 2 * j, (j & 1) ? b2 : b0, sw, sx + 8,
                              accumulate | j);
            }
          };
          if (whole && third) issue(std::integral_constant<int, kXAtoms>{}, std::true_type{});
          else if (whole) issue(std::integral_constant<int, kXAtoms>{}, std::false_type{});
          else if (third) issue(std::integral_constant<int, 1>{}, std::true_type{});
          else issue(std::integral_constant<int, 1>{}, std::false_type{});
          tc_commit_pair(empty_own + 8u * stage);
          tc_commit_pair(empty_peer + 8u * stage);
        }
        __syncwarp();
        accumulate = 1;
        if (++stage == kPStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elected) {
        tc_commit_pair(accf_own);
        tc_commit_pair(accf_peer);
      }
      __syncwarp();
      acc_phase ^= 1u;
    }
    if (elected) {
      tc_commit_pair(mapa_shared(smem_u32(&drain_bar), 0));
      volatile int never = 0;
      mbar_wait(&drain_bar, 0, &never);
    }
    __syncwarp();
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, part = (warp - 2) >> 2;
    const int n_in = quad * 32 + lane;
    const uint32_t tacc = tmem + ((uint32_t)(quad * 32) << 16) + part * 128;
    const uint32_t acce_leader = mapa_shared(smem_u32(&acc_empty_bar), 0);
    uint32_t acc_phase = 0;
    for (int t = t_first; t < num_tiles; t += t_step) {
      const MxTile c = mx_tile(p, segs, t);
      const int n = (c.wt * 2 + (int)rank) * kXBM + n_in;
      const float bias = !PLAIN && p.bias && n < p.N ? p.bias[(size_t)c.e * p.N + n] : 0.0f;
      // loaded before the accumulator is ready
      const int cnt = c.tokens - part * 128, m0 = c.row0 + part * 128;
      float weights[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) weights[i] = mx_load_weight<PLAIN>(p, m0 + 32 * i, cnt - 32 * i);
      if (!mbar_wait(&acc_full_bar, acc_phase, abort_flag)) {
        mx_give_up_pair(p.status, abort_flag, peer_abort);
        break;
      }
      tc_fence_after();
      bool held = true;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(acce_leader);
        held = false;
      };
      if (T::size == 2 && p.pairs && cnt > 0) {
        // drain the thread's 128 columns into 64 packed words and hand the
        // accumulator back before any store
        uint32_t w[64];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t r[32];
          tmem_ld32(tacc + 32 * i, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            if constexpr (T::size == 2)
              w[16 * i + j / 2] = T::pack(mx_value<PLAIN>(r[j], mx_weight<PLAIN>(weights[i], j), bias),
                                          mx_value<PLAIN>(r[j + 1], mx_weight<PLAIN>(weights[i], j + 1), bias));
          }
        }
        release();
        uint16_t* at = static_cast<uint16_t*>(p.y) + (size_t)(m0 + (n & 1)) * (size_t)p.y_stride + (n & ~1);
        const size_t step = 2 * (size_t)p.y_stride;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          mx_store_pair(p, w[i], at, cnt - 2 * i, n);
          at += step;
        }
      } else {
        // fp32 (or unaligned) outputs do not fit the registers at once: the
        // accumulator waits while all but the last 32 columns are stored (64 at
        // a time measured slower, 92.7 us against 80.8 at 8192 x 4096 x 6144
        // fp32: twice the straight-line code)
#pragma unroll 1
        for (int col = 0; col < 128 && col < cnt; col += 32) {
          uint32_t r[32];
          tmem_ld32(tacc + col, r);
          tmem_ld_wait();
          if (col + 32 >= 128 || col + 32 >= cnt) release();
          const float h = col == 0 ? weights[0] : col == 32 ? weights[1] : col == 64 ? weights[2] : weights[3];
          mx_store32<T, PLAIN>(p, r, m0 + col, min(32, cnt - col), n, bias, h);
        }
      }
      if (held) release();
      acc_phase ^= 1u;
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other may still arrive on its barriers or
  // the leader's MMAs may still read its shared memory
  cluster_sync_all();
  if (*abort_flag) {
    // copies issued before a give-up may still be landing here: they finish within microseconds
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Opts a kernel into the largest dynamic shared memory, once per device.
template <auto Kernel>
static nvfp4_status opt_in_smem(int bytes = kXMaxSmem) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  NV_CHECK(check_cuda(cudaGetDevice(&dev), "cudaGetDevice"));
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 0 || dev >= 64 || !done[dev]) {
    NV_CHECK(check_cuda(cudaFuncSetAttribute((const void*)Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             bytes),
                        "cudaFuncSetAttribute"));
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  return NVFP4_OK;
}

struct MxGemmArgs {
  const uint8_t *a_codes = nullptr, *a_scales = nullptr, *b_codes = nullptr, *b_scales = nullptr;
  int M = 0, N = 0, K = 0, E = 0;
  const int32_t *expert_offsets = nullptr, *expert_counts = nullptr;
  const float *row_weight = nullptr, *bias = nullptr;
  int out_dtype = 0;
  void* y = nullptr;
  long long y_stride = 0;
  uint32_t* status = nullptr;
  bool early_b = false;
  // unquantised a, for a fused product (x_rows of them, x_stride elements apart)
  const void* x = nullptr;
  const int32_t* perm = nullptr;
  int x_rows = 0, x_dtype = 0;
  long long x_stride = 0;
  bool x_wide = false;
};

// Tile width, pipeline depth and K splits of a product (host arithmetic).
struct MxPlan {
  int nt, stages, splits, ctas_per_sm, n_acc;
  bool pair;
};

// Tiles of up to 128 tokens on one CTA, or of 384 on a pair: the kind whose
// waves are estimated to end first, fitted to measurements (one B200, us).
// One CTA has its SM to itself while that gives every tile an SM, else two
// share one.  Measured, waves (of 148 tiles, 296 shared, 74 pairs): us
//   K = 6144 (24 stages)   alone   1: 12.5  2: 20.7  3: 29.4
//                          shared  1: 15.8  2: 26.3  (128 tiles: 14.1)
//                          pairs   1: 18.7  2: 29.6  3: 41.5
//   K = 1024 (4 stages)    alone   1: 5.8   2: 8.4
//                          shared  1: 7.3
//                          pairs   1: 9.4   2: 14.0
// and 16 experts of 32 tokens, 6144 x 2048 (768 tiles): alone 25.3, shared
// 22.4.  (256 tokens a tile, one wave of 148 at K = 6144, took 15.1 to 16.1.)
static MxPlan plan_mx_gemm(int M, int N, int K, int E, int sms) {
  const int kt = (mx_groups(K) + kXAtoms - 1) / kXAtoms;
  const int n_wt = (N + kXBM - 1) / kXBM;
  const int experts = std::max(1, E);
  // tokens an expert, taken as even; grouped rows hold up to 127 of padding an
  // expert (moe_route's capacity has that many)
  const long long per = E == 0 ? M : std::max(16ll, (long long)M / E - 127);
  const long long tiles = (long long)n_wt * experts * ((per + kXNT - 1) / kXNT);
  const bool shared = tiles > sms;
  const double us = shared ? 4.6 + (double)((tiles + 2 * sms - 1) / (2 * sms)) * (0.43 * kt + 0.9) : 5.4 + 0.30 * kt;
  const long long pairs = (long long)((n_wt + 1) / 2) * experts * ((per + kPNT - 1) / kPNT);
  const double pair_us = 6.5 + (double)((pairs + sms / 2 - 1) / (sms / 2)) * (0.32 * kt + 3.3);
  MxPlan pl;
  pl.splits = pl.ctas_per_sm = pl.n_acc = 1;
  pl.pair = pair_us < us && E <= kPMaxE;
  if (pl.pair) {
    pl.nt = kPNT;
    pl.stages = kPStages;
    return pl;
  }
  // a single token tile is no wider than its tokens
  pl.nt = E == 0 && M <= kXNT ? (M + 15) / 16 * 16 : kXNT;
  // Few tokens: two CTAs on an SM, and K split over a cluster while there is
  // an SM for each of its CTAs.  Measured at N = K = 6144 (48 tiles) and one
  // token, splits of 1, 2, 3, 4, 6, 8: 10.8, 7.8, 7.6, 7.0, 11.4, 11.2 us; at N
  // = 1024 (8 tiles) 10.2, 6.9, 5.8, 5.1, 4.7, 4.4; at N = 5001, K = 2010 (40
  // tiles) 6.0, 5.7, 5.5, 6.6, 6.7, 11.0.  One rule for all of them: it takes 3
  // splits at 48 tiles and at 40, where 4 gain 0.6 us and lose 1.1, and stops at
  // 4, where 8 tiles would still gain 0.7 from 8.  Wider tiles, at one CTA an SM (128 tokens, 48
  // tiles): 12.2, 11.2, then 17 and more, as clusters of three and more no
  // longer fit at once; with 16 tiles (100 x 2048 x 6144) 11.6, 9.3, 7.8, 7.2,
  // 7.5, 13.4.  Joining 128 columns costs 2 us: at 8 stages (128 x 4096 x 2048)
  // one split takes 6.8 us, two 7.4, at 16 (128 x 6144 x 4096) 9.5 and 9.1.
  const int table = mx_segment_bytes(E), stage = mx_stage_bytes(pl.nt);
  // (a table of very many experts leaves two CTAs too few stages each)
  pl.ctas_per_sm = (pl.nt <= 64 || shared) && (kXSmemPair - 1024 - table) / stage >= 3 ? 2 : 1;
  pl.n_acc = pl.nt <= 64 || pl.ctas_per_sm == 1 ? 2 : 1;
  pl.stages = std::min(kXMaxStages, ((pl.ctas_per_sm == 2 ? kXSmemPair : kXMaxSmem) - 1024 - table) / stage);
  if (E == 0) {
    const long long all = (long long)n_wt * ((M + pl.nt - 1) / pl.nt);
    const long long most = pl.nt <= 64 ? kXMaxSplits : kt < 12 ? 1 : all * 4 <= sms / 2 ? kXMaxSplits : 2;
    pl.splits = (int)std::max(1ll, std::min({most, sms / all, (long long)(kt + 1) / 2}));
  }
  return pl;
}

// The plan of a product that quantises its own tokens, from the plan of one
// that does not; false where there is none or it would be slower.  It takes a
// single token tile, a tile a CTA, and a's share of K beside three stages (four
// where K is split) at least.  Every CTA converts the tokens for itself, which
// costs 0.4 us a pass (32 units of 128 elements, 16 of fp32; more where rows are
// not 16-byte aligned) where the quantiser's launch costs 2 on the GPU and 2.5
// on the host.
// Measured, tokens: us fused, us with the quantiser's kernel
//   bf16  1024 x 6144 (6 stages a CTA)    1: 5.4, 7.2   8: 5.7, 7.4  16: 7.0, 7.6
//         6144 x 6144 (8 stages)          1: 7.9, 9.5   8: 8.8, 9.9  12: 10.1, 10.0
//         12288 x 4096 (16 stages)        1: 9.9, 11.0  6: 10.5, 11.1  8: 11.4, 11.1
//         18000 x 6144 (24 stages)        1: 13.8, 15.1 4: 14.1, 15.1  6: 15.3, 15.2
//         20000 x 5000 (20 stages; three in flight)                     1: 14.5, 14.9
//         3000 x 20000 (20 stages, split; three in flight, not taken)   1: 12.9, 12.1
//   fp32  6144 x 6144                     4: 8.7, 9.8   6: 9.7, 9.8    8: 10.8, 9.9
//   rows at odd elements, 6144 x 6144     bf16 8: 9.3, 9.8  12: 11.0, 9.9
//                                         fp32 4: 8.8, 9.8   6: 10.5, 9.9
static bool fuse_quantiser(MxPlan& pl, int M, int N, int K, int E, bool wide, int dtype, int sms) {
  if (E != 0 || pl.pair || M > kXFuseTokens) return false;
  const long long ctas = (long long)(N + kXBM - 1) / kXBM * pl.splits;
  const int kt = (mx_groups(K) + kXAtoms - 1) / kXAtoms, nkt = (kt + pl.splits - 1) / pl.splits;
  if (ctas > 2ll * sms || nkt > kXFuseStages) return false;
  const int pass = dtype == MXFP4_DTYPE_F32 ? fuse_pass<F32>() : fuse_pass<Bf16>();
  if (nkt * 2 * M > pass * (wide ? 6 : 4)) return false;
  const int per_sm = pl.splits > 1 || ctas > sms ? 2 : 1;    // (clusters fit at two CTAs an SM)
  const int stages = ((per_sm == 2 ? kXSmemPair : kXMaxSmem) - 1024 - kXFuseSmem - nkt * mx_fused_a_bytes(pl.nt)) /
                     kXFuseStageBytes;
  if (stages < (pl.splits > 1 ? 4 : 3)) return false;
  pl.ctas_per_sm = per_sm;
  pl.n_acc = 1;
  pl.stages = std::min(kXMaxStages, stages);
  return true;
}

template <typename T, bool PLAIN, bool FUSED>
static nvfp4_status run_mx_gemm(const MxPlan& pl, int sms, const CUtensorMap& tmW,
                                const CUtensorMap& tmX, const CUtensorMap& tmX32, const MxGemmParams& p,
                                long long tiles, cudaStream_t s) {
  constexpr auto kernel = mx_gemm_kernel<T, PLAIN, FUSED>;
  NV_CHECK(opt_in_smem<kernel>(FUSED ? kXMaxSmem - kXFuseSmem : kXMaxSmem));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (pl.splits > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)pl.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  cfg.blockDim = dim3(kXThreads);
  cfg.gridDim = dim3((unsigned)(pl.splits > 1 ? tiles * pl.splits
                                              : std::max(1ll, std::min<long long>(tiles, (long long)sms * pl.ctas_per_sm))));
  cfg.dynamicSmemBytes = FUSED ? (size_t)pl.stages * kXFuseStageBytes +
                                     (size_t)((p.kt_total + pl.splits - 1) / pl.splits) * mx_fused_a_bytes(pl.nt) + 1024
                               : (size_t)pl.stages * mx_stage_bytes(pl.nt) + mx_segment_bytes(p.E) + 1024;
  cfg.stream = s;
  return check_cuda(cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, tmX32, p), "mx_gemm_kernel");
}

template <typename T, bool PLAIN>
static nvfp4_status run_mx_gemm_pair(const MxPairMaps& tm, const MxGemmParams& p, long long tiles, cudaStream_t s) {
  constexpr auto kernel = mx_gemm_pair_kernel<T, PLAIN>;
  NV_CHECK(opt_in_smem<kernel>());
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = kPStages * kPStageBytes + mx_segment_bytes(p.E) + 1024;
  cfg.stream = s;
  // the grid is persistent: as many pairs as can be resident at once
  static std::mutex mu;
  static int resident[64] = {};
  int dev = 0, n = 0;
  NV_CHECK(check_cuda(cudaGetDevice(&dev), "cudaGetDevice"));
  {
    std::lock_guard<std::mutex> lock(mu);
    const bool kept = dev >= 0 && dev < 64;
    n = kept ? resident[dev] : 0;
    if (n == 0) {
      int sms = 0;
      NV_CHECK(device_sm_count(&sms));
      cfg.gridDim = dim3(2 * (sms / 2));
      NV_CHECK(check_cuda(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg),
                          "cudaOccupancyMaxActiveClusters"));
      NV_REQUIRE(n >= 1, NVFP4_ERR_CUDA, "mx_gemm_pair_kernel: no cluster of two CTAs can be resident");
      if (kept) resident[dev] = n;
    }
  }
  cfg.gridDim = dim3((unsigned)(2 * std::max(1ll, std::min<long long>(n, tiles))));
  cfg.numAttrs = 2;
  return check_cuda(cudaLaunchKernelEx(&cfg, kernel, tm, p), "mx_gemm_pair_kernel");
}

// Calls f(output type tag, whether there is neither bias nor row weight).
template <typename F>
static nvfp4_status with_output(const MxGemmArgs& a, F&& f) {
  auto by_plain = [&](auto tag) -> nvfp4_status {
    return a.bias || a.row_weight ? f(tag, std::false_type{}) : f(tag, std::true_type{});
  };
  if (a.out_dtype == MXFP4_DTYPE_BF16) return by_plain(Bf16{});
  if (a.out_dtype == MXFP4_DTYPE_F16) return by_plain(F16{});
  return by_plain(F32{});
}

static nvfp4_status launch_mx_gemm(const MxGemmArgs& a, const MxPlan& pl, int sms, cudaStream_t s) {
  MxGemmParams p;
  p.M = a.M;
  p.N = a.N;
  p.E = a.E;
  p.groups = mx_groups(a.K);
  p.kt_total = (p.groups + kXAtoms - 1) / kXAtoms;
  p.n_wt = pl.pair ? (a.N + 2 * kXBM - 1) / (2 * kXBM) : (a.N + kXBM - 1) / kXBM;
  p.nt = pl.nt;
  p.n_tt = a.E ? 0 : (a.M + pl.nt - 1) / pl.nt;
  p.stages = pl.stages;
  p.n_acc = pl.n_acc;
  p.splits = pl.splits;
  p.early_b = a.early_b;
  const int elem = mx_elem_size(a.out_dtype), access = row_access_bytes(a.y, a.M > 1 ? a.y_stride * elem : 0, elem);
  p.pairs = elem == 2 && access >= 4;
  p.quads = access >= 4 * elem;
  p.expert_offsets = a.expert_offsets;
  p.expert_counts = a.expert_counts;
  p.a_sf = a.a_scales;
  p.b_sf = a.b_scales;
  p.row_weight = a.row_weight;
  p.bias = a.bias;
  p.y = a.y;
  p.y_stride = a.y_stride;
  p.status = a.status;
  p.x = static_cast<const uint8_t*>(a.x);
  // tiles at most: each expert may end in a partly filled token tile
  const long long tiles = (long long)p.n_wt * (a.E ? (a.M + pl.nt - 1) / pl.nt + a.E : p.n_tt);
  const uint64_t inner = (uint64_t)mx_row_bytes(a.K);
  if (pl.pair) {
    MxPairMaps tm;
    const uint64_t brows = (uint64_t)std::max(1, a.E) * (uint64_t)a.N;
    NV_CHECK(make_tmap_2d(&tm.w, a.b_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner, brows, inner, kXRowBytes, kXBM));
    NV_CHECK(make_tmap_2d(&tm.x, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner, (uint64_t)a.M, inner, kXRowBytes, 128));
    NV_CHECK(make_tmap_2d(&tm.x64, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner, (uint64_t)a.M, inner, kXRowBytes, 64));
    // scale atoms as rows of 128 words; a box that reaches past the last atom
    // of a row tile reads the next tile's (or zeros), which no MMA uses
    NV_CHECK(make_tmap_2d(&tm.sfw, a.b_scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 128,
                          (brows + 127) / 128 * (uint64_t)p.groups, kAtomBytes, 128, kXAtoms, false));
    NV_CHECK(make_tmap_2d(&tm.sfx, a.a_scales, CU_TENSOR_MAP_DATA_TYPE_UINT32, 128,
                          ((uint64_t)a.M + 127) / 128 * (uint64_t)p.groups, kAtomBytes, 128, kXAtoms, false));
    return with_output(a, [&](auto tag, auto plain) -> nvfp4_status {
      return run_mx_gemm_pair<decltype(tag), decltype(plain)::value>(tm, p, tiles, s);
    });
  }
  CUtensorMap tmW, tmX, tmX32;
  NV_CHECK(make_tmap_2d(&tmW, a.b_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner,
                        (uint64_t)std::max(1, a.E) * (uint64_t)a.N, inner, kXRowBytes, kXBM));
  if (a.x) {
    p.perm = a.perm;
    p.x_rows = a.x_rows;
    p.x_dtype = a.x_dtype;
    p.x_wide = a.x_wide;
    p.K = a.K;
    p.x_stride = a.x_stride * mx_elem_size(a.x_dtype);
    return with_output(a, [&](auto tag, auto plain) -> nvfp4_status {
      return run_mx_gemm<decltype(tag), decltype(plain)::value, true>(pl, sms, tmW, tmW, tmW, p, tiles, s);
    });
  }
  NV_CHECK(make_tmap_2d(&tmX, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner, (uint64_t)a.M, inner, kXRowBytes,
                        (uint32_t)pl.nt));
  if (a.E) {
    NV_CHECK(make_tmap_2d(&tmX32, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner, (uint64_t)a.M, inner, kXRowBytes,
                          32));
  } else {
    tmX32 = tmX;
  }
  return with_output(a, [&](auto tag, auto plain) -> nvfp4_status {
    return run_mx_gemm<decltype(tag), decltype(plain)::value, false>(pl, sms, tmW, tmX, tmX32, p, tiles, s);
  });
}

static nvfp4_status check_product(const char* name, int M, const uint8_t* b_codes, const uint8_t* b_scales, int N,
                                  int K, int E, const int32_t* offsets, const int32_t* counts,
                                  const float* row_weight, const float* bias, int out_dtype, const void* y,
                                  long long y_stride) {
  NV_REQUIRE(M >= 0 && N >= 1 && K >= 1, NVFP4_ERR_INVALID_ARG, "%s: M=%d N=%d K=%d", name, M, N, K);
  NV_REQUIRE(M <= (1 << 30) && N <= (1 << 30) && K <= (1 << 30), NVFP4_ERR_UNSUPPORTED_SHAPE,
             "%s: M=%d, N=%d or K=%d is above 2^30", name, M, N, K);
  NV_REQUIRE(E >= 0 && E <= kXMaxE, NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: E=%d is not in [0, %d]", name, E, kXMaxE);
  NV_REQUIRE((E > 0) == (offsets != nullptr) && (E > 0 || !counts), NVFP4_ERR_INVALID_ARG,
             "%s: expert_offsets (and expert_counts) go with E >= 1, E=%d", name, E);
  NV_REQUIRE(E == 0 || N % kXBM == 0, NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: N=%d per expert must be a multiple of 128",
             name, N);
  NV_REQUIRE((long long)std::max(1, E) * N < (1ll << 31), NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: E * N = %lld rows of b",
             name, (long long)std::max(1, E) * N);
  // tile counts stay 32-bit: 128 x 128 outputs a tile at least, 8 K splits at most
  NV_REQUIRE(((long long)M / 128 + E + 1) * (N / 128 + 1) < (1ll << 28), NVFP4_ERR_UNSUPPORTED_SHAPE,
             "%s: M=%d N=%d is too large", name, M, N);
  NV_REQUIRE(mx_dtype_ok(out_dtype), NVFP4_ERR_INVALID_ARG, "%s: unknown output dtype %d", name, out_dtype);
  NV_REQUIRE(M <= 1 || y_stride >= N, NVFP4_ERR_INVALID_ARG, "%s: y stride %lld is below N=%d", name, y_stride, N);
  NV_REQUIRE(M == 0 || (b_codes && b_scales && y), NVFP4_ERR_INVALID_ARG, "%s: a required pointer is NULL", name);
  NV_REQUIRE(aligned(b_codes, 16) && aligned(b_scales, 16), NVFP4_ERR_INVALID_ARG,
             "%s: codes and scales need 16-byte alignment", name);
  NV_REQUIRE(aligned(y, mx_elem_size(out_dtype)) && aligned(row_weight, 4) && aligned(bias, 4) && aligned(offsets, 4) &&
                 aligned(counts, 4),
             NVFP4_ERR_INVALID_ARG, "%s: a tensor is not aligned to its elements", name);
  return NVFP4_OK;
}

}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" size_t mxfp4_matmul_workspace_size(void) { return 256; }

extern "C" nvfp4_status mxfp4_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int M, const uint8_t* b_codes,
                                     const uint8_t* b_scales, int N, int K, int E, const int32_t* expert_offsets,
                                     const int32_t* expert_counts, const float* row_weight, const float* bias,
                                     int out_dtype, void* y, long long y_stride, void* ws, size_t ws_bytes,
                                     void* stream) {
  NV_CHECK(check_product("mxfp4_matmul", M, b_codes, b_scales, N, K, E, expert_offsets, expert_counts, row_weight,
                         bias, out_dtype, y, y_stride));
  if (M == 0) return NVFP4_OK;
  NV_REQUIRE(a_codes && a_scales, NVFP4_ERR_INVALID_ARG, "mxfp4_matmul: a required pointer is NULL");
  NV_REQUIRE(aligned(a_codes, 16) && aligned(a_scales, 16), NVFP4_ERR_INVALID_ARG,
             "mxfp4_matmul: codes and scales need 16-byte alignment");
  const size_t need = mxfp4_matmul_workspace_size();
  NV_REQUIRE(ws && ws_bytes >= need && aligned(ws, 256), NVFP4_ERR_WORKSPACE,
             "mxfp4_matmul: needs a 256-byte aligned workspace of %zu bytes", need);
  MxGemmArgs g;
  g.a_codes = a_codes; g.a_scales = a_scales; g.b_codes = b_codes; g.b_scales = b_scales;
  g.M = M; g.N = N; g.K = K; g.E = E;
  g.expert_offsets = expert_offsets; g.expert_counts = expert_counts;
  g.row_weight = row_weight; g.bias = bias;
  g.out_dtype = out_dtype; g.y = y; g.y_stride = y_stride;
  g.status = static_cast<uint32_t*>(ws);
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  return launch_mx_gemm(g, plan_mx_gemm(M, N, K, E, sms), sms, as_stream(stream));
}

struct MxLinearScratch {
  uint32_t* status;
  uint8_t *codes, *scales;
};
static MxLinearScratch carve_linear(Carver& c, int M, int K) {
  MxLinearScratch l;
  l.status = c.take<uint32_t>(64);
  l.codes = c.take<uint8_t>((size_t)M * mx_row_bytes(K));
  l.scales = c.take<uint8_t>(mxfp4_scale_bytes(M, K, NVFP4_LAYOUT_TILED));
  return l;
}

extern "C" size_t mxfp4_linear_workspace_size(int M, int K) {
  if (M < 0 || K < 1) return 0;
  Carver c(nullptr);
  carve_linear(c, M, K);
  return c.size();
}

extern "C" nvfp4_status mxfp4_linear(const void* x, int dtype, int rows, long long row_stride, const int32_t* perm,
                                     int perm_rows, const uint8_t* b_codes, const uint8_t* b_scales, int N, int K,
                                     int E, const int32_t* expert_offsets, const int32_t* expert_counts,
                                     const float* row_weight, const float* bias, int out_dtype, void* y,
                                     long long y_stride, void* ws, size_t ws_bytes, void* stream) {
  NV_CHECK(check_mx_source("mxfp4_linear", x, dtype, rows, K, row_stride));
  NV_REQUIRE(!perm || perm_rows >= 0, NVFP4_ERR_INVALID_ARG, "mxfp4_linear: perm_rows=%d", perm_rows);
  NV_REQUIRE(aligned(perm, 4), NVFP4_ERR_INVALID_ARG, "mxfp4_linear: perm is not aligned to its elements");
  const int M = perm ? perm_rows : rows;
  NV_CHECK(check_product("mxfp4_linear", M, b_codes, b_scales, N, K, E, expert_offsets, expert_counts, row_weight,
                         bias, out_dtype, y, y_stride));
  if (M == 0) return NVFP4_OK;
  const size_t need = mxfp4_linear_workspace_size(M, K);
  NV_REQUIRE(ws && ws_bytes >= need && aligned(ws, 256), NVFP4_ERR_WORKSPACE,
             "mxfp4_linear: needs a 256-byte aligned workspace of %zu bytes", need);
  Carver c(ws);
  const MxLinearScratch l = carve_linear(c, M, K);
  MxGemmArgs g;
  g.a_codes = l.codes; g.a_scales = l.scales; g.b_codes = b_codes; g.b_scales = b_scales;
  g.M = M; g.N = N; g.K = K; g.E = E;
  g.expert_offsets = expert_offsets; g.expert_counts = expert_counts;
  g.row_weight = row_weight; g.bias = bias;
  g.out_dtype = out_dtype; g.y = y; g.y_stride = y_stride;
  g.status = l.status;
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  MxPlan pl = plan_mx_gemm(M, N, K, E, sms);
  cudaStream_t s = as_stream(stream);
  // (a fused product reads x while it writes y)
  const int elem = mx_elem_size(dtype);
  const bool wide = row_access_bytes(x, rows > 1 ? row_stride * elem : 0, elem) >= 16;
  if (rows > 0 && !overlap(x, rows, row_stride, K, elem, y, M, y_stride, N, mx_elem_size(out_dtype)) &&
      fuse_quantiser(pl, M, N, K, E, wide, dtype, sms)) {
    g.x = x;
    g.perm = perm;
    g.x_rows = rows;
    g.x_dtype = dtype;
    g.x_stride = row_stride;
    g.x_wide = wide;
    return launch_mx_gemm(g, pl, sms, s);
  }
  // b may load before the quantiser has finished: the quantiser itself starts
  // only behind everything queued earlier, which may have written b
  g.early_b = true;
  NV_CHECK(launch_mx_quantize(x, dtype, rows, K, row_stride, perm, M, NVFP4_LAYOUT_TILED, l.codes, l.scales, s,
                              expert_offsets, expert_counts, E));
  return launch_mx_gemm(g, pl, sms, s);
}

extern "C" int nvfp4_test_mxfp4_plan(int M, int N, int K, int E, int* splits, int* pair, int* stages) {
  if (M < 1 || N < 1 || K < 1 || E < 0 || M > (1 << 30) || N > (1 << 30) || K > (1 << 30) || E > kXMaxE) return -1;
  const MxPlan pl = plan_mx_gemm(M, N, K, E, 148);
  if (splits) *splits = pl.splits;
  if (pair) *pair = pl.pair ? 1 : 0;
  if (stages) *stages = pl.stages;
  return pl.nt;
}

extern "C" int nvfp4_test_mxfp4_residency(int M, int N, int K, int E, int* smem_bytes, int* tmem_columns) {
  if (M < 1 || N < 1 || K < 1 || E < 0 || M > (1 << 30) || N > (1 << 30) || K > (1 << 30) || E > kXMaxE) return -1;
  const MxPlan pl = plan_mx_gemm(M, N, K, E, 148);
  if (smem_bytes)
    *smem_bytes = pl.stages * (pl.pair ? kPStageBytes : mx_stage_bytes(pl.nt)) + mx_segment_bytes(E) + 1024;
  if (tmem_columns) *tmem_columns = pl.pair ? 512 : (int)mx_tmem_columns(pl.nt, pl.n_acc);
  return pl.ctas_per_sm;
}

extern "C" int nvfp4_test_mxfp4_fuses(int M, int N, int K, int dtype, int wide, int* stages, int* ctas_per_sm) {
  if (M < 1 || N < 1 || K < 1 || M > (1 << 30) || N > (1 << 30) || K > (1 << 30) || !mx_dtype_ok(dtype)) return -1;
  MxPlan pl = plan_mx_gemm(M, N, K, 0, 148);
  if (!fuse_quantiser(pl, M, N, K, 0, wide != 0, dtype, 148)) return 0;
  if (stages) *stages = pl.stages;
  if (ctas_per_sm) *ctas_per_sm = pl.ctas_per_sm;
  return 1;
}

extern "C" int nvfp4_test_mxfp4_segments(const int32_t* offsets, const int32_t* counts, int M, int E, int* row0,
                                         int* rows) {
  if (!offsets || !row0 || !rows || M < 0 || E < 1 || E > kXMaxE) return -1;
  for (int e = 0; e < E; ++e) {
    const MxSegment s = mx_segment(offsets, counts, M, e);
    row0[e] = s.row0;
    rows[e] = s.rows;
  }
  return 0;
}
