// MXFP4 products on the 5th-generation tensor cores (tcgen05, sm_100a):
// y[m][n] = row_weight[m] * (sum_k a[m][k] b[n][k] + bias[n]), dense or
// grouped by expert.
//
// The block scales are applied inside the MMA (kind::mxf4, scale_vec::2X: two
// E8M0 bytes per row and 64-element step), the products of E2M1 values under
// powers of two are exact and accumulate in fp32, so the one rounding that
// the definition has is the store.
//
// Orientation: the 128 rows of an MMA tile (the tensor-memory lanes) are rows
// of b, its N columns are rows of a ("tokens").  A decoding step's few tokens
// are then a narrow N (16 columns) instead of a 128-row tile that is nearly
// empty, and a warp's 32 lanes hold 32 neighbouring outputs of one token, so
// y leaves in whole sectors straight from registers for any N.
//
// One CTA per tile of 128 b rows x up to 256 tokens; warp 0 issues the loads
// (TMA for codes, bulk copies for scale atoms), warp 1 the MMAs, warps 2..9
// drain the accumulator.  A K stage is 256 elements: 128-byte code rows in the
// 128-byte swizzle, two scale atoms per 128 rows.
//
// Few tiles (a decoding step) split K over a cluster of CTAs: each leaves its
// fp32 partial sums in its own shared memory and, behind a cluster barrier,
// rank r adds the columns r, r + S, ... of all of them in rank order and
// stores them, so the result does not depend on scheduling and takes no
// second kernel and no workspace.
#include <algorithm>
#include <mutex>

#include "mx.cuh"

namespace nvfp4moe {

constexpr int kXBM = 128;                        // b rows per tile
constexpr int kXMaxNT = 256;                     // tokens per tile, at most
constexpr int kXBK = 256;                        // K elements per stage
constexpr int kXRowBytes = kXBK / 2;             // 128 bytes of codes per row and stage
constexpr int kXWBytes = kXBM * kXRowBytes;      // 16 KiB
constexpr int kXAtoms = kXBK / kMxGroup;         // 2 scale atoms per 128 rows and stage
constexpr int kXSfBytes = kXAtoms * kAtomBytes;  // 1 KiB
constexpr int kXThreads = 320;
constexpr int kXEpiWarps = 8;
constexpr int kXMaxStages = 8;
constexpr int kXMaxE = 1024;
// Dynamic shared memory of a CTA that has an SM to itself, and of one of two
// on an SM (228 KiB less 1 KiB a CTA; the static part is below 4.5 KiB).
constexpr int kXMaxSmem = 227 * 1024 - 4608;
constexpr int kXSmemPair = 228 * 1024 / 2 - 1024 - 4608;

struct MxGemmParams {
  int M, N, E;               // E = 0: dense
  int groups;                // scale atoms along K
  int kt_total;              // K stages
  int n_wt, n_tt;            // b tiles (per expert), token tiles (dense)
  int nt;                    // tokens per tile
  int stages;
  int splits;                // K splits (CTAs per cluster)
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
};

// One stage: b codes, token codes, b scales, token scales (1 KiB per started
// 128 tokens).
__host__ __device__ constexpr int mx_sf_tiles(int nt) { return (nt + 127) / 128; }
__host__ __device__ constexpr int mx_stage_bytes(int nt) {
  return kXWBytes + (nt * kXRowBytes + 1023) / 1024 * 1024 + kXSfBytes * (1 + mx_sf_tiles(nt));
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
NVDEV float ld_shared_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// A tile of the work list: its expert, its first token row, its tokens and
// its b tile.
struct MxTile {
  int e, row0, tokens, wt;
};

// First tile group (128.. tokens of one expert) of every expert, as an
// exclusive prefix in start[0..E], from device-side offsets that are not
// trusted: a segment is clamped to [0, M] and its tokens to the segment.
struct MxSegment {
  int row0, tokens;
};
NVDEV MxSegment mx_segment(const MxGemmParams& p, int e) {
  MxSegment g;
  const int lo = min(max(p.expert_offsets[e], 0), p.M);
  const int hi = min(max(p.expert_offsets[e + 1], lo), p.M);
  g.row0 = lo & ~127;                            // a multiple of 128 by contract; never past the scale tiles
  int n = hi - g.row0;
  if (p.expert_counts) n = min(n, max(p.expert_counts[e], 0));
  g.tokens = n;
  return g;
}
NVDEV void mx_scan_segments(const MxGemmParams& p, int* start) {
  if ((threadIdx.x >> 5) == 0) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int v = 0;
      if (e < p.E) v = (mx_segment(p, e).tokens + p.nt - 1) / p.nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (e < p.E) start[e + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) start[0] = 0;
  }
  __syncthreads();
}
NVDEV MxTile mx_tile(const MxGemmParams& p, const int* start, int t) {
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
    if (start[mid] <= g) lo = mid; else hi = mid - 1;
  }
  const MxSegment s = mx_segment(p, lo);
  const int j = g - start[lo];
  c.e = lo;
  c.row0 = s.row0 + j * p.nt;
  c.tokens = min(p.nt, s.tokens - j * p.nt);
  return c;
}

template <typename T>
NVDEV void mx_store(void* y, size_t i, float v) {
  if constexpr (T::size == 2) static_cast<uint16_t*>(y)[i] = T::one(v);
  else static_cast<float*>(y)[i] = v;
}

template <typename T>
__global__ void __launch_bounds__(kXThreads, 2)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ CUtensorMap tmX32, const MxGemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kXMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[kXMaxStages];
  __shared__ __align__(8) uint64_t acc_full_bar;
  __shared__ __align__(8) uint64_t acc_empty_bar;
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  __shared__ int seg_start[kXMaxE + 1];
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nt_pad = max(p.nt, 32);                          // accumulator columns
  const uint32_t need = (uint32_t)nt_pad + 4 * kXAtoms * (1 + 2);
  const uint32_t tcols = need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
  const int stage_bytes = mx_stage_bytes(p.nt);
  const int x_bytes = (p.nt * kXRowBytes + 1023) / 1024 * 1024;
  // this CTA's share of K
  const int rank = p.splits > 1 ? (int)cluster_ctarank() : 0;
  const int kt0 = (int)((long long)p.kt_total * rank / p.splits);
  const int nkt = (int)((long long)p.kt_total * (rank + 1) / p.splits) - kt0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&acc_full_bar, 1);
    mbar_init(&acc_empty_bar, kXEpiWarps);
    mbar_init(&drain_bar, 1);
    abort_s = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmX32);
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

  // Dense calls whose b nobody is still writing fill the pipeline with b
  // before the previous kernel (the quantiser of a) has finished.
  int early = 0;
  if (p.early_b && t_first < p.n_wt * p.n_tt) early = min(p.stages, nkt);
  if (warp == 0 && early && elect_one()) {
    for (int i = 0; i < early; ++i) load_b(t_first % p.n_wt, 0, kt0 + i, i);
  }
  __syncwarp();
  griddep_wait();
  griddep_launch();
  // first kernel of a call: the status word is cleared here, before any wait
  // of this call can give up
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;

  int num_tiles;
  if (p.E == 0) {
    num_tiles = p.n_wt * p.n_tt;
  } else {
    mx_scan_segments(p, seg_start);
    num_tiles = seg_start[p.E] * p.n_wt;
  }

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint32_t elected = elect_one();
    int stage = 0, issued = 0;
    uint32_t phase = 0, filled = 0, fill_parity = 0;
    bool ok = true;
    for (int t = t_first; ok && t < num_tiles; t += t_step) {
      const MxTile c = mx_tile(p, seg_start, t);
      // token rows in 32-row boxes where a tile is not full (dense tiles:
      // rows past M read as zeros and move no bytes)
      const bool whole = p.E == 0 || c.tokens > p.nt - 32;
      const int boxes = (c.tokens + 31) / 32;
      const uint32_t xb = (uint32_t)(whole ? p.nt : boxes * 32) * kXRowBytes;
      const int sft = mx_sf_tiles(c.tokens);
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
          mbar_arrive_expect_tx(&full_bar[stage], kXWBytes + xb + sf_bytes * (uint32_t)(1 + sft));
          if (issued >= early) load_b(c.wt, c.e, kt, stage);
          if (whole) {
            tma_load_2d(sX, &tmX, kt * kXRowBytes, c.row0, &full_bar[stage]);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(sX + b * 32 * kXRowBytes, &tmX32, kt * kXRowBytes, c.row0 + 32 * b, &full_bar[stage]);
          }
          for (int h = 0; h < sft; ++h)
            bulk_load(sSFX + h * kXSfBytes, p.a_sf + (size_t)(c.row0 / kRowTile + h) * sf_tile + (size_t)kt * kXSfBytes,
                      sf_bytes, &full_bar[stage]);
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
    const uint64_t w0 = sdesc_sw128(s0), x0 = sdesc_sw128(s0 + kXWBytes);
    const uint64_t sfw0 = sdesc_scale_atom(s0 + kXWBytes + x_bytes);
    const uint64_t sfx0 = sdesc_scale_atom(s0 + kXWBytes + x_bytes + kXSfBytes);
    const uint64_t stage_step = (uint64_t)stage_bytes >> 4;
    constexpr uint64_t kAtomStep = kAtomBytes >> 4, kSfStep = kXSfBytes >> 4;
    const uint32_t sfw_t = tmem + (uint32_t)nt_pad, sfx_t = sfw_t + 4 * kXAtoms;
    int stage = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int t = t_first; ok && t < num_tiles; t += t_step) {
      const MxTile c = mx_tile(p, seg_start, t);
      const int n_mma = (c.tokens + 15) & ~15;
      const bool two = c.tokens > kRowTile;
      const uint32_t id0 = idesc_mxf4(kXBM, n_mma, 0), id2 = idesc_mxf4(kXBM, n_mma, 2);
      ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty_bar, acc_phase ^ 1u, abort_flag));
      if (!ok) {
        if (elected) {
          *abort_flag = 1;
          atomicExch(p.status, kDevTimeout);
        }
        break;
      }
      tc_fence_after();
      for (int i = 0; i < nkt; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort_flag));
        if (!ok) {
          if (elected) {
            *abort_flag = 1;
            atomicExch(p.status, kDevTimeout);
          }
          break;
        }
        const int atoms = min(kXAtoms, p.groups - (kt0 + i) * kXAtoms);
        if (elected) {
          const uint64_t d = (uint64_t)stage * stage_step;
#pragma unroll
          for (int j = 0; j < kXAtoms; ++j) {
            if (j < atoms) {
              tc_cp_scale_atom(sfw_t + 4 * j, sfw0 + d + j * kAtomStep);
              tc_cp_scale_atom(sfx_t + 8 * j, sfx0 + d + j * kAtomStep);
              if (two) tc_cp_scale_atom(sfx_t + 8 * j + 4, sfx0 + d + kSfStep + j * kAtomStep);
            }
          }
#pragma unroll
          for (int j = 0; j < 2 * kXAtoms; ++j)      // 64 elements = 32 bytes of K per MMA, two per atom
            if (j < 2 * atoms)
              mma_mxf4(tmem, w0 + d + 2 * j, x0 + d + 2 * j, (j & 1) ? id2 : id0, sfw_t + 4 * (j >> 1),
                       sfx_t + 8 * (j >> 1), (i | j) != 0);
          tc_commit(&empty_bar[stage]);
        }
        __syncwarp();
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elected) tc_commit(&acc_full_bar);
      __syncwarp();
      acc_phase ^= 1u;
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
    uint32_t acc_phase = 0;
    for (int t = t_first; t < num_tiles; t += t_step) {
      const MxTile c = mx_tile(p, seg_start, t);
      const int n = c.wt * kXBM + n_in;
      const bool n_ok = n < p.N;
      const float bias = p.bias && n_ok && p.splits == 1 ? p.bias[(size_t)c.e * p.N + n] : 0.0f;
      if (!mbar_wait(&acc_full_bar, acc_phase, abort_flag)) {
        *abort_flag = 1;
        atomicExch(p.status, kDevTimeout);
        break;
      }
      tc_fence_after();
      for (int col = half * 32; col < c.tokens; col += 64) {
        uint32_t r[32];
        tmem_ld32(tacc + col, r);
        tmem_ld_wait();
        const int cnt = min(32, c.tokens - col);
        if (p.splits > 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < cnt) red[(col + i) * kXBM + n_in] = __uint_as_float(r[i]);
        } else if (n_ok) {
          const size_t base = (size_t)(c.row0 + col) * (size_t)p.y_stride + n;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < cnt) {
              float v = __fadd_rn(__uint_as_float(r[i]), bias);
              if (p.row_weight) v = __fmul_rn(v, p.row_weight[c.row0 + col + i]);
              mx_store<T>(p.y, base + (size_t)i * (size_t)p.y_stride, v);
            }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty_bar);
      acc_phase ^= 1u;
    }
    __syncwarp();
  }
  if (p.splits > 1) {
    // one tile per cluster (the grid has splits CTAs per tile)
    cluster_sync_all();                                      // every rank's partial sums are in place
    if (warp >= 2 && t_first < num_tiles) {
      const MxTile c = mx_tile(p, seg_start, t_first);
      const int tid = threadIdx.x - 64, n_in = tid & (kXBM - 1);
      const int n = c.wt * kXBM + n_in;
      if (n < p.N) {
        const float bias = p.bias ? p.bias[(size_t)c.e * p.N + n] : 0.0f;
        const uint32_t red = smem_u32(smem);
        for (int m = rank + p.splits * (tid >> 7); m < c.tokens; m += p.splits * 2) {
          const uint32_t at = red + (uint32_t)(m * kXBM + n_in) * 4u;
          float v = ld_shared_cluster_f32(mapa_shared(at, 0));
          for (int q = 1; q < p.splits; ++q) v = __fadd_rn(v, ld_shared_cluster_f32(mapa_shared(at, (uint32_t)q)));
          v = __fadd_rn(v, bias);
          if (p.row_weight) v = __fmul_rn(v, p.row_weight[c.row0 + m]);
          mx_store<T>(p.y, (size_t)(c.row0 + m) * (size_t)p.y_stride + n, v);
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

// Opts a kernel into the largest dynamic shared memory, once per device.
template <auto Kernel>
static nvfp4_status opt_in_smem() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  NV_CHECK(check_cuda(cudaGetDevice(&dev), "cudaGetDevice"));
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 0 || dev >= 64 || !done[dev]) {
    NV_CHECK(check_cuda(cudaFuncSetAttribute((const void*)Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kXMaxSmem),
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
};

// Tile width, pipeline depth and K splits of a product (host arithmetic).
struct MxPlan {
  int nt, stages, splits, ctas_per_sm;
};
static MxPlan plan_mx_gemm(int M, int N, int K, int E, int sms) {
  MxPlan pl;
  const int n_wt = (N + kXBM - 1) / kXBM;
  const int kt = (mx_groups(K) + kXAtoms - 1) / kXAtoms;
  if (E == 0 && M <= kXMaxNT) {
    pl.nt = (M + 15) / 16 * 16;
  } else {
    const long long wide = (long long)n_wt * std::max(1, E) * ((M / std::max(1, E) + kXMaxNT - 1) / kXMaxNT);
    pl.nt = wide < sms ? 128 : kXMaxNT;
  }
  pl.ctas_per_sm = pl.nt <= 64 ? 2 : 1;
  const int room = (pl.ctas_per_sm == 2 ? kXSmemPair : kXMaxSmem) - 1024;
  pl.stages = std::min(kXMaxStages, room / mx_stage_bytes(pl.nt));
  pl.splits = 1;
  if (E == 0) {
    const long long tiles = (long long)n_wt * ((M + pl.nt - 1) / pl.nt);
    if (tiles < sms) pl.splits = (int)std::min<long long>({8, (long long)sms * pl.ctas_per_sm / tiles, (kt + 1) / 2});
    pl.splits = std::max(1, pl.splits);
  }
  return pl;
}

template <typename T>
static nvfp4_status run_mx_gemm(const MxGemmArgs& a, const MxPlan& pl, int sms, const CUtensorMap& tmW,
                                const CUtensorMap& tmX, const CUtensorMap& tmX32, const MxGemmParams& p,
                                long long tiles, cudaStream_t s) {
  NV_CHECK(opt_in_smem<mx_gemm_kernel<T>>());
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
  cfg.dynamicSmemBytes = (size_t)pl.stages * mx_stage_bytes(pl.nt) + 1024;
  cfg.stream = s;
  (void)a;
  return check_cuda(cudaLaunchKernelEx(&cfg, mx_gemm_kernel<T>, tmW, tmX, tmX32, p), "mx_gemm_kernel");
}

static nvfp4_status launch_mx_gemm(const MxGemmArgs& a, cudaStream_t s) {
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  const MxPlan pl = plan_mx_gemm(a.M, a.N, a.K, a.E, sms);
  MxGemmParams p;
  p.M = a.M;
  p.N = a.N;
  p.E = a.E;
  p.groups = mx_groups(a.K);
  p.kt_total = (p.groups + kXAtoms - 1) / kXAtoms;
  p.n_wt = (a.N + kXBM - 1) / kXBM;
  p.nt = pl.nt;
  p.n_tt = a.E ? 0 : (a.M + pl.nt - 1) / pl.nt;
  p.stages = pl.stages;
  p.splits = pl.splits;
  p.early_b = a.early_b && a.E == 0;
  p.expert_offsets = a.expert_offsets;
  p.expert_counts = a.expert_counts;
  p.a_sf = a.a_scales;
  p.b_sf = a.b_scales;
  p.row_weight = a.row_weight;
  p.bias = a.bias;
  p.y = a.y;
  p.y_stride = a.y_stride;
  p.status = a.status;
  // tiles at most: each expert may end in a partly filled token tile
  const long long tiles = (long long)p.n_wt * (a.E ? (a.M + pl.nt - 1) / pl.nt + a.E : p.n_tt);
  const uint64_t inner = (uint64_t)mx_row_bytes(a.K);
  CUtensorMap tmW, tmX, tmX32;
  NV_CHECK(make_tmap_2d(&tmW, a.b_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner,
                        (uint64_t)std::max(1, a.E) * (uint64_t)a.N, inner, kXRowBytes, kXBM));
  NV_CHECK(make_tmap_2d(&tmX, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner, (uint64_t)a.M, inner, kXRowBytes,
                        (uint32_t)pl.nt));
  if (a.E) {
    NV_CHECK(make_tmap_2d(&tmX32, a.a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, inner, (uint64_t)a.M, inner, kXRowBytes,
                          32));
  } else {
    tmX32 = tmX;
  }
  switch (a.out_dtype) {
    case MXFP4_DTYPE_BF16: return run_mx_gemm<Bf16>(a, pl, sms, tmW, tmX, tmX32, p, tiles, s);
    case MXFP4_DTYPE_F16: return run_mx_gemm<F16>(a, pl, sms, tmW, tmX, tmX32, p, tiles, s);
    default: return run_mx_gemm<F32>(a, pl, sms, tmW, tmX, tmX32, p, tiles, s);
  }
}

static nvfp4_status check_product(const char* name, int M, const uint8_t* b_codes, const uint8_t* b_scales, int N,
                                  int K, int E, const int32_t* offsets, const int32_t* counts,
                                  const float* row_weight, const float* bias, int out_dtype, const void* y,
                                  long long y_stride) {
  NV_REQUIRE(M >= 0 && N >= 1 && K >= 1, NVFP4_ERR_INVALID_ARG, "%s: M=%d N=%d K=%d", name, M, N, K);
  NV_REQUIRE(K <= (1 << 30) && N <= (1 << 30), NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: N=%d or K=%d is above 2^30", name, N,
             K);
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
  return launch_mx_gemm(g, as_stream(stream));
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
  // b may load before the quantiser has finished: the quantiser itself starts
  // only behind everything queued earlier, which may have written b
  g.early_b = true;
  cudaStream_t s = as_stream(stream);
  NV_CHECK(launch_mx_quantize(x, dtype, rows, K, row_stride, perm, M, NVFP4_LAYOUT_TILED, l.codes, l.scales, s));
  return launch_mx_gemm(g, s);
}
