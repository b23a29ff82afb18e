// Load-balance loss of the router, per-expert counts, and the gradient.
//
// Forward, two kernels.  balance_pieces_kernel streams the logits once: a
// group of lanes holds one token's row, takes its softmax (or sigmoid shares)
// in registers and adds it to per-lane sums; a block covers a fixed chunk of
// tokens and leaves, for every (chunk, sequence) piece it meets, the piece's
// probability sums, counts and tokens.  Pieces are numbered chunk + sequence:
// going along the tokens either the chunk or the sequence advances, so the
// numbers are distinct, and chunks + S entries hold them for any lengths.
// balance_finish_kernel adds each sequence's pieces in order; its last block
// adds the sequences.  Every sum has a fixed order.
//
// Backward, one kernel: the same row arithmetic, with the experts' shares f
// of the row's sequence held in registers while the sequence lasts.
//
// Bound: HBM (logits in; gradient out), with one exponential (softmax) or one
// exponential and one reciprocal (sigmoid) per element behind it; below some
// ten thousand tokens the chain of loads, joins and launches.  Measured on one
// B200 (fp32, 128 experts, top-8): 262,144 tokens forward 38 us (3.7 TB/s),
// backward 50 us (5.3 TB/s); 65,536 tokens 19 and 14 us (inputs in L2); 16
// tokens of 80 experts 3.8 and 2.7 us.  With four logits a lane and row instead of
// sixteen (five shuffles for each maximum and sum), a reciprocal a logit for
// softmax too and the choices counted before the rows, 65,536 tokens took 57
// and 31 us.
#include <algorithm>
#include <type_traits>

#include "mx.cuh"
#include "../../include/moe_balance.h"

namespace nvfp4moe {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalMaxE = 1024;
constexpr int kBalMaxK = 32;
constexpr int kBalOneBlock = 16384;      // logits

struct BalanceShape {
  int T, E, S, k;
  int lanes;                  // lanes per row, a power of two
  long long stride;           // logits row stride, elements
  const int32_t* seq_offsets; // null: one sequence
  const uint8_t* mask;        // null: every token
};

NVDEV int seq_begin(const BalanceShape& b, int s) {
  return b.seq_offsets ? min(max(__ldg(b.seq_offsets + s), 0), b.T) : (s > 0 ? b.T : 0);
}
// The last sequence that starts at or before token t, or -1.
NVDEV int seq_of(const BalanceShape& b, int t) {
  int lo = -1, hi = b.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_begin(b, mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Four neighbouring logits from element e of a row; -inf past E.
template <typename T, bool VEC>
NVDEV void load4(const void* logits, long long row, int e, int E, bool live, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = -INFINITY;
  if (!live || e >= E) return;
  if constexpr (VEC) {
    if constexpr (T::size == 4) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(logits) + row + e));
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + row + e));
      v[0] = T::lo(u.x); v[1] = T::hi(u.x); v[2] = T::lo(u.y); v[3] = T::hi(u.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i < E) {
        if constexpr (T::size == 4) v[i] = __ldg(static_cast<const float*>(logits) + row + e + i);
        else v[i] = T::from(__ldg(static_cast<const uint16_t*>(logits) + row + e + i));
      }
  }
}

template <int N>
NVDEV float row_max(const float* v, int lanes) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  for (int o = lanes >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
NVDEV float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
NVDEV float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// l -> the row's scores up to a common factor (in place): exp(l - max), or
// sigma(l), and where asked d = dlog(score)/dl (1, or sigma(-l)).
// Softmax: exp2((l - max) log2(e)), whose two roundings move a share p by about
// |log p| 2^-23 relative.  (The difference comes first: l log2(e) of the
// type's lowest value, a usual mask, is no fp32 number.)
// Sigmoid: while the row's largest logit is above -60 the sigmas are taken as
// they are (one that underflows is below 1e-12 of the largest); below it
// sigma(l) is exp(l) to the last bit of fp32, and the shares are a softmax,
// which nothing underflows.  1 - sigma is taken as t sigma with t = exp(-l)
// for l >= 0, where 1 - sigma would cancel.
// -inf (a masked expert, or past E) gives 0 by itself; a row of nothing else
// has max = -inf and is measured from 0 instead.
template <int N, int SCORE, bool GRAD>
NVDEV void row_scores(float* l, float* d, int lanes) {
  const float m = row_max<N>(l, lanes);
  if (SCORE == MOE_BALANCE_SOFTMAX || m < -60.0f) {
    const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      l[i] = ex2_approx((l[i] - from) * kLog2e);
      if (GRAD) d[i] = 1.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float t = ex2_approx(-l[i] * kLog2e);
      const float sg = rcp_approx(1.0f + t);
      if (GRAD) d[i] = l[i] < 0.0f ? 1.0f - sg : t * sg;
      l[i] = sg;
    }
  }
  __syncwarp();
}
// 1 / the row's sum of scores; 0 for a row without any.
NVDEV float share_factor(float z) { return z == 0.0f ? 0.0f : rcp_approx(z); }

struct BalancePieces {
  float* probs;       // [pieces][E]
  int32_t* counts;    // [pieces][E]
  int32_t* tokens;    // [pieces]
  uint32_t* status;   // [0] status word, [1] finished blocks
};

// f = counts * share_unit: E / (k n).
NVDEV float share_unit(const BalanceShape& b, int n) { return (float)b.E / ((float)b.k * (float)n); }

struct BalanceOut {
  float coeff;
  float* loss;        // [1]
  int32_t* counts;    // [S][E]
  int32_t* tokens;    // [S + 1]
  float* probs;       // [S][E]
};

// V x 4 logits a lane; UR rows in flight per group of lanes.  ONE: a single
// block takes every token (chunk >= T) and writes the results itself.
template <typename T, bool VEC, int V, int UR, int SCORE, bool ONE>
__global__ void __launch_bounds__(kBalThreads, V <= 4 ? 3 : 2)
    balance_pieces_kernel(const void* __restrict__ logits, const int32_t* __restrict__ topk_idx, const BalanceShape b,
                          int chunk, const BalancePieces out, const BalanceOut res) {
  extern __shared__ float s_sum[];                          // [warps][E], then int counts [E]
  __shared__ int s_tokens;
  __shared__ double s_dot[kBalWarps];
  int32_t* s_cnt = reinterpret_cast<int32_t*>(s_sum + kBalWarps * b.E);
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0 && threadIdx.x < 2) out.status[threadIdx.x] = 0u;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int L = b.lanes, l = lane & (L - 1), g = lane / L, G = 32 / L;
  const int c0 = (int)min((long long)blockIdx.x * chunk, (long long)b.T);
  const int c1 = (int)min((long long)c0 + chunk, (long long)b.T);
  if (!ONE && c0 >= c1) return;
  double dot = 0.0;                                         // ONE: this thread's experts, every sequence
  int full = 0;
  for (int s = ONE ? 0 : max(seq_of(b, c0), 0); s < b.S; ++s) {
    const int s0 = seq_begin(b, s);
    if (!ONE && s0 >= c1) break;
    const int r0 = max(c0, s0), r1 = min(c1, seq_begin(b, s + 1));
    if (!ONE && r0 >= r1) continue;
    __syncthreads();                                        // the last piece has left shared memory
    for (int e = threadIdx.x; e < b.E; e += kBalThreads) s_cnt[e] = 0;
    if (threadIdx.x == 0) s_tokens = 0;
    __syncthreads();
    int kept = 0;
    float acc[V * 4];
#pragma unroll
    for (int i = 0; i < V * 4; ++i) acc[i] = 0.0f;
    for (int base = r0 + warp * G; base < r1; base += kBalWarps * G * UR) {
      float v[UR][V * 4];
      int choice[UR];
      bool live[UR];
#pragma unroll
      for (int u = 0; u < UR; ++u) {
        const int t = base + u * kBalWarps * G + g;
        live[u] = t < r1;
        // a masked token's logits are read, so that no load waits for the mask, and not used
        const uint8_t m = live[u] && b.mask ? __ldg(b.mask + t) : 1;
        choice[u] = live[u] && l < b.k ? __ldg(topk_idx + (size_t)t * b.k + l) : -1;
#pragma unroll
        for (int i = 0; i < V; ++i)
          load4<T, VEC>(logits, (long long)t * b.stride, (i * L + l) * 4, b.E, live[u], v[u] + 4 * i);
        live[u] = live[u] && m;
      }
#pragma unroll
      for (int u = 0; u < UR; ++u) {
        row_scores<V * 4, SCORE, false>(v[u], nullptr, L);
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < V * 4; ++i) z += v[u][i];
        for (int o = L >> 1; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (live[u]) {
          const float inv = share_factor(z);
#pragma unroll
          for (int i = 0; i < V * 4; ++i) acc[i] = __fmaf_rn(v[u][i], inv, acc[i]);
          // the choices: integer atomics, whose order does not matter
          if (choice[u] >= 0 && choice[u] < b.E) atomicAdd(&s_cnt[choice[u]], 1);
          for (int j = l + L; j < b.k; j += L) {
            const int e = __ldg(topk_idx + (size_t)(base + u * kBalWarps * G + g) * b.k + j);
            if (e >= 0 && e < b.E) atomicAdd(&s_cnt[e], 1);
          }
          if (l == 0) ++kept;
        }
        __syncwarp();
      }
    }
    // lanes of the warp that hold the same experts, then the warps in order
#pragma unroll
    for (int i = 0; i < V * 4; ++i)
      for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (g == 0) {
#pragma unroll
      for (int i = 0; i < V * 4; ++i) {
        const int e = ((i >> 2) * L + l) * 4 + (i & 3);
        if (e < b.E) s_sum[warp * b.E + e] = acc[i];
      }
    }
    kept = __reduce_add_sync(0xffffffffu, kept);
    if (lane == 0 && kept) atomicAdd(&s_tokens, kept);
    __syncthreads();
    const size_t piece = (size_t)blockIdx.x + s;
    const int n = s_tokens;
    for (int e = threadIdx.x; e < b.E; e += kBalThreads) {
      float z = 0.0f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) z += s_sum[w * b.E + e];
      const int c = s_cnt[e];
      if constexpr (ONE) {
        const float mean = n > 0 ? z / (float)n : 0.0f;
        res.counts[(size_t)s * b.E + e] = c;
        res.probs[(size_t)s * b.E + e] = mean;
        if (n > 0) dot += (double)((float)c * share_unit(b, n) * mean);
      } else {
        out.probs[piece * b.E + e] = z;
        out.counts[piece * b.E + e] = c;
      }
    }
    if constexpr (ONE) full += n > 0;
    if (threadIdx.x == 0) (ONE ? res.tokens[s] : out.tokens[piece]) = n;
  }
  if constexpr (ONE) {
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_dot[warp] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      dot = 0.0;
      for (int w = 0; w < kBalWarps; ++w) dot += s_dot[w];
      *res.loss = full ? res.coeff / (float)full * (float)dot : 0.0f;
      res.tokens[b.S] = full;
    }
  }
}

// One block per (sequence, 32 experts): warp w adds pieces w, w + 32, ...,
// eight loads in flight; the warps' sums join in warp order.
constexpr int kFinThreads = 1024, kFinWarps = kFinThreads / 32;
__global__ void __launch_bounds__(kFinThreads) balance_finish_kernel(const BalanceShape b, int chunk,
                                                                     const BalancePieces in, double* __restrict__ dots,
                                                                     const BalanceOut res) {
  __shared__ double s_p[kFinWarps][33];                     // padded: read by columns
  __shared__ int32_t s_c[kFinWarps][33];
  __shared__ int s_n[kFinWarps];
  __shared__ bool s_last;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int eg = gridDim.y, s = blockIdx.x, e = blockIdx.y * 32 + lane;
  const int r0 = seq_begin(b, s), r1 = seq_begin(b, s + 1);
  double p = 0.0;
  int c = 0, n = 0;
  if (r0 < r1) {
    const int first = r0 / chunk, last = (r1 - 1) / chunk;
    for (int i0 = first + warp; i0 <= last; i0 += kFinWarps * 8) {
      float vp[8];
      int vc[8], vn[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kFinWarps;
        const size_t piece = (size_t)min(i, last) + s;
        const bool in_range = i <= last;
        vp[u] = in_range && e < b.E ? in.probs[piece * b.E + e] : 0.0f;
        vc[u] = in_range && e < b.E ? in.counts[piece * b.E + e] : 0;
        vn[u] = in_range ? in.tokens[piece] : 0;             // the same in every lane
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        p += (double)vp[u];
        c += vc[u];
        n += vn[u];
      }
    }
  }
  s_p[warp][lane] = p;
  s_c[warp][lane] = c;
  if (lane == 0) s_n[warp] = n;
  __syncthreads();
  // warp w now joins expert w's 32 partial sums, in the same tree every time
  p = s_p[lane][warp];
  c = __reduce_add_sync(0xffffffffu, s_c[lane][warp]);
  n = __reduce_add_sync(0xffffffffu, s_n[lane]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
  __syncthreads();
  if (lane == 0) {
    const int e = blockIdx.y * 32 + warp;
    const float mean = n > 0 ? (float)p / (float)n : 0.0f;
    if (e < b.E) {
      res.counts[(size_t)s * b.E + e] = c;
      res.probs[(size_t)s * b.E + e] = mean;
    }
    s_p[0][warp] = n > 0 ? (double)((float)c * share_unit(b, n) * mean) : 0.0;
  }
  __syncthreads();
  if (warp == 0) {
    double dot = s_p[0][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) {
      dots[(size_t)s * eg + blockIdx.y] = dot;
      if (blockIdx.y == 0) res.tokens[s] = n;
      __threadfence();
      s_last = atomicAdd(&in.status[1], 1u) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  // the last block to finish adds the sequences, in a fixed order
  __threadfence();
  double z = 0.0;
  int full = 0;
  for (long long i = threadIdx.x; i < (long long)b.S * eg; i += kFinThreads) z += __ldcg(dots + i);
  for (int i = threadIdx.x; i < b.S; i += kFinThreads) full += __ldcg(res.tokens + i) > 0;
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  full = __reduce_add_sync(0xffffffffu, full);
  __syncthreads();
  if (lane == 0) {
    s_p[warp][0] = z;
    s_n[warp] = full;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    z = 0.0;
    full = 0;
    for (int w = 0; w < kFinWarps; ++w) {
      z += s_p[w][0];
      full += s_n[w];
    }
    *res.loss = full ? res.coeff / (float)full * (float)z : 0.0f;
    res.tokens[b.S] = full;
  }
}

template <typename T, bool VEC, int V, int UR, int SCORE>
__global__ void __launch_bounds__(kBalThreads, V <= 4 ? 3 : 2) balance_backward_kernel(const void* __restrict__ logits,
                                                                       const BalanceShape b, int rows_per_warp,
                                                                       float coeff, const int32_t* __restrict__ counts,
                                                                       const int32_t* __restrict__ tokens,
                                                                       const float* __restrict__ grad_loss,
                                                                       void* __restrict__ dlogits,
                                                                       long long grad_stride) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int L = b.lanes, l = lane & (L - 1), g = lane / L, G = 32 / L;
  const long long w0 = ((long long)blockIdx.x * kBalWarps + warp) * rows_per_warp;
  const int r1 = (int)min(w0 + rows_per_warp, (long long)b.T);
  if (w0 >= b.T) return;
  const float up = *grad_loss;
  const int full = tokens[b.S];
  // this group's sequence: the tokens [s0, s1) that its shares f hold for
  int s0 = 0, s1 = 0;
  float f[V * 4], scale = 0.0f;
#pragma unroll
  for (int i = 0; i < V * 4; ++i) f[i] = 0.0f;
  auto enter = [&](int t) {
    const int s = seq_of(b, t);
    scale = 0.0f;
    s0 = s1 = 0;
    if (s >= 0 && t < seq_begin(b, s + 1)) {
      s0 = seq_begin(b, s);
      s1 = seq_begin(b, s + 1);
      int c[V * 4];
#pragma unroll
      for (int i = 0; i < V * 4; ++i) {
        const int e = ((i >> 2) * L + l) * 4 + (i & 3);
        c[i] = e < b.E ? __ldg(counts + (size_t)s * b.E + e) : 0;
      }
      const int n = __ldg(tokens + s);
      const float unit = n > 0 ? share_unit(b, n) : 0.0f;
      scale = n > 0 && full > 0 ? up * coeff / ((float)full * (float)n) : 0.0f;
#pragma unroll
      for (int i = 0; i < V * 4; ++i) f[i] = (float)c[i] * unit;
    }
  };
  for (int base = (int)w0; base < r1; base += G * UR) {
    float v[UR][V * 4];
    bool live[UR];
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const int t = base + u * G + g;
      live[u] = t < r1;
      const uint8_t m = live[u] && b.mask ? __ldg(b.mask + t) : 1;
#pragma unroll
      for (int i = 0; i < V; ++i)
        load4<T, VEC>(logits, (long long)t * b.stride, (i * L + l) * 4, b.E, live[u], v[u] + 4 * i);
      live[u] = live[u] && m;
    }
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const int t = base + u * G + g;
      if (live[u] && !(t >= s0 && t < s1)) enter(t);
      const bool in_seq = live[u] && t >= s0 && t < s1;
      __syncwarp();
      float d[V * 4];
      row_scores<V * 4, SCORE, true>(v[u], d, L);
      float z = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < V * 4; ++i) {
        z += v[u][i];
        dot = __fmaf_rn(f[i], v[u][i], dot);
      }
      for (int o = L >> 1; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float inv = share_factor(z);
      dot *= inv;
      const float by = scale * inv;
      if (t < r1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = (i * L + l) * 4;
          if (e >= b.E) continue;
          float o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = in_seq ? by * v[u][4 * i + j] * (f[4 * i + j] - dot) * d[4 * i + j] : 0.0f;
          const long long at = (long long)t * grad_stride + e;
          if constexpr (VEC) {
            if constexpr (T::size == 4)
              *reinterpret_cast<float4*>(static_cast<float*>(dlogits) + at) = make_float4(o[0], o[1], o[2], o[3]);
            else
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dlogits) + at) =
                  make_uint2(T::pack(o[0], o[1]), T::pack(o[2], o[3]));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (e + j < b.E) {
                if constexpr (T::size == 4) static_cast<float*>(dlogits)[at + j] = o[j];
                else static_cast<uint16_t*>(dlogits)[at + j] = T::one(o[j]);
              }
          }
        }
      }
    }
  }
}

// Lanes per row: the fewest (a power of two) that hold it in at most 16
// logits each; a row's maximum and sums then cost few shuffles (at 128
// experts 3 a row and lane instead of 5, and 16 logits a lane to share them
// instead of 4).
static inline int balance_lanes(int E) {
  const int quads = (E + 3) / 4;
  int l = 1;
  while (l < 32 && l * 4 < quads) l <<= 1;
  return l;
}
// Tokens per block of the forward: about three blocks an SM (what fits at
// once), whole warps of rows.
static inline int balance_chunk(int T, int E) {
  const int step = kBalWarps * (32 / balance_lanes(E));
  return std::max(1, (int)(((long long)T + 148ll * 3 * step - 1) / (148ll * 3 * step))) * step;
}
// Few logits: one block does the whole forward, one launch instead of two.
// Measured, one block against two kernels (us): 16 x 80 3.7 and 8.8, 64 x 80
// 4.1 and 8.9, 128 x 128 6.3 and 9.5, 256 x 128 9.4 and 9.6, 512 x 128 15.5
// and 9.5.  It walks its sequences one after the other, hence at most 64.
static inline bool balance_one_block(int T, int E, int S) { return (long long)T * E <= kBalOneBlock && S <= 64; }

struct BalanceScratch {
  uint32_t* status;
  BalancePieces pieces;
  double* dots;
};
static BalanceScratch carve_balance(Carver& c, int T, int E, int S) {
  BalanceScratch w;
  const int chunk = balance_chunk(T, E);
  const size_t pieces = (size_t)((T + chunk - 1) / chunk) + (size_t)S;
  w.status = c.take<uint32_t>(64);
  w.pieces.status = w.status;
  w.pieces.probs = c.take<float>(pieces * E);
  w.pieces.counts = c.take<int32_t>(pieces * E);
  w.pieces.tokens = c.take<int32_t>(pieces);
  w.dots = c.take<double>((size_t)S * ((E + 31) / 32));
  return w;
}

static nvfp4_status check_balance(const char* name, const void* logits, int dtype, int T, int E, long long stride,
                                  int k, int score, int S, const int32_t* seq_offsets) {
  NV_REQUIRE(mx_dtype_ok(dtype), NVFP4_ERR_INVALID_ARG, "%s: unknown dtype %d", name, dtype);
  NV_REQUIRE(score == MOE_BALANCE_SIGMOID || score == MOE_BALANCE_SOFTMAX, NVFP4_ERR_INVALID_ARG,
             "%s: unknown score %d", name, score);
  NV_REQUIRE(T >= 0 && S >= 1, NVFP4_ERR_INVALID_ARG, "%s: T=%d S=%d", name, T, S);
  NV_REQUIRE(T <= (1 << 30) && S <= (1 << 24), NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: T=%d or S=%d is too large", name, T,
             S);
  NV_REQUIRE(E >= 1 && E <= kBalMaxE && k >= 1 && k <= kBalMaxK, NVFP4_ERR_UNSUPPORTED_SHAPE,
             "%s: needs 1 <= E <= %d and 1 <= k <= %d (E=%d k=%d)", name, kBalMaxE, kBalMaxK, E, k);
  NV_REQUIRE(seq_offsets || S == 1, NVFP4_ERR_INVALID_ARG, "%s: S=%d sequences need seq_offsets", name, S);
  NV_REQUIRE(T == 0 || logits, NVFP4_ERR_INVALID_ARG, "%s: logits is NULL", name);
  NV_REQUIRE(T <= 1 || stride >= E, NVFP4_ERR_INVALID_ARG, "%s: row stride %lld is below E=%d", name, stride, E);
  NV_REQUIRE(aligned(logits, mx_elem_size(dtype)) && aligned(seq_offsets, 4), NVFP4_ERR_INVALID_ARG,
             "%s: a tensor is not aligned to its elements", name);
  return NVFP4_OK;
}

// Calls f(type tag, vector loads allowed, quads of logits per lane, score).
template <typename F>
static nvfp4_status with_balance(int dtype, bool vec, int E, int score, F&& f) {
  const int quads = ((E + 3) / 4 + balance_lanes(E) - 1) / balance_lanes(E);
  auto by_score = [&](auto tag, auto vv, auto v) -> nvfp4_status {
    if (score == MOE_BALANCE_SOFTMAX) return f(tag, vv, v, std::integral_constant<int, MOE_BALANCE_SOFTMAX>{});
    return f(tag, vv, v, std::integral_constant<int, MOE_BALANCE_SIGMOID>{});
  };
  auto by_v = [&](auto tag, auto vv) -> nvfp4_status {
    if (quads <= 1) return by_score(tag, vv, std::integral_constant<int, 1>{});
    if (quads <= 2) return by_score(tag, vv, std::integral_constant<int, 2>{});
    if (quads <= 3) return by_score(tag, vv, std::integral_constant<int, 3>{});
    if (quads <= 4) return by_score(tag, vv, std::integral_constant<int, 4>{});
    return by_score(tag, vv, std::integral_constant<int, 8>{});
  };
  auto by_vec = [&](auto tag) -> nvfp4_status {
    return vec ? by_v(tag, std::true_type{}) : by_v(tag, std::false_type{});
  };
  if (dtype == MXFP4_DTYPE_BF16) return by_vec(Bf16{});
  if (dtype == MXFP4_DTYPE_F16) return by_vec(F16{});
  return by_vec(F32{});
}
// Rows in flight per group of lanes.
constexpr int balance_rows(int v) { return v <= 1 ? 4 : v <= 4 ? 2 : 1; }
// Whether rows may be read or written four elements at a time.
static inline bool balance_vec(const void* p, long long stride, int T, int E, int elem) {
  return E % 4 == 0 && row_access_bytes(p, T > 1 ? stride * elem : 0, elem) >= 4 * elem;
}

}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" size_t moe_balance_loss_workspace_size(int T, int E, int S) {
  if (T < 0 || T > (1 << 30) || E < 1 || E > kBalMaxE || S < 1 || S > (1 << 24)) return 0;
  Carver c(nullptr);
  carve_balance(c, T, E, S);
  return c.size();
}

extern "C" nvfp4_status moe_balance_loss(const void* logits, int dtype, int T, int E, long long row_stride,
                                         const int32_t* topk_idx, int k, int score, const uint8_t* token_mask,
                                         const int32_t* seq_offsets, int S, float coeff, float* loss, int32_t* counts,
                                         int32_t* tokens, float* probs, void* ws, size_t ws_bytes, void* stream) {
  NV_CHECK(check_balance("moe_balance_loss", logits, dtype, T, E, row_stride, k, score, S, seq_offsets));
  NV_REQUIRE((T == 0 || topk_idx) && loss && counts && tokens && probs, NVFP4_ERR_INVALID_ARG,
             "moe_balance_loss: a required pointer is NULL");
  NV_REQUIRE(aligned(topk_idx, 4) && aligned(loss, 4) && aligned(counts, 4) && aligned(tokens, 4) && aligned(probs, 4),
             NVFP4_ERR_INVALID_ARG, "moe_balance_loss: a tensor is not aligned to its elements");
  const size_t need = moe_balance_loss_workspace_size(T, E, S);
  NV_REQUIRE(ws && ws_bytes >= need && aligned(ws, 256), NVFP4_ERR_WORKSPACE,
             "moe_balance_loss: needs a 256-byte aligned workspace of %zu bytes", need);
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  cudaStream_t s = as_stream(stream);
  Carver c(ws);
  const BalanceScratch w = carve_balance(c, T, E, S);
  const int chunk = balance_chunk(T, E);
  const BalanceShape b{T, E, S, k, balance_lanes(E), row_stride, seq_offsets, token_mask};
  const bool one = balance_one_block(T, E, S);
  const BalanceOut res{coeff, loss, counts, tokens, probs};
  const dim3 grid(one ? 1u : (unsigned)std::max(1, (T + chunk - 1) / chunk));
  const size_t smem = (size_t)(kBalWarps + 1) * E * 4;
  NV_CHECK(with_balance(dtype, balance_vec(logits, row_stride, T, E, mx_elem_size(dtype)), E, score,
                        [&](auto tag, auto vec, auto v, auto sc) -> nvfp4_status {
                          constexpr int V = decltype(v)::value, SC = decltype(sc)::value;
                          using TT = decltype(tag);
                          constexpr bool VEC = decltype(vec)::value;
                          return launch_dependent(
                              "balance_pieces_kernel",
                              one ? balance_pieces_kernel<TT, VEC, V, balance_rows(V), SC, true>
                                  : balance_pieces_kernel<TT, VEC, V, balance_rows(V), SC, false>,
                              grid, dim3(kBalThreads), smem, s, logits, topk_idx, b, one ? std::max(T, 1) : chunk,
                              w.pieces, res);
                        }));
  if (one) return NVFP4_OK;
  return launch_dependent("balance_finish_kernel", balance_finish_kernel, dim3((unsigned)S, (unsigned)((E + 31) / 32)),
                          dim3(kFinThreads), 0, s, b, chunk, w.pieces, w.dots, res);
}

extern "C" nvfp4_status moe_balance_loss_backward(const void* logits, int dtype, int T, int E, long long row_stride,
                                                  int k, int score, const uint8_t* token_mask,
                                                  const int32_t* seq_offsets, int S, float coeff,
                                                  const int32_t* counts, const int32_t* tokens,
                                                  const float* grad_loss, void* dlogits, long long grad_stride,
                                                  void* stream) {
  NV_CHECK(check_balance("moe_balance_loss_backward", logits, dtype, T, E, row_stride, k, score, S, seq_offsets));
  if (T == 0) return NVFP4_OK;
  NV_REQUIRE(counts && tokens && grad_loss && dlogits, NVFP4_ERR_INVALID_ARG,
             "moe_balance_loss_backward: a required pointer is NULL");
  NV_REQUIRE(dlogits != logits, NVFP4_ERR_INVALID_ARG,
             "moe_balance_loss_backward: dlogits may not take the place of logits");
  NV_REQUIRE(T <= 1 || grad_stride >= E, NVFP4_ERR_INVALID_ARG,
             "moe_balance_loss_backward: gradient stride %lld is below E=%d", grad_stride, E);
  NV_REQUIRE(aligned(dlogits, mx_elem_size(dtype)) && aligned(counts, 4) && aligned(tokens, 4) &&
                 aligned(grad_loss, 4),
             NVFP4_ERR_INVALID_ARG, "moe_balance_loss_backward: a tensor is not aligned to its elements");
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  const BalanceShape b{T, E, S, k, balance_lanes(E), row_stride, seq_offsets, token_mask};
  const int elem = mx_elem_size(dtype);
  const bool vec = balance_vec(logits, row_stride, T, E, elem) && balance_vec(dlogits, grad_stride, T, E, elem);
  // about three blocks an SM (what fits at once); a warp takes neighbouring
  // rows, so that it seldom changes sequence
  const int per_iter = 32 / b.lanes;
  const long long warps = (long long)sms * 3 * kBalWarps;
  const int rows_per_warp = (int)(((T + warps - 1) / warps + per_iter - 1) / per_iter) * per_iter;
  const long long rows_per_block = (long long)rows_per_warp * kBalWarps;
  const dim3 grid((unsigned)((T + rows_per_block - 1) / rows_per_block));
  return with_balance(dtype, vec, E, score, [&](auto tag, auto vv, auto v, auto sc) -> nvfp4_status {
    constexpr int V = decltype(v)::value;
    return launch_dependent(
        "balance_backward_kernel",
        balance_backward_kernel<decltype(tag), decltype(vv)::value, V, balance_rows(V), decltype(sc)::value>, grid,
        dim3(kBalThreads), 0, as_stream(stream), logits, b, rows_per_warp, coeff, counts, tokens, grad_loss, dlogits,
        grad_stride);
  });
}
