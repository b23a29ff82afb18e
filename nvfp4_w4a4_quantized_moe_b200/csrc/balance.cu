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
// Bound: HBM (logits in; gradient out) behind a dozen instructions an element,
// one exponential (softmax) or one exponential and one reciprocal (sigmoid)
// among them; below some ten thousand tokens the chain of loads, joins and
// launches.  Measured on one B200 (top-8, us forward and backward, logits from
// HBM):
//                                               softmax                 sigmoid
//                                          fp32        bf16        fp32        bf16
//   262,144 x 128, 33 sequences, mask   38.7, 50.3  36.8, 36.4  42.5, 53.5  42.7, 43.7
//   65,531 x 128, 17 sequences, mask    21.5, 15.5  19.2, 12.5  21.5, 16.5  20.3, 14.4
//   65,531 x 128, one sequence          16.5, 14.6  15.7, 10.9  17.4, 15.4  16.9, 13.0
//   262,144 x 80, one sequence          32.7, 38.4  30.9, 30.0  35.3, 42.1  34.5, 35.4
//   8,192 x 80, one sequence             8.9,  3.7   9.3,  3.8   9.2,  3.9   9.4,  4.2
//   16 x 80                              3.4,  2.6   3.4,  2.6   3.5,  2.7   3.5,  2.6
// What brought it there: four logits a lane and row (five shuffles for each
// maximum and sum), a reciprocal a logit for softmax too and the choices counted
// before the rows, 57 and 31 us at 65,536 tokens fp32; sixteen a lane 23 and 17
// (bf16 22 and 16: 433 instructions a warp's row group); pairs of fp32 in one
// instruction, one fused operation before an exponential, loads without
// branches, a row ahead, and smaller blocks of the finish, the table above.
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

// A lane's share of a row: V quads of neighbouring logits, quad i from element
// (i L + l) 4 on, as they are in memory.  Every lane loads, without a branch:
// past the row's end from inside it (row_values puts -inf there).
template <typename T, int V> struct RowWords { uint32_t w[V * T::size]; };
template <typename T, bool VEC, int V>
NVDEV void load_row(const uint8_t* row, int l, int L, int E, RowWords<T, V>& r) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = (i * L + l) * 4;
    if constexpr (VEC) {
      const uint8_t* p = row + min(e, E - 4) * T::size;
      if constexpr (T::size == 4) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
        r.w[4 * i] = u.x; r.w[4 * i + 1] = u.y; r.w[4 * i + 2] = u.z; r.w[4 * i + 3] = u.w;
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        r.w[2 * i] = u.x; r.w[2 * i + 1] = u.y;
      }
    } else if constexpr (T::size == 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[4 * i + j] = __ldg(reinterpret_cast<const uint32_t*>(row) + min(e + j, E - 1));
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        r.w[2 * i + j] = (uint32_t)__ldg(p + min(e + 2 * j, E - 1)) | ((uint32_t)__ldg(p + min(e + 2 * j + 1, E - 1)) << 16);
    }
  }
}
// Its values in pairs (packed fp32 instructions take two at once).
template <typename T, int V>
NVDEV void row_values(const RowWords<T, V>& r, int l, int L, int E, uint64_t* v) {
#pragma unroll
  for (int i = 0; i < V * 2; ++i) {
    if constexpr (T::size == 4) v[i] = pack_f32x2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    else v[i] = pack_f32x2(T::lo(r.w[i]), T::hi(r.w[i]));
  }
  if (V * 4 * L != E) {
#pragma unroll
    for (int i = 0; i < V * 2; ++i) {
      const int e = ((i >> 1) * L + l) * 4 + (i & 1) * 2;
      v[i] = pack_f32x2(e < E ? lo_f32(v[i]) : -INFINITY, e + 1 < E ? hi_f32(v[i]) : -INFINITY);
    }
  }
}

// Over the L lanes of a row.
NVDEV float group_max(float m, int L) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < L) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
NVDEV float group_sum(float z, int L) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < L) z += __shfl_xor_sync(0xffffffffu, z, o);
  return z;
}
NVDEV uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
NVDEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
NVDEV uint64_t twice(float a) { return pack_f32x2(a, a); }
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
// Softmax: exp2(l log2(e) - max log2(e)) in one fused operation an element.
// The rounding of max log2(e) is a common factor of the row (below 2^0.01 while
// |max| < 65536) and leaves the shares; the other moves a share p by about
// |log p| 2^-24 relative.  Beyond that, and for a row whose max is no number,
// exp2((l - max) log2(e)): l log2(e) of the type's lowest value, a usual mask,
// is no fp32 number, and is 0 in either form.
// Sigmoid: while the row's largest logit is above -60 the sigmas are taken as
// they are (one that underflows is below 1e-12 of the largest); below it
// sigma(l) is exp(l) to the last bit of fp32, and the shares are a softmax,
// which nothing underflows.  1 - sigma is taken as t sigma with t = exp(-l)
// for l >= 0, where 1 - sigma would cancel.
// -inf (a masked expert, or past E) gives 0 by itself; a row of nothing else
// has max = -inf and is measured from 0 instead.
template <int N, int SCORE, bool GRAD>
NVDEV void row_scores(uint64_t* l, uint64_t* d, int L) {
  float m = fmaxf(lo_f32(l[0]), hi_f32(l[0]));
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, fmaxf(lo_f32(l[i]), hi_f32(l[i])));
  m = group_max(m, L);
  if (SCORE == MOE_BALANCE_SOFTMAX || m < -60.0f) {
    if (fabsf(m) < 65536.0f) {
      const uint64_t by = twice(kLog2e), from = twice(-m * kLog2e);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint64_t x = fma_f32x2(l[i], by, from);
        l[i] = pack_f32x2(ex2_approx(lo_f32(x)), ex2_approx(hi_f32(x)));
      }
    } else {
      const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < N; ++i)
        l[i] = pack_f32x2(ex2_approx((lo_f32(l[i]) - from) * kLog2e), ex2_approx((hi_f32(l[i]) - from) * kLog2e));
    }
    if (GRAD && SCORE != MOE_BALANCE_SOFTMAX) {
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = twice(1.0f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t x = mul_f32x2(l[i], twice(-kLog2e));
      const uint64_t t = pack_f32x2(ex2_approx(lo_f32(x)), ex2_approx(hi_f32(x)));
      const uint64_t t1 = add_f32x2(t, twice(1.0f));
      const float s0 = rcp_approx(lo_f32(t1)), s1 = rcp_approx(hi_f32(t1));
      if (GRAD)
        d[i] = pack_f32x2(lo_f32(l[i]) < 0.0f ? 1.0f - s0 : lo_f32(t) * s0, hi_f32(l[i]) < 0.0f ? 1.0f - s1 : hi_f32(t) * s1);
      l[i] = pack_f32x2(s0, s1);
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

// Whether the forward's registers hold the next rows beside those at work: 32
// words of a row do not fit (32768 x 1024 fp32: 60.4 us ahead, 46.2 not), nor
// do 16 with the addresses of single elements (65536 x 127 fp32: 25.1, 21.6).
template <typename T, bool VEC, int V> constexpr bool loads_ahead() { return T::size == 2 || (VEC && V <= 4); }

// V x 4 logits a lane; UR rows at once per group of lanes.  ONE: a single
// block takes every token (chunk >= T) and writes the results itself.
template <typename T, bool VEC, int V, int UR, int SCORE, bool ONE>
__global__ void __launch_bounds__(kBalThreads, ONE ? 1 : V <= 4 ? 3 : 2)
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
    uint64_t acc2[V * 2];
#pragma unroll
    for (int i = 0; i < V * 2; ++i) acc2[i] = 0;
    // the next rows load while these are worked on
    RowWords<T, V> w[2][UR];
    int choice[2][UR];
    bool live[2][UR];
    auto load = [&](auto buf, int base) {
      constexpr int B = decltype(buf)::value;
#pragma unroll
      for (int u = 0; u < UR; ++u) {
        const int t = base + u * kBalWarps * G + g, at = min(t, r1 - 1);
        // a masked token's logits are read, so that no load waits for the mask, and not used
        const uint8_t m = b.mask ? __ldg(b.mask + at) : 1;
        choice[B][u] = l < b.k ? __ldg(topk_idx + (size_t)at * b.k + l) : -1;
        load_row<T, VEC, V>(static_cast<const uint8_t*>(logits) + (size_t)at * (size_t)b.stride * T::size, l, L, b.E,
                            w[B][u]);
        live[B][u] = t < r1 && m;
      }
    };
    auto work = [&](auto buf, int base) {
      constexpr int B = decltype(buf)::value;
#pragma unroll
      for (int u = 0; u < UR; ++u) {
        uint64_t v[V * 2];
        row_values<T, V>(w[B][u], l, L, b.E, v);
        row_scores<V * 2, SCORE, false>(v, nullptr, L);
        uint64_t z2 = v[0];
#pragma unroll
        for (int i = 1; i < V * 2; ++i) z2 = add_f32x2(z2, v[i]);
        const float z = group_sum(lo_f32(z2) + hi_f32(z2), L);
        if (live[B][u]) {
          const uint64_t inv = twice(share_factor(z));
#pragma unroll
          for (int i = 0; i < V * 2; ++i) acc2[i] = fma_f32x2(v[i], inv, acc2[i]);
          // the choices: integer atomics, whose order does not matter
          if ((unsigned)choice[B][u] < (unsigned)b.E) atomicAdd(&s_cnt[choice[B][u]], 1);
          for (int j = l + L; j < b.k; j += L) {
            const int e = __ldg(topk_idx + (size_t)(base + u * kBalWarps * G + g) * b.k + j);
            if ((unsigned)e < (unsigned)b.E) atomicAdd(&s_cnt[e], 1);
          }
          if (l == 0) ++kept;
        }
        __syncwarp();
      }
    };
    using B0 = std::integral_constant<int, 0>;
    using B1 = std::integral_constant<int, 1>;
    const int step = kBalWarps * G * UR;
    int base = r0 + warp * G;
    if constexpr (loads_ahead<T, VEC, V>() || ONE) {
      if (base < r1) load(B0{}, base);
#pragma unroll 1
      for (; base < r1; base += 2 * step) {
        if (base + step < r1) load(B1{}, base + step);
        work(B0{}, base);
        if (base + step >= r1) break;
        if (base + 2 * step < r1) load(B0{}, base + 2 * step);
        work(B1{}, base + step);
      }
    } else {
#pragma unroll 1
      for (; base < r1; base += step) {
        load(B0{}, base);
        work(B0{}, base);
      }
    }
    float acc[V * 4];
#pragma unroll
    for (int i = 0; i < V * 2; ++i) {
      acc[2 * i] = lo_f32(acc2[i]);
      acc[2 * i + 1] = hi_f32(acc2[i]);
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

// One block per (sequence, FE experts): a group of FE lanes adds every
// (256 / FE)-th piece, sixteen loads of each kind in flight; groups and warps
// join in a fixed order.
constexpr int kFinThreads = 256, kFinWarps = kFinThreads / 32, kFinLoads = 16;
template <int kFinE>
__global__ void __launch_bounds__(kFinThreads) balance_finish_kernel(const BalanceShape b, int chunk,
                                                                     const BalancePieces in, double* __restrict__ dots,
                                                                     const BalanceOut res) {
  constexpr int kFinSlots = kFinThreads / kFinE;
  __shared__ double s_p[kFinWarps][kFinE];
  __shared__ int s_c[kFinWarps][kFinE], s_n[kFinWarps];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int eg = gridDim.y, s = blockIdx.x, le = lane & (kFinE - 1), e = blockIdx.y * kFinE + le;
  const int slot = threadIdx.x / kFinE;
  // (the previous kernel ran behind whatever wrote the offsets)
  const int r0 = seq_begin(b, s), r1 = seq_begin(b, s + 1);
  griddep_wait();
  griddep_launch();
  double p = 0.0;
  int c = 0, n = 0;
  if (r0 < r1) {
    const int first = r0 / chunk, last = (r1 - 1) / chunk;
    for (int i0 = first + slot; i0 <= last; i0 += kFinSlots * kFinLoads) {
      float vp[kFinLoads];
      int vc[kFinLoads], vn[kFinLoads];
#pragma unroll
      for (int u = 0; u < kFinLoads; ++u) {
        const int i = i0 + u * kFinSlots;
        const size_t piece = (size_t)i + s;
        vp[u] = i <= last && e < b.E ? in.probs[piece * b.E + e] : 0.0f;
        vc[u] = i <= last && e < b.E ? in.counts[piece * b.E + e] : 0;
        vn[u] = i <= last ? in.tokens[piece] : 0;            // the same in the group's lanes
      }
#pragma unroll
      for (int u = 0; u < kFinLoads; ++u) {
        p += (double)vp[u];
        c += vc[u];
        n += vn[u];
      }
    }
  }
#pragma unroll
  for (int o = kFinE; o < 32; o <<= 1) {
    p += __shfl_xor_sync(0xffffffffu, p, o);
    c += __shfl_xor_sync(0xffffffffu, c, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (lane < kFinE) {
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    if (lane == 0) s_n[warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    p = 0.0;
    c = n = 0;
#pragma unroll
    for (int w = 0; w < kFinWarps; ++w) {
      p += s_p[w][le];
      c += s_c[w][le];
      n += s_n[w];
    }
    const float mean = n > 0 ? (float)p / (float)n : 0.0f;
    const bool mine = lane < kFinE && e < b.E;
    if (mine) {
      res.counts[(size_t)s * b.E + e] = c;
      res.probs[(size_t)s * b.E + e] = mean;
    }
    double dot = mine && n > 0 ? (double)((float)c * share_unit(b, n) * mean) : 0.0;
#pragma unroll
    for (int o = kFinE / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
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
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  full = __reduce_add_sync(0xffffffffu, full);
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

// Blocks per SM of the backward: fp32 rows in two buffers, their shares and
// derivatives take more than the 80 registers that three leave (two against
// three at 65,531 x 128 fp32: softmax 15.6 and 16.9 us, sigmoid 16.5 and 18.7;
// bf16 at 262,144 x 128: 39.5 and 36.5).
constexpr int balance_backward_blocks(int v, int size) { return v <= 4 && size == 2 ? 3 : 2; }
template <typename T, bool VEC, int V, int UR, int SCORE>
__global__ void __launch_bounds__(kBalThreads, balance_backward_blocks(V, T::size))
    balance_backward_kernel(const void* __restrict__ logits, const BalanceShape b, int rows_per_warp, float coeff,
                            const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
                            const float* __restrict__ grad_loss, void* __restrict__ dlogits, long long grad_stride) {
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
  float scale = 0.0f;
  uint64_t f[V * 2];
#pragma unroll
  for (int i = 0; i < V * 2; ++i) f[i] = 0;
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
      for (int i = 0; i < V * 2; ++i) f[i] = pack_f32x2((float)c[2 * i] * unit, (float)c[2 * i + 1] * unit);
    }
  };
  // the next rows load while these are worked on
  RowWords<T, V> w[2][UR];
  bool live[2][UR];
  auto load = [&](auto buf, int base) {
    constexpr int B = decltype(buf)::value;
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const int t = base + u * G + g, at = min(t, r1 - 1);
      const uint8_t m = b.mask ? __ldg(b.mask + at) : 1;
      load_row<T, VEC, V>(static_cast<const uint8_t*>(logits) + (size_t)at * (size_t)b.stride * T::size, l, L, b.E,
                          w[B][u]);
      live[B][u] = t < r1 && m;
    }
  };
  auto work = [&](auto buf, int base) {
    constexpr int B = decltype(buf)::value;
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const int t = base + u * G + g;
      if (live[B][u] && !(t >= s0 && t < s1)) enter(t);
      const bool in_seq = live[B][u] && t >= s0 && t < s1;
      __syncwarp();
      uint64_t v[V * 2], d[V * 2];
      row_values<T, V>(w[B][u], l, L, b.E, v);
      row_scores<V * 2, SCORE, true>(v, d, L);
      uint64_t z2 = v[0], dot2 = mul_f32x2(f[0], v[0]);
#pragma unroll
      for (int i = 1; i < V * 2; ++i) {
        z2 = add_f32x2(z2, v[i]);
        dot2 = fma_f32x2(f[i], v[i], dot2);
      }
      const float inv = share_factor(group_sum(lo_f32(z2) + hi_f32(z2), L));
      const uint64_t dot = twice(-inv * group_sum(lo_f32(dot2) + hi_f32(dot2), L)), by = twice(scale * inv);
      if (t < r1) {
        uint8_t* out = static_cast<uint8_t*>(dlogits) + (size_t)t * (size_t)grad_stride * T::size;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = (i * L + l) * 4;
          if (e >= b.E) continue;
          uint64_t o[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            o[j] = mul_f32x2(mul_f32x2(by, v[2 * i + j]), add_f32x2(f[2 * i + j], dot));
            if (SCORE != MOE_BALANCE_SOFTMAX) o[j] = mul_f32x2(o[j], d[2 * i + j]);
            o[j] = in_seq ? o[j] : 0;
          }
          if constexpr (VEC) {
            if constexpr (T::size == 4)
              *reinterpret_cast<ulonglong2*>(out + e * 4) = make_ulonglong2(o[0], o[1]);
            else
              *reinterpret_cast<uint2*>(out + e * 2) =
                  make_uint2(T::pack(lo_f32(o[0]), hi_f32(o[0])), T::pack(lo_f32(o[1]), hi_f32(o[1])));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (e + j < b.E) {
                const float x = j & 1 ? hi_f32(o[j >> 1]) : lo_f32(o[j >> 1]);
                if constexpr (T::size == 4) reinterpret_cast<float*>(out)[e + j] = x;
                else reinterpret_cast<uint16_t*>(out)[e + j] = T::one(x);
              }
          }
        }
      }
    }
  };
  using B0 = std::integral_constant<int, 0>;
  using B1 = std::integral_constant<int, 1>;
  const int step = G * UR;
  int base = (int)w0;
  if constexpr (T::size == 2 || V <= 4) {
    load(B0{}, base);
#pragma unroll 1
    for (; base < r1; base += 2 * step) {
      if (base + step < r1) load(B1{}, base + step);
      work(B0{}, base);
      if (base + step >= r1) break;
      if (base + 2 * step < r1) load(B0{}, base + 2 * step);
      work(B1{}, base + step);
    }
  } else {
#pragma unroll 1
    for (; base < r1; base += step) {
      load(B0{}, base);
      work(B0{}, base);
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
// Measured, one block against two kernels (us): 16 x 80 3.5 and 7.8, 64 x 80
// 4.3 and 7.9, 128 x 128 6.2 and 8.5, 192 x 128 7.7 and 8.4, 256 x 128 9.1 and
// 8.4, 512 x 128 14.7 and 8.1: the limit of 16,384 logits lies below the
// crossing, which was not sought closer than between 24,576 and 32,768.  The
// block walks its sequences one after the other, 2.3
// us each (128 x 128 in 20: 50 and 27, in 60: 144 and 47), hence at most two.
static inline bool balance_one_block(int T, int E, int S) { return (long long)T * E <= kBalOneBlock && S <= 2; }

// Experts per block of the finish: few where that leaves few blocks, as all of
// them meet at one counter.
static inline int balance_finish_experts(int E, int S) { return (long long)S * ((E + 7) / 8) <= 128 ? 8 : 32; }

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
  w.dots = c.take<double>((size_t)S * ((E + balance_finish_experts(E, S) - 1) / balance_finish_experts(E, S)));
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
// Each number of quads has its kernel: with four in place of one, two and three
// (whose further logits are -inf) 65,536 tokens, fp32 softmax and bf16 sigmoid,
// took, us forward and backward, own kernel against four quads:
//   4 experts (1)    8.5, 2.5 and 10.9, 2.8     8.4, 2.6 and 11.5, 3.9
//   8 experts (2)    8.8, 3.0 and 10.7, 3.2     8.6, 2.9 and 11.1, 4.1
//   40 experts (3)   12.6, 6.7 and 13.8, 7.4    12.9, 7.3 and 13.9, 8.7
//   80 experts (3)   15.4, 10.3 and 16.6, 11.0  15.1, 11.2 and 17.4, 13.4
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
// Rows that a group of lanes takes at once (as many again are being loaded).
constexpr int balance_rows(int v) { return v <= 1 ? 2 : 1; }
// Whether rows may be read or written four elements at a time.
static inline bool balance_vec(const void* p, long long stride, int T, int E, int elem) {
  return E % 4 == 0 && row_access_bytes(p, T > 1 ? stride * elem : 0, elem) >= 4 * elem;
}

// Whether the gradient may share elements with the logits, whose rows are
// loaded ahead of the stores.  Matrices whose memory meets are apart when they
// are different columns of one buffer: equal strides, and the one's row between
// the other's row and the next.
static bool shares_elements(const void* logits, long long stride, const void* dlogits, long long grad_stride, int T,
                            int E, int elem) {
  if (!overlap(logits, T, stride, E, elem, dlogits, T, grad_stride, E, elem)) return false;
  if (T <= 1 || stride != grad_stride) return true;
  const long long pitch = stride * elem, width = (long long)E * elem;
  const long long by = (long long)(reinterpret_cast<intptr_t>(dlogits) - reinterpret_cast<intptr_t>(logits));
  const long long column = (by % pitch + pitch) % pitch;
  return column < width || column + width > pitch;
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
  const int fe = balance_finish_experts(E, S);
  return launch_dependent("balance_finish_kernel", fe == 8 ? balance_finish_kernel<8> : balance_finish_kernel<32>,
                          dim3((unsigned)S, (unsigned)((E + fe - 1) / fe)), dim3(kFinThreads), 0, s, b, chunk, w.pieces,
                          w.dots, res);
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
  NV_REQUIRE(T <= 1 || grad_stride >= E, NVFP4_ERR_INVALID_ARG,
             "moe_balance_loss_backward: gradient stride %lld is below E=%d", grad_stride, E);
  const int elem = mx_elem_size(dtype);
  NV_REQUIRE(!shares_elements(logits, row_stride, dlogits, grad_stride, T, E, elem), NVFP4_ERR_INVALID_ARG,
             "moe_balance_loss_backward: dlogits may not take the place of logits, whole or in part");
  NV_REQUIRE(aligned(dlogits, elem) && aligned(counts, 4) && aligned(tokens, 4) &&
                 aligned(grad_loss, 4),
             NVFP4_ERR_INVALID_ARG, "moe_balance_loss_backward: a tensor is not aligned to its elements");
  int sms = 0;
  NV_CHECK(device_sm_count(&sms));
  const BalanceShape b{T, E, S, k, balance_lanes(E), row_stride, seq_offsets, token_mask};
  const bool vec = balance_vec(logits, row_stride, T, E, elem) && balance_vec(dlogits, grad_stride, T, E, elem);
  return with_balance(dtype, vec, E, score, [&](auto tag, auto vv, auto v, auto sc) -> nvfp4_status {
    using TT = decltype(tag);
    constexpr int V = decltype(v)::value;
    // what fits an SM at once; a warp takes neighbouring rows, so that it
    // seldom changes sequence
    const int per_iter = 32 / b.lanes;
    const long long warps = (long long)sms * balance_backward_blocks(V, TT::size) * kBalWarps;
    const int rows_per_warp = (int)(((T + warps - 1) / warps + per_iter - 1) / per_iter) * per_iter;
    const long long rows_per_block = (long long)rows_per_warp * kBalWarps;
    const dim3 grid((unsigned)((T + rows_per_block - 1) / rows_per_block));
    return launch_dependent(
        "balance_backward_kernel",
        balance_backward_kernel<TT, decltype(vv)::value, V, balance_rows(V), decltype(sc)::value>, grid,
        dim3(kBalThreads), 0, as_stream(stream), logits, b, rows_per_warp, coeff, counts, tokens, grad_loss, dlogits,
        grad_stride);
  });
}
