// Balance loss of the router and its gradient. Per token t of a sequence of n
// tokens, with s_e the score of expert e (sigmoid of the logit, as the router's,
// or exp for softmax), the share is p_e = s_e / sum_j s_j, and per sequence
//   counts[e] = (token, slot) pairs that chose e       f_e = counts[e] E / (K n)
//   prob[e] = mean_t p_e                               loss = coef sum_e f_e prob[e]
//   d loss / d logit_e = coef / n (f_e - sum_j f_j p_j) p_e (1 - sigma(logit_e))
// (softmax: without the last factor; the counts have no gradient).
//
// L = 2 (up to 8 experts), 4, 8, 16 (past 128) or 32 lanes (past 256) take a token: a
// warp up to sixteen at a time, with fewer steps of shuffles for a token's sum, and
// no idle lanes where E is small (450209 x 8: 61 -> 23 us). A lane's sums over the
// tokens are of fixed experts and stay in registers. Few logits take one launch, a
// cluster of blocks per sequence. Else a block takes a strip of tokens, and for each
// sequence in it writes one row of partial sums (row strip + sequence: unique, since
// both only grow), and a second launch adds a sequence's rows in a fixed order, eight
// blocks of a cluster sharing the experts. The logits are read once. Many tokens are
// bound by waits (65536 x 256 in 29 sequences: 22 us, of them 4 the second launch;
// bytes 10.2): the first launch issues in 43% of its cycles, DRAM is at 41%, and of a
// warp's time between two instructions a third is for loaded logits, an eighth each
// for shuffles and exponentials and for barriers, a seventh the instructions' own
// latency. Few tokens are bound by the launch (64 x 192: 4.3 us).
// The gradient reads and writes each logit once: 65536 x 256 with an addend 34 us at
// 5.9 TB/s, 8192 x 192 5.6.
//
// Scores that are all small (every logit far below 0) keep their ratios: where a
// token's sum is below 2^-25 the shares are taken relative to the largest. A token
// whose scores are all 0 (every logit -infinity) adds nothing and gets a zero gradient.
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kSumWarps = 16, kSumThreads = 32 * kSumWarps;
constexpr int kGradWarps = 8, kGradThreads = 32 * kGradWarps;
constexpr int kFinalMost = 1024, kFinalCluster = 8;
constexpr int kIdsAhead = 8;            // ids that a thread loads at a time
constexpr int kNoId = 1 << 30;          // past the last pair

struct BalanceParams {
  int T, E, K, B, strip;
  float coef;
  const float* logits;
  const int32_t* topk_idx;
  const int32_t* seq;  // [B+1], or nullptr: one sequence of all tokens
  int32_t* counts;     // [B, E]
  float* prob;         // [B, E]
  float* loss;         // [B]
  float* part;         // [strips + B, E] sums of shares, then as many counts
  int32_t* part_n;
  int* status;
  const float* dloss;  // [B]
  const float* add;    // [T, E] or nullptr
  float* dlogits;      // [T, E]
};

__device__ __forceinline__ int seq_start(const BalanceParams& p, int b) {
  const int v = p.seq ? __ldcg(p.seq + b) : (b == 0 ? 0 : p.T);
  return v < 0 ? 0 : (v > p.T ? p.T : v);
}
// The first sequence that ends past token t (B: none), by a warp: 32 probes at a time.
__device__ int first_sequence(const BalanceParams& p, int t, int lane) {
  int lo = 0, hi = p.B;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const bool past = b >= hi || seq_start(p, b + 1) > t;
    const unsigned m = __ballot_sync(0xFFFFFFFFu, past);
    const int first = m ? __ffs(m) - 1 : 32;  // the first probe that ends past t
    const int new_hi = lo + first * step, new_lo = first ? lo + (first - 1) * step + 1 : lo;
    hi = new_hi < hi ? new_hi : hi;
    lo = new_lo < hi ? new_lo : hi;
  }
  return lo;
}

// Ends of the sequences from one on, 32 loaded at a time by a warp that walks them
// (84 x 56 in 63 sequences: 20 us of the gradient's were loads one after another).
struct Ends {
  const BalanceParams& p;
  const int lane;
  int base, v;
  __device__ __forceinline__ Ends(const BalanceParams& p_, int first, int lane_) : p(p_), lane(lane_) { take(first); }
  __device__ __forceinline__ void take(int b) {
    base = b;
    v = seq_start(p, b + lane + 1 < p.B ? b + lane + 1 : p.B);
  }
  __device__ __forceinline__ int operator()(int b) {
    if (b - base >= 32) take(b);
    return __shfl_sync(0xFFFFFFFFu, v, b - base);
  }
};

// Sum and maximum over the L lanes that hold a token.
template <int L = 32>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Loads that stay where they are written (a group of tokens ahead of their use).
__device__ __forceinline__ float load_now(const float* p) {
  float v;
  asm volatile("ld.global.cs.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 load_now(const float4* p) {
  float4 v;
  asm volatile("ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

// What a kernel's template holds: L lanes per token with V experts each; FOURS (E
// a multiple of 4): groups of four neighbours, loaded at once; FULL: E = L V.
template <int L_, int V_, bool FOURS_, bool FULL_>
struct Shape {
  static constexpr int L = L_, V = V_;
  static constexpr bool FOURS = FOURS_, FULL = FULL_;
  static constexpr int kTokens = 32 / L;  // of a warp at a time
  static __device__ __forceinline__ int expert(int j, int sub) { return FOURS ? 4 * (sub + L * (j >> 2)) + (j & 3) : sub + L * j; }
  static __device__ __forceinline__ bool is(int j, int sub, int E) { return FULL || expert(j, sub) < E; }
  static __device__ __forceinline__ void load(float (&x)[V], const float* row, int E, int sub, float fill) {
    if constexpr (FOURS) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float4 v = is(j, sub, E) ? load_now(reinterpret_cast<const float4*>(row + expert(j, sub))) : make_float4(fill, fill, fill, fill);
        x[j] = v.x;
        x[j + 1] = v.y;
        x[j + 2] = v.z;
        x[j + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = is(j, sub, E) ? load_now(row + expert(j, sub)) : fill;
    }
  }
};

// exp(x) to 2 + 1.2 |x| ulp (the product with log2 e is rounded) and 1 / x to 2,
// results below 2^-126 as 0: two instructions and one, where the forms that keep
// subnormals take five.
__device__ __forceinline__ float exp_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A token's scores from its logits (in place; `row`: where they came from), and 1
// over their sum: the shares are their products. With SLOPE also d log(score) / d logit.
template <class S, bool SOFTMAX, bool SLOPE>
__device__ __forceinline__ float scores(float (&x)[S::V], float (&slope)[SLOPE ? S::V : 1], const float* row, int E, int sub) {
  constexpr int V = S::V;
  // exp(x - the largest): scores that underflow keep their ratios.
  auto relative = [&] {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, x[j]);
    top = lanes_max<S::L>(top);
    if (top == -INFINITY) top = 0.0f;  // all scores 0
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = S::is(j, sub, E) ? exp_fast(x[j] - top) : 0.0f;
      sum += x[j];
    }
    return lanes_sum<S::L>(sum);
  };
  float sum = 0.0f;
  if (SOFTMAX) {
    sum = relative();
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float a = exp_fast(-fabsf(x[j])), d = rcp_fast(1.0f + a), ad = a * d;
      const bool up = x[j] >= 0.0f;
      if (SLOPE) slope[SLOPE ? j : 0] = up ? ad : d;
      x[j] = S::is(j, sub, E) ? (up ? d : ad) : 0.0f;
      sum += x[j];
    }
    sum = lanes_sum<S::L>(sum);
    // Below 2^-25 sigma(x) is exp(x) to half an ulp, and scores far below the largest
    // would be flushed to 0 although their shares are not: from the logits once more.
    const bool tiny = sum < 2.98023224e-8f;
    if (__any_sync(0xFFFFFFFFu, tiny)) {
      float sg[V];
#pragma unroll
      for (int j = 0; j < V; ++j) sg[j] = x[j];
      S::load(x, row, E, sub, -INFINITY);
      const float sum2 = relative();
      if (tiny) {
        sum = sum2;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = sg[j];
      }
    }
  }
  return sum == 0.0f ? 0.0f : 1.0f / sum;  // a NaN stays
}

// A block's part of a sequence, tokens lo .. hi - 1: their counts are added to hist
// [E], and the sums of their shares written to sums [warps][E].
template <class S, bool SOFTMAX>
__device__ __forceinline__ void accumulate(const BalanceParams& p, int lo, int hi, float* sums, int32_t* hist) {
  constexpr int V = S::V, L = S::L;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, E = p.E;
  // U groups of tokens at a time, the next ones' logits on their way meanwhile: 64 KB
  // per SM in flight (32 KB: 13 of the 22 us of 65536 x 256 were waits).
  constexpr int U = V <= 4 ? 8 : (V <= 8 ? 4 : (V <= 16 ? 2 : 1)), kStep = kSumWarps * S::kTokens;
  float next[U][V];
  auto load = [&](int t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u * kStep >= hi) break;
      const int at = t + u * kStep + lane / L;
      S::load(next[u], p.logits + (size_t)(at < hi ? at : lo) * E, E, sub, -INFINITY);
    }
  };
  load(lo + warp * S::kTokens);
  // The counts. Up to 16 experts one ballot each, as their words would be added to
  // by many lanes at once.
  const int32_t* ids = p.topk_idx + (size_t)lo * p.K;
  const long long pairs = (long long)(hi - lo) * p.K;
  int mine = 0;
  for (long long i0 = threadIdx.x; i0 - lane < pairs; i0 += kIdsAhead * kSumThreads) {
    int id[kIdsAhead];
#pragma unroll
    for (int k = 0; k < kIdsAhead; ++k) {
      const long long i = i0 + k * kSumThreads;
      id[k] = i < pairs ? __ldcs(ids + i) : kNoId;
    }
#pragma unroll
    for (int k = 0; k < kIdsAhead; ++k) {
      if (i0 + k * kSumThreads < pairs && (id[k] < 0 || id[k] >= E)) atomicCAS(p.status, 0, MOE_DEV_BAD_EXPERT_ID);
      if (E <= 16) {
        for (int e = 0; e < E; ++e) {
          const int n = __popc(__ballot_sync(0xFFFFFFFFu, id[k] == e));
          if (lane == e) mine += n;
        }
      } else if (id[k] >= 0 && id[k] < E) {
        atomicAdd(hist + id[k], 1);
      }
    }
  }
  if (E <= 16 && lane < E) atomicAdd(hist + lane, mine);
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
  for (int t = lo + warp * S::kTokens; t < hi; t += U * kStep) {
    float x[U][V], unused[1];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < V; ++j) x[u][j] = next[u][j];
    if (t + U * kStep < hi) load(t + U * kStep);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u * kStep >= hi) break;
      const bool live = t + u * kStep + lane / L < hi;
      float inv = scores<S, SOFTMAX, false>(x[u], unused, p.logits + (size_t)(live ? t + u * kStep + lane / L : lo) * E, E, sub);
      if (!live) inv = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = fmaf(live ? x[u][j] : 0.0f, inv, acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
    if (lane < L && S::is(j, sub, E)) sums[warp * E + S::expert(j, sub)] = acc[j];
  }
}

template <class S, bool SOFTMAX>
__global__ void __launch_bounds__(kSumThreads, 1) balance_sum_kernel(const BalanceParams p) {
  extern __shared__ float smem[];
  float* sums = smem;                                                 // [warps][E]
  int32_t* hist = reinterpret_cast<int32_t*>(smem + kSumWarps * p.E);  // [E]
  __shared__ int first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.E;
  wait_for_previous_launch();
  allow_next_launch();
  const int t0 = blockIdx.x * p.strip, t1 = t0 + p.strip < p.T ? t0 + p.strip : p.T;
  if (warp == 0) {
    const int b = p.seq ? first_sequence(p, t0, lane) : 0;
    if (lane == 0) first = b;
  }
  for (int e = threadIdx.x; e < E; e += kSumThreads) hist[e] = 0;
  __syncthreads();
  int b = first;
  Ends ends(p, b, lane);
  for (int a, z = b < p.B ? seq_start(p, b) : 0; b < p.B; ++b) {
    a = z;
    z = ends(b);
    if (a >= t1) break;
    const int lo = a > t0 ? a : t0, hi = z < t1 ? z : t1;
    if (lo >= hi) continue;
    accumulate<S, SOFTMAX>(p, lo, hi, sums, hist);
    __syncthreads();
    const size_t row = ((size_t)blockIdx.x + b) * E;
    for (int e = threadIdx.x; e < E; e += kSumThreads) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kSumWarps; ++w) s += sums[w * E + e];
      p.part[row + e] = s;
      p.part_n[row + e] = hist[e];
      hist[e] = 0;
    }
    __syncthreads();
  }
}

// The two halves of a cluster's barrier, for work in between.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A cluster per sequence, its blocks taking runs of 32 experts by turns.
__global__ void __launch_bounds__(kFinalMost) balance_final_kernel(const BalanceParams p) {
  const int kWarps = blockDim.x / 32;  // a power of two
  __shared__ float ps[kFinalMost];
  __shared__ int pn[kFinalMost];
  __shared__ float share[kFinalCluster];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E;
  const uint32_t rank = cluster_ctarank();
  const int b = (int)cluster_id_x(), nranks = (int)(gridDim.x / ncluster_x());
  wait_for_previous_launch();
  allow_next_launch();
  cluster_arrive();  // waited for before the first block's shared memory is written
  const int a = seq_start(p, b), z = seq_start(p, b + 1), n = z > a ? z - a : 0;
  const int s0 = n ? a / p.strip : 0, s1 = n ? (z - 1) / p.strip + 1 : 0;
  const float inv_n = n ? 1.0f / (float)n : 0.0f, per = (float)E * inv_n / (float)p.K;
  float loss = 0.0f;
  for (int e0 = (int)rank * 32; e0 < E; e0 += 32 * nranks) {
    const int e = e0 + lane;
    float s = 0.0f;
    int c = 0;
    if (e < E) {
#pragma unroll 5
      for (int i = s0 + warp; i < s1; i += kWarps) {
        s += __ldcg(p.part + ((size_t)i + b) * E + e);
        c += __ldcg(p.part_n + ((size_t)i + b) * E + e);
      }
    }
    // Halves are added until one warp's are left.
    for (int half = kWarps / 2; half > 0; half >>= 1) {
      ps[threadIdx.x] = s;
      pn[threadIdx.x] = c;
      __syncthreads();
      if (warp < half) {
        s += ps[threadIdx.x + 32 * half];
        c += pn[threadIdx.x + 32 * half];
      }
      __syncthreads();
    }
    if (warp == 0 && e < E) {
      const float prob = s * inv_n;
      p.counts[(size_t)b * E + e] = c;
      p.prob[(size_t)b * E + e] = prob;
      loss += (float)c * per * prob;
    }
  }
  __syncwarp();
  cluster_wait();
  if (warp == 0) {
    loss = lanes_sum(loss);
    if (lane == 0) {
      const uint32_t at = mapa_shared(smem_u32(share + rank), 0);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(loss) : "memory");
    }
  }
  __syncwarp();
  cluster_sync_all();
  if (rank == 0 && threadIdx.x == 0) {
    float l = 0.0f;
    for (int r = 0; r < nranks; ++r) l += share[r];
    p.loss[b] = p.coef * l;
  }
}

// Both in one launch, for few logits: a cluster takes a sequence, each block a run of
// its tokens, and the first block adds their sums from their shared memories.
template <class S, bool SOFTMAX>
__global__ void __launch_bounds__(kSumThreads, 1) balance_one_kernel(const BalanceParams p) {
  extern __shared__ float smem[];
  float* sums = smem;
  int32_t* hist = reinterpret_cast<int32_t*>(smem + kSumWarps * p.E);
  __shared__ float share[kSumWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.E;
  const int rank = (int)cluster_ctarank(), b = (int)cluster_id_x(), nranks = (int)(gridDim.x / ncluster_x());
  wait_for_previous_launch();
  allow_next_launch();
  const int a = seq_start(p, b), z = seq_start(p, b + 1), n = z > a ? z - a : 0;
  for (int e = threadIdx.x; e < E; e += kSumThreads) hist[e] = 0;
  __syncthreads();
  const int run = (n + nranks - 1) / nranks, lo = a + rank * run, hi = z - lo < run ? z : lo + run;
  if (lo < hi) accumulate<S, SOFTMAX>(p, lo, hi, sums, hist);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSumThreads) {
    float s = 0.0f;
    if (lo < hi) {
#pragma unroll
      for (int w = 0; w < kSumWarps; ++w) s += sums[w * E + e];
    }
    sums[e] = s;
  }
  cluster_sync_all();
  if (rank == 0) {
    const float inv_n = n ? 1.0f / (float)n : 0.0f, per = (float)E * inv_n / (float)p.K;
    float loss = 0.0f;
    for (int e = threadIdx.x; e < E; e += kSumThreads) {
      float s = 0.0f;
      int c = 0;
#pragma unroll 8
      for (int r = 0; r < nranks; ++r) {
        s += __int_as_float(ld_shared_cluster_s32(mapa_shared(smem_u32(sums + e), r)));
        c += ld_shared_cluster_s32(mapa_shared(smem_u32(hist + e), r));
      }
      const float prob = s * inv_n;
      p.counts[(size_t)b * E + e] = c;
      p.prob[(size_t)b * E + e] = prob;
      loss += (float)c * per * prob;
    }
    loss = lanes_sum(loss);
    if (lane == 0) share[warp] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
      float l = 0.0f;
      for (int w = 0; w < kSumWarps; ++w) l += share[w];
      p.loss[b] = p.coef * l;
    }
  }
  __syncwarp();
  cluster_sync_all();  // the sums are read
}

template <class S, bool SOFTMAX>
__global__ void __launch_bounds__(kGradThreads, S::V > 16 ? 1 : 2) balance_grad_kernel(const BalanceParams p) {
  constexpr int V = S::V, L = S::L;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, E = p.E;
  wait_for_previous_launch();
  allow_next_launch();
  // A run of tokens per warp, so that where sequences are short each warp walks its own.
  const int run = p.strip / kGradWarps, t0 = blockIdx.x * p.strip + warp * run, t1 = t0 + run < p.T ? t0 + run : p.T;
  if (t0 >= t1) return;
  int b = p.seq ? first_sequence(p, t0, lane) : 0;
  Ends ends(p, b, lane);
  for (int a, z = b < p.B ? seq_start(p, b) : 0; b < p.B; ++b) {
    a = z;
    z = ends(b);
    if (a >= t1) break;
    const int lo = a > t0 ? a : t0, hi = z < t1 ? z : t1;
    if (lo >= hi) continue;
    const float inv_n = 1.0f / (float)(z - a), per = (float)E * inv_n / (float)p.K;
    const float w = __ldcg(p.dloss + b) * p.coef * inv_n;
    float f[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      f[j] = S::is(j, sub, E) ? (float)__ldcg(p.counts + (size_t)b * E + S::expert(j, sub)) * per : 0.0f;
    // The next tokens' logits are on their way meanwhile (52362 x 241, sigmoid: 74 -> 25 us).
    float next[V];
    auto load = [&](int t) { S::load(next, p.logits + (size_t)(t + lane / L < hi ? t + lane / L : t) * E, E, sub, -INFINITY); };
    load(lo);
    for (int t = lo; t < hi; t += S::kTokens) {
      const bool live = t + lane / L < hi;
      const size_t at = (size_t)(live ? t + lane / L : t) * E;
      float x[V], slope[V], add[V];
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = next[j];
      if (p.add) S::load(add, p.add + at, E, sub, 0.0f);
      if (t + S::kTokens < hi) load(t + S::kTokens);
      const float inv = scores<S, SOFTMAX, true>(x, slope, p.logits + at, E, sub);
      float c = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) c = fmaf(f[j], x[j], c);
      c = lanes_sum<L>(c) * inv;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float d = w * (f[j] - c) * (x[j] * inv);
        if (!SOFTMAX) d *= slope[j];
        x[j] = p.add ? d + add[j] : d;
      }
      float* row = p.dlogits + at;
      if (!live) {
      } else if constexpr (S::FOURS) {
#pragma unroll
        for (int j = 0; j < V; j += 4)
          if (S::is(j, sub, E)) __stcs(reinterpret_cast<float4*>(row + S::expert(j, sub)), make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]));
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (S::is(j, sub, E)) __stcs(row + S::expert(j, sub), x[j]);
      }
    }
  }
}

enum Pass { kSum, kOne, kGrad };
// blocks: of the grid; kOne: of a sequence.
template <int PASS, bool SOFTMAX, class S>
cudaError_t run(const BalanceParams& p, int blocks, cudaStream_t s) {
  if constexpr (PASS == kGrad) return launch_dependent(balance_grad_kernel<S, SOFTMAX>, blocks, kGradThreads, 0, s, true, 1, p);
  const size_t smem = (size_t)(kSumWarps + 1) * p.E * 4;
  if constexpr (PASS == kOne) return launch_dependent(balance_one_kernel<S, SOFTMAX>, p.B * blocks, kSumThreads, smem, s, true, blocks, p);
  return launch_dependent(balance_sum_kernel<S, SOFTMAX>, blocks, kSumThreads, smem, s, true, 1, p);
}
template <int PASS, bool SOFTMAX, int L, int V>
cudaError_t fit(const BalanceParams& p, int blocks, cudaStream_t s) {
  if (p.E == L * V && V % 4 == 0) return run<PASS, SOFTMAX, Shape<L, V, V % 4 == 0, V % 4 == 0>>(p, blocks, s);
  if (p.E % 4 == 0 && V % 4 == 0) return run<PASS, SOFTMAX, Shape<L, V, V % 4 == 0, false>>(p, blocks, s);
  return run<PASS, SOFTMAX, Shape<L, V, false, false>>(p, blocks, s);
}
// Values per lane: the least of these that hold E, so that few loads and exponentials are of no expert.
template <int PASS, bool SOFTMAX>
cudaError_t pick(const BalanceParams& p, int blocks, cudaStream_t s) {
  if (p.E <= 8) return fit<PASS, SOFTMAX, 2, 4>(p, blocks, s);
  if (p.E <= 16) return fit<PASS, SOFTMAX, 4, 4>(p, blocks, s);
  if (p.E <= 32) return fit<PASS, SOFTMAX, 8, 4>(p, blocks, s);
  if (p.E <= 64) return fit<PASS, SOFTMAX, 8, 8>(p, blocks, s);
  if (p.E <= 128) return fit<PASS, SOFTMAX, 8, 16>(p, blocks, s);
  if (p.E <= 192) return fit<PASS, SOFTMAX, 16, 12>(p, blocks, s);
  if (p.E <= 256) return fit<PASS, SOFTMAX, 16, 16>(p, blocks, s);
  if (p.E <= 512) return fit<PASS, SOFTMAX, 32, 16>(p, blocks, s);
  return fit<PASS, SOFTMAX, 32, 32>(p, blocks, s);
}
template <int PASS>
cudaError_t pick(const BalanceParams& p, bool softmax, int blocks, cudaStream_t s) {
  return softmax ? pick<PASS, true>(p, blocks, s) : pick<PASS, false>(p, blocks, s);
}

BalanceParams params_of(const BalanceArgs& a, int strip) {
  BalanceParams p = {};
  p.T = a.T;
  p.E = a.E;
  p.K = a.K;
  p.B = a.B;
  p.strip = strip;
  p.coef = a.coef;
  p.logits = a.logits;
  p.topk_idx = a.topk_idx;
  p.seq = a.seq;
  p.counts = a.counts;
  p.prob = a.prob;
  p.loss = a.loss;
  p.status = a.status;
  p.dloss = a.dloss;
  p.add = a.add;
  p.dlogits = a.dlogits;
  return p;
}

// Tokens per block of the sums: one per warp at least, and at most
// 152 blocks, one per SM, so that the second launch has few rows to add.
int sum_strip(int T) {
  const int n = (T + 151) / 152;
  return n > kSumWarps ? n : kSumWarps;
}
int sum_strips(int T) { return (T + sum_strip(T) - 1) / sum_strip(T); }

}  // namespace

cudaError_t balance_prepare_device() {
  // Past 512 experts the sums take more shared memory than a launch may without asking.
  const int most = (kSumWarps + 1) * 1024 * 4;
  auto allow = [&](auto kernel) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most); };
  using A = Shape<32, 32, true, true>;
  using B = Shape<32, 32, true, false>;
  using C = Shape<32, 32, false, false>;
  const cudaError_t errs[] = {
      allow(balance_sum_kernel<A, false>), allow(balance_sum_kernel<A, true>), allow(balance_sum_kernel<B, false>),
      allow(balance_sum_kernel<B, true>),  allow(balance_sum_kernel<C, false>), allow(balance_sum_kernel<C, true>),
      allow(balance_one_kernel<A, false>), allow(balance_one_kernel<A, true>), allow(balance_one_kernel<B, false>),
      allow(balance_one_kernel<B, true>),  allow(balance_one_kernel<C, false>), allow(balance_one_kernel<C, true>)};
  for (cudaError_t e : errs)
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

size_t balance_scratch_bytes(int T, int E, int B) { return ((size_t)sum_strips(T) + B) * E * 8; }

cudaError_t launch_balance_loss(const BalanceArgs& a, cudaStream_t s) {
  BalanceParams p = params_of(a, sum_strip(a.T));
  const int strips = sum_strips(a.T);
  p.part = static_cast<float*>(a.scratch);
  p.part_n = reinterpret_cast<int32_t*>(p.part + ((size_t)strips + a.B) * a.E);
  // One launch where a cluster of up to eight blocks is enough even if one sequence has
  // all tokens (its length is known on the device alone). In a graph, two launches and
  // one, us: 512 x 192 5.6, 4.8; 1024 x 256 6.4, 6.3; 8192 x 192 8.0, 19.0. With many
  // sequences a strip's blocks take them one by one, and more is worth it: 84 x 56 in 63
  // 20.3, 5.0; 8192 x 64 in 17 with nearly all tokens in the first 26.9, 10.6. The bound
  // is for such batches: past it even sequences would be better off in one launch too
  // (8192 x 64 in 64 9.2, 5.3; 2000 x 64 in 200 10.0, 5.8; 20000 x 64 in 1000 19.1, 18.4).
  int cluster = 8;
  while (cluster > 1 && a.B * cluster > 152) cluster /= 2;
  if ((long long)a.T * a.E <= (a.B == 1 ? 1 << 14 : 1 << 16) * (long long)cluster) return pick<kOne>(p, a.softmax, cluster, s);
  if (strips > 0) {
    const cudaError_t e = pick<kSum>(p, a.softmax, strips, s);
    if (e != cudaSuccess) return e;
  }
  // A warp for about five of a sequence's rows (152 for one sequence), a block for 32 experts.
  int warps = 4, blocks = 1;
  while (warps < kFinalMost / 32 && warps * 5 < strips / a.B) warps *= 2;
  while (blocks < kFinalCluster && blocks * 32 < a.E) blocks *= 2;
  return launch_dependent(balance_final_kernel, a.B * blocks, 32 * warps, 0, s, true, blocks, p);
}

cudaError_t launch_balance_loss_backward(const BalanceArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  // Eight tokens per warp at least, so that a lane's f is loaded for several and a
  // small batch takes one wave of blocks (8192 x 192: 6.5 us; four 7.9, two 10.5),
  // more once four blocks of each SM are at work.
  // A warp takes 16 tokens at a time of up to 8 experts, fewer of more.
  const int least = a.E <= 8 ? 16 : 8, per_warp = (a.T + 608 * kGradWarps - 1) / (608 * kGradWarps);
  const int strip = kGradWarps * (per_warp > least ? (per_warp + least - 1) / least * least : least);
  const int strips = (a.T + strip - 1) / strip;
  const BalanceParams p = params_of(a, strip);
  return pick<kGrad>(p, a.softmax, strips, s);
}

}  // namespace moe
