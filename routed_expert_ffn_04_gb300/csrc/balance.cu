// Balance loss of the router and its gradient. Per token t of a sequence of n
// tokens, with s_e the score of expert e (sigmoid of the logit, as the router's,
// or exp for softmax), the share is p_e = s_e / sum_j s_j, and per sequence
//   counts[e] = (token, slot) pairs that chose e       f_e = counts[e] E / (K n)
//   prob[e] = mean_t p_e                               loss = coef sum_e f_e prob[e]
//   d loss / d logit_e = coef / n (f_e - sum_j f_j p_j) p_e (1 - sigma(logit_e))
// (softmax: without the last factor; the counts have no gradient).
//
// A warp takes a token: its lanes hold the experts lane, lane + 32, ... (or pairs
// of neighbours), so a lane's sums over the tokens are of fixed experts and stay in registers. A
// block takes a strip of tokens, and for each sequence in it writes one row of
// partial sums (row strip + sequence: unique, since both only grow). A second
// launch adds a sequence's rows in a fixed order, eight blocks of a cluster
// sharing the experts. The logits are read once; what bounds it is HBM for many
// tokens and the two launches for few.
//
// Scores that all underflow (every logit far below 0) keep their ratios: the
// shares are then taken relative to the largest. A token whose scores are all 0
// (every logit -infinity) adds nothing and gets a zero gradient.
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kSumWarps = 16, kSumThreads = 32 * kSumWarps;
constexpr int kGradWarps = 8, kGradThreads = 32 * kGradWarps;
constexpr int kFinalThreads = 256, kFinalCluster = 8;

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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Expert of a lane's value j. FULL (E = 32 V): pairs of neighbours, loaded at
// once, and no lane's value is of no expert.
template <bool FULL>
__device__ __forceinline__ int expert_of(int j, int lane) {
  return FULL ? 64 * (j >> 1) + 2 * lane + (j & 1) : lane + 32 * j;
}

// exp(x) and 1 / x to 2 ulp, tiny results as 0: two instructions each, where the
// forms that keep subnormals take five (with them and the checks of lanes past E
// a token of 256 experts took 238 instructions).
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

// A token's scores from its logits (in place), and 1 over their sum: the shares
// are their products. With SLOPE also d log(score) / d logit.
template <int V, bool SOFTMAX, bool SLOPE, bool FULL>
__device__ __forceinline__ float scores(float (&x)[V], float (&slope)[V], int E, int lane) {
  auto is = [&](int j) { return FULL || expert_of<FULL>(j, lane) < E; };
  // exp(x - the largest): scores that underflow keep their ratios.
  auto relative = [&] {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, x[j]);
    top = warp_max(top);
    if (top == -INFINITY) top = 0.0f;  // all scores 0
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = is(j) ? exp_fast(x[j] - top) : 0.0f;
      sum += x[j];
    }
    return warp_sum(sum);
  };
  float sum = 0.0f;
  if (SOFTMAX) {
    sum = relative();
  } else {
    float sg[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float a = exp_fast(-fabsf(x[j])), d = rcp_fast(1.0f + a), ad = a * d;
      const bool up = x[j] >= 0.0f;
      if (SLOPE) slope[j] = up ? ad : d;
      sg[j] = is(j) ? (up ? d : ad) : 0.0f;
      sum += sg[j];
    }
    sum = warp_sum(sum);
    if (sum < 1e-30f) {  // sigma(x) = exp(x) here
      sum = relative();
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = sg[j];
    }
  }
  return sum == 0.0f ? 0.0f : 1.0f / sum;  // a NaN stays
}

template <int V, bool FULL>
__device__ __forceinline__ void load_row(float (&x)[V], const float* row, int E, int lane, float fill) {
  if (FULL) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 v = __ldcs(reinterpret_cast<const float2*>(row + expert_of<true>(j, lane)));
      x[j] = v.x;
      x[j + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = lane + 32 * j < E ? __ldcs(row + lane + 32 * j) : fill;
  }
}

// Tokens that a warp takes at a time.
template <int V>
constexpr int kAtOnce = V <= 8 ? 2 : 1;

template <int V, bool SOFTMAX, bool FULL>
__global__ void __launch_bounds__(kSumThreads) balance_sum_kernel(const BalanceParams p) {
  extern __shared__ float smem[];
  float* sums = smem;                                                 // [warps][E]
  int32_t* hist = reinterpret_cast<int32_t*>(smem + kSumWarps * p.E);  // [E]
  __shared__ int first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.E;
  wait_for_previous_launch();
  allow_next_launch();
  const int t0 = blockIdx.x * p.strip, t1 = t0 + p.strip < p.T ? t0 + p.strip : p.T;
  if (warp == 0) {
    const int b = first_sequence(p, t0, lane);
    if (lane == 0) first = b;
  }
  for (int e = threadIdx.x; e < E; e += kSumThreads) hist[e] = 0;
  __syncthreads();
  for (int b = first; b < p.B; ++b) {
    const int a = seq_start(p, b), z = seq_start(p, b + 1);
    if (a >= t1) break;
    const int lo = a > t0 ? a : t0, hi = z < t1 ? z : t1;
    if (lo >= hi) continue;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    for (int t = lo + warp; t < hi; t += kAtOnce<V> * kSumWarps) {
      float x[kAtOnce<V>][V], unused[V];
      int id[kAtOnce<V>];
#pragma unroll
      for (int k = 0; k < kAtOnce<V>; ++k) {
        const int at = t + k * kSumWarps < hi ? t + k * kSumWarps : t;
        load_row<V, FULL>(x[k], p.logits + (size_t)at * E, E, lane, -INFINITY);
        id[k] = lane < p.K ? __ldcs(p.topk_idx + (size_t)at * p.K + lane) : 0;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce<V>; ++k) {
        if (t + k * kSumWarps >= hi) break;
        if (lane < p.K) {
          if (id[k] >= 0 && id[k] < E) atomicAdd(hist + id[k], 1);
          else atomicCAS(p.status, 0, MOE_DEV_BAD_EXPERT_ID);
        }
        const float inv = scores<V, SOFTMAX, false, FULL>(x[k], unused, E, lane);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(x[k][j], inv, acc[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert_of<FULL>(j, lane);
      if (e < E) sums[warp * E + e] = acc[j];
    }
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

// A cluster per sequence, each block every eighth run of 32 experts.
__global__ void __launch_bounds__(kFinalThreads) balance_final_kernel(const BalanceParams p) {
  __shared__ float ps[kFinalThreads];
  __shared__ int pn[kFinalThreads];
  __shared__ float share[kFinalCluster];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E;
  const uint32_t rank = cluster_ctarank();
  const int b = (int)cluster_id_x();
  wait_for_previous_launch();
  allow_next_launch();
  const int a = seq_start(p, b), z = seq_start(p, b + 1), n = z > a ? z - a : 0;
  const int s0 = n ? a / p.strip : 0, s1 = n ? (z - 1) / p.strip + 1 : 0;
  const float inv_n = n ? 1.0f / (float)n : 0.0f, per = (float)E * inv_n / (float)p.K;
  float loss = 0.0f;
  for (int e0 = (int)rank * 32; e0 < E; e0 += 32 * kFinalCluster) {
    const int e = e0 + lane;
    float s = 0.0f;
    int c = 0;
    if (e < E) {
#pragma unroll 4
      for (int i = s0 + warp; i < s1; i += kFinalThreads / 32) {
        s += __ldcg(p.part + ((size_t)i + b) * E + e);
        c += __ldcg(p.part_n + ((size_t)i + b) * E + e);
      }
    }
    ps[threadIdx.x] = s;
    pn[threadIdx.x] = c;
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kFinalThreads / 32; ++w) {
        s += ps[w * 32 + lane];
        c += pn[w * 32 + lane];
      }
      if (e < E) {
        const float prob = s * inv_n;
        p.counts[(size_t)b * E + e] = c;
        p.prob[(size_t)b * E + e] = prob;
        loss += (float)c * per * prob;
      }
    }
    __syncthreads();
  }
  if (warp == 0) {
    loss = warp_sum(loss);
    if (lane == 0) {
      const uint32_t at = mapa_shared(smem_u32(share + rank), 0);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(loss) : "memory");
    }
  }
  __syncwarp();
  cluster_sync_all();
  if (rank == 0 && threadIdx.x == 0) {
    float l = 0.0f;
    for (int r = 0; r < kFinalCluster; ++r) l += share[r];
    p.loss[b] = p.coef * l;
  }
}

template <int V, bool SOFTMAX, bool FULL>
__global__ void __launch_bounds__(kGradThreads) balance_grad_kernel(const BalanceParams p) {
  __shared__ int first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.E;
  wait_for_previous_launch();
  allow_next_launch();
  const int t0 = blockIdx.x * p.strip, t1 = t0 + p.strip < p.T ? t0 + p.strip : p.T;
  if (warp == 0) {
    const int b = first_sequence(p, t0, lane);
    if (lane == 0) first = b;
  }
  __syncthreads();
  for (int b = first; b < p.B; ++b) {
    const int a = seq_start(p, b), z = seq_start(p, b + 1);
    if (a >= t1) break;
    const int lo = a > t0 ? a : t0, hi = z < t1 ? z : t1;
    if (lo + warp >= hi) continue;
    const float inv_n = 1.0f / (float)(z - a), per = (float)E * inv_n / (float)p.K;
    const float w = __ldcg(p.dloss + b) * p.coef * inv_n;
    float f[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = expert_of<FULL>(j, lane);
      f[j] = e < E ? (float)__ldcg(p.counts + (size_t)b * E + e) * per : 0.0f;
    }
    for (int t0 = lo + warp; t0 < hi; t0 += kAtOnce<V> * kGradWarps) {
      float x[kAtOnce<V>][V], add[kAtOnce<V>][V], slope[V];
#pragma unroll
      for (int k = 0; k < kAtOnce<V>; ++k) {
        const int at = t0 + k * kGradWarps < hi ? t0 + k * kGradWarps : t0;
        load_row<V, FULL>(x[k], p.logits + (size_t)at * E, E, lane, -INFINITY);
        if (p.add) load_row<V, FULL>(add[k], p.add + (size_t)at * E, E, lane, 0.0f);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce<V>; ++k) {
        const int t = t0 + k * kGradWarps;
        if (t >= hi) break;
        const float inv = scores<V, SOFTMAX, true, FULL>(x[k], slope, E, lane);
        float c = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) c = fmaf(f[j], x[k][j], c);
        c = warp_sum(c) * inv;
        float* row = p.dlogits + (size_t)t * E;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float d = w * (f[j] - c) * (x[k][j] * inv);
          if (!SOFTMAX) d *= slope[j];
          x[k][j] = p.add ? d + add[k][j] : d;
        }
        if (FULL) {
#pragma unroll
          for (int j = 0; j < V; j += 2)
            __stcs(reinterpret_cast<float2*>(row + expert_of<true>(j, lane)), make_float2(x[k][j], x[k][j + 1]));
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (lane + 32 * j < E) __stcs(row + lane + 32 * j, x[k][j]);
        }
      }
    }
  }
}

template <bool GRAD, int V, bool SOFTMAX, bool FULL>
cudaError_t run(const BalanceParams& p, int strips, cudaStream_t s) {
  if (GRAD) return launch_dependent(balance_grad_kernel<V, SOFTMAX, FULL>, strips, kGradThreads, 0, s, true, 1, p);
  const size_t smem = (size_t)(kSumWarps + 1) * p.E * 4;
  return launch_dependent(balance_sum_kernel<V, SOFTMAX, FULL>, strips, kSumThreads, smem, s, true, 1, p);
}
// Values per lane: the least that hold E, so that few lanes' loads and exponentials are of no expert.
template <bool GRAD, bool SOFTMAX, int V>
cudaError_t fit(const BalanceParams& p, int strips, cudaStream_t s) {
  return p.E == 32 * V ? run<GRAD, V, SOFTMAX, true>(p, strips, s) : run<GRAD, V, SOFTMAX, false>(p, strips, s);
}
template <bool GRAD, bool SOFTMAX>
cudaError_t pick(const BalanceParams& p, int strips, cudaStream_t s) {
  if (p.E <= 64) return fit<GRAD, SOFTMAX, 2>(p, strips, s);
  if (p.E <= 128) return fit<GRAD, SOFTMAX, 4>(p, strips, s);
  if (p.E <= 192) return fit<GRAD, SOFTMAX, 6>(p, strips, s);
  if (p.E <= 256) return fit<GRAD, SOFTMAX, 8>(p, strips, s);
  if (p.E <= 512) return fit<GRAD, SOFTMAX, 16>(p, strips, s);
  return fit<GRAD, SOFTMAX, 32>(p, strips, s);
}
template <bool GRAD>
cudaError_t pick(const BalanceParams& p, bool softmax, int strips, cudaStream_t s) {
  return softmax ? pick<GRAD, true>(p, strips, s) : pick<GRAD, false>(p, strips, s);
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

// Tokens per block of the sums: two per warp at least, and at most about 300
// blocks, so that the second launch has few rows to add.
int sum_strip(int T) {
  const int n = (T + 303) / 304;
  return n > 2 * kSumWarps ? n : 2 * kSumWarps;
}
int sum_strips(int T) { return (T + sum_strip(T) - 1) / sum_strip(T); }

}  // namespace

cudaError_t balance_prepare_device() {
  const int most = (kSumWarps + 1) * 1024 * 4;
  const cudaError_t errs[] = {
      cudaFuncSetAttribute(balance_sum_kernel<32, false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most),
      cudaFuncSetAttribute(balance_sum_kernel<32, true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most),
      cudaFuncSetAttribute(balance_sum_kernel<32, false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most),
      cudaFuncSetAttribute(balance_sum_kernel<32, true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most)};
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
  if (strips > 0) {
    const cudaError_t e = pick<false>(p, a.softmax, strips, s);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(balance_final_kernel, a.B * kFinalCluster, kFinalThreads, 0, s, true, kFinalCluster, p);
}

cudaError_t launch_balance_loss_backward(const BalanceArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  // Four tokens per warp, more (so that a lane's f is loaded for several) once two
  // blocks of each SM are at work.
  const int per_warp = (a.T + 304 * kGradWarps - 1) / (304 * kGradWarps), strip = kGradWarps * (per_warp > 4 ? per_warp : 4);
  const int strips = (a.T + strip - 1) / strip;
  const BalanceParams p = params_of(a, strip);
  return pick<true>(p, a.softmax, strips, s);
}

}  // namespace moe
