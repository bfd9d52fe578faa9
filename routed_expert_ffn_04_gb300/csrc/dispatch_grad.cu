// Gradient of the token dispatch: of the weighted combine (step 4), of the
// routing weights (step 1) and of the permutation (step 2). p(t,k) is
// flat_to_perm[t*K + k], sigma_k the sigmoid of the k-th chosen expert's logit.
//
//   combine: out[t] = sum_k w[t,k] y[p(t,k)] + shared[t]
//     dy[p(t,k)] = w[t,k] * dout[t];  dw[t,k] = <dout[t], y[p(t,k)]>;  dshared = dout
//   routing: w_k = scaling * sigma_k / S, S = sum_j sigma_j (route_norm), or scaling * sigma_k
//     dl_k = scaling * r_k (1 - sigma_k) * sum_j r_j (dw_k - dw_j),  r_k = sigma_k / S   (route_norm)
//     dl_k = scaling * sigma_k (1 - sigma_k) * dw_k                                      (else)
//     and 0 for the experts that were not chosen. The differences dw_k - dw_j
//     are taken before the sum, which keeps the digits that dw_k S - sum_j
//     sigma_j dw_j would cancel; the sigmoids are divided by S one by one, since
//     1 / S^2 passes fp32's range where they are small (logits near -88).
//   permutation: x_perm[p(t,k)] = x[t]
//     dx[t] = sum_k dx_perm[p(t,k)] + dx_add[t]
//
// Bound: HBM. The combine's gradient reads the K fp32 rows of y once and
// writes the K bf16 rows of dy; dout[t] is read once per token. Sums are fp32
// in a fixed order (no atomics); dy and dx are rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kMaxK = 32;
constexpr int kBatch = 8;  // permutation: rows a thread holds in flight

__device__ __forceinline__ void unpack8(const uint4& a, float (&f)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Slot k's expert in lane k of a warp (-1 in the others, and for an id out of
// range), with its logit.
struct SlotLogit {
  int e;
  float l;
};
__device__ __forceinline__ SlotLogit load_slot(const float* logits, const int32_t* idx,
                                               int E, int K, int* status) {
  const int lane = threadIdx.x & 31;
  SlotLogit s = {-1, 0.0f};
  if (lane < K) {
    const int e = idx[lane];
    if ((unsigned)e < (unsigned)E) s = {e, logits[e]};
    else atomicCAS(status, 0, MOE_DEV_BAD_EXPERT_ID);
  }
  return s;
}
// r_k, or sigma_k without route_norm, and 1 - sigma_k (0 where there is no expert).
struct SlotWeight {
  float r, om;
};
__device__ __forceinline__ SlotWeight slot_weight(SlotLogit s, int route_norm) {
  SlotWeight w = {0.0f, 0.0f};
  if (s.e >= 0) w = {1.0f / (1.0f + expf(-s.l)), 1.0f / (1.0f + expf(s.l))};
  if (route_norm) {
    float S = w.r;  // summed as the forward does
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) S += __shfl_xor_sync(0xFFFFFFFFu, S, off);
    w.r /= S;
  }
  return w;
}
// The chosen experts' dlogits of one token, by one warp; lane k holds slot k's
// dw. The row has been zeroed before (and that is visible to this warp).
__device__ __forceinline__ void route_grad_warp(int e, SlotWeight w, float dw, int K, float scaling, int route_norm,
                                                float* dlogits) {
  float d = dw;
  if (route_norm) {
    d = 0.0f;
    for (int j = 0; j < K; ++j) d = fmaf(__shfl_sync(0xFFFFFFFFu, w.r, j), dw - __shfl_sync(0xFFFFFFFFu, dw, j), d);
  }
  if (e >= 0) dlogits[e] = scaling * w.r * w.om * d;
}

// One warp per (token, slot): it reads the token's dout and one y row, writes
// the dy row and keeps the dot product; nothing is exchanged until the end, so
// every warp's loads stay in flight. dout[t] comes from L1 for the token's
// other warps. A block has one token's slots, or several tokens' when a token
// has few. (One block per token whose threads hold all eight rows' columns took
// 367 us at 8192 tokens x 8 slots x 4096.)
//
// Runs of 256 columns that a warp has in flight: eight where one wave of blocks
// holds everything, since a row's round trips are then the whole time, and in
// many waves of long rows; else two, which leaves room for twice the warps.
//   us for two / eight runs (8 slots, operands from HBM)
//   H       61 tokens     152            304            608            8192
//   512     4.1 / 4.2     4.5 / 4.6      5.3 / 5.4      6.3 / 8.6
//   1024    5.0 / 4.6     5.8 / 5.1      6.7 / 6.3      8.5 / 10.4     74 / 97
//   4096    9.3 / 6.9     11.0 / 8.9     14.1 / 13.4    23.2 / 23.7    251 / 248
// Around the second rule (8192 tokens but where given): H = 2048 130 / 138, 3136
// 204 / 200, 4096 of 2432 tokens 78.3 / 77.0, 6144 of 4096 tokens 188 / 185.
// 248 us are 6.79 TB/s, a copy's rate.
constexpr int kMaxWarps = 16;  // per block

template <int kUnroll>  // 256-column runs a warp has in flight
__global__ void __launch_bounds__(32 * kMaxWarps) combine_bwd_kernel(
    const __nv_bfloat16* dout, const float* y, const float* topk_w, const int32_t* f2p, int T, int K, int H, int E,
    int slot_warps, int tokens, float scaling, int route_norm, const int32_t* topk_idx, const float* logits,
    __nv_bfloat16* dy, float* dtopk_w, float* dlogits, int* status) {
  allow_next_launch();
  wait_for_previous_launch();
  __shared__ float dots[kMaxK];  // [token][slot]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sw = warp % slot_warps, tok = warp / slot_warps;
  const int t = blockIdx.x * tokens + tok;
  const int H8 = H >> 3;
  SlotLogit slot = {-1, 0.0f};
  if (t < T) {
    if (dlogits) {
      if (sw == 0) slot = load_slot(logits + (size_t)t * E, topk_idx + (size_t)t * K, E, K, status);
      for (int e = sw * 32 + lane; e < E; e += 32 * slot_warps) dlogits[(size_t)t * E + e] = 0.0f;
    }
    const uint4* drow = reinterpret_cast<const uint4*>(dout + (size_t)t * H);
    for (int k = sw; k < K; k += slot_warps) {
      const size_t f = (size_t)t * K + k;
      int32_t p = f2p[f];
      const float w = topk_w[f];
      if ((unsigned)p >= (unsigned)(T * K)) {
        // -1: a pair that the permutation dropped and has reported already.
        if (p != -1 && lane == 0) atomicCAS(status, 0, MOE_DEV_BAD_PERM_INDEX);
        p = -1;
      }
      float acc = 0.0f;
      if (p >= 0) {
        const float4* yr = reinterpret_cast<const float4*>(y + (size_t)p * H);
        uint4* dyr = reinterpret_cast<uint4*>(dy + (size_t)p * H);
        for (int c = lane; c < H8; c += 32 * kUnroll) {
          uint4 d[kUnroll];
          float4 v[kUnroll][2];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int cc = c + u * 32;
            if (cc < H8) {
              d[u] = drow[cc];
              v[u][0] = __ldcs(yr + 2 * cc);
              v[u][1] = __ldcs(yr + 2 * cc + 1);
            }
          }
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int cc = c + u * 32;
            if (cc >= H8) break;
            float g[8], o[8];
            unpack8(d[u], g);
            acc = fmaf(g[0], v[u][0].x, acc);
            acc = fmaf(g[1], v[u][0].y, acc);
            acc = fmaf(g[2], v[u][0].z, acc);
            acc = fmaf(g[3], v[u][0].w, acc);
            acc = fmaf(g[4], v[u][1].x, acc);
            acc = fmaf(g[5], v[u][1].y, acc);
            acc = fmaf(g[6], v[u][1].z, acc);
            acc = fmaf(g[7], v[u][1].w, acc);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = w * g[i];
            dyr[cc] = pack8(o);
          }
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, off);
      if (lane == 0) dots[tok * K + k] = acc;
    }
  }
  SlotWeight weight = {0.0f, 0.0f};
  if (dlogits && sw == 0) weight = slot_weight(slot, route_norm);  // while the token's other warps finish
  __syncthreads();
  if (sw != 0 || t >= T) return;  // one warp per token
  const float dw = lane < K ? dots[tok * K + lane] : 0.0f;
  if (lane < K) dtopk_w[(size_t)t * K + lane] = dw;
  if (dlogits) route_grad_warp(slot.e, weight, dw, K, scaling, route_norm, dlogits + (size_t)t * E);
}

// The routing's gradient alone: one warp per token (8192 tokens, 8 of 192: 4.0 us
// in a graph, 1.0 of them for its bytes).
__global__ void __launch_bounds__(256) route_bwd_kernel(const float* __restrict__ logits,
                                                        const int32_t* __restrict__ topk_idx,
                                                        const float* __restrict__ dtopk_w, int T, int E, int K,
                                                        float scaling, int route_norm, float* __restrict__ dlogits,
                                                        int* status) {
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= T) return;
  float* dl = dlogits + (size_t)t * E;
  for (int e = lane; e < E; e += 32) dl[e] = 0.0f;
  __syncwarp();
  const SlotLogit slot = load_slot(logits + (size_t)t * E, topk_idx + (size_t)t * K, E, K, status);
  route_grad_warp(slot.e, slot_weight(slot, route_norm), lane < K ? dtopk_w[(size_t)t * K + lane] : 0.0f, K, scaling,
                  route_norm, dl);
}

// dx: a work unit is one token's chunk of 8 * blockDim columns; a thread adds
// its 8 columns of the K rows (batches of 8 loads in flight), k ascending.
// 8192 tokens x 8 rows x 4096 with dx_add: 99.6 us (6.74 TB/s, a copy's rate).
__global__ void __launch_bounds__(256) permute_bwd_kernel(const __nv_bfloat16* dxp, const int32_t* f2p, int T, int K,
                                                          int H, int chunks, const __nv_bfloat16* add,
                                                          __nv_bfloat16* dx, int* status) {
  __shared__ int32_t sp[kMaxK];
  allow_next_launch();
  wait_for_previous_launch();
  const long long u = blockIdx.x;
  const int t = (int)(u / chunks);
  const int c = (int)(u - (long long)t * chunks) * blockDim.x + threadIdx.x;
  if (threadIdx.x < K) {
    int32_t p = f2p[(size_t)t * K + threadIdx.x];
    if ((unsigned)p >= (unsigned)(T * K)) {
      if (p != -1) atomicCAS(status, 0, MOE_DEV_BAD_PERM_INDEX);
      p = -1;
    }
    sp[threadIdx.x] = p;
  }
  __syncthreads();
  if (c >= (H >> 3)) return;
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.0f;
  uint4 a = make_uint4(0u, 0u, 0u, 0u);
  if (add) a = reinterpret_cast<const uint4*>(add + (size_t)t * H)[c];
  for (int k0 = 0; k0 < K; k0 += kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int p = k0 + j < K ? sp[k0 + j] : -1;
      v[j] = p >= 0 ? reinterpret_cast<const uint4*>(dxp + (size_t)p * H)[c] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      float f[8];
      unpack8(v[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += f[i];
    }
  }
  float f[8];
  unpack8(a, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] += f[i];
  reinterpret_cast<uint4*>(dx + (size_t)t * H)[c] = pack8(s);
}

}  // namespace

cudaError_t launch_combine_backward(const CombineGradArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int slot_warps = a.K < kMaxWarps ? a.K : kMaxWarps;
  const int tokens = slot_warps <= 4 ? 8 / slot_warps : 1;
  const int grid = (a.T + tokens - 1) / tokens;
  const int threads = 32 * slot_warps * tokens;
  const double waves = (double)grid * threads / (512.0 * a.num_sms);  // of the wide form: 512 threads per SM
  const bool wide = waves <= 1 ? a.H > 512 : waves >= 8 && a.H >= 4096;
  return launch_dependent(wide ? combine_bwd_kernel<8> : combine_bwd_kernel<2>, grid, threads, 0, s, true, 1,
                          static_cast<const __nv_bfloat16*>(a.dout), a.y_perm, a.topk_w, a.flat_to_perm, a.T, a.K, a.H,
                          a.E, slot_warps, tokens, a.scaling, a.route_norm, a.topk_idx, a.logits,
                          static_cast<__nv_bfloat16*>(a.dy_perm), a.dtopk_w, a.dlogits, a.status);
}

cudaError_t launch_route_backward(const float* logits, const int32_t* topk_idx, const float* dtopk_w, int T, int E,
                                  int K, float scaling, int route_norm, float* dlogits, int* status, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  route_bwd_kernel<<<(T + 7) / 8, 256, 0, s>>>(logits, topk_idx, dtopk_w, T, E, K, scaling, route_norm, dlogits, status);
  return cudaGetLastError();
}

cudaError_t launch_permute_backward(const void* dx_perm, const int32_t* flat_to_perm, int T, int K, int H,
                                    const void* dx_add, void* dx, int* status, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  int threads = (H / 8 + 31) / 32 * 32;
  threads = threads > 256 ? 256 : threads;
  const int chunks = (H / 8 + threads - 1) / threads;
  const long long grid = (long long)T * chunks;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch_dependent(permute_bwd_kernel, (int)grid, threads, 0, s, true, 1,
                          static_cast<const __nv_bfloat16*>(dx_perm), flat_to_perm, T, K, H, chunks,
                          static_cast<const __nv_bfloat16*>(dx_add), static_cast<__nv_bfloat16*>(dx), status);
}

}  // namespace moe
