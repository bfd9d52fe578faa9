// Residual add + RMS norm in front of the MoE layer, with the layer's input
// forms as outputs (bf16 rows for the router, MXFP8 codes and E8M0 scales for
// the experts), and its backward pass.
//
//   s = x + residual;  h_out = s rounded to the residual's type
//   rstd = 1 / sqrt(mean(s^2) + eps);  n = s * rstd * w
//   out = bf16(n);  (q, q_scale) = the MX blocks of n (32 along the row)
// backward, with xhat = h * rstd and g = dout * w:
//   dh = rstd * (g - xhat * mean(g * xhat)) + dh_in;  dw = sum_rows dout * xhat
//
// Sums and the norm's factors are fp32; every output is rounded once from the
// fp32 value (q from n itself, not from its bf16 rounding).
//
// Bound: HBM. One pass: a row's elements stay in the registers of the threads
// that loaded them (8 consecutive columns per vector), so each input is read
// once. Rows of at most 1024 columns take one warp each, longer rows (up to
// 16384) one block each. Every thread reads its elements of a row before it
// writes them, so the outputs may overwrite the inputs of their own type.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "mx.cuh"

namespace moe {
namespace {

constexpr int kWarpRowCols = 1024;  // rows up to this many columns: one warp each
constexpr int kWarpRows = 8;        // such rows per block

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// Sum over the block (warp shuffles, then one exchange through `part`, which
// the caller alternates between two buffers when it calls repeatedly).
__device__ __forceinline__ float block_sum(float v, float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  v = warp_sum(v);
  if (lane == 0) part[warp] = v;
  __syncthreads();
  return warp_sum(lane < nw ? part[lane] : 0.0f);
}

// Eight consecutive elements, as raw vectors and as fp32.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// The MX block of 32 columns that four neighbouring lanes hold (8 each): their
// codes, and the block's scale code (the same in all four). The largest |v| is
// taken over the bit patterns, so a NaN or an infinity is the block's largest
// and a NaN stays one (code 0x7F).
__device__ __forceinline__ uint2 mx_block(const float (&f)[8], int& scale_code) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  uint2 q = make_uint2(0u, 0u);
  scale_code = 0;
  if (m != 0) {
    const int sexp = mx_shared_exp(__uint_as_float(m));
    scale_code = sexp + 127;
    const float inv = pow2f(-sexp);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * inv, f[2 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    q = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  }
  return q;
}

// ------------------------------------------------------------------ forward
template <typename RT, int NV, bool WARP_ROW, bool MX>
__global__ void __launch_bounds__(WARP_ROW ? 32 * kWarpRows : 512) add_rmsnorm_kernel(long long rows, int H, const __nv_bfloat16* x,
                                   const RT* residual, const __nv_bfloat16* __restrict__ w, float eps, RT* h_out, __nv_bfloat16* out,
                                   uint8_t* __restrict__ q, uint8_t* __restrict__ q_scale,
                                   float* __restrict__ rstd_out) {
  __shared__ float part[32];
  const int tid = WARP_ROW ? (threadIdx.x & 31) : threadIdx.x;
  const int nt = WARP_ROW ? 32 : blockDim.x;
  const long long row = WARP_ROW ? (long long)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : (long long)blockIdx.x;
  if (WARP_ROW && row >= rows) return;
  const size_t at = (size_t)row * H;
  Vec8<__nv_bfloat16> vx[NV], vw[NV];
  Vec8<RT> vr[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * nt + tid) * 8;
    vx[v].zero();
    vr[v].zero();
    vw[v].zero();
    if (c < H) {
      vx[v].load(x + at + c);
      if (residual) vr[v].load(residual + at + c);
      vw[v].load(w + c);
    }
  }
  float s[NV][8], ss = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float r[8];
    vx[v].unpack(s[v]);
    vr[v].unpack(r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[v][j] += r[j];
      ss = fmaf(s[v][j], s[v][j], ss);
    }
  }
  if (h_out) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * nt + tid) * 8;
      if (c < H) Vec8<RT>::store(h_out + at + c, s[v]);
    }
  }
  ss = WARP_ROW ? warp_sum(ss) : block_sum(ss, part);
  const float rstd = 1.0f / sqrtf(ss / (float)H + eps);
  if (rstd_out && tid == 0) rstd_out[row] = rstd;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * nt + tid) * 8;
    float g[8];
    vw[v].unpack(g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = s[v][j] * rstd * g[j];
    if (out && c < H) Vec8<__nv_bfloat16>::store(out + at + c, g);
    if (MX) {  // H % 32 == 0: a block's four lanes are all inside the row or all outside
      int code;
      const uint2 words = mx_block(g, code);
      if (c < H) {
        *reinterpret_cast<uint2*>(q + at + c) = words;
        if ((tid & 3) == 0) q_scale[(at + c) >> 5] = (uint8_t)code;
      }
    }
  }
}

// Any H (rows not 16-byte aligned): one block per row, element by element,
// two passes over the row's inputs.
template <typename RT>
__global__ void add_rmsnorm_any_kernel(int H, const __nv_bfloat16* x, const RT* residual,
                                       const __nv_bfloat16* __restrict__ w, float eps, RT* h_out, __nv_bfloat16* out,
                                       float* __restrict__ rstd_out) {
  __shared__ float part[32];
  const size_t at = (size_t)blockIdx.x * H;
  float ss = 0.0f;
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    const float s = to_f32(x[at + c]) + (residual ? to_f32(residual[at + c]) : 0.0f);
    ss = fmaf(s, s, ss);
  }
  ss = block_sum(ss, part);
  const float rstd = 1.0f / sqrtf(ss / (float)H + eps);
  if (rstd_out && threadIdx.x == 0) rstd_out[blockIdx.x] = rstd;
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    const float s = to_f32(x[at + c]) + (residual ? to_f32(residual[at + c]) : 0.0f);
    if (h_out) put(h_out + at + c, s);
    if (out) put(out + at + c, s * rstd * to_f32(w[c]));
  }
}

// ----------------------------------------------------------------- backward
// A fixed number of blocks walks the rows, so each thread keeps its columns'
// dw in registers; the blocks' partial sums go to `part_dw` [gridDim, H] and
// a second kernel adds them in block order (no atomics: the result does not
// change from run to run).
template <typename RT, int NV, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 32 * kWarpRows : 512) add_rmsnorm_bwd_kernel(long long rows, int H, const __nv_bfloat16* dout,
                                       const RT* dh_in, const RT* h, const __nv_bfloat16* __restrict__ w,
                                       const float* __restrict__ rstd, RT* dh, __nv_bfloat16* dx,
                                       float* __restrict__ part_dw) {
  __shared__ float part[2][32];
  extern __shared__ float warp_dw[];  // WARP_ROW: [kWarpRows][H]
  const int tid = WARP_ROW ? (threadIdx.x & 31) : threadIdx.x;
  const int nt = WARP_ROW ? 32 : blockDim.x;
  const long long first = WARP_ROW ? (long long)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : (long long)blockIdx.x;
  const long long step = WARP_ROW ? (long long)gridDim.x * kWarpRows : (long long)gridDim.x;
  float dw[NV][8];
  Vec8<__nv_bfloat16> vw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * nt + tid) * 8;
    vw[v].zero();
    if (c < H) vw[v].load(w + c);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = 0.0f;
  }
  const float inv_h = 1.0f / (float)H;
  int buf = 0;
  for (long long row = first; row < rows; row += step, buf ^= 1) {
    const size_t at = (size_t)row * H;
    Vec8<__nv_bfloat16> vd[NV];
    Vec8<RT> vh[NV], vi[NV];
    const float rs = rstd[row];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * nt + tid) * 8;
      vd[v].zero();
      vh[v].zero();
      vi[v].zero();
      if (c < H) {
        vd[v].load(dout + at + c);
        vh[v].load(h + at + c);
        if (dh_in) vi[v].load(dh_in + at + c);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float d[8], xh[8], g[8];
      vd[v].unpack(d);
      vh[v].unpack(xh);
      vw[v].unpack(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[j] *= rs;
        dw[v][j] = fmaf(d[j], xh[j], dw[v][j]);
        dot = fmaf(d[j] * g[j], xh[j], dot);
      }
    }
    dot = WARP_ROW ? warp_sum(dot) : block_sum(dot, part[buf]);
    const float m = dot * inv_h;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * nt + tid) * 8;
      if (c >= H) continue;
      float d[8], xh[8], g[8], r[8];
      vd[v].unpack(d);
      vh[v].unpack(xh);
      vw[v].unpack(g);
      vi[v].unpack(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = fmaf(rs, d[j] * g[j] - xh[j] * rs * m, r[j]);
      Vec8<RT>::store(dh + at + c, r);
      if (dx) Vec8<__nv_bfloat16>::store(dx + at + c, r);
    }
  }
  if (!part_dw) return;
  float* mine = part_dw + (size_t)blockIdx.x * H;
  if (WARP_ROW) {
    float* sw = warp_dw + (threadIdx.x >> 5) * H;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * nt + tid) * 8;
      if (c < H) Vec8<float>::store(sw + c, dw[v]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarpRows; ++k) t += warp_dw[k * H + c];
      mine[c] = t;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * nt + tid) * 8;
      if (c < H) Vec8<float>::store(mine + c, dw[v]);
    }
  }
}

// Any H: one block per row for dh; dw by columns in the second kernel below.
template <typename RT>
__global__ void add_rmsnorm_bwd_any_kernel(long long rows, int H, const __nv_bfloat16* dout, const RT* dh_in,
                                           const RT* h, const __nv_bfloat16* __restrict__ w,
                                           const float* __restrict__ rstd, RT* dh, __nv_bfloat16* dx) {
  __shared__ float part[2][32];
  int buf = 0;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x, buf ^= 1) {
    const size_t at = (size_t)row * H;
    const float rs = rstd[row];
    float dot = 0.0f;
    for (int c = threadIdx.x; c < H; c += blockDim.x)
      dot = fmaf(to_f32(dout[at + c]) * to_f32(w[c]), to_f32(h[at + c]) * rs, dot);
    const float m = block_sum(dot, part[buf]) / (float)H;
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
      const float r = rs * (to_f32(dout[at + c]) * to_f32(w[c]) - to_f32(h[at + c]) * rs * m) +
                      (dh_in ? to_f32(dh_in[at + c]) : 0.0f);
      put(dh + at + c, r);
      if (dx) put(dx + at + c, r);
    }
  }
}
// part_dw[b, c] = sum over block b's rows of dout * h * rstd. Run before the
// kernel above, whose dh may overwrite h or dout in place.
template <typename RT>
__global__ void add_rmsnorm_dw_any_kernel(long long rows, int H, const __nv_bfloat16* __restrict__ dout,
                                          const RT* __restrict__ h, const float* __restrict__ rstd,
                                          float* __restrict__ part_dw) {
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    float t = 0.0f;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x)
      t = fmaf(to_f32(dout[(size_t)row * H + c]), to_f32(h[(size_t)row * H + c]) * rstd[row], t);
    part_dw[(size_t)blockIdx.x * H + c] = t;
  }
}

// dw[c] = sum of part[0 .. n-1][c] in a fixed order: 32 columns per block, 8
// threads per column over every eighth partial, then those 8 in order.
__global__ void __launch_bounds__(256) sum_partials_kernel(const float* __restrict__ part, int n, int H,
                                                           float* __restrict__ dw) {
  __shared__ float s[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float t = 0.0f;
  if (c < H)
    for (int i = k; i < n; i += 8) t += part[(size_t)i * H + c];
  s[k][threadIdx.x & 31] = t;
  __syncthreads();
  if (k == 0 && c < H) {
    t = s[0][threadIdx.x];
#pragma unroll
    for (int j = 1; j < 8; ++j) t += s[j][threadIdx.x];
    dw[c] = t;
  }
}

// Threads of a block that holds one row in NV vectors of 8 per thread.
int row_threads(int H, int nv) { return ((H + 8 * nv - 1) / (8 * nv) + 31) / 32 * 32; }

template <typename RT, bool MX>
cudaError_t run_norm(const NormArgs& a, cudaStream_t s) {
  const auto* x = static_cast<const __nv_bfloat16*>(a.x);
  const auto* r = static_cast<const RT*>(a.residual);
  const auto* w = static_cast<const __nv_bfloat16*>(a.weight);
  auto* ho = static_cast<RT*>(a.h_out);
  auto* out = static_cast<__nv_bfloat16*>(a.out);
  if (a.H % 8) {
    add_rmsnorm_any_kernel<RT><<<(unsigned)a.rows, 256, 0, s>>>(a.H, x, r, w, a.eps, ho, out, a.rstd);
    return cudaGetLastError();
  }
#define MOE_NORM(NV, WR, GRID, THREADS)                                                                           \
  add_rmsnorm_kernel<RT, NV, WR, MX><<<(unsigned)(GRID), (THREADS), 0, s>>>(a.rows, a.H, x, r, w, a.eps, ho, out, \
                                                                          a.q, a.q_scale, a.rstd)
  if (a.H <= kWarpRowCols) {
    const long long grid = (a.rows + kWarpRows - 1) / kWarpRows;
    if (a.H <= 256) MOE_NORM(1, true, grid, 32 * kWarpRows);
    else if (a.H <= 512) MOE_NORM(2, true, grid, 32 * kWarpRows);
    else MOE_NORM(4, true, grid, 32 * kWarpRows);
  } else if (a.H <= 8192) {
    MOE_NORM(2, false, a.rows, row_threads(a.H, 2));
  } else {
    MOE_NORM(4, false, a.rows, row_threads(a.H, 4));
  }
#undef MOE_NORM
  return cudaGetLastError();
}

template <typename RT>
cudaError_t run_norm_bwd(const NormGradArgs& a, cudaStream_t s) {
  const auto* dout = static_cast<const __nv_bfloat16*>(a.dout);
  const auto* di = static_cast<const RT*>(a.dh_in);
  const auto* h = static_cast<const RT*>(a.h);
  const auto* w = static_cast<const __nv_bfloat16*>(a.weight);
  auto* dh = static_cast<RT*>(a.dh);
  auto* dx = static_cast<__nv_bfloat16*>(a.dx);
  float* part = a.dweight ? a.partials : nullptr;
  const int n = norm_grad_blocks(a.rows, a.H);
  if (a.H % 8) {
    if (part) add_rmsnorm_dw_any_kernel<RT><<<n, 256, 0, s>>>(a.rows, a.H, dout, h, a.rstd, part);
    add_rmsnorm_bwd_any_kernel<RT><<<n, 256, 0, s>>>(a.rows, a.H, dout, di, h, w, a.rstd, dh, dx);
  } else {
#define MOE_NORM(NV, WR, THREADS, SMEM)                                                                           \
  add_rmsnorm_bwd_kernel<RT, NV, WR><<<n, (THREADS), (SMEM), s>>>(a.rows, a.H, dout, di, h, w, a.rstd, dh, dx, part)
    if (a.H <= kWarpRowCols) {
      const int smem = part ? kWarpRows * a.H * 4 : 0;
      if (a.H <= 256) MOE_NORM(1, true, 32 * kWarpRows, smem);
      else if (a.H <= 512) MOE_NORM(2, true, 32 * kWarpRows, smem);
      else MOE_NORM(4, true, 32 * kWarpRows, smem);
    } else if (a.H <= 8192) {
      MOE_NORM(2, false, row_threads(a.H, 2), 0);
    } else {
      MOE_NORM(4, false, row_threads(a.H, 4), 0);
    }
#undef MOE_NORM
  }
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.dweight) {
    sum_partials_kernel<<<(a.H + 31) / 32, 256, 0, s>>>(part, n, a.H, a.dweight);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

// Blocks of the backward pass: two per SM of a GB300 (152), fewer when the
// rows are fewer. A constant, so dw's summation order is the same everywhere.
int norm_grad_blocks(long long rows, int H) {
  const long long units = (H % 8 == 0 && H <= kWarpRowCols) ? (rows + kWarpRows - 1) / kWarpRows : rows;
  return (int)(units < 304 ? units : 304);
}

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (a.q) return a.res_f32 ? run_norm<float, true>(a, s) : run_norm<__nv_bfloat16, true>(a, s);
  return a.res_f32 ? run_norm<float, false>(a, s) : run_norm<__nv_bfloat16, false>(a, s);
}

cudaError_t launch_add_rmsnorm_backward(const NormGradArgs& a, cudaStream_t s) {
  if (a.rows == 0)
    return a.dweight ? cudaMemsetAsync(a.dweight, 0, (size_t)a.H * 4, s) : cudaSuccess;
  return a.res_f32 ? run_norm_bwd<float>(a, s) : run_norm_bwd<__nv_bfloat16>(a, s);
}

}  // namespace moe
