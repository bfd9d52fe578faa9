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
// once (8192 x 4096 with MXFP8 output: 44.9 us, 6.7 TB/s, the copy rate). Rows of
// at most 1024 columns take one warp each, longer rows (up to
// 16384) one block each. Every thread reads its elements of a row before it
// writes them, so the outputs may overwrite the inputs of their own type.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "internal.h"
#include "launch.cuh"
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
                                   const RT* residual, const __nv_bfloat16* w, float eps, RT* h_out, __nv_bfloat16* out,
                                   uint8_t* q, uint8_t* q_scale, float* rstd_out) {
  __shared__ float part[32];
  allow_next_launch();
  wait_for_previous_launch();
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
//
// A row's sum needs the whole row before its first output, so loads that wait
// for the previous row would leave the memory idle in between. Each thread
// therefore copies its own columns of the next rows into shared memory
// (cp.async) and reads back only what it copied, twice: for the sum and for
// the outputs. A block is several groups of threads, each with a row of its
// own and a barrier of its own (a group of 32 needs none); 32 columns per
// thread keep the groups small and the sum's exchange cheap. 8192 x 4096 in
// bf16: 47 us (40 at a copy's rate), 3 of them until the partial sums are added.
constexpr int kPieces = 3;
template <typename RT, int NV>
struct BwdShape {
  // 16-byte pieces of one vector of 8 columns: dout, h, and a bf16 dh_in. (An
  // fp32 dh_in would take the room of a row more in flight: it is prefetched
  // into L2 when the row's copies start and loaded a row ahead, or, where that
  // would take too many registers, while its row is summed.)
  static constexpr int RP = sizeof(RT) / 2;
  static constexpr bool RING_IN = RP == 1, AHEAD = !RING_IN && NV <= 2;
  static constexpr int PIECES = kPieces;
};
// Rows a group holds: four or three where they fit in `room` bytes, else two
// (at most 192 KB: 512 threads of 4 vectors).
int bwd_stages(int bytes_per_thread, int threads, int room) {
  const int row = bytes_per_thread * threads;
  return 4 * row <= room ? 4 : (3 * row <= room ? 3 : 2);
}

__device__ __forceinline__ void copy16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))),
               "l"(g)
               : "memory");
}

template <typename RT, int NV, int STAGES>
__global__ void __launch_bounds__(512)
    add_rmsnorm_bwd_kernel(long long rows, int H, int nt, const __nv_bfloat16* dout, const RT* dh_in, const RT* h,
                           const __nv_bfloat16* w, const float* rstd, RT* dh, __nv_bfloat16* dx, float* part_dw) {
  wait_for_previous_launch();
  using Sh = BwdShape<RT, NV>;
  __shared__ float part[2][16];  // [buffer][warp of the block]
  extern __shared__ uint4 ring[];  // [stage][vector][piece][thread]; at the end the groups' dw
  const int group = threadIdx.x / nt, groups = blockDim.x / nt, tid = threadIdx.x - group * nt;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group_warps = nt >> 5;
  const long long first = (long long)blockIdx.x * groups + group, step = (long long)gridDim.x * groups;
  auto slot = [&](int st, int v, int piece) {
    return ring + ((st * NV + v) * Sh::PIECES + piece) * blockDim.x + threadIdx.x;
  };
  auto fetch = [&](int st, long long row) {
    if (row < rows) {
      const size_t at = (size_t)row * H;
      const __nv_bfloat16* pd = dout + at;
      const RT *ph = h + at, *pi = dh_in + at;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * nt + tid) * 8;
        if (c >= H) continue;
        copy16(slot(st, v, 0), pd + c);
#pragma unroll
        for (int i = 0; i < Sh::RP; ++i) {
          copy16(slot(st, v, 1 + i), reinterpret_cast<const uint4*>(ph + c) + i);
          if (Sh::RING_IN && dh_in) copy16(slot(st, v, 1 + Sh::RP + i), reinterpret_cast<const uint4*>(pi + c) + i);
        }
        if (!Sh::RING_IN && dh_in && (lane & 3) == 0)  // four lanes' columns are one 128-byte line
          asm volatile("prefetch.global.L2 [%0];" ::"l"(pi + c));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i, first + i * step);
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
  int buf = 0, st = 0;
  float rs = first < rows ? rstd[first] : 0.0f;
  Vec8<RT> vi[Sh::RING_IN ? 1 : NV], vi_next[Sh::AHEAD ? NV : 1];
  auto load_in = [&](Vec8<RT>* to, long long row) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * nt + tid) * 8;
      to[v].zero();
      if (dh_in && c < H && row < rows) to[v].load(dh_in + (size_t)row * H + c);
    }
  };
  if (Sh::AHEAD) load_in(vi_next, first);
  for (long long row = first; row < rows; row += step, buf ^= 1) {
    const float rs_next = row + step < rows ? rstd[row + step] : 0.0f;  // a row ahead, like the copies
    fetch(st == 0 ? STAGES - 1 : st - 1, row + (STAGES - 1) * step);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    const size_t at = (size_t)row * H;
    if (Sh::AHEAD) {
#pragma unroll
      for (int v = 0; v < NV; ++v) vi[v] = vi_next[Sh::AHEAD ? v : 0];
      load_in(vi_next, row + step);
    } else if (!Sh::RING_IN) {
      load_in(vi, row);
    }
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if ((v * nt + tid) * 8 >= H) continue;
      Vec8<__nv_bfloat16> vd;
      Vec8<RT> vh;
      vd.a = *slot(st, v, 0);
#pragma unroll
      for (int i = 0; i < Sh::RP; ++i) reinterpret_cast<uint4*>(&vh)[i] = *slot(st, v, 1 + i);
      float d[8], xh[8], g[8];
      vd.unpack(d);
      vh.unpack(xh);
      vw[v].unpack(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = d[j] * (xh[j] * rs);
        dw[v][j] += t;
        dot = fmaf(t, g[j], dot);
      }
    }
    dot = warp_sum(dot);
    if (group_warps > 1) {
      if (lane == 0) part[buf][warp] = dot;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(nt) : "memory");
      dot = warp_sum(lane < group_warps ? part[buf][group * group_warps + lane] : 0.0f);
    }
    const float m = dot * inv_h * rs * rs;  // dh = rs g - h rs^2 mean(g xhat) + dh_in
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * nt + tid) * 8;
      if (c >= H) continue;
      Vec8<__nv_bfloat16> vd;
      Vec8<RT> vh;
      vd.a = *slot(st, v, 0);
#pragma unroll
      for (int i = 0; i < Sh::RP; ++i) reinterpret_cast<uint4*>(&vh)[i] = *slot(st, v, 1 + i);
      Vec8<RT>& in = vi[Sh::RING_IN ? 0 : v];
      if (Sh::RING_IN) {
        in.zero();
        if (dh_in) *reinterpret_cast<uint4*>(&in) = *slot(st, v, 2);
      }
      float d[8], hh[8], g[8], r[8];
      vd.unpack(d);
      vh.unpack(hh);
      vw[v].unpack(g);
      in.unpack(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = fmaf(rs, d[j] * g[j], r[j] - hh[j] * m);
      Vec8<RT>::store(dh + at + c, r);
      if (dx) Vec8<__nv_bfloat16>::store(dx + at + c, r);
    }
    st = st + 1 == STAGES ? 0 : st + 1;
    rs = rs_next;
  }
  if (!part_dw) return;
  allow_next_launch();
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();  // every group is done with the ring
  float* mine = part_dw + (size_t)blockIdx.x * H;
  float* all = reinterpret_cast<float*>(ring);  // [groups][H]
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * nt + tid) * 8;
    if (c < H) Vec8<float>::store(groups > 1 ? all + group * H + c : mine + c, dw[v]);
  }
  if (groups == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    float t = all[c];
    for (int k = 1; k < groups; ++k) t += all[k * H + c];
    mine[c] = t;
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

// dw[c] = sum of part[0 .. n-1][c] in a fixed order: 32 columns per block, 32
// threads per column over every 32nd partial, then those 32 in order. (`part` is
// written while this kernel may already run: no read-only loads of it, which
// the compiler may move up past the wait.)
__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* part, int n, int H, float* dw) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, k = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  allow_next_launch();
  wait_for_previous_launch();
  float t = 0.0f;
  if (c < H) {
#pragma unroll 4
    for (int i = k; i < n; i += 32) t += __ldcg(part + (size_t)i * H + c);
  }
  s[k][x] = t;
  __syncthreads();
  t = warp_sum(s[x][k]);  // the column of this warp: blockIdx.x * 32 + k
  if (x == 0 && blockIdx.x * 32 + k < H) dw[blockIdx.x * 32 + k] = t;
}

// Threads of a block that holds one row in NV vectors of 8 per thread.
int row_threads(int H, int nv) { return ((H + 8 * nv - 1) / (8 * nv) + 31) / 32 * 32; }

// Backward: vectors of 8 columns per thread (an fp32 row of up to 8192 columns
// takes two, for its wider loads).
int norm_grad_vectors(int H, bool f32) { return H <= 256 ? 1 : (H <= 512 || (f32 && H <= 8192) ? 2 : 4); }

// Its blocks and the row groups of each: a block per row while there are no more
// than two per SM; then one block per SM of 512 threads for bf16 rows, which
// halves the partial sums (1000 x 4096 13.2 -> 11.8 us, 8192 x 4096 48.7 ->
// 47.0, 300 to 1000 x 512 4% slower), and two of 256 for fp32 rows of up to 4096
// columns, which is within 5% of one either way (us, two / one: 1000 x 512 6.7 /
// 6.6, 8192 x 512 16.8 / 17.3, 1000 x 2048 11.2 / 10.6, 8192 x 2048 49.3 / 48.3,
// 1000 x 4096 19.6 / 20.2, 3000 x 4096 38.8 / 39.1, 8192 x 4096 89.9 / 88.4).
// Longer fp32 rows have a block of up to 512 threads: 3000 x 8192 69 us, with
// four vectors in each of 256 threads 77. A function of the shape alone, so dw's
// summation order is the same everywhere.
constexpr int kSms = 152;  // of a GB300
struct BwdGrid {
  int blocks, groups, room;  // room: of a block's ring
};
BwdGrid norm_grad_grid(long long rows, int H, bool f32) {
  constexpr int kOne = 192 * 1024, kTwo = 112 * 1024;  // blocks per SM
  const int nt = row_threads(H, norm_grad_vectors(H, f32)), per_sm = f32 && nt <= 256 ? 2 : 1;
  if (rows <= 2 * kSms) return {(int)rows, 1, rows <= kSms || nt > 256 ? kOne : kTwo};
  if (H % 8) return {2 * kSms, 1, 0};  // no ring
  const int g = 512 / per_sm / nt, groups = g < 1 ? 1 : g;
  const long long units = (rows + groups - 1) / groups;
  return {(int)(units < per_sm * kSms ? units : per_sm * kSms), groups, per_sm == 2 ? kTwo : kOne};
}

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
#define MOE_NORM(NV, WR, GRID, THREADS)                                                                              \
  return launch_dependent(add_rmsnorm_kernel<RT, NV, WR, MX>, (int)(GRID), (THREADS), 0, s, true, 1, a.rows, a.H, x, r, \
                          w, a.eps, ho, out, a.q, a.q_scale, a.rstd)
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
  const BwdGrid g = norm_grad_grid(a.rows, a.H, a.res_f32);
  const int n = g.blocks;
  cudaError_t e = cudaSuccess;
  if (a.H % 8) {
    if (part) add_rmsnorm_dw_any_kernel<RT><<<n, 256, 0, s>>>(a.rows, a.H, dout, h, a.rstd, part);
    add_rmsnorm_bwd_any_kernel<RT><<<n, 256, 0, s>>>(a.rows, a.H, dout, di, h, w, a.rstd, dh, dx);
    e = cudaGetLastError();
  } else {
    const int nv = norm_grad_vectors(a.H, a.res_f32), nt = row_threads(a.H, nv);
    const int threads = g.groups * nt, bytes = nv * kPieces * 16, stages = bwd_stages(bytes, threads, g.room);
#define MOE_NORM(NV, ST)                                                                                      \
  if (nv == NV && stages == ST)                                                                               \
  e = launch_dependent(add_rmsnorm_bwd_kernel<RT, NV, ST>, n, threads, (size_t)ST * bytes * threads, s, true, 1, a.rows, \
                       a.H, nt, dout, di, h, w, a.rstd, dh, dx, part)
    MOE_NORM(1, 4);
    MOE_NORM(2, 4);
    MOE_NORM(4, 4);
    MOE_NORM(4, 3);
    MOE_NORM(4, 2);
#undef MOE_NORM
  }
  if (e == cudaSuccess && a.dweight)
    e = launch_dependent(sum_partials_kernel, (a.H + 31) / 32, 1024, 0, s, true, /*cluster=*/1, part, n, a.H,
                         a.dweight);
  return e;
}

template <typename RT>
cudaError_t set_all_bwd_smem() {
  const void* kernels[] = {reinterpret_cast<const void*>(add_rmsnorm_bwd_kernel<RT, 1, 4>),
                           reinterpret_cast<const void*>(add_rmsnorm_bwd_kernel<RT, 2, 4>),
                           reinterpret_cast<const void*>(add_rmsnorm_bwd_kernel<RT, 4, 4>),
                           reinterpret_cast<const void*>(add_rmsnorm_bwd_kernel<RT, 4, 3>),
                           reinterpret_cast<const void*>(add_rmsnorm_bwd_kernel<RT, 4, 2>)};
  for (const void* k : kernels) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 192 * 1024);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t norm_prepare_device() {
  const cudaError_t e = set_all_bwd_smem<float>();
  return e != cudaSuccess ? e : set_all_bwd_smem<__nv_bfloat16>();
}

// Blocks of the backward pass: rows of partial sums in its workspace.
int norm_grad_blocks(long long rows, int H, bool f32) { return norm_grad_grid(rows, H, f32).blocks; }

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
