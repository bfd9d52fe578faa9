// Quantisers to E4M3 with one fp32 scale per block of 128 (fp8.cuh has the rule),
// of bf16 or fp32 matrices:
//   rows     128 values of a row share a scale      (a product's activations)
//   squares  128 rows x 128 columns share a scale   (weights)
//   columns  128 rows of a group, one column        (the weight gradient's
//            operands: the reduction runs over the rows; each group starts at a
//            multiple of 128 rows of the result, and zero rows fill its last block)
// One pass: a block's values stay in registers between its maximum and its
// codes. Floors are of HBM, 2 (4) bytes in and 1 out per value; the rows take 75% of
// the issue slots beside it (maxima of two bf16 values at a time: 23.6 -> 18.4 us).
// 33.6 million bf16 values (floor 15 us): rows of 4096 18.1, squares 18.6, columns of
// uneven groups 23.0; fp32 (24.9): rows 27.9, squares 33.6, columns 34.2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

// 16 bytes of input: eight bf16 or four fp32 values.
template <bool F32>
struct Vec {
  static constexpr int kN = F32 ? 4 : 8;
  uint4 raw;
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = F32 ? (&raw.x)[i] : (&raw.x)[i >> 1];
    return __uint_as_float(F32 ? w : ((i & 1) ? (w & 0xFFFF0000u) : (w << 16)));
  }
  // |values| as bits that order as they do, per value: bf16 ones two to a word.
  static constexpr uint32_t kAbs = F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
  static __device__ __forceinline__ uint32_t max_of(uint32_t a, uint32_t b) { return F32 ? (a > b ? a : b) : __vmaxu2(a, b); }
  // The largest of a word's values, as fp8_abs_bits.
  static __device__ __forceinline__ uint32_t whole(uint32_t t) {
    if (F32) return t;
    const uint32_t hi = t & 0xFFFF0000u, lo = t << 16;
    return hi > lo ? hi : lo;
  }
  __device__ __forceinline__ uint32_t amax_bits() const {
    return whole(max_of(max_of(raw.x & kAbs, raw.y & kAbs), max_of(raw.z & kAbs, raw.w & kAbs)));
  }
  template <bool SMALL>
  __device__ __forceinline__ void store(uint8_t* q, const Fp8Block& b) const {
    const uint32_t lo = b.code4<SMALL>(at(0), at(1), at(2), at(3));
    if (F32) *reinterpret_cast<uint32_t*>(q) = lo;
    else *reinterpret_cast<uint2*>(q) = make_uint2(lo, b.code4<SMALL>(at(4 & (kN - 1)), at(5 & (kN - 1)), at(6 & (kN - 1)), at(7 & (kN - 1))));
  }
};

// ---------------------------------------------------------------- rows
// A block of a row per 16 lanes (bf16) or warp (fp32), kInFlight of them loading
// at a time. WHOLE: rows of whole blocks, so that block b is values 128 b .. of
// the matrix; else a thread finds its first block's row by one division and
// steps from there (with a division per block they took half as long again).
constexpr int kRowThreads = 256;
constexpr int kInFlight = 4;

template <bool F32, bool WHOLE>
__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const uint8_t* x, long long blocks, int cols, int nb,
                                                                    int step_rows, int step_blocks, uint8_t* q, float* scale) {
  constexpr int kN = Vec<F32>::kN, kLanes = 128 / kN, kEsize = F32 ? 4 : 2;
  constexpr int kGroups = kRowThreads / kLanes;  // blocks that the thread block works on at a time
  wait_for_previous_launch();
  allow_next_launch();
  const int sub = threadIdx.x % kLanes;
  const long long first = (long long)blockIdx.x * (kGroups * kInFlight) + threadIdx.x / kLanes;
  long long row = WHOLE ? 0 : (blocks <= 0x7FFFFFFF ? (int)first / nb : first / nb);
  int blk = WHOLE ? 0 : (int)(first - row * nb);
  Vec<F32> v[kInFlight];
  long long at[kInFlight];
#pragma unroll
  for (int j = 0; j < kInFlight; ++j) {
    const long long b = first + (long long)j * kGroups;
    const int col = blk * 128 + sub * kN;
    v[j].raw = make_uint4(0, 0, 0, 0);
    at[j] = -1;
    if (b < blocks && (WHOLE || col < cols)) {
      at[j] = WHOLE ? b * 128 + sub * kN : row * cols + col;
      v[j].raw = __ldcs(reinterpret_cast<const uint4*>(x + at[j] * kEsize));
    }
    row += step_rows;
    blk += step_blocks;
    if (blk >= nb) {
      blk -= nb;
      ++row;
    }
  }
  auto amax_of = [](const Vec<F32>& x) {  // over the lanes of a block
    uint32_t top = x.amax_bits();
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      const uint32_t u = __shfl_xor_sync(0xFFFFFFFFu, top, o);
      top = u > top ? u : top;
    }
    return top;
  };
  bool small = false;
#pragma unroll
  for (int j = 0; j < kInFlight; ++j) {
    const Fp8Block b(fp8_scale(amax_of(v[j])));
    small |= b.small();
    if (at[j] >= 0) {
      v[j].template store<false>(q + at[j], b);
      if (sub == 0) scale[first + (long long)j * kGroups] = b.scale;
    }
  }
  if (!__any_sync(0xFFFFFFFFu, small)) return;
  // Rare: the codes of small scales once more, from x, so that the values above need
  // not be kept for it (8192 x 4096 bf16 in a graph: 16.0 us without this, 17.5 with
  // kept values, 16.2 so).
#pragma unroll 1
  for (int j = 0; j < kInFlight; ++j) {
    const long long b = first + (long long)j * kGroups, r = WHOLE ? 0 : b / nb;
    const int col = (WHOLE ? 0 : (int)(b - r * nb) * 128) + sub * kN;
    const long long to = WHOLE ? b * 128 + col : r * cols + col;
    const bool mine = b < blocks && (WHOLE || col < cols);
    Vec<F32> again;
    again.raw = make_uint4(0, 0, 0, 0);
    if (mine) again.raw = *reinterpret_cast<const uint4*>(x + to * kEsize);
    const Fp8Block k(fp8_scale(amax_of(again)));
    if (mine && k.small()) again.template store<true>(q + to, k);
  }
}

// ---------------------------------------------------------------- 128 x 128 tiles
// A thread block holds a tile, 64 values per thread: rows a 16th (bf16) or an 8th
// (fp32) of the tile apart.
constexpr int kTileThreads = 256;
constexpr int kMaxGroups = 1024;

template <bool F32, int COLS = 128>
struct TileRegs {
  static constexpr int kThreads = kTileThreads * COLS / 128;
  static constexpr int kN = Vec<F32>::kN, kLanes = COLS / kN, kStep = kThreads / kLanes, kRows = 128 / kStep;
  Vec<F32> v[kRows];
  int col, row;  // of this thread's first value in the tile
  __device__ __forceinline__ TileRegs() : col(threadIdx.x % kLanes * kN), row(threadIdx.x / kLanes) {}
  // x: the tile's first element; rows and columns past `nr`, `nc` are zeros.
  __device__ __forceinline__ void load(const uint8_t* x, long long ld, int nr, int nc) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = row + i * kStep;
      v[i].raw = make_uint4(0, 0, 0, 0);
      if (r < nr && col < nc) v[i].raw = __ldcs(reinterpret_cast<const uint4*>(x + (r * ld + col) * (F32 ? 4 : 2)));
    }
  }
};

template <bool F32>
__global__ void __launch_bounds__(kTileThreads)
    quantize_squares_kernel(const uint8_t* x, int rows, int cols, int row_blocks, int col_blocks, uint8_t* q, float* scale) {
  __shared__ uint32_t tops[kTileThreads / 32];
  wait_for_previous_launch();
  allow_next_launch();
  const int cb = blockIdx.x % col_blocks;
  const long long rb_all = blockIdx.x / col_blocks;  // of all matrices
  const long long mat = rb_all / row_blocks;
  const int rb = (int)(rb_all - mat * row_blocks);
  const long long at = (mat * rows + rb * 128ll) * cols + cb * 128;
  const int nr = rows - rb * 128, nc = cols - cb * 128;
  TileRegs<F32> t;
  t.load(x + at * (F32 ? 4 : 2), cols, nr, nc);
  using V = Vec<F32>;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < TileRegs<F32>::kRows; ++i) {
    const uint4 r = t.v[i].raw;
    top = V::max_of(top, V::max_of(V::max_of(r.x & V::kAbs, r.y & V::kAbs), V::max_of(r.z & V::kAbs, r.w & V::kAbs)));
  }
  top = V::whole(top);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
  top = tops[threadIdx.x & 7];
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  const Fp8Block blk(fp8_scale(top));
  if (threadIdx.x == 0) scale[blockIdx.x] = blk.scale;
  fp8_by_size(blk.small(), [&](auto s) {
#pragma unroll
    for (int i = 0; i < TileRegs<F32>::kRows; ++i) {
      const int r = t.row + i * TileRegs<F32>::kStep;
      if (r < nr && t.col < nc) t.v[i].template store<decltype(s)::value>(q + at + (long long)r * cols + t.col, blk);
    }
  });
}

// Tiles of 128 rows x kCols: twice the thread blocks per SM of tiles of 128 columns,
// whose loads, maxima and codes alternate (24.9 -> 22.7 us; of 32 columns 27.2).
constexpr int kCols = 64, kColThreads = TileRegs<false, kCols>::kThreads;

template <bool F32>
__global__ void __launch_bounds__(kColThreads, F32 ? 4 : 6)
    quantize_columns_kernel(const uint8_t* x, int rows, int cols, const int32_t* offsets, int G, uint8_t* q, float* scale) {
  using T = TileRegs<F32, kCols>;
  __shared__ __align__(16) uint32_t part[T::kStep][kCols];
  __shared__ __align__(16) float scales[kCols], invs[kCols];
  __shared__ int where[2], starts[kMaxGroups + 1];
  wait_for_previous_launch();
  allow_next_launch();
  // The group whose blocks of 128 rows this one is of: every lane of a warp takes
  // some groups, and the one whose blocks end past blockIdx.x looks for it.
  for (int g = threadIdx.x; g <= G; g += kColThreads) {
    const int v = offsets ? __ldcg(offsets + g) : (g == 0 ? 0 : rows);
    starts[g] = v < 0 ? 0 : (v > rows ? rows : v);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (G + 31) / 32, b = lane * per < G ? lane * per : G, e = b + per < G ? b + per : G;
    auto blocks = [&](int g) { return starts[g + 1] > starts[g] ? (starts[g + 1] - starts[g] + 127) / 128 : 0; };
    int mine = 0;
    for (int g = b; g < e; ++g) mine += blocks(g);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += u;
    }
    const int want = blockIdx.x;
    if (lane == 31 && want >= incl) where[1] = -1;
    if (want < incl && want >= incl - mine) {
      int at = incl - mine;
      for (int g = b; g < e; ++g) {
        const int n = blocks(g);
        if (want < at + n) {
          where[0] = starts[g] + (want - at) * 128;
          where[1] = starts[g + 1] - where[0];
          break;
        }
        at += n;
      }
    }
  }
  __syncthreads();
  const int row0 = where[0], nr = where[1];
  if (nr < 0) return;  // behind the last group
  for (int cb = blockIdx.y; cb * kCols < cols; cb += gridDim.y) {
    const int nc = cols - cb * kCols;
    T t;
    t.load(x + ((long long)row0 * cols + cb * kCols) * (F32 ? 4 : 2), cols, nr, nc);
    using V = Vec<F32>;
    uint32_t top[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      top[w] = 0;
#pragma unroll
      for (int i = 0; i < T::kRows; ++i) top[w] = V::max_of(top[w], (&t.v[i].raw.x)[w] & V::kAbs);
    }
    uint4* mine = reinterpret_cast<uint4*>(&part[t.row][t.col]);
    if (F32) {
      mine[0] = make_uint4(top[0], top[1], top[2], top[3]);
    } else {
      mine[0] = make_uint4(top[0] << 16, top[0] & 0xFFFF0000u, top[1] << 16, top[1] & 0xFFFF0000u);
      mine[1] = make_uint4(top[2] << 16, top[2] & 0xFFFF0000u, top[3] << 16, top[3] & 0xFFFF0000u);
    }
    __syncthreads();
    bool small = false;
    if (threadIdx.x < kCols) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < T::kStep; ++i) {
        const uint32_t a = part[i][threadIdx.x];
        m = a > m ? a : m;
      }
      const Fp8Block blk(fp8_scale(m));
      scales[threadIdx.x] = blk.scale;
      invs[threadIdx.x] = blk.inv;
      small = blk.small();
      if ((int)threadIdx.x < nc) scale[(long long)blockIdx.x * cols + cb * kCols + threadIdx.x] = blk.scale;
    }
    small = __syncthreads_or(small);
    if (t.col < nc) {
      uint8_t* at = q + ((long long)blockIdx.x * 128 + t.row) * cols + cb * kCols + t.col;
      // Four columns at a time, so that four scales and reciprocals are in registers.
      uint32_t w[T::kRows][T::kN / 4];
#pragma unroll
      for (int h = 0; h < T::kN / 4; ++h) {
        const float4 s4 = *reinterpret_cast<const float4*>(scales + t.col + 4 * h);
        const float4 i4 = *reinterpret_cast<const float4*>(invs + t.col + 4 * h);
        const Fp8Block b0(s4.x, i4.x), b1(s4.y, i4.y), b2(s4.z, i4.z), b3(s4.w, i4.w);
        fp8_by_size(small, [&](auto any) {
          constexpr bool S = decltype(any)::value;
#pragma unroll
          for (int i = 0; i < T::kRows; ++i) {
            const Vec<F32>& v = t.v[i];
            w[i][h] = fp8_pack4(b0.over<S>(v.at(4 * h)), b1.over<S>(v.at(4 * h + 1)), b2.over<S>(v.at(4 * h + 2)), b3.over<S>(v.at(4 * h + 3)));
          }
        });
      }
#pragma unroll
      for (int i = 0; i < T::kRows; ++i) {
        uint8_t* d = at + (long long)i * T::kStep * cols;
        if (F32) *reinterpret_cast<uint32_t*>(d) = w[i][0];
        else *reinterpret_cast<uint2*>(d) = make_uint2(w[i][0], w[i][T::kN / 4 - 1]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_fp8_quantize_rows(const void* x, bool f32, int64_t rows, int cols, uint8_t* q, float* scale,
                                     cudaStream_t s) {
  const int nb = fp8_blocks(cols);
  if (rows == 0) return cudaSuccess;
  const int groups = kRowThreads / (f32 ? 32 : 16);
  const long long blocks = rows * nb, per = (long long)groups * kInFlight, grid = (blocks + per - 1) / per;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  const uint8_t* in = static_cast<const uint8_t*>(x);
  auto run = [&](auto* kernel) {
    return launch_dependent(kernel, (int)grid, kRowThreads, 0, s, true, 1, in, blocks, cols, nb, groups / nb, groups % nb, q, scale);
  };
  if (cols % 128 == 0) return f32 ? run(quantize_rows_kernel<true, true>) : run(quantize_rows_kernel<false, true>);
  return f32 ? run(quantize_rows_kernel<true, false>) : run(quantize_rows_kernel<false, false>);
}

cudaError_t launch_fp8_quantize_squares(const void* x, bool f32, int64_t batch, int rows, int cols, uint8_t* q,
                                        float* scale, cudaStream_t s) {
  const int rb = fp8_blocks(rows), cb = fp8_blocks(cols);
  const long long grid = batch * rb * cb;
  if (grid == 0) return cudaSuccess;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  const uint8_t* in = static_cast<const uint8_t*>(x);
  return f32 ? launch_dependent(quantize_squares_kernel<true>, (int)grid, kTileThreads, 0, s, true, 1, in, rows, cols, rb, cb, q, scale)
             : launch_dependent(quantize_squares_kernel<false>, (int)grid, kTileThreads, 0, s, true, 1, in, rows, cols, rb, cb, q, scale);
}

cudaError_t launch_fp8_quantize_columns(const void* x, bool f32, int rows, int cols, const int32_t* offsets, int G,
                                        uint8_t* q, float* scale, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int blocks = (int)(fp8_padded_rows(rows, G) / 128), cb = (cols + kCols - 1) / kCols;
  // About two thousand thread blocks share the column blocks of each row block, so
  // that each looks for its group once for several of them.
  const int share = (2048 + blocks - 1) / blocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)(cb < share ? cb : share), 1);
  cfg.blockDim = dim3(kColThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const uint8_t* in = static_cast<const uint8_t*>(x);
  return f32 ? cudaLaunchKernelEx(&cfg, quantize_columns_kernel<true>, in, rows, cols, offsets, G, q, scale)
             : cudaLaunchKernelEx(&cfg, quantize_columns_kernel<false>, in, rows, cols, offsets, G, q, scale);
}

}  // namespace moe
