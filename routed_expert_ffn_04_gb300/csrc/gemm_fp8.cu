// Products in 8-bit floating point with one fp32 scale per block of 128, over
// groups of rows (experts). For the rows r of group g, with `^` the values that
// E4M3 codes and their scales stand for:
//   FORWARD:      out[r, n] = sum_k a^[r, k] w^[g][n, k]
//   TRANSPOSED:   out[r, n] = sum_k a^[r, k] w^[g][k, n]     (the gradient of an input)
//   GATE_UP:      h = silu(a^ wg^[g]^T) (a^ wu^[g]^T), out as codes and scales per 1 x 128
//   WEIGHT_GRAD:  dw[g][n, k] = sum_r dy^[r, n] a^[r, k]
// Scales: a per row and 128 of k, w per 128 x 128; WEIGHT_GRAD's operands per
// column and 128 rows of a group (which starts at a multiple of 128 of them).
//
// Within a block of 128 of the reduction the scales are one factor per result,
//   out[r, n] = sum_kb (sa[r, kb] sw[n / 128, kb]) sum_{k in kb} qa[r, k] qw[n, k],
// so the tensor cores sum a block's codes (tcgen05.mma kind::f8f6f4, fp32 sums
// of exact products), and after each block the epilogue's warps take the partial
// sums out of TMEM and add them, times the factor, to accumulators in registers.
// fp32 scales cannot go through the block-scaled kinds, which take powers of two.
//
// A tile is 128 rows x 256 columns on one CTA (cta_group::1): 48 KB of operands per
// block of 128, and two buffers of 256 columns of TMEM for partial sums. A thread's
// accumulators are 128 columns of one row: its factor is one number per block (two
// for GATE_UP). Rows (tokens) as M make the factor, SwiGLU and the quantisation of a
// row of h local to a thread. Tiles of 256 rows on pairs of CTAs (cta_group::2)
// load a third less, but each block then waits for the slower CTA's epilogue, a
// group of 341 rows takes 512 and one of few rows leaves a CTA idle: 192 such
// groups took 990 us (GATE_UP) and 684 (FORWARD), on single CTAs 809 and 544; 4 rows
// each, 449 and 361; dense 8192 x 4096 x 4096 113 and 111.
//
// TRANSPOSED and WEIGHT_GRAD read operands MN-major from the row-major tensors,
// with no transposed copy: a box of 128 columns x 128 rows lands as 128 rows of
// 128 swizzled bytes, 8 rows (1024 bytes) per step of the layout, 32 rows per MMA.
//
// PARTS: where few tiles leave SMs idle, the four or eight CTAs of a cluster share a
// tile, each a part of the reduction. Each CTA then takes a slice of the columns
// from the others, through the idle ring by asynchronous stores, and adds the parts
// in their order (7 rows, K 4096, N 1536: 15.2 -> 7.5 us). Whole copies of a slice
// instead were better past 64 rows only (128: 17.3 -> 14.3; 1: 9.0 -> 9.7).
//
// What bounds it: of few rows HBM; of many the epilogue, which adds a block in about
// 700 cycles (265 for the additions of a scheduler's two warps and 100-280 for its
// reads of TMEM, which hardly overlap, and the barriers) against 512 of MMAs, and the
// tile's own end (GATE_UP: 4000 cycles of SwiGLU and codes, half of them waits for
// exp and the quotient). Measured, H 4096, I 1536, 192 groups, 341 rows each and (in
// brackets) routed ones of that mean:
//   GATE_UP      809 us, 2.0 PFLOP/s (908); of 4 rows 361 us, 6.7 TB/s
//   FORWARD      544 us, 1.5 PFLOP/s and 4.4 TB/s (573; 2.4 GB, 1.1 of fp32 results)
//   WEIGHT_GRAD  773 us (777; 2.8 GB, of them 2.4 of bf16 results)
//   FORWARD      dense 8192 x 4096 x 4096 118 us, 2.3 PFLOP/s
// TRANSPOSED with a short reduction is bound by neither: 16384 uneven rows of 64
// groups, K 768, N 2048 take 46 us, 1500 cycles a block, in which the MMAs are at work
// a third of the time, instructions issue in 37% and L2 hands out 27% of its rate.
//
// Roles (12 warps, each walking its tiles in step): 0 loads, 1 issues the MMAs, 2
// and 3 multiply each block's scales into factors ahead of the epilogue, 4-11 are
// the epilogue: TMEM lanes 32 (w % 4) .., columns 128 ((w - 4) / 4) ... Every wait is
// bounded; on expiry the CTA records a code in the status word, lets its copies and
// MMAs end, frees TMEM and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "fp8.cuh"
#include "gemm_grad.cuh"
#include "gemm_sched.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxGroups = 1024;
constexpr int kMaxSmem = 232448;  // 227 KB dynamic shared memory per CTA
constexpr int kTileBytes = 128 * 128;  // of 128 rows (columns) and a block of 128 of the reduction
constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
// Registers per thread: 168 at launch (three warps in each quarter of the SM),
// then a first warpgroup of loads, MMAs and scales hands most of its own to the
// two of the epilogue, whose accumulators take 128: 128 x 56 + 256 x 224 = 384 x 168.
constexpr int kRegsLaunch = 168, kRegsFew = 56, kRegsMany = 224;
static_assert(128 * kRegsFew + 32 * kEpiWarps * kRegsMany == kThreads * kRegsLaunch, "registers");
constexpr int kStgBlock = 4096;  // staging: 32 rows of 128 bytes
// The ring, of stages of A (128 rows) and B (256), and staging per warp: GATE_UP's
// rows of a warp are 64 bytes of codes, the others' 256 or 512, 128 at a time. Four
// stages instead of three: 828 -> 809 us for GATE_UP's 341 rows.
constexpr int ring_bytes(int mode) { return (mode == kFp8GateUp ? 12 : 10) * kTileBytes; }
constexpr int stg_warp(int mode) { return mode == kFp8GateUp ? kStgBlock / 2 : kStgBlock; }
// Rows of A in a stage where no group has more, for one more stage (the MMAs read on
// past them, rows whose results nobody takes).
constexpr int kNarrowRows = 32;
constexpr int stages(int mode, bool narrow) {
  return ring_bytes(mode) / ((narrow ? kNarrowRows * 128 : kTileBytes) + 2 * kTileBytes);
}
constexpr int kScaleWarp0 = 2, kScaleWarps = 2;
constexpr int kFactorSlots = 4;               // blocks whose factors are kept
constexpr int kFactors = 384;                 // of a block: rows' (twice, or once and 256 columns')
constexpr int kColBytes = kFactorSlots * kFactors * 4 + 2048;  // and GATE_UP's row maxima: two slots of two parts
constexpr int kMostStages = 5;
constexpr int kBars = 2 * kMostStages + 5 + 4 + kEpiWarps;
constexpr int kBarBytes = (8 * kBars + 8 + 15) / 16 * 16;  // and the TMEM address and the abort flag
constexpr int kTableBytes = (kMaxGroups + 8) * 4 * 2;
constexpr int smem_of(int mode) {
  return 1024 + ring_bytes(mode) + kEpiWarps * stg_warp(mode) + kColBytes + kBarBytes + kTableBytes;
}
static_assert(smem_of(kFp8GateUp) <= kMaxSmem && smem_of(kFp8Forward) <= kMaxSmem, "shared memory");
static_assert(stages(kFp8GateUp, true) <= kMostStages && stages(kFp8Forward, true) <= kMostStages, "barriers");

struct Fp8Params {
  const int32_t* offsets;  // [G+1] or nullptr
  int G, rows;
  int N;                // columns of the result (GATE_UP: of h; WEIGHT_GRAD: rows of dw)
  int K;                // reduction (WEIGHT_GRAD: columns of dw)
  const float *sa, *sb, *sb1;  // FORWARD ..: a's, w's (gate's), up's; WEIGHT_GRAD: dy's, a's
  void* out;
  int out_f32;
  float* out_scale;     // GATE_UP
  int* status;
  uint64_t limit_ns;
};

// a: boxes of 128, 64, 32 and 16 rows (WEIGHT_GRAD: a[0] alone, of dy). out: 32
// rows of 128 bytes (GATE_UP: of 64).
struct Fp8Maps {
  CUtensorMap a[4], b0, b1, out;
};

// D (+)= A B, E4M3 inputs, fp32 accumulator (M = 128, K = 32).
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: fp32 D, E4M3 A and B.
constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// MN-major operand: 128 columns' rows of the reduction 128 bytes apart, groups of 8
// rows 1024 bytes; 32 rows are 4096 bytes.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kTileBytes >> 4) << 16;  // the next 128 columns (of B)
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Loads of the scales that stay where they are written: the compiler moves
// others down to their use, a tile or four blocks later, and waits there.
__device__ __forceinline__ float load_now(const float* p) {
  float v;
  asm volatile("ld.global.ca.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 load_now(const float4* p) {
  float4 v;
  asm volatile("ld.global.ca.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// x sigma(x) to 4 + 1.2 |x| ulp (exp's argument is rounded), and the approximate
// quotient, which is 0 past 2^126: gates below -87.3 give 0 instead of -1e-36 and less.
__device__ __forceinline__ float silu_fast(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// Bounded wait by a whole warp. The waits suspend: polling took issue slots from
// the epilogue (a tenth of the time of gate and up at 192 x 341 rows).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, int code,
                                          uint64_t limit_ns) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, status, code, limit_ns)) != 0;
}
// The same for what other CTAs of the cluster have stored (st_async): the wait
// acquires at this CTA's scope, which does not order their stores before reads
// here, so the phase is looked at once more, acquiring at the cluster's.
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status,
                                                  int code, uint64_t limit_ns) {
  if (!warp_wait(bar, parity, abort_flag, status, code, limit_ns)) return false;
  mbar_acquire_cluster(bar, parity);
  return true;
}

// ---- tensor maps (3-D: a group's matrix is cut off at its own edge)
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
  }();
  return fn;
}
// Boxes of row_bytes (the swizzle too: 64 or 128) x box_rows x 1 of [groups, outer, inner] elements of esize bytes
// (1, 2 bf16, 4 fp32).
bool make_map(CUtensorMap* m, const void* ptr, int esize, uint64_t inner, uint64_t outer, uint64_t groups, int row_bytes,
              uint32_t box_rows) {
  if (!encode_tiled()) return false;
  const cuuint64_t dims[3] = {inner, outer, groups};
  const cuuint64_t strides[2] = {inner * esize, inner * outer * esize};
  const cuuint32_t box[3] = {(cuuint32_t)(row_bytes / esize), box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType type = esize == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  return encode_tiled()(m, type, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Store to the shared memory of a CTA of the cluster (addresses from mapa_shared)
// that counts its 4 bytes on a barrier there: no release, which would wait for
// this SM's other memory traffic (3000 cycles).
__device__ __forceinline__ void st_async(uint32_t cluster_addr, uint32_t v, uint32_t cluster_bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(cluster_addr), "r"(v),
               "r"(cluster_bar)
               : "memory");
}

__device__ __forceinline__ void st_async4(uint32_t cluster_addr, float4 v, uint32_t cluster_bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   cluster_addr),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(cluster_bar)
               : "memory");
}

// A tile: group, its first row (WEIGHT_GRAD: of the padded rows), the rows it
// has there, first row and column, blocks of the reduction and the first of them
// (PARTS: this CTA's).
struct Tile {
  int g, row0, nrows, m0, n0, kb, k0;
};

// PARTS > 1: a cluster of as many CTAs has one tile, each a part of the reduction.
template <int MODE, int PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_fp8_kernel(const __grid_constant__ Fp8Maps m, const Fp8Params p) {
  constexpr bool kA_MN = MODE == kFp8WeightGrad, kB_MN = MODE == kFp8WeightGrad || MODE == kFp8Transposed;
  constexpr int kCols = MODE == kFp8GateUp ? 128 : 256;  // result columns per tile
  constexpr int kWide = stages(MODE, false), kStages = stages(MODE, true);  // kStages: the most
  constexpr int kStgWarp = stg_warp(MODE), kStgBytes = kEpiWarps * kStgWarp, kRing = ring_bytes(MODE);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
  uint8_t* base = smem_raw + pad;
  const uint32_t sm0 = raw_addr + pad;
  // Shared memory: A ring | B ring | staging | factors, maxima | barriers | tables.
  uint8_t* staging = base + kRing;
  float* factors = reinterpret_cast<float*>(staging + kStgBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStgBytes + kColBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* tile_start = reinterpret_cast<int32_t*>(staging + kStgBytes + kColBytes + kBarBytes);
  int32_t* row_start = tile_start + kMaxGroups + 8;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMostStages + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * kMostStages + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * kMostStages + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kMostStages + 4);
  auto join_bar = [&](int q) { return bar0 + 8u * (2 * kMostStages + 5 + q); };   // GATE_UP: a tile's maxima are there
  auto slice_bar = [&](int w) { return bar0 + 8u * (2 * kMostStages + 9 + w); };  // PARTS: a warp's slices are

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = PARTS > 1 ? (int)cluster_ctarank() : 0;
  const int worker = PARTS > 1 ? (int)cluster_id_x() : (int)blockIdx.x, workers = PARTS > 1 ? (int)ncluster_x() : (int)gridDim.x;
  const int G = p.G;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1 + kScaleWarps);
      mbar_init(tempty_bar(a), kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    for (int i = 0; i < 4; ++i) mbar_init(join_bar(i), 2);  // the two warps of 32 rows
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(slice_bar(i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  wait_for_previous_launch();
  allow_next_launch();
  for (int g = threadIdx.x; g <= G; g += kThreads) {
    const int v = p.offsets ? __ldcg(p.offsets + g) : (g == 0 ? 0 : p.rows);
    row_start[g] = v < 0 ? 0 : (v > p.rows ? p.rows : v);
  }
  __syncthreads();
  int most = 0;  // rows of a group
  const int n_wt = MODE == kFp8WeightGrad ? (p.N + 127) / 128 : (p.N + kCols - 1) / kCols, n_kt = (p.K + 255) / 256;
  for (int g = threadIdx.x; g < G; g += kThreads) {
    const int n = row_start[g + 1] - row_start[g];
    most = n > most ? n : most;
    // WEIGHT_GRAD: blocks of 128 rows before the group; else tiles before it.
    tile_start[g] = MODE == kFp8WeightGrad ? (n > 0 ? (n + 127) / 128 : 0) : (n > 0 ? n_wt * ((n + 127) / 128) : 0);
  }
  const bool narrow = !__syncthreads_or(MODE == kFp8WeightGrad || most > kNarrowRows);
  const int nstages = narrow ? kStages : kWide;
  const uint32_t a_step = narrow ? kNarrowRows * 128 : kTileBytes, b_ring = sm0 + nstages * a_step;
  if (warp == 0) scan_warp(tile_start, G, lane);
  tc_fence_before();
  __syncthreads();
  if (PARTS > 1) cluster_sync_all();  // the other CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // PARTS: at most one tile per cluster.
  const int all = MODE == kFp8WeightGrad ? G * n_wt * n_kt : tile_start[G], total = PARTS > 1 && all > workers ? workers : all;

  auto decode = [&](int tile) {
    Tile t;
    if (MODE == kFp8WeightGrad) {
      const int per = n_wt * n_kt;
      t.g = tile / per;
      const int at = tile - t.g * per;
      t.m0 = at / n_kt * 128;
      t.n0 = (at - at / n_kt * n_kt) * 256;
      t.row0 = tile_start[t.g] * 128;
      t.nrows = row_start[t.g + 1] - row_start[t.g];
      t.kb = t.nrows > 0 ? (t.nrows + 127) / 128 : 0;
      t.k0 = 0;
      return t;
    }
    int lo = 0, hi = G;  // tile_start[lo] <= tile < tile_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_start[mid] <= tile) lo = mid; else hi = mid;
    }
    t.g = lo;
    const int n = row_start[lo + 1] - row_start[lo], n_tt = (n + 127) / 128;
    const int local = tile - tile_start[lo], wt = local / n_tt;
    t.m0 = (local - wt * n_tt) * 128;
    t.n0 = wt * kCols;
    t.row0 = row_start[lo] + t.m0;
    t.nrows = n - t.m0;
    t.k0 = 0;
    t.kb = (p.K + 127) / 128;
    if (PARTS > 1) {
      const int per = (t.kb + PARTS - 1) / PARTS, left = t.kb - part * per;
      t.k0 = part * per;
      t.kb = left < 0 ? 0 : (left < per ? left : per);
    }
    return t;
  };
  auto box_of = [&](int n) { return n > 64 ? 128 : (n > 32 ? 64 : (n > 16 ? 32 : 16)); };  // rows of A that are loaded

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      Ring rg;
      bool ok = true;
      for (int tile = worker; ok && tile < total; tile += workers) {
        const Tile t = decode(tile);
        const int box = kA_MN ? 128 : box_of(t.nrows);
        const uint32_t bytes = (uint32_t)box * 128u + 2u * kTileBytes;
        const CUtensorMap* amap = &m.a[box == 128 ? 0 : (box == 64 ? 1 : (box == 32 ? 2 : 3))];
        for (int kb = 0; kb < t.kb; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty_bar(rg.s), rg.ph ^ 1u, abort_flag, p.status,
                                                         MOE_DEV_TIMEOUT_PRODUCER, p.limit_ns))) {
            ok = false;
            break;
          }
          const uint32_t bar = full_bar(rg.s);
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, bytes);
            const uint32_t da = sm0 + rg.s * a_step, db = b_ring + rg.s * 2 * kTileBytes, db1 = db + kTileBytes;
            const int k = (t.k0 + kb) * 128, r = t.row0 + kb * 128;
            if (kA_MN) {
              tma_load_3d(da, amap, bar, t.m0, r, 0);
              tma_load_3d(db, &m.b0, bar, t.n0, r, 0);
              tma_load_3d(db1, &m.b0, bar, t.n0 + 128, r, 0);
            } else {
              tma_load_3d(da, amap, bar, k, t.row0, 0);
              if (MODE == kFp8GateUp) {
                tma_load_3d(db, &m.b0, bar, k, t.n0, t.g);
                tma_load_3d(db1, &m.b1, bar, k, t.n0, t.g);
              } else if (kB_MN) {
                tma_load_3d(db, &m.b0, bar, t.n0, k, t.g);
                tma_load_3d(db1, &m.b0, bar, t.n0 + 128, k, t.g);
              } else {
                tma_load_3d(db, &m.b0, bar, k, t.n0, t.g);
                tma_load_3d(db1, &m.b0, bar, k, t.n0 + 128, t.g);
              }
            }
          }
          __syncwarp();
          rg.next(nstages);
        }
      }
      if (!ok) {  // let copies already issued land before the CTA leaves: 5 ms
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 5000000ull) {
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdesc = idesc_e4m3(128, 256, kA_MN, kB_MN);
      constexpr uint32_t kStepA = kA_MN ? 4096 >> 4 : 32 >> 4, kStepB = kB_MN ? 4096 >> 4 : 32 >> 4;  // 32 of k
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return warp_wait(bar, parity, abort_flag, p.status, MOE_DEV_TIMEOUT_MMA, p.limit_ns);
      };
      Ring rg;
      Ring acc;  // TMEM buffer of the block
      bool ok = true, issued = false;
      for (int tile = worker; ok && tile < total; tile += workers) {
        const Tile t = decode(tile);
        for (int kb = 0; kb < t.kb; ++kb) {
          const uint64_t da = kA_MN ? mn_desc(sm0 + rg.s * a_step) : sw128_kmajor_desc(sm0 + rg.s * a_step);
          const uint64_t db = kB_MN ? mn_desc(b_ring + rg.s * 2 * kTileBytes) : sw128_kmajor_desc(b_ring + rg.s * 2 * kTileBytes);
          if (!wait_all(full_bar(rg.s), rg.ph) || !wait_all(tempty_bar(acc.s), acc.ph ^ 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc.s * 256);
          if (elect_one()) {
            umma_e4m3(d, da, db, kIdesc, 0u);
#pragma unroll
            for (int k = 1; k < 4; ++k) umma_e4m3(d, da + k * kStepA, db + k * kStepB, kIdesc, 1u);
            umma_commit(empty_bar(rg.s));
            umma_commit(tfull_bar(acc.s));
          }
          __syncwarp();
          issued = true;
          rg.next(nstages);
          acc.next(2);
        }
      }
      if (!ok && issued && lane == 0) {  // every issued MMA is done before TMEM is freed
        umma_commit(drain_bar);
        drain_wait(drain_bar, 0, 200000000ull);
      }
    } else {
      // ------------------------------------------------------------ scales
      // The factors of each block for the epilogue: rows' for columns 0-127 and
      // 128-255 (GATE_UP: gates, ups), or rows' and columns' (WEIGHT_GRAD). A
      // block's factors complete its phase of tfull together with its MMAs. Slot
      // j % 4 is free when block j - 2 is complete: its MMAs waited for the
      // epilogue to be done with block j - 4. Loads run four blocks (WEIGHT_GRAD:
      // one) ahead.
      const int kbs = fp8_blocks(p.K), nbs = fp8_blocks(p.N);  // scales per row of a; blocks of w's columns
      const int s0 = (warp - kScaleWarp0) * 64 + lane;          // rows s0 and s0 + 32 of this CTA's 128
      Ring acc;
      int slot = 0;
      bool ok = true;
      auto hand_over = [&](auto&& write) {
        ok = warp_wait(tfull_bar(acc.s), acc.ph ^ 1u, abort_flag, p.status, MOE_DEV_TIMEOUT_EPILOGUE, p.limit_ns);
        if (!ok) return;
        write(factors + slot * kFactors);
        __syncwarp();
        if (lane == 0) mbar_arrive(tfull_bar(acc.s));
        slot = (slot + 1) % kFactorSlots;
        acc.next(2);
      };
      for (int tile = worker; ok && tile < total; tile += workers) {
        const Tile t = decode(tile);
        if (MODE == kFp8WeightGrad) {
          const int n0 = t.m0 + s0, n1 = n0 + 32, c0 = t.n0 + (warp - kScaleWarp0) * 128 + 4 * lane;
          const int c = c0 < p.K ? c0 : p.K - 4;
          const int r0 = n0 < p.N ? n0 : p.N - 1, r1 = n1 < p.N ? n1 : p.N - 1;
          const int blocks = p.rows / 128 + G;  // that there are; offsets that fall could ask for more
          struct Block {
            float a, b;
            float4 c;
          };
          auto load = [&](int kb) {
            const int at = t.row0 / 128 + (kb < t.kb ? kb : t.kb - 1);
            const size_t blk = (size_t)(at < blocks ? at : blocks - 1);
            return Block{load_now(p.sa + blk * p.N + r0), load_now(p.sa + blk * p.N + r1),
                         load_now(reinterpret_cast<const float4*>(p.sb + blk * p.K + c))};
          };
          if (t.kb == 0) continue;
          Block next = load(0);
          for (int kb = 0; ok && kb < t.kb; ++kb) {
            const Block cur = next;
            next = load(kb + 1);
            hand_over([&](float* f) {
              f[s0] = cur.a;
              f[s0 + 32] = cur.b;
              *reinterpret_cast<float4*>(f + 128 + (warp - kScaleWarp0) * 128 + 4 * lane) = cur.c;
            });
          }
        } else {
          // Rows past the group's end take its last row's scales: their results are not stored.
          const int last = t.nrows - 1;
          if (PARTS > 1 && t.kb == 0) continue;
          const float* sa0 = p.sa + (size_t)(t.row0 + (s0 < last ? s0 : last)) * kbs + t.k0;
          const float* sa1 = p.sa + (size_t)(t.row0 + (s0 + 32 < last ? s0 + 32 : last)) * kbs + t.k0;
          const int left = kbs - t.k0;  // blocks from this part's first on
          auto load_a = [&](const float* sa, int kb) {
            const int e = left - 1;
            return make_float4(load_now(sa + (kb < e ? kb : e)), load_now(sa + (kb + 1 < e ? kb + 1 : e)),
                               load_now(sa + (kb + 2 < e ? kb + 2 : e)), load_now(sa + (kb + 3 < e ? kb + 3 : e)));
          };
          const int nb = t.n0 / 128, nb1 = MODE == kFp8GateUp || nb + 1 == nbs ? nb : nb + 1;
          auto load_w = [&](const float* sb, int n, int kb) {  // a lane each for 32 blocks
            const int k = t.k0 + (kb + lane < left ? kb + lane : left - 1);
            return load_now(sb + (MODE == kFp8Transposed ? ((size_t)t.g * kbs + k) * nbs + n : ((size_t)t.g * nbs + n) * kbs + k));
          };
          const float* sb1 = MODE == kFp8GateUp ? p.sb1 : p.sb;
          float4 n0 = load_a(sa0, 0), n1 = load_a(sa1, 0);
          float w = 0.f, w1 = 0.f, w_next = load_w(p.sb, nb, 0), w1_next = load_w(sb1, nb1, 0);
          for (int kb0 = 0; ok && kb0 < t.kb; kb0 += 4) {
            if ((kb0 & 31) == 0) {
              w = w_next;
              w1 = w1_next;
              w_next = load_w(p.sb, nb, kb0 + 32);
              w1_next = load_w(sb1, nb1, kb0 + 32);
            }
            float4 c0 = n0, c1 = n1;
            n0 = load_a(sa0, kb0 + 4);
            n1 = load_a(sa1, kb0 + 4);
            const int stop = t.kb - kb0 < 4 ? t.kb : kb0 + 4;
            for (int kb = kb0; ok && kb < stop; ++kb) {
              const float x = __shfl_sync(0xFFFFFFFFu, w, kb & 31), y = __shfl_sync(0xFFFFFFFFu, w1, kb & 31);
              hand_over([&](float* f) {
                f[s0] = c0.x * x;
                f[s0 + 32] = c1.x * x;
                f[128 + s0] = c0.x * y;
                f[128 + s0 + 32] = c1.x * y;
              });
              c0 = make_float4(c0.y, c0.z, c0.w, 0.f);
              c1 = make_float4(c1.y, c1.z, c1.w, 0.f);
            }
          }
        }
      }
    }
    __syncwarp();
    if (PARTS > 1 && worker < total) cluster_sync_all();
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
    const int q = warp & 3;                      // this warp may access TMEM lanes 32q .. 32q+31
    const int half = (warp - kEpiWarp0) >> 2;    // its 128 columns (GATE_UP: 64 of gate, 64 of up)
    uint8_t* stg = staging + (warp - kEpiWarp0) * kStgWarp;
    bool idle = false;  // PARTS: the cluster's rings are
    auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(buf));
    };
    Ring acc;
    bool ok = true;
    int slot = 0;
    uint32_t joined = 0;  // GATE_UP: tiles whose maxima were put together
    for (int tile = worker; ok && tile < total; tile += workers) {
      const Tile c_t = decode(tile);
      const int r0 = q * 32;  // this warp's first row of the tile
      if (MODE != kFp8WeightGrad && c_t.nrows <= r0) {  // none of this warp's rows: keep step
        for (int kb = 0; ok && kb < c_t.kb; ++kb) {
          ok = warp_wait(tfull_bar(acc.s), acc.ph, abort_flag, p.status, MOE_DEV_TIMEOUT_EPILOGUE, p.limit_ns);
          if (ok) release(acc.s);
          acc.next(2);
          slot = (slot + 1) % kFactorSlots;
        }
        continue;
      }
      const int col0 = (MODE == kFp8GateUp ? 64 : 128) * half;  // the first column that this warp adds
      // The accumulators live in the loops below: nothing but their end and the results
      // read them, so that no copies join them with another path's.
      float sum[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sum[i] = 0.f;
      // 32 columns of a block's partial sums on their way while the 32 before are
      // added, over the blocks' borders too: the next block's wait and its first
      // load come before this one's last additions.
      uint32_t v0[32], v1[32];
      uint32_t u[2][16];  // WEIGHT_GRAD: 16 columns at a time
      uint32_t tb = 0;
      auto begin = [&] {  // wait for a block and load its first columns
        if (!warp_wait(tfull_bar(acc.s), acc.ph, abort_flag, p.status, MOE_DEV_TIMEOUT_EPILOGUE, p.limit_ns)) return false;
        tc_fence_after();
        tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc.s * 256 + col0);
        if constexpr (MODE == kFp8WeightGrad) tmem_ld_32x32b_x16(tb, u[0]);
        else tmem_ld_32x32b_x32(tb, v0);
        return true;
      };
      auto arrived = [&](uint32_t (&x)[32]) {  // used behind the wait only
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(x[i]));
      };
      float f0 = 0.f, f1 = 0.f;  // the row's factors of the block (GATE_UP: the gates', the ups')
      const float* f = nullptr;
      auto take_factors = [&] {
        f = factors + slot * kFactors;
        slot = (slot + 1) % kFactorSlots;
        f0 = f[(MODE == kFp8GateUp || MODE == kFp8WeightGrad ? 0 : half * 128) + q * 32 + lane];
        f1 = MODE == kFp8GateUp ? f[128 + q * 32 + lane] : f0;
        f += 128 + 128 * half;  // WEIGHT_GRAD: the columns'
      };
      auto add = [&](int c, float y, const uint32_t (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[32 * c + i] = fmaf(__uint_as_float(v[i]), y, sum[32 * c + i]);
      };
      if (c_t.kb > 0 && !begin()) goto done;
      if constexpr (MODE == kFp8WeightGrad) {
        // Columns' factors as well. They are read before the wait for their columns
        // (which the compiler moves no load across): with 32 columns at a time there
        // were no registers for that, and each read was waited for (192 x 341 rows, in
        // tiles of 256 rows on pairs of CTAs: 871 -> 788 us; on single ones 773). Every
        // lane reads all 128, which fills the shared memory's port (648 us without); TMEM
        // loads of 16 lanes x 256 bits, with which a lane has four rows and a quarter of
        // the columns, were no faster (798, 64 columns at a time 817).
#pragma unroll 1
        for (int kb = 0; kb < c_t.kb; ++kb) {
          take_factors();
          const float y = f0;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float4 z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = *reinterpret_cast<const float4*>(f + 16 * c + 4 * i);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(u[c & 1][i]));
            if (c < 7) {
              tmem_ld_32x32b_x16(tb + 16 * (c + 1), u[(c & 1) ^ 1]);
            } else {
              release(acc.s);
              acc.next(2);
              if (kb + 1 < c_t.kb && !begin()) goto done;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float* a = sum + 16 * c + 4 * i;
              const uint32_t* v = u[c & 1] + 4 * i;
              a[0] = fmaf(__uint_as_float(v[0]), y * z[i].x, a[0]);
              a[1] = fmaf(__uint_as_float(v[1]), y * z[i].y, a[1]);
              a[2] = fmaf(__uint_as_float(v[2]), y * z[i].z, a[2]);
              a[3] = fmaf(__uint_as_float(v[3]), y * z[i].w, a[3]);
            }
          }
        }
      } else {
        auto at = [&](int c) { return tb + (MODE == kFp8GateUp ? (c & 1) * 32 + (c >> 1) * 128 : 32 * c); };
#pragma unroll 1
        for (int kb = 0; kb < c_t.kb; ++kb) {
          take_factors();
          arrived(v0);
          tmem_ld_32x32b_x32(at(1), v1);
          add(0, f0, v0);
          arrived(v1);
          tmem_ld_32x32b_x32(at(2), v0);
          add(1, f0, v1);
          arrived(v0);
          tmem_ld_32x32b_x32(at(3), v1);
          add(2, f1, v0);
          arrived(v1);
          release(acc.s);
          acc.next(2);
          if (kb + 1 < c_t.kb && !begin()) goto done;
          add(3, f1, v1);
        }
      }
      if constexpr (PARTS > 1) {
        // The parts' sums are put together: each CTA takes a slice of every warp's
        // columns, a warp's 32 rows of it from the same warp of the other CTAs, through
        // its ring, which is idle by then (16 bytes of 32 rows at a time: 512 bytes in
        // order).
        constexpr int kKinds = MODE == kFp8GateUp ? 2 : 1;       // gates and ups
        constexpr int kN = 32 / kKinds, kPer = kN / PARTS;       // groups of four columns: of the warp, of a slice
        cluster_sync_all();
        idle = true;
        auto place = [&](int from, int c) { return base + ((from * kEpiWarps + warp - kEpiWarp0) * (kPer * kKinds) + c) * 512 + lane * 16; };
        const uint32_t bar = slice_bar(warp - kEpiWarp0);
        if (lane == 0) mbar_arrive_expect_tx(bar, PARTS * kPer * kKinds * 512);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const int to = c % kN / kPer;
          st_async4(mapa_shared(smem_u32(place(part, c / kN * kPer + c % kPer)), to),
                    make_float4(sum[4 * c], sum[4 * c + 1], sum[4 * c + 2], sum[4 * c + 3]), mapa_shared(bar, to));
        }
        if (!warp_wait_cluster(bar, 0, abort_flag, p.status, MOE_DEV_TIMEOUT_EPILOGUE, p.limit_ns)) goto done;
        float x[4 * kPer * kKinds];
#pragma unroll
        for (int c = 0; c < kPer * kKinds; ++c) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < PARTS; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(place(i, c));
            v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
          }
          x[4 * c] = v.x;
          x[4 * c + 1] = v.y;
          x[4 * c + 2] = v.z;
          x[4 * c + 3] = v.w;
        }
        const int r = r0 + lane, first = c_t.n0 + col0 + part * kPer * 4;
        const bool live = r < c_t.nrows;
        const size_t row = (size_t)(c_t.row0 + r) * p.N + first;
        if constexpr (MODE == kFp8GateUp) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 4 * kPer; ++i) {
            x[i] = silu_fast(x[i]) * x[4 * kPer + i];
            const uint32_t b = fp8_abs_bits(x[i]);
            top = b > top ? b : top;
          }
          // The maxima of each CTA's warps go to all CTAs, behind the slices.
          uint32_t* tops = reinterpret_cast<uint32_t*>(base + 8 * kTileBytes) + q * 32 + lane;
          if (lane == 0) {
            if (half == 0) mbar_arrive_expect_tx(join_bar(q), PARTS * 2 * 32 * 4);
            else mbar_arrive(join_bar(q));
          }
#pragma unroll
          for (int to = 0; to < PARTS; ++to)
            st_async(mapa_shared(smem_u32(tops + (2 * part + half) * 128), to), top, mapa_shared(join_bar(q), to));
          if (!warp_wait_cluster(join_bar(q), 0, abort_flag, p.status, MOE_DEV_TIMEOUT_EPILOGUE, p.limit_ns)) goto done;
#pragma unroll
          for (int i = 0; i < 2 * PARTS; ++i) {
            const uint32_t t = tops[i * 128];
            top = t > top ? t : top;
          }
          const Fp8Block blk(fp8_scale(top));
          if (live && half == 0 && part == 0) p.out_scale[(size_t)(c_t.row0 + r) * fp8_blocks(p.N) + c_t.n0 / 128] = blk.scale;
          fp8_by_size(blk.small(), [&](auto small) {
#pragma unroll
            for (int c = 0; c < kPer; ++c)
              if (live && first + 4 * c < p.N)
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row + 4 * c) =
                    blk.code4<decltype(small)::value>(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          });
        } else {
#pragma unroll
          for (int c = 0; c < kPer; ++c) {
            if (!live || first + 4 * c >= p.N) break;
            if (p.out_f32)
              *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row + 4 * c) =
                  make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
            else
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row + 4 * c) =
                  make_uint2(pack_bf16(x[4 * c], x[4 * c + 1]), pack_bf16(x[4 * c + 2], x[4 * c + 3]));
          }
        }
        __syncwarp();
        continue;
      }
      // Results go out by TMA from the warp's staging (the tensor maps' swizzles),
      // while the next tile is summed: stores from the warps held them up for as
      // long as three blocks (an SM stores 32 bytes a cycle). A group's last rows,
      // fewer than 32, are stored by the warp; WEIGHT_GRAD's map ends where a
      // group's matrix does.
      const int live_rows = MODE == kFp8WeightGrad ? p.N - c_t.m0 : c_t.nrows;
      const bool whole = MODE == kFp8WeightGrad || r0 + 32 <= live_rows;
      const int width = MODE == kFp8WeightGrad ? p.K : p.N;
      auto reuse = [&] {  // the staging's last copies have left
        if (lane == 0) bulk_wait_group_read0();
        __syncwarp();
      };
      // The staging: `bytes` (64 or 128) of each row, from column col of `esize` bytes on.
      auto send = [&](int bytes, int esize, int col) {
        if (whole) {
          if (lane == 0 && col < width && r0 < live_rows) {
            if (MODE == kFp8WeightGrad) tma_store_3d(&m.out, smem_u32(stg), col, c_t.m0 + r0, c_t.g);
            else tma_store_3d(&m.out, smem_u32(stg), col, c_t.row0 + r0, 0);
            bulk_commit_group();
          }
          return;
        }
        const int per = bytes / 16, c = col + 16 / esize * (lane % per);  // 16-byte chunks of a row
        uint8_t* out = static_cast<uint8_t*>(p.out) + ((size_t)(c_t.row0 + r0) * width + c) * esize;
        for (int i = lane / per; i < 32; i += 32 / per) {
          const int chunk = (lane % per) ^ (bytes == 128 ? i & 7 : (i >> 1) & 3);
          const uint4 v = *reinterpret_cast<const uint4*>(stg + i * bytes + 16 * chunk);
          if (c < width && r0 + i < live_rows) *reinterpret_cast<uint4*>(out + (size_t)i * width * esize) = v;
        }
      };
      if (MODE == kFp8GateUp) {
        // h of 64 columns; the block's largest is the largest of the two warps', in two
        // slots by turns: the other warp may still read the last tile's.
        uint32_t top = 0;
        auto finish = [&](float g, float u) {
          const float x = silu_fast(g) * u;
          const uint32_t b = fp8_abs_bits(x);
          top = b > top ? b : top;
          return x;
        };
        uint32_t* tops = reinterpret_cast<uint32_t*>(factors + kFactorSlots * kFactors) + q * 32 + lane;
#pragma unroll
        for (int i = 0; i < 64; ++i) sum[i] = finish(sum[i], sum[64 + i]);
        tops += (joined & 1) * 256;
        tops[half * 128] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(join_bar(q));
        ok = warp_wait(join_bar(q), joined & 1u, abort_flag, p.status, MOE_DEV_TIMEOUT_EPILOGUE, p.limit_ns);
        if (!ok) goto done;
        ++joined;
        const uint32_t other = *reinterpret_cast<volatile uint32_t*>(tops + (half ^ 1) * 128);
        top = other > top ? other : top;
        const float scale = fp8_scale(top);
        const int r = r0 + lane;
        if (half == 0 && r < c_t.nrows)
          p.out_scale[(size_t)(c_t.row0 + r) * fp8_blocks(p.N) + c_t.n0 / 128] = scale;
        const Fp8Block blk(scale);
        reuse();
        fp8_by_size(blk.small(), [&](auto small) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 16 codes
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 16 * c + 4 * i;
              w[i] = blk.code4<decltype(small)::value>(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
            }
            *reinterpret_cast<uint4*>(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        });
        fence_proxy_async_smem();
        __syncwarp();
        send(64, 1, c_t.n0 + col0);
      } else {
        const int c0 = c_t.n0 + col0;
        uint8_t* mine = stg + lane * 128;
        if (p.out_f32) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {  // 32 columns
            reuse();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float* x = sum + 32 * g + 4 * j;
              *reinterpret_cast<float4*>(mine + ((j ^ (lane & 7)) << 4)) = make_float4(x[0], x[1], x[2], x[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            send(128, 4, c0 + 32 * g);
          }
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g) {  // 64
            reuse();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float* x = sum + 64 * g + 8 * j;
              *reinterpret_cast<uint4*>(mine + ((j ^ (lane & 7)) << 4)) =
                  make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            send(128, 2, c0 + 64 * g);
          }
        }
      }
    }
  done:
    tmem_ld_wait();
    bulk_wait_group0();
    __syncwarp();
    if (PARTS > 1 && worker < total && !idle) cluster_sync_all();
  }

  // The CTAs of a cluster arrive here only when their roles are done (every wait is
  // bounded), so none leaves while another may still write to its shared memory.
  tc_fence_before();
  __syncwarp();
  if (PARTS > 1) {
    cluster_sync_all();
    if (*abort_flag) {  // the others' last stores and arrivals here land: 5 ms
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 5000000ull) {
      }
    }
  } else {
    __syncthreads();
  }
  __syncwarp();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// CTAs that share each tile's reduction, where there are few tiles: as many as make
// one wave (clusters of eight: 15, of four: 36 and more). The exchange of the sums
// costs about 2 us for up to 32 rows (K = 4096, 15 tiles: 15.3 us, in four parts 9.0,
// in eight 8.2; K = 1024: 7.1, 6.7, 6.9; 30 tiles 7.2, 7.4), 4 for 64 (K = 2048 and
// 1024, 30 tiles: 10.6, in four parts 11.2; 16 tiles 10.4, 10.0 and 7.5, 9.3), 8 for
// 128 (K = 4096: 16.9, 17.3). The order of the sums is the parts', so the sizes and the
// device decide, not how many SMs the call may take: few tiles take one wave of the
// device all the same.
int parts_of(long long tiles, int rows, int blocks, int num_sms) {
  if (rows > 64 || tiles > 36 || blocks < (rows > 32 ? 20 : 10)) return 1;
  if (tiles <= 15 && blocks >= 24 && 8 * tiles <= num_sms) return 8;
  return 4 * tiles <= num_sms ? 4 : 1;
}

template <int MODE>
cudaError_t run_fp8(const Fp8GemmArgs& a, cudaStream_t s) {
  const int G = a.offsets ? a.G : 1;
  Fp8Maps m = {};
  bool ok = true;
  if (MODE == kFp8WeightGrad) {
    const uint64_t P = fp8_padded_rows(a.rows, G);
    ok = make_map(&m.a[0], a.a, 1, a.N, P, 1, 128, 128) && make_map(&m.b0, a.w0, 1, a.K, P, 1, 128, 128);
    for (int i = 1; i < 4; ++i) m.a[i] = m.a[0];
  } else {
    for (int i = 0; ok && i < 4; ++i) ok = make_map(&m.a[i], a.a, 1, a.K, a.rows, 1, 128, 128u >> i);
    const uint64_t inner = MODE == kFp8Transposed ? a.N : a.K, outer = MODE == kFp8Transposed ? a.K : a.N;
    ok = ok && make_map(&m.b0, a.w0, 1, inner, outer, G, 128, 128);
    if (MODE == kFp8GateUp) ok = ok && make_map(&m.b1, a.w1, 1, inner, outer, G, 128, 128);
  }
  if (MODE != kFp8GateUp) m.b1 = m.b0;
  if (MODE == kFp8GateUp) ok = ok && make_map(&m.out, a.out, 1, a.N, a.rows, 1, 64, 32);
  else if (MODE == kFp8WeightGrad) ok = ok && make_map(&m.out, a.out, a.out_f32 ? 4 : 2, a.K, a.N, G, 128, 32);
  else ok = ok && make_map(&m.out, a.out, a.out_f32 ? 4 : 2, a.N, a.rows, 1, 128, 32);
  if (!ok) return cudaErrorInvalidValue;
  Fp8Params p = {};
  p.offsets = a.offsets;
  p.G = G;
  p.rows = a.rows;
  p.N = a.N;
  p.K = a.K;
  p.sa = a.a_scale;
  p.sb = a.s0;
  p.sb1 = a.s1;
  p.out = a.out;
  p.out_f32 = a.out_f32;
  p.out_scale = a.out_scale;
  p.status = a.status;
  p.limit_ns = a.wait_limit_ns;
  const int cols = MODE == kFp8GateUp ? 128 : 256;
  const long long n_wt = (a.N + cols - 1) / cols;
  auto launch = [&](auto kernel, long long tiles, int parts) {
    const long long grid = parts > 1 ? parts * tiles : (tiles < a.num_sms ? tiles : a.num_sms);
    return launch_dependent(kernel, (int)grid, kThreads, smem_of(MODE), s, true, /*cluster=*/parts, m, p);
  };
  if constexpr (MODE == kFp8WeightGrad) {
    return launch(grouped_gemm_fp8_kernel<MODE, 1>, (long long)G * ((a.N + 127) / 128) * ((a.K + 255) / 256), 1);
  } else {
    const long long tiles = n_wt * (a.rows / 128 + (G < a.rows ? G : a.rows));  // at most: of groups that have rows
    const int parts = parts_of(tiles, a.rows, fp8_blocks(a.K), a.device_sms);
    if (parts == 8) return launch(grouped_gemm_fp8_kernel<MODE, 8>, tiles, 8);
    if (parts == 4) return launch(grouped_gemm_fp8_kernel<MODE, 4>, tiles, 4);
    return launch(grouped_gemm_fp8_kernel<MODE, 1>, tiles, 1);
  }
}

template <int MODE, int PARTS>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(grouped_gemm_fp8_kernel<MODE, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(MODE));
}

}  // namespace

cudaError_t gemm_fp8_prepare_device() {
  const cudaError_t errs[] = {allow_smem<kFp8Forward, 1>(),    allow_smem<kFp8Forward, 4>(),    allow_smem<kFp8Forward, 8>(),
                              allow_smem<kFp8Transposed, 1>(), allow_smem<kFp8Transposed, 4>(), allow_smem<kFp8Transposed, 8>(),
                              allow_smem<kFp8GateUp, 1>(),     allow_smem<kFp8GateUp, 4>(),     allow_smem<kFp8GateUp, 8>(),
                              allow_smem<kFp8WeightGrad, 1>()};
  for (cudaError_t e : errs)
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, int mode, cudaStream_t s) {
  if (mode != kFp8WeightGrad && a.rows == 0) return cudaSuccess;
  switch (mode) {
    case kFp8Forward: return run_fp8<kFp8Forward>(a, s);
    case kFp8Transposed: return run_fp8<kFp8Transposed>(a, s);
    case kFp8GateUp: return run_fp8<kFp8GateUp>(a, s);
    case kFp8WeightGrad: return run_fp8<kFp8WeightGrad>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace moe
