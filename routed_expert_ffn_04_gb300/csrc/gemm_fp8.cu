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
// A tile is 256 rows x 256 columns on a pair of CTAs (the two SMs of a TPC,
// cta_group::2): each CTA holds 128 rows of A and half of B, 32 KB per block of
// 128, and its TMEM the partial sums of its 128 rows, double-buffered (2 x 256
// columns, all of it). A thread's accumulators are 128 columns of one row: its
// factor is one number per block (two for GATE_UP). Rows (tokens) as M make the
// factor, SwiGLU and the quantisation of a row of h local to a thread; a group's
// last tile costs its whole MMAs (341 rows take 512), which matters only past 256
// rows per group, below that the weights' bytes take longer (16 KB per SM and
// block: 700 cycles of its share of HBM against 512 of MMAs).
//
// TRANSPOSED and WEIGHT_GRAD read operands MN-major from the row-major tensors,
// with no transposed copy: a box of 128 columns x 128 rows lands as 128 rows of
// 128 swizzled bytes, 8 rows (1024 bytes) per step of the layout, 32 rows per MMA.
//
// Roles per CTA (12 warps, each walking its tiles in step): 0 loads, 1 (of the
// even CTA, the leader) issues the pair's MMAs, 4-11 are the epilogue: TMEM lanes
// 32 (w % 4) .., columns 128 ((w - 4) / 4) ... Both CTAs' copies of a stage
// complete on the leader's full barrier. Every wait is bounded; on expiry the
// CTA records a code in the status word, lets its copies and MMAs end, frees
// TMEM and exits.
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
constexpr int kHalf = 128 * 128;  // a CTA's A, or B, of a stage
constexpr int kStages = 5;
constexpr int kEpiWarps = 8;
constexpr int kEpiWarp0 = 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
// Registers per thread: 168 at launch (three warps in each quarter of the SM),
// then a first warpgroup of loads and MMAs hands most of its own to the two of
// the epilogue, whose accumulators take 128: 128 x 56 + 256 x 224 = 384 x 168.
constexpr int kRegsFew = 56, kRegsMany = 224;
static_assert(128 * kRegsFew + 32 * kEpiWarps * kRegsMany == kThreads * 168, "registers");
constexpr int kStgBytes = kEpiWarps * 4096;   // staging: 32 rows of 128 bytes per warp
constexpr int kColBytes = kEpiWarps * 2 * 512;  // WEIGHT_GRAD: column factors of a block, twice; GATE_UP: row maxima
constexpr int kBars = 2 * kStages + 5;
constexpr int kBarBytes = 8 * kBars + 8;  // and the TMEM address and the abort flag
constexpr int kTableBytes = (kMaxGroups + 8) * 4 * 2;
constexpr int kSmem = 1024 + 2 * kStages * kHalf + kStgBytes + kColBytes + kBarBytes + kTableBytes;
constexpr uint16_t kPairMask = 0x3;
static_assert(kSmem <= kMaxSmem && kBarBytes % 16 == 0, "shared memory");

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

// a: boxes of 128, 64, 32 and 16 rows (WEIGHT_GRAD: a[0] alone, of dy).
struct Fp8Maps {
  CUtensorMap a[4], b0, b1;
};

// D (+)= A B over the CTA pair, E4M3 inputs, fp32 accumulator (M = 256, K = 32).
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: fp32 D, E4M3 A and B.
constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// MN-major operand of 128 columns: rows of the reduction 128 bytes apart, groups
// of 8 rows 1024 bytes; 32 rows are 4096 bytes.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kHalf >> 4) << 16;  // the next 128 columns: there are none
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                                 int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Two fp32 at a time. volatile: they stay behind the wait for their TMEM load.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ void add_scaled(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t factor) {
  asm volatile(
      "{\n\t.reg .b64 p;\n\t"
      "mov.b64 p, {%1, %2};\n\t"
      "fma.rn.f32x2 %0, p, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(factor));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A tile: group, its first row (WEIGHT_GRAD: of the padded rows), the rows it
// has there, first column, blocks of the reduction.
struct Tile {
  int g, row0, nrows, m0, n0, kb;
};

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_fp8_kernel(const __grid_constant__ Fp8Maps m, const Fp8Params p) {
  constexpr bool kA_MN = MODE == kFp8WeightGrad, kB_MN = MODE == kFp8WeightGrad || MODE == kFp8Transposed;
  constexpr int kCols = MODE == kFp8GateUp ? 128 : 256;  // result columns per tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
  uint8_t* base = smem_raw + pad;
  const uint32_t sm0 = raw_addr + pad;
  // Shared memory (the same in both CTAs): A ring | B ring | staging | column factors | barriers | tables.
  const uint32_t b_ring = sm0 + kStages * kHalf;
  uint8_t* staging = base + 2 * kStages * kHalf;
  float* cols = reinterpret_cast<float*>(staging + kStgBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStgBytes + kColBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* tile_start = reinterpret_cast<int32_t*>(staging + kStgBytes + kColBytes + kBarBytes);
  int32_t* row_start = tile_start + kMaxGroups + 8;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };                    // leader: both CTAs' stage s
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };       // each CTA
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * kStages + a); };   // each CTA
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * kStages + 2 + a); };  // leader
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: leader
  const int pair = (int)cluster_id_x(), npairs = (int)ncluster_x();
  const int G = p.G;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {  // one warp of each CTA of the pair, together
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  wait_for_previous_launch();
  allow_next_launch();
  for (int g = threadIdx.x; g <= G; g += kThreads) {
    const int v = p.offsets ? __ldcg(p.offsets + g) : (g == 0 ? 0 : p.rows);
    row_start[g] = v < 0 ? 0 : (v > p.rows ? p.rows : v);
  }
  __syncthreads();
  const int n_wt = (p.N + kCols - 1) / kCols, n_kt = (p.K + 255) / 256;
  for (int g = threadIdx.x; g < G; g += kThreads) {
    const int n = row_start[g + 1] - row_start[g];
    // WEIGHT_GRAD: blocks of 128 rows before the group; else tiles before it.
    tile_start[g] = MODE == kFp8WeightGrad ? (n > 0 ? (n + 127) / 128 : 0) : (n > 0 ? n_wt * ((n + 255) / 256) : 0);
  }
  __syncthreads();
  if (warp == 0) scan_warp(tile_start, G, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers and TMEM are there
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = MODE == kFp8WeightGrad ? G * n_wt * n_kt : tile_start[G];

  auto decode = [&](int tile) {
    Tile t;
    if (MODE == kFp8WeightGrad) {
      const int per = n_wt * n_kt;
      t.g = tile / per;
      const int at = tile - t.g * per;
      t.m0 = at / n_kt * 256;
      t.n0 = (at - at / n_kt * n_kt) * 256;
      t.row0 = tile_start[t.g] * 128;
      t.nrows = row_start[t.g + 1] - row_start[t.g];
      t.kb = t.nrows > 0 ? (t.nrows + 127) / 128 : 0;
      return t;
    }
    int lo = 0, hi = G;  // tile_start[lo] <= tile < tile_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_start[mid] <= tile) lo = mid; else hi = mid;
    }
    t.g = lo;
    const int n = row_start[lo + 1] - row_start[lo], n_tt = (n + 255) / 256;
    const int local = tile - tile_start[lo], wt = local / n_tt;
    t.m0 = (local - wt * n_tt) * 256;
    t.n0 = wt * kCols;
    t.row0 = row_start[lo] + t.m0;
    t.nrows = n - t.m0;
    t.kb = (p.K + 127) / 128;
    return t;
  };
  // Rows of A that CTA r of the pair has in a tile, and the box that covers them (0: none).
  auto rows_of = [&](const Tile& t, int r) {
    const int n = t.nrows - 128 * r;
    return n < 0 ? 0 : (n > 128 ? 128 : n);
  };
  auto box_of = [&](int n) { return n > 64 ? 128 : (n > 32 ? 64 : (n > 16 ? 32 : (n > 0 ? 16 : 0))); };

  if (warp < kEpiWarp0) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    Ring rg;
    bool ok = true;
    for (int tile = pair; ok && tile < total; tile += npairs) {
      const Tile t = decode(tile);
      const int box = kA_MN ? 128 : box_of(rows_of(t, (int)rank));
      const int boxes = kA_MN ? 256 : box_of(rows_of(t, 0)) + box_of(rows_of(t, 1));
      const uint32_t bytes = (uint32_t)boxes * 128u + 2u * kHalf;
      const CUtensorMap* amap = &m.a[kA_MN || box == 128 ? 0 : (box == 64 ? 1 : (box == 32 ? 2 : 3))];
      const CUtensorMap* bmap = MODE == kFp8GateUp && rank == 1 ? &m.b1 : &m.b0;
      const int bn = t.n0 + (MODE == kFp8GateUp ? 0 : (int)rank * 128);
      for (int kb = 0; kb < t.kb; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty_bar(rg.s), rg.ph ^ 1u, abort_flag, p.status,
                                                       MOE_DEV_TIMEOUT_PRODUCER, p.limit_ns))) {
          ok = false;
          break;
        }
        const uint32_t full = full_bar(rg.s);
        const uint32_t bar = rank == 0 ? full : mapa_shared(full, 0);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(bar, bytes);  // both CTAs' bytes (the other's may land first)
          const uint32_t da = sm0 + rg.s * kHalf, db = b_ring + rg.s * kHalf;
          if (kA_MN) {
            tma_load_2d_pair(da, amap, bar, t.m0 + (int)rank * 128, t.row0 + kb * 128);
            tma_load_2d_pair(db, bmap, bar, bn, t.row0 + kb * 128);
          } else {
            if (box) tma_load_2d_pair(da, amap, bar, kb * 128, t.row0 + (int)rank * 128);
            if (kB_MN) tma_load_3d_pair(db, bmap, bar, bn, kb * 128, t.g);
            else tma_load_3d_pair(db, bmap, bar, kb * 128, bn, t.g);
          }
        }
        __syncwarp();
        rg.next(kStages);
      }
    }
    if (!ok) {  // let copies already issued land before the CTA leaves: 5 ms
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 5000000ull) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      constexpr uint32_t kIdesc = idesc_e4m3(256, 256, kA_MN, kB_MN);
      constexpr uint32_t kStepA = kA_MN ? 4096 >> 4 : 32 >> 4, kStepB = kB_MN ? 4096 >> 4 : 32 >> 4;  // 32 of k
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
        return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, p.status, MOE_DEV_TIMEOUT_MMA,
                                                         p.limit_ns)) != 0;
      };
      Ring rg;
      Ring acc;  // TMEM buffer of the block
      bool ok = true, issued = false;
      for (int tile = pair; ok && tile < total; tile += npairs) {
        const Tile t = decode(tile);
        for (int kb = 0; kb < t.kb; ++kb) {
          const uint64_t da = kA_MN ? mn_desc(sm0 + rg.s * kHalf) : sw128_kmajor_desc(sm0 + rg.s * kHalf);
          const uint64_t db = kB_MN ? mn_desc(b_ring + rg.s * kHalf) : sw128_kmajor_desc(b_ring + rg.s * kHalf);
          if (!wait_all(tempty_bar(acc.s), acc.ph ^ 1u) || !wait_all(full_bar(rg.s), rg.ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc.s * 256);
          if (elect_one()) {
            umma_e4m3_pair(d, da, db, kIdesc, 0u);
#pragma unroll
            for (int k = 1; k < 4; ++k) umma_e4m3_pair(d, da + k * kStepA, db + k * kStepB, kIdesc, 1u);
            umma_commit_pair_mc(empty_bar(rg.s), kPairMask);
            umma_commit_pair_mc(tfull_bar(acc.s), kPairMask);
          }
          __syncwarp();
          issued = true;
          rg.next(kStages);
          acc.next(2);
        }
      }
      if (!ok && issued && lane == 0) {  // every issued MMA is done before TMEM is freed
        umma_commit_pair(drain_bar);
        drain_wait(drain_bar, 0, 200000000ull);
      }
    }
  }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
    const int q = warp & 3;                      // this warp may access TMEM lanes 32q .. 32q+31
    const int half = (warp - kEpiWarp0) >> 2;    // its 128 columns (GATE_UP: 64 of gate, 64 of up)
    uint8_t* stg = staging + (half * 4 + q) * 4096;
    float* colf = cols + (half * 4 + q) * 256;   // WEIGHT_GRAD: two blocks' factors
    const int kbs = fp8_blocks(p.K);             // a's scales per row
    const int nbs = fp8_blocks(p.N);
    const bool vec = (kbs & 3) == 0;
    const uint32_t tempty0 = rank == 0 ? tempty_bar(0) : mapa_shared(tempty_bar(0), 0);
    auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(tempty0 + 8u * buf);
        else mbar_arrive_remote(tempty0 + 8u * buf);
      }
    };
    Ring acc;
    int ok = 1, seq = 0;
    for (int tile = pair; ok && tile < total; tile += npairs, ++seq) {
      const Tile t = decode(tile);
      const int r = (int)rank * 128 + q * 32 + lane;  // row of the tile
      uint64_t sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      // One block: wait, take the partial sums out, 32 columns loading while 32 are added.
      auto block = [&](auto&& factor) {
        if (lane == 0)
          ok = mbar_wait_bounded(tfull_bar(acc.s), acc.ph, abort_flag, p.status, MOE_DEV_TIMEOUT_EPILOGUE, p.limit_ns) ? 1 : 0;
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) return;
        tc_fence_after();
        const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc.s * 256);
        // GATE_UP: columns 64 half .. of the gates (0-127) and of the ups (128-255).
        auto at = [&](int c) { return MODE == kFp8GateUp ? tb + 64 * half + (c & 1) * 32 + (c >> 1) * 128 : tb + 128 * half + 32 * c; };
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(at(0), v[0]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < 3) tmem_ld_32x32b_x32(at(c + 1), v[(c + 1) & 1]);
          else release(acc.s);
#pragma unroll
          for (int i = 0; i < 16; ++i) add_scaled(sum[16 * c + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], factor(c, i));
          if (c < 3) tmem_ld_wait();
        }
        acc.next(2);
      };
      if (MODE != kFp8WeightGrad) {
        const bool live = r < t.nrows;
        if (t.nrows <= (int)rank * 128 + q * 32) {  // none of this warp's rows: keep step
          for (int kb = 0; ok && kb < t.kb; ++kb) {
            if (lane == 0)
              ok = mbar_wait_bounded(tfull_bar(acc.s), acc.ph, abort_flag, p.status, MOE_DEV_TIMEOUT_EPILOGUE, p.limit_ns) ? 1 : 0;
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (ok) release(acc.s);
            acc.next(2);
          }
          continue;
        } else {
          const float* sa = p.sa + (size_t)(t.row0 + r) * kbs;
          auto load4 = [&](int kb) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!live || kb >= kbs) return v;
            if (vec) return __ldca(reinterpret_cast<const float4*>(sa + kb));
            v.x = __ldca(sa + kb);
            if (kb + 1 < kbs) v.y = __ldca(sa + kb + 1);
            if (kb + 2 < kbs) v.z = __ldca(sa + kb + 2);
            if (kb + 3 < kbs) v.w = __ldca(sa + kb + 3);
            return v;
          };
          // w's scales of this warp's 128 columns: block nb, every kb.
          const int nb0 = t.n0 / 128 + (MODE == kFp8GateUp ? 0 : half), nb = nb0 < nbs ? nb0 : nbs - 1;
          const size_t step = MODE == kFp8Transposed ? nbs : 1;
          const size_t first = MODE == kFp8Transposed ? (size_t)t.g * kbs * nbs + nb : ((size_t)t.g * nbs + nb) * kbs;
          float4 next = load4(0);
          float wl = 0.f, wl1 = 0.f;
          for (int kb0 = 0; ok && kb0 < t.kb; kb0 += 4) {
            if ((kb0 & 31) == 0) {  // a lane each for the next 32 blocks
              const int kb = kb0 + lane;
              wl = kb < t.kb ? __ldca(p.sb + first + kb * step) : 0.f;
              if (MODE == kFp8GateUp) wl1 = kb < t.kb ? __ldca(p.sb1 + first + kb * step) : 0.f;
            }
            float4 cur = next;
            next = load4(kb0 + 4);
            const int stop = t.kb - kb0 < 4 ? t.kb : kb0 + 4;
#pragma unroll 1
            for (int kb = kb0; ok && kb < stop; ++kb) {
              const float f0 = cur.x * __shfl_sync(0xFFFFFFFFu, wl, kb & 31);
              const uint64_t g0 = pack2(f0, f0);
              if (MODE == kFp8GateUp) {
                const float f1 = cur.x * __shfl_sync(0xFFFFFFFFu, wl1, kb & 31);
                const uint64_t g1 = pack2(f1, f1);
                block([&](int c, int) { return c < 2 ? g0 : g1; });
              } else {
                block([&](int, int) { return g0; });
              }
              cur = make_float4(cur.y, cur.z, cur.w, 0.f);
            }
          }
        }
      } else {
        const int n = t.m0 + r, c0 = t.n0 + 128 * half;
        const size_t blk = (size_t)tile_start[t.g];
        auto load_row = [&](int kb) { return kb < t.kb && n < p.N ? __ldca(p.sa + (blk + kb) * p.N + n) : 0.f; };
        auto load_col = [&](int kb) {
          const int c = c0 + 4 * lane;
          return kb < t.kb && c < p.K ? __ldca(reinterpret_cast<const float4*>(p.sb + (blk + kb) * p.K + c))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        float row = load_row(0);
        float4 col = load_col(0);
        for (int kb = 0; ok && kb < t.kb; ++kb) {
          float* slot = colf + (kb & 1) * 128;
          *reinterpret_cast<float4*>(slot + 4 * lane) = col;
          __syncwarp();
          const uint64_t f = pack2(row, row);
          row = load_row(kb + 1);
          col = load_col(kb + 1);
          block([&](int c, int i) { return mul2(f, *reinterpret_cast<const uint64_t*>(slot + 32 * c + 2 * i)); });
        }
        __syncwarp();
      }
      if (!ok) break;

      const int live_rows = MODE == kFp8WeightGrad ? p.N - t.m0 : t.nrows;
      const int r0 = (int)rank * 128 + q * 32;  // this warp's first row of the tile
      if (MODE == kFp8GateUp) {
        // h of 64 columns; the block's largest is the larger of the two halves'.
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 g = unpack2(sum[i]), u = unpack2(sum[32 + i]);
          const float a = silu_f(g.x) * u.x, b = silu_f(g.y) * u.y;
          sum[i] = pack2(a, b);
          const uint32_t x = fp8_abs_bits(a), y = fp8_abs_bits(b);
          top = x > top ? x : top;
          top = y > top ? y : top;
        }
        // Two slots by turns: the other warp may still read the last tile's.
        uint32_t* tops = reinterpret_cast<uint32_t*>(cols) + (seq & 1) * 256;
        tops[half * 128 + q * 32 + lane] = top;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
        const uint32_t other = tops[(half ^ 1) * 128 + q * 32 + lane];
        const float scale = fp8_scale(top > other ? top : other);
        if (half == 0 && r < t.nrows) p.out_scale[(size_t)(t.row0 + r) * nbs + t.n0 / 128] = scale;
        const Fp8Block blk(scale);
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 16 codes: chunk c of the row's 64 bytes, at c ^ (row / 2) % 4
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = unpack2(sum[8 * c + 2 * i]), b = unpack2(sum[8 * c + 2 * i + 1]);
            w[i] = blk.code4(a.x, a.y, b.x, b.y);
          }
          *reinterpret_cast<uint4*>(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        uint8_t* out = static_cast<uint8_t*>(p.out);
        const int col = t.n0 + 64 * half + 16 * (lane & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // eight rows' 64 bytes per instruction
          const int i = 8 * j + (lane >> 2);
          const uint4 v = *reinterpret_cast<const uint4*>(stg + i * 64 + (((lane & 3) ^ ((i >> 1) & 3)) << 4));
          if (r0 + i < t.nrows && col < p.N) *reinterpret_cast<uint4*>(out + (size_t)(t.row0 + r0 + i) * p.N + col) = v;
        }
        __syncwarp();
      } else {
        // Through the warp's staging, 128 bytes of each of 32 rows at a time (16-byte
        // chunk j of row i at j ^ i % 8), then four whole rows per store instruction.
        const size_t row_first = MODE == kFp8WeightGrad ? (size_t)t.g * p.N + t.m0 : (size_t)t.row0;
        const int width = MODE == kFp8WeightGrad ? p.K : p.N;
        const int c0 = t.n0 + 128 * half;
        auto flush = [&](uint8_t* at, int esize, int col) {  // at: this lane's column in row row_first + r0
          __syncwarp();
          const bool in = col < width;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int i = 4 * j + (lane >> 3);
            const uint4 v = *reinterpret_cast<const uint4*>(stg + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
            if (in && r0 + i < live_rows) *reinterpret_cast<uint4*>(at + (size_t)i * width * esize) = v;
          }
          __syncwarp();
        };
        uint8_t* srow = stg + lane * 128;
        if (p.out_f32) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c0 + 32 * c >= width) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 a = unpack2(sum[16 * c + 2 * j]), b = unpack2(sum[16 * c + 2 * j + 1]);
              *reinterpret_cast<float4*>(srow + ((j ^ (lane & 7)) << 4)) = make_float4(a.x, a.y, b.x, b.y);
            }
            const int col = c0 + 32 * c + 4 * (lane & 7);
            flush(static_cast<uint8_t*>(p.out) + ((row_first + r0) * width + col) * 4, 4, col);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (c0 + 64 * c >= width) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 a = unpack2(sum[32 * c + 4 * j + i]);
                w[i] = pack_bf16(a.x, a.y);
              }
              *reinterpret_cast<uint4*>(srow + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            const int col = c0 + 64 * c + 8 * (lane & 7);
            flush(static_cast<uint8_t*>(p.out) + ((row_first + r0) * width + col) * 2, 2, col);
          }
        }
      }
    }
  }

  // Both CTAs arrive here only when their roles are done (every wait is
  // bounded), so neither frees TMEM or leaves while the other may still touch
  // its shared memory or barriers.
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int MODE>
cudaError_t run_fp8(const Fp8GemmArgs& a, cudaStream_t s) {
  const int G = a.offsets ? a.G : 1;
  Fp8Maps m = {};
  bool ok = true;
  if (MODE == kFp8WeightGrad) {
    const uint64_t P = fp8_padded_rows(a.rows, G);
    ok = make_tmap_u8(&m.a[0], a.a, a.N, P, 128) && make_tmap_u8(&m.b0, a.w0, a.K, P, 128);
    for (int i = 1; i < 4; ++i) m.a[i] = m.a[0];
  } else {
    for (int i = 0; ok && i < 4; ++i) ok = make_tmap_u8(&m.a[i], a.a, a.K, a.rows, 128u >> i);
    const uint64_t inner = MODE == kFp8Transposed ? a.N : a.K, outer = MODE == kFp8Transposed ? a.K : a.N;
    ok = ok && make_tmap_u8_3d(&m.b0, a.w0, inner, outer, G, 128);
    if (MODE == kFp8GateUp) ok = ok && make_tmap_u8_3d(&m.b1, a.w1, inner, outer, G, 128);
  }
  if (MODE != kFp8GateUp) m.b1 = m.b0;
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
  const long long tiles = MODE == kFp8WeightGrad ? G * n_wt * ((a.K + 255) / 256) : n_wt * (a.rows / 256 + G);
  const long long most = a.num_sms / 2;
  const int pairs = (int)(tiles < most ? tiles : most);
  if (pairs < 1) return cudaErrorInvalidValue;
  return launch_dependent(grouped_gemm_fp8_kernel<MODE>, 2 * pairs, kThreads, kSmem, s, true, /*cluster=*/2, m, p);
}

}  // namespace

cudaError_t gemm_fp8_prepare_device() {
  const cudaError_t errs[] = {
      cudaFuncSetAttribute(grouped_gemm_fp8_kernel<kFp8Forward>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem),
      cudaFuncSetAttribute(grouped_gemm_fp8_kernel<kFp8Transposed>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem),
      cudaFuncSetAttribute(grouped_gemm_fp8_kernel<kFp8GateUp>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem),
      cudaFuncSetAttribute(grouped_gemm_fp8_kernel<kFp8WeightGrad>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)};
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
