// Gradient of the grouped SwiGLU expert products (step 3), bf16 operands, fp32
// accumulation on the 5th-generation tensor cores. For the rows r of group g,
// with a the rows' inputs and dy the gradient of their outputs:
//
//   gate = a Wg^T, up = a Wu^T, h = silu(gate) * up, y = h Wd^T   (the forward)
//   Q  (DOWN):   q = dy Wd                                        [rows, I] fp32
//   GU (SWIGLU): gate and up once more, then
//                h = silu(gate) up;  du = q silu(gate);
//                dg = q up sigma(gate) (1 + gate (1 - sigma(gate)))  [rows, I] bf16
//   DX (INPUT):  da = dg Wg + du Wu                               [rows, H] bf16
//   and, in gemm_grad_dw.cu, dWd = dy^T h;  dWg = dg^T a;  dWu = du^T a   per group
//
// 16 rows H I FLOP in all: 12 for the gradient and 4 to recompute gate and up,
// which the forward does not keep. q stays fp32 between the launches; h, dg
// and du are rounded to bf16 once, as the tensor cores read them (the results
// are then 2.35e-3 of their norm off, 1.7e-3 of it by their own rounding to
// bf16; low halves in a second product would double the MMAs of DX and DW,
// which keep the tensor cores busy for 60 to 70% of their time).
//
// One kernel, three modes. Persistent, a pair of CTAs on the two SMs of a TPC
// per tile (tcgen05 .cta_group::2): the weights are the M = 256 rows of the MMA,
// 128 in each SM, and a chunk of up to 256 of the group's rows (tokens) is N,
// half loaded by each SM. A group of n rows is cut into ceil(n / 256) chunks of
// about one size, each rounded up to 32: 341 rows take 192 + 160. With the
// tokens as M instead, a tile of 128 rows on one SM, 341 rows take 384, and an
// SM takes in 48 KB per 64 elements of the reduction for 512 cycles of MMAs
// (it can take in about 64 bytes a cycle); the pair's tile costs it at most
// 32 KB. In TMEM an accumulator's lane is a weight row (an output feature), its
// column a token; two accumulators of 256 columns.
//
// Operands. The forward's weights are K-major for the forward products; Q and
// DX reduce over their other axis, so they are read MN-major from the same
// row-major tensors, with no transposed copy: a box of 64 columns x 64 rows
// lands as 64 rows (the reduction axis) of 128 swizzled bytes, the tensor
// cores' MN-major operand layout, and the instruction descriptor's transpose
// bit is set.
//   mode  A (M: weights)                   B (N: tokens)              reduction
//   Q     Wd columns, MN-major             dy rows, K-major           H
//   GU    64 Wg rows, 64 Wu rows, K-major  a rows, K-major            H
//   DX    Wg, then Wu columns, MN-major    dg rows, then du rows      I, twice
//
// Roles per CTA (12 warps, each walking its tiles in step with warp-uniform
// values and one elected lane issuing): 0 loads A's boxes and arms the stage,
// 6 and 7 load B's (a box costs its issuer 100 to 150 cycles, a stage's MMAs
// take 330 at 341 rows per group), 1 (of the
// even CTA, the leader) issues the pair's MMAs, 2-5 and 8-11 are the epilogue,
// 32 accumulator lanes and every other block of 32 tokens each. Both CTAs'
// copies of a stage complete on the leader's full barrier. In GU lanes 0-63
// hold the gates and 64-127 the ups of the same 64 features: the warps of lane
// quarters q and q + 2 exchange half of each block through shared memory and
// finish 16 tokens each.
//
// Measured at 192 experts x 341 rows, H = 4096, I = 1536 (short runs): Q 0.63,
// GU 1.24, DX 1.18 ms. Alone, their HBM traffic (3.4, 6.4 and 5.8 GB, mostly
// the weights, once per launch) takes 0.50, 0.94 and 0.85 ms at a copy's rate,
// and their MMAs 0.38, 0.75 and 0.75. Tiles of two chunks that share a stage of
// weights read 29% less from L2, but leave no accumulator for the next tile
// while the epilogue reads theirs: 0.60, 1.29 and 1.08 ms, and 7% more for the
// pass at uneven loads. A ring of more and smaller stages where the chunks are
// short changed nothing.
//
// Every wait is bounded; on expiry the CTA records an error code in the status
// word, lets its in-flight copies and MMAs end, frees TMEM and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "gemm_grad.cuh"
#include "gemm_sched.cuh"
#include "internal.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

enum GradMode { kQ = 0, kGU = 1, kDX = 2 };

constexpr int kBK = 64;  // reduction elements per stage
constexpr int kMaxGroups = 1024;
constexpr int kMaxSmem = 232448;  // 227 KB dynamic shared memory per CTA
constexpr int kMaxN = 256;        // tokens per tile
constexpr int kABytes = 128 * 128;         // 128 weight rows (or columns) x 64
constexpr int kBBytes = kMaxN / 2 * 128;   // half of the tokens x 64
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kStages = 6;
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kExchange = kEpiWarps * 2048;  // GU: per epilogue warp 16 tokens x 32 features
constexpr int kBarBytes = 8 * (2 * kStages + 5) + 24;
constexpr int kTableBytes = (kMaxGroups + 8) * (4 + 4 + 2 + 2);  // tile starts, row starts, padding, order
constexpr int kSmem = 1024 + kStages * kStageBytes + kExchange + kBarBytes + kTableBytes;
constexpr uint16_t kPairMask = 0x3;
static_assert(kBarBytes % 16 == 0 && kSmem <= kMaxSmem, "shared memory");

struct GradParams {
  KParams k;              // offsets, G, rows, status, limit_ns; N = weight rows or columns (output features)
  int H, I;
  int num_kb;             // stages per tile (Q, GU: H / 64; DX: 2 I / 64)
  float* q;               // [rows, I]
  __nv_bfloat16 *h, *dg, *du;  // [prows, I], padded (padded_rows)
  int prows;
  bool after_dw;          // DX: the launch before is the weight gradients', else GU
  ChainWords chain;
  int* odd;               // set where gate or q is not finite
  __nv_bfloat16* da;      // [rows, H]
};

// a0 / a1: the weights; b0 / b1: the rows, in boxes of 64, 32, 16 and 8 rows.
// Q: Wd; dy. GU: Wg, Wu; a. DX: Wg, Wu; dg, du.
struct GradMaps {
  CUtensorMap a0, a1, b0[4], b1[4];
};
__device__ __forceinline__ int pow2_below(int n) { return 1 << (31 - __clz(n - 1)); }  // the largest, n >= 2
__device__ __forceinline__ int box_map(int rows) { return __clz(rows) - 25; }

// Tokens of chunk c of a group of n rows: [first, first + count), and the MMA's
// N. (A chunk is at most 256, so the last one is never empty.)
struct Chunk {
  int first, count, N;
};
__device__ __forceinline__ Chunk chunk_of(int n, int c) {
  const int chunks = (n + kMaxN - 1) / kMaxN;
  const int size = ((n + chunks - 1) / chunks + 31) & ~31;
  Chunk k;
  k.first = c * size;
  k.count = n - k.first < size ? n - k.first : size;
  k.N = (k.count + 31) & ~31;
  return k;
}

// All threads of `threads` (a multiple of 32) agree: true if every one says so.
__device__ __forceinline__ bool agree(int id, int threads, bool mine) {
  int all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 q, %3, 0;\n\t"
      "bar.red.and.pred p, %1, %2, q;\n\t"
      "selp.s32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"((int)mine)
      : "memory");
  return all != 0;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_grad_kernel(const __grid_constant__ GradMaps m, const GradParams p) {
  constexpr int kTileM = MODE == kGU ? 128 : 256;  // output features per pair tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
  uint8_t* base = smem_raw + pad;
  const uint32_t base_u32 = raw_addr + pad;
  // Shared memory (the same in both CTAs): ring | exchange | barriers | tables.
  float* exchange = reinterpret_cast<float*>(base + kStages * kStageBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + kStages * kStageBytes + kExchange);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* early_flag = abort_flag + 1;
  int32_t* tile_start = reinterpret_cast<int32_t*>(base + kStages * kStageBytes + kExchange + kBarBytes);
  int32_t* row_start = tile_start + kMaxGroups + 8;
  // Group g's first row in h, dg and du (gemm_grad.cuh) is row_start[g] -
  // row_start[0] + pad_extra[g].
  uint16_t* pad_extra = reinterpret_cast<uint16_t*>(row_start + kMaxGroups + 8);
  // Groups by the size of their chunks, largest first; tile_start is in that
  // order. Tiles are dealt to the pairs forwards and backwards in turn, which
  // keeps the pairs' shares of unequal tiles within a fraction of a tile.
  uint16_t* order = pad_extra + kMaxGroups + 8;
  int32_t* pads = reinterpret_cast<int32_t*>(base);  // until the loop starts
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };                       // leader: both CTAs' stage s
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };          // each CTA
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * kStages + a); };      // each CTA
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * kStages + 2 + a); };  // leader
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: leader
  const int pair = (int)cluster_id_x(), npairs = (int)ncluster_x();
  const int G = p.k.G;
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
  // Blocks of the launch before may still be running (programmatic dependent
  // launch). Q waits for its end, here, and publishes that it has: the caller's
  // operands are complete. GU and DX need no more than that to begin; DX after
  // the weight gradients finds the word that those publish, and with it GU's
  // results.
  if (MODE == kQ) {
    wait_for_previous_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      *p.odd = 0;
      *p.chain.gu_done = 0;
      publish(p.chain.inputs_ready, p.chain.call);
    }
  } else {
    wait_until_published(MODE == kDX && p.after_dw ? p.chain.gu_done : p.chain.inputs_ready, p.chain.call, early_flag);
  }
  allow_next_launch();

  // ---- tables: row starts; tile_start[g] = tiles of groups before g; padding.
  fill_row_start_coherent(p.k, row_start, threadIdx.x, kThreads);
  const int n_wt = (p.k.N + kTileM - 1) / kTileM;
  __syncthreads();
  auto rows_of = [&](int g) {
    const int n = row_start[g + 1] - row_start[g];
    return n > 0 ? n : 0;
  };
  int32_t* sizes = pads + kMaxGroups + 8;  // until the loop starts
  for (int g = threadIdx.x; g < G; g += kThreads) {
    const int n = rows_of(g);
    pads[g] = pad16(n) - n;
    sizes[g] = n > 0 ? chunk_of(n, 0).N : 0;
  }
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += kThreads) {
    const int size = sizes[g];
    int at = 0;
    for (int j = 0; j < G; ++j) {
      const int o = sizes[j];
      at += (o > size || (o == size && j < g)) ? 1 : 0;
    }
    order[at] = (uint16_t)g;
    tile_start[at] = n_wt * ((rows_of(g) + kMaxN - 1) / kMaxN);
  }
  __syncthreads();
  if (warp == 0) scan_warp(tile_start, G, lane);
  if (warp == 2) {
    scan_warp(pads, G, lane);
    __syncwarp();
    for (int g = lane; g < G; g += 32) pad_extra[g] = (uint16_t)pads[g];
  }
  // pads' bytes become a stage: written by the async proxy from here on.
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers and TMEM are there
  tc_fence_after();
  // Each role waits for the end of the launch before where it first needs its
  // results, or where it would start to wait for a role that does. GU's operands
  // do not come from Q, only its epilogue's q does: two tiles of MMAs fit before
  // it. In DX a ring of weights does; after the weight gradients, which let it
  // start when GU is done, DX waits for nothing but, at the end, for them. Every
  // CTA waits, so a launch's end is the end of all before it. Against every
  // thread of every launch waiting for the launch before at its top (us): 128
  // tokens, 2 of 8 experts, H = 1024, I = 512 44.5 -> 31.6; 64 tokens, 2 of 16,
  // H = 512, I = 256 35.5 -> 23.5; 40 tokens, 3 of 20, H = 1600, I = 1024 130 ->
  // 116; 2048 tokens, 4 of 64, H = 4096, I = 1536 1210 -> 1140; 341 rows for each
  // of 192 experts the same.
  const bool at_once = MODE == kDX && p.after_dw;
  const uint32_t tmem_base = *tmem_slot;
  const int total = tile_start[G];
  auto tile_of = [&](int i) { return i * npairs + ((i & 1) ? npairs - 1 - pair : pair); };
  const int rounds = (total + npairs - 1) / npairs;
  const int my_tiles = rounds > 0 && tile_of(rounds - 1) >= total ? rounds - 1 : rounds;  // the last round may be short

  // This pair's tiles, decoded 32 at a time, one by each lane of a role's warp,
  // and read back by shuffles.
  struct Tile {
    int g, wt, row, prow, count, N, npad;  // npad: count and the zero rows after a group's last token
  };
  auto decode = [&](int i) {
    Tile t = {};
    if (i >= my_tiles) return t;
    const int tile = tile_of(i);
    int lo = 0, hi = G;  // tile_start[lo] <= tile < tile_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_start[mid] <= tile) lo = mid; else hi = mid;
    }
    const int local = tile - tile_start[lo];
    lo = order[lo];
    const int n = rows_of(lo), chunks = (n + kMaxN - 1) / kMaxN;
    t.g = lo;
    t.wt = local / chunks;
    const Chunk c = chunk_of(n, local - t.wt * chunks);
    t.row = row_start[lo] + c.first;
    t.prow = row_start[lo] - row_start[0] + pad_extra[lo] + c.first;
    t.count = c.count;
    t.N = c.N;
    t.npad = c.first + c.count == n ? pad16(n) - c.first : c.count;
    return t;
  };
  auto at_tile = [&](int v, int i) { return __shfl_sync(0xFFFFFFFFu, v, i & 31); };

  if (warp == 0 || warp == 6 || warp == 7) {
    // ------------------------------------------------------------ producers
    const bool is_a = warp == 0;
    const uint32_t bar_base = rank == 0 ? bar0 : mapa_shared(bar0, 0);  // the leader's full barriers
    Ring rg;
    bool ok = true;
    Tile mine = {};
    for (int i = 0; ok && i < my_tiles; ++i) {
      if (MODE == kDX ? i == 0 && !is_a && !at_once : MODE == kGU && i == 2) wait_for_previous_launch();
      if ((i & 31) == 0) mine = decode(i + lane);
      const int g = at_tile(mine.g, i), wt = at_tile(mine.wt, i), half = at_tile(mine.N, i) >> 1;
      const int row = at_tile(MODE == kDX ? mine.prow : mine.row, i) + (int)rank * half;
      // B's `half` rows (a multiple of 16, at most 128): the largest power of
      // two below that by warp 6, the rest by warp 7. Both have a box in every
      // stage: a warp without one could fall behind by two rounds of the ring,
      // where a wait by parity would miss the phase that it waits for.
      const int most = pow2_below(half), rest = half - most, second_box = pow2_below(rest + 1);
      const int at = warp == 6 ? 0 : most, box = warp == 6 ? most : second_box;
      const int extra = warp == 6 ? 0 : rest - second_box;  // 48 = 32 + 16
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (MODE == kDX && is_a && !at_once && i * p.num_kb + kb == kStages) wait_for_previous_launch();
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty_bar(rg.s), rg.ph ^ 1u, abort_flag, p.k.status,
                                                       MOE_DEV_TIMEOUT_PRODUCER, p.k.limit_ns))) {
          ok = false;
          break;
        }
        // DX: the first half of the stages is dg Wg, the second du Wu.
        const bool second = MODE == kDX && kb >= (p.num_kb >> 1);
        const int kx = (second ? kb - (p.num_kb >> 1) : kb) * kBK;
        const uint32_t bar = bar_base + 8u * rg.s;
        const uint32_t sa = base_u32 + rg.s * kStageBytes, sb = sa + kABytes;
        if (elect_one()) {
          if (is_a) {
            // Both CTAs' bytes (the other's may land first).
            if (rank == 0) mbar_arrive_expect_tx(full_bar(rg.s), 2u * (kABytes + (uint32_t)half * 128u));
            if (MODE == kGU) {
              const int f = g * p.I + wt * kTileM + (int)rank * 64;
              tma_load_2d_pair(sa, &m.a0, bar, kx, f);
              tma_load_2d_pair(sa + kChunk, &m.a1, bar, kx, f);
            } else {
              const CUtensorMap* map = second ? &m.a1 : &m.a0;
              const int f = wt * kTileM + (int)rank * 128, krow = g * (MODE == kQ ? p.H : p.I) + kx;
              tma_load_2d_pair(sa, map, bar, f, krow);
              tma_load_2d_pair(sa + kChunk, map, bar, f + 64, krow);
            }
          } else {
            const CUtensorMap* map = second ? m.b1 : m.b0;
            tma_load_2d_pair(sb + at * 128, map + box_map(box), bar, kx, row + at);
            if (extra) tma_load_2d_pair(sb + (at + box) * 128, map + box_map(extra), bar, kx, row + at + box);
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
      constexpr uint32_t kIdesc = idesc_bf16_f32(256, 0) | (MODE == kGU ? 0u : 1u << 15);
      constexpr uint32_t kStepA = MODE == kGU ? 32 >> 4 : 2048 >> 4, kStepB = 32 >> 4;
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
        return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, p.k.status, MOE_DEV_TIMEOUT_MMA,
                                                         p.k.limit_ns)) != 0;
      };
      Ring rg;
      bool ok = true, issued = false;
      int n32 = 0;
      for (int i = 0; ok && i < my_tiles; ++i) {
        if (i == (MODE == kGU ? 2 : 0) && !at_once) wait_for_previous_launch();
        if ((i & 31) == 0) n32 = decode(i + lane).N;
        const int N = at_tile(n32, i);
        const int acc = i & 1;
        const uint32_t ap = (uint32_t)(i >> 1) & 1u;
        if (!wait_all(tempty_bar(acc), ap ^ 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc * kMaxN);
        const uint32_t idesc = kIdesc | (uint32_t)(N >> 3) << 17;
        for (int kb = 0; kb < p.num_kb; ++kb) {
          const uint32_t sa = base_u32 + rg.s * kStageBytes;
          const uint64_t da = MODE == kGU ? sw128_kmajor_desc(sa) : sw128_mnmajor_desc(sa);
          const uint64_t db = sw128_kmajor_desc(sa + kABytes);
          if (!wait_all(full_bar(rg.s), rg.ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            umma_bf16_pair(d, da, db, idesc, kb ? 1u : 0u);
#pragma unroll
            for (int k = 1; k < kBK / 16; ++k) umma_bf16_pair(d, da + k * kStepA, db + k * kStepB, idesc, 1u);
            umma_commit_pair_mc(empty_bar(rg.s), kPairMask);
          }
          __syncwarp();
          issued = true;
          rg.next(kStages);
        }
        if (!ok) break;
        if (elect_one()) umma_commit_pair_mc(tfull_bar(acc), kPairMask);
        __syncwarp();
      }
      if (!ok && issued && lane == 0) {  // every issued MMA is done before TMEM is freed
        umma_commit_pair(drain_bar);
        drain_wait(drain_bar, 0, 200000000ull);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;             // this warp may access TMEM lanes 32q .. 32q+31
    const int half = warp >= 8 ? 1 : 0;  // its blocks of 32 tokens: every other one
    const int partners = 1 + (q & 1) + 2 * half;  // named barrier of warps q and q ^ 2
    Tile mine = {};
    float odd = 0.0f;  // GU: turns NaN where a gate or q is not finite
    if (!at_once) wait_for_previous_launch();
    for (int i = 0; i < my_tiles; ++i) {
      if ((i & 31) == 0) mine = decode(i + lane);
      const int wt = at_tile(mine.wt, i), count = at_tile(mine.count, i), N = at_tile(mine.N, i);
      const int row = at_tile(mine.row, i), prow = at_tile(mine.prow, i);
      int npad = at_tile(mine.npad, i);
      if (prow < 0 || npad > p.prows - prow) npad = 0;  // (offsets that decrease: no store outside)
      const int acc = i & 1;
      const uint32_t ap = (uint32_t)(i >> 1) & 1u;
      const int gu_f0 = wt * kTileM + (int)rank * 64;
      if (MODE == kGU && gu_f0 < p.I) {
        // This CTA's q of the tile (256 bytes a token) into L2 while the tile's
        // MMAs run: q is larger than L2, and from HBM a block's loads took 5000
        // cycles under load, longer than everything else here.
        const char* qt = reinterpret_cast<const char*>(p.q + (size_t)row * p.I + gu_f0);
        for (int x = (half * 4 + q) * 32 + lane; x < 2 * count; x += 32 * kEpiWarps)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(qt + (size_t)(x >> 1) * p.I * 4 + (x & 1) * 128));
      }
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded(tfull_bar(acc), ap, abort_flag, p.k.status, MOE_DEV_TIMEOUT_EPILOGUE, p.k.limit_ns) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (MODE == kGU) ok = agree(partners, 64, ok != 0);  // partners leave together
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kMaxN);
      if (MODE == kGU) {
        const int f0 = gu_f0 + (q & 1) * 32;  // (64 features: all inside I or none)
        const bool gate_warp = q < 2;
        const int j0 = gate_warp ? 0 : 16;  // the 16 tokens of a block that this warp finishes
        float* mine_ex = exchange + (half * 4 + q) * 512;
        const float* other_ex = exchange + (half * 4 + (q ^ 2)) * 512 + lane;
        uint16_t* stg = reinterpret_cast<uint16_t*>(mine_ex);
        if (f0 < p.I) {
          const float* qp = p.q + (size_t)(row + j0) * p.I + f0 + lane;
          float nq[16];  // q of the next block's 16 tokens
          auto load_q = [&](int c) {
            const float* at = qp + (size_t)c * p.I;
#pragma unroll
            for (int j = 0; j < 16; ++j, at += p.I) nq[j] = c + j0 + j < count ? *at : 0.0f;
          };
          load_q(32 * half);
#pragma unroll 1
          for (int c = 32 * half; c < N; c += 64) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tb + c, v);
            tmem_ld_wait();
            float own[16], other[16], qv[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              own[j] = __uint_as_float(gate_warp ? v[j] : v[16 + j]);
              mine_ex[j * 32 + lane] = __uint_as_float(gate_warp ? v[16 + j] : v[j]);
              qv[j] = nq[j];
            }
            if (c + 64 < N) load_q(c + 64);
            named_sync(partners, 64);
#pragma unroll
            for (int j = 0; j < 16; ++j) other[j] = other_ex[j * 32];
            named_sync(partners, 64);  // both have read: each buffer is its warp's own again
            // The 16 x 32 results of h and dg, then of du, go out through that
            // buffer: 64-byte rows, eight tokens per store instruction.
            const int live = count - (c + j0);  // tokens of the group among the 16
            uint32_t du[8];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float gt = gate_warp ? own[j] : other[j], up = gate_warp ? other[j] : own[j];
              const float sg = __fdividef(1.0f, 1.0f + __expf(-gt));
              const float act = gt * sg, qs = qv[j] * sg;
              // An infinity or NaN in the row of a or of dy leaves none of its
              // gate values, or of its q values, finite. (One of the next
              // group's, in a token past this one's, does no harm.)
              odd = fmaf(0.0f, gt, fmaf(0.0f, qv[j], odd));
              uint16_t h = __bfloat16_as_ushort(__float2bfloat16_rn(act * up));
              uint16_t dg = __bfloat16_as_ushort(__float2bfloat16_rn(qs * up * fmaf(gt, 1.0f - sg, 1.0f)));
              uint16_t d = __bfloat16_as_ushort(__float2bfloat16_rn(qs * gt));
              if (j >= live) h = dg = d = 0;
              stg[j * 32 + lane] = h;
              stg[512 + j * 32 + lane] = dg;
              du[j >> 1] = j & 1 ? du[j >> 1] | (uint32_t)d << 16 : (uint32_t)d;
            }
            const size_t at = (size_t)(prow + c + j0) * p.I + f0 + (lane & 3) * 8;
            auto put = [&](__nv_bfloat16* dst, const uint16_t* src) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int t = (lane >> 2) + 8 * u;
                if (c + j0 + t < npad)
                  *reinterpret_cast<uint4*>(dst + at + (size_t)t * p.I) =
                      *reinterpret_cast<const uint4*>(src + t * 32 + (lane & 3) * 8);
              }
            };
            __syncwarp();
            put(p.h, stg);
            put(p.dg, stg + 512);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 16; ++j) stg[j * 32 + lane] = (uint16_t)(du[j >> 1] >> (16 * (j & 1)));
            __syncwarp();
            put(p.du, stg);
            __syncwarp();
          }
        }
      } else {
        const int cols = MODE == kQ ? p.I : p.H;
        const int f0 = wt * kTileM + (int)rank * 128 + q * 32;  // (32 features: all inside or none)
        if (f0 < cols) {
          const size_t at = (size_t)row * cols + f0 + lane;
          auto put = [&](size_t o, uint32_t v) {
            if (MODE == kQ) p.q[o] = __uint_as_float(v);
            else p.da[o] = __float2bfloat16_rn(__uint_as_float(v));
          };
#pragma unroll 1
          for (int c = 32 * half; c < count; c += 64) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(tb + c, v);
            tmem_ld_wait();
            size_t o = at + (size_t)c * cols;
            if (c + 32 <= count) {
#pragma unroll
              for (int j = 0; j < 32; ++j, o += cols) put(o, v[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j, o += cols)
                if (c + j < count) put(o, v[j]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(tempty_bar(acc));
        else mbar_arrive_remote(mapa_shared(tempty_bar(acc), 0));
      }
    }
    if (MODE == kGU && odd != 0.0f) *p.odd = 1;
  }

  if (at_once) wait_for_previous_launch();
  // DX ends the chain. (A thread that has waited; a block of DX that finds the
  // word cleared waits itself.)
  if (MODE == kDX && blockIdx.x == 0 && warp == 2 && lane == 0) *p.chain.inputs_ready = 0;
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

// row_chunks: an upper bound on the groups' chunks.
template <int MODE>
int pairs_of(const GradParams& p, long long row_chunks, int num_sms) {
  constexpr int kTileM = MODE == kGU ? 128 : 256;
  const long long tiles = row_chunks * ((p.k.N + kTileM - 1) / kTileM);
  return (int)(tiles < num_sms / 2 ? tiles : num_sms / 2);
}

template <int MODE>
cudaError_t run_mode(const GradMaps& m, const GradParams& p, long long row_chunks, int num_sms, cudaStream_t s) {
  const int pairs = pairs_of<MODE>(p, row_chunks, num_sms);
  if (pairs < 1) return cudaErrorInvalidValue;
  return launch_dependent(grouped_grad_kernel<MODE>, 2 * pairs, kThreads, kSmem, s, true, /*cluster=*/2, m, p);
}

template <int MODE>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(grouped_grad_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

// The maps of a [rows, cols] tensor in boxes of 64, 32, 16 and 8 rows.
bool row_maps(CUtensorMap (&m)[4], const void* ptr, uint64_t cols, uint64_t rows) {
  for (int i = 0; i < 4; ++i)
    if (!make_tmap_bf16(&m[i], ptr, cols, rows, 64u >> i)) return false;
  return true;
}

}  // namespace

cudaError_t gemm_grad_prepare_device() {
  const cudaError_t errs[] = {set_smem<kQ>(), set_smem<kGU>(), set_smem<kDX>(), gemm_grad_dw_prepare_device()};
  for (cudaError_t e : errs)
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

cudaError_t launch_grouped_swiglu_backward(const GroupedGradArgs& a, cudaStream_t s) {
  const int G = a.offsets ? a.G : 1, H = a.H, I = a.I;
  const bool want_dw = a.dw_gate != nullptr;
  if (a.rows == 0) {  // no operand to map: every weight gradient is zero
    cudaError_t e = cudaSuccess;
    const size_t bytes = (size_t)G * H * I * 2;
    for (void* d : {a.dw_gate, a.dw_up, a.dw_down})
      if (d && e == cudaSuccess) e = cudaMemsetAsync(d, 0, bytes, s);
    return e;
  }
  GradParams p = {};
  p.k.offsets = a.offsets;
  p.k.G = G;
  p.k.rows = a.rows;
  p.k.status = a.status;
  p.k.limit_ns = a.wait_limit_ns;
  p.k.fold_group = -1;
  p.H = H;
  p.I = I;
  p.q = a.q;
  p.h = static_cast<__nv_bfloat16*>(a.h);
  p.dg = static_cast<__nv_bfloat16*>(a.dg);
  p.du = static_cast<__nv_bfloat16*>(a.du);
  p.prows = (int)padded_rows(a.rows, G);
  p.odd = a.odd;
  p.chain = a.chain;
  p.da = static_cast<__nv_bfloat16*>(a.da);
  const uint64_t R = a.rows, P = p.prows, GI = (uint64_t)G * I, GH = (uint64_t)G * H;
  const long long row_chunks = (a.rows + kMaxN - 1) / kMaxN + (long long)G;  // at most: one short chunk per group
  cudaError_t e = cudaSuccess;
  {
    GradMaps m = {};
    if (!make_tmap_bf16(&m.a0, a.w_down, I, GH, 64) || !row_maps(m.b0, a.dy, H, R)) return cudaErrorInvalidValue;
    p.k.N = I;
    p.num_kb = H / kBK;
    e = run_mode<kQ>(m, p, row_chunks, a.num_sms, s);
  }
  if (e == cudaSuccess) {
    GradMaps m = {};
    if (!make_tmap_bf16(&m.a0, a.w_gate, H, GI, 64) || !make_tmap_bf16(&m.a1, a.w_up, H, GI, 64) ||
        !row_maps(m.b0, a.a, H, R))
      return cudaErrorInvalidValue;
    p.k.N = I;
    p.num_kb = H / kBK;
    e = run_mode<kGU>(m, p, row_chunks, a.num_sms, s);
  }
  p.k.N = H;
  p.num_kb = 2 * (I / kBK);
  p.after_dw = want_dw;
  if (e == cudaSuccess && want_dw)
    e = launch_grouped_weight_grad(a, a.da ? pairs_of<kDX>(p, row_chunks, a.num_sms) : 0, s);
  if (e == cudaSuccess && a.da) {
    GradMaps m = {};
    if (!make_tmap_bf16(&m.a0, a.w_gate, H, GI, 64) || !make_tmap_bf16(&m.a1, a.w_up, H, GI, 64) ||
        !row_maps(m.b0, a.dg, I, P) || !row_maps(m.b1, a.du, I, P))
      return cudaErrorInvalidValue;
    e = run_mode<kDX>(m, p, row_chunks, a.num_sms, s);
  }
  return e;
}

}  // namespace moe
