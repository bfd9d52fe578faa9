// Weight gradients of the grouped SwiGLU expert products, per group g:
//   dWd[g] = dy^T h   [H, I]      dWg[g] = dg^T a,  dWu[g] = du^T a   [I, H]
// The reduction runs over the group's rows (rows offsets[g] .. offsets[g+1]-1),
// bf16 operands, fp32 accumulation, bf16 results.
//
// Both operands are read MN-major from row-major tensors (boxes of 64 columns
// by 64 rows, see gemm_grad.cu). Tiles of 256 x 256 results are computed by a
// pair of CTAs on the two SMs of a TPC (tcgen05 .cta_group::2): each holds 128
// of the M columns and half of the N columns, 32 KB per 64 rows, and in its
// TMEM its 128 rows of the result, double-buffered.
//
// Why pairs: an SM takes in about 64 bytes a cycle for loads and 32 for stores,
// and a result tile is short here (rows per expert / 16 MMAs). A 128 x 256 tile
// on one SM costs 48 KB of loads per 64 rows, which with the result's 64 KB
// outlasts its MMAs; the pair's tile costs each SM 32 KB for the same MMAs.
//
// Work is dealt in strips: up to four tiles of one group side by side, which
// share their A columns. A group of up to 64 rows per stage of the A ring (384)
// keeps A in shared memory for the whole strip, and its later tiles load only
// B: 16 KB per 64 rows. Longer groups, which are bound by their MMAs, have
// strips of one tile; so do all when there are few (fewer than eight strips per
// pair), to keep the pairs' shares even.
//
// Measured at 192 experts x 341 rows, H = 4096, I = 1536 (short runs): one SM
// per tile 2.45 ms, pairs 2.30, tiles decoded by lanes 2.22, no clearing 1.96,
// strips 1.89, stores from the warps instead of by TMA 1.83 (8.9 GB of HBM
// traffic: 1.32 ms at a copy's rate; 2.47 TFLOP: 1.33 ms at the burst rate of
// a large bf16 product).
//
// A group's rows end anywhere; the MMA runs in steps of 16 rows. One operand of
// each product is h, dg or du, whose groups are followed by zero rows up to a
// multiple of 16, so whatever finite rows of the next group the other operand
// holds there adds nothing. A zero times an infinity or NaN would: when the
// launch before has met one (p.odd), the rows past the group's end are
// cleared in shared memory first (the careful way: 0.26 ms more at the
// size above, as every tile's last stage waits for it). The launch before looks
// at groups' rows alone, and rows after the last group may hold anything: a
// group whose last step reaches one of them always goes the careful way. A
// group without rows gives zero gradients.
//
// Roles per CTA (12 warps): 0 loads A's boxes and arms the stage; 6 loads B's;
// 1 (of the even CTA, the leader) issues the pair's MMAs; 11 clears ragged
// stages (the careful way); 2-5 and 7-10 store the result, 32 rows by 64 columns at a time. A
// stage's copies in both CTAs complete on the leader's full barrier; a ragged
// stage's on each CTA's own tail barrier, whose clearing warp then arrives on
// the leader's full barrier. Every wait is bounded.
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

constexpr int kBK = 64;  // rows per stage
constexpr int kMaxGroups = 1024;
constexpr int kMaxSmem = 232448;       // 227 KB dynamic shared memory per CTA
constexpr int kHalfBytes = 2 * kChunk;  // a stage of A, or of B: two chunks of 64 columns
constexpr int kMaxStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 384;
constexpr int kEpiBytes = kEpiWarps * 4096;  // 32 rows of 128 bytes per warp
constexpr int kBarBytes = 8 * (6 * kMaxStages + 5) + 24;  // and the TMEM address and two flags
constexpr uint16_t kPairMask = 0x3;

constexpr int table_bytes(int G) { return ((G + 1) * 4 + 2 * G + 2 * G + 15) / 16 * 16; }
constexpr int smem_bytes(int G, int stages) {
  return 1024 + 2 * stages * kHalfBytes + kEpiBytes + kBarBytes + table_bytes(G);
}
// Six stages, or five when the tables of many groups (more than 211) need the room.
constexpr int ring_stages(int G) { return smem_bytes(G, kMaxStages) <= kMaxSmem ? kMaxStages : kMaxStages - 1; }
static_assert(kBarBytes % 16 == 0, "the tables follow the barriers");
static_assert(smem_bytes(kMaxGroups, kMaxStages - 1) <= kMaxSmem, "shared memory");

struct DwParams {
  KParams k;  // offsets, G, rows, status, limit_ns
  int H, I;
  __nv_bfloat16* dw[3];  // dWd, dWg, dWu
  int stages;
  const int* odd;              // not 0: a row of a or dy may hold an infinity or NaN
  ChainWords chain;
  bool last;                   // of the chain: no DX follows
  // Strips: [0] of groups longer than the ring, one tile each; [1] of the others.
  struct Cut {
    int per_group;        // strips of a group: nd of dWd, then ng of dWg, then ng of dWu
    int nd, ng;
    int parts_d, parts_g;  // strips per row of tiles
    int len_d, len_g;      // tiles per strip
    uint32_t r_group, r_d, r_g;  // floor(2^32 / d) of per_group, parts_d, parts_g (div_by)
  } cut[2];
};

// A = dy, dg, du; B = h, then a twice. Three box heights each (64, 32 and 16
// rows): a group's last stage takes the lowest that covers its rows.
struct DwMaps {
  CUtensorMap dy[3], dg[3], du[3], h[3], a[3];
};

// Arrive on a barrier of another CTA of the cluster, releasing this CTA's
// writes (the wait's other half: mbar_acquire_cluster).
__device__ __forceinline__ void mbar_arrive_remote_release(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    grouped_weight_grad_kernel(const __grid_constant__ DwMaps m, const DwParams p) {
  const int NS = p.stages, G = p.k.G;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
  uint8_t* base = smem_raw + pad;
  const uint32_t base_u32 = raw_addr + pad;
  // Shared memory (the same in both CTAs): A ring | B ring | epilogue staging | barriers | tables.
  const uint32_t b_ring = base_u32 + NS * kHalfBytes;
  uint8_t* epi_stage = base + 2 * NS * kHalfBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi_stage + kEpiBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 6 * kMaxStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* row_start = reinterpret_cast<int32_t*>(epi_stage + kEpiBytes + kBarBytes);
  // Group g's first row in h, dg and du (gemm_grad.cuh) is row_start[g] -
  // row_start[0] + pad_extra[g].
  uint16_t* pad_extra = reinterpret_cast<uint16_t*>(row_start + G + 1);
  uint16_t* order = pad_extra + G;
  int32_t* pads = reinterpret_cast<int32_t*>(epi_stage);  // until the loop starts
  const uint32_t bar0 = smem_u32(bars);
  // Of A's ring (ab = 0) and B's (ab = 1).
  auto full_bar = [&](int ab, int s) { return bar0 + 8u * (ab * kMaxStages + s); };        // leader: both CTAs' stage s
  auto empty_bar = [&](int ab, int s) { return bar0 + 8u * ((2 + ab) * kMaxStages + s); };  // each CTA
  auto tail_bar = [&](int ab, int s) { return bar0 + 8u * ((4 + ab) * kMaxStages + s); };   // each CTA: a ragged stage
  auto tfull_bar = [&](int a) { return bar0 + 8u * (6 * kMaxStages + a); };                 // each CTA
  auto tempty_bar = [&](int a) { return bar0 + 8u * (6 * kMaxStages + 2 + a); };            // leader
  const uint32_t drain_bar = bar0 + 8u * (6 * kMaxStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: leader
  const int pair = (int)cluster_id_x(), npairs = (int)ncluster_x();

  wait_until_published(p.chain.inputs_ready, p.chain.call, abort_flag + 1);
  fill_row_start_coherent(p.k, row_start, threadIdx.x, kThreads);
  int* longs = reinterpret_cast<int*>(epi_stage) + kMaxGroups + 8;  // until the loop starts
  if (threadIdx.x == 0) *longs = 0;
  __syncthreads();
  // order[rank] = group, by length, longest first (equal lengths by number).
  // Tiles are dealt to the pairs in that order, forwards and backwards in turn,
  // which keeps their shares of unequal groups within a fraction of a tile.
  for (int g = threadIdx.x; g < G; g += kThreads) {
    const int n = row_start[g + 1] - row_start[g];
    int at = 0;
    for (int j = 0; j < G; ++j) {
      const int o = row_start[j + 1] - row_start[j];
      at += (o > n || (o == n && j < g)) ? 1 : 0;
    }
    order[at] = (uint16_t)g;
    pads[g] = n > 0 ? pad16(n) - n : 0;
    if (n > NS * kBK) atomicAdd(longs, 1);
  }
  if (threadIdx.x == 0) {
    for (int ab = 0; ab < 2; ++ab)
      for (int s = 0; s < NS; ++s) {
        mbar_init(full_bar(ab, s), 2);
        mbar_init(empty_bar(ab, s), 1);
        mbar_init(tail_bar(ab, s), 1);
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
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    scan_warp(pads, G, lane);
    __syncwarp();
    for (int g = lane; g < G; g += 32) pad_extra[g] = (uint16_t)pads[g];
  }
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers and TMEM are there
  tc_fence_after();
  // DX, the next launch, needs GU's results and not these: it may start now.
  wait_for_previous_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    publish(p.chain.gu_done, p.chain.call);
    if (p.last) *p.chain.inputs_ready = 0;
  }
  allow_next_launch();
  const bool careful = *static_cast<const volatile int*>(p.odd) != 0;
  const uint32_t tmem_base = *tmem_slot;
  const int n_long = *longs, long_strips = n_long * p.cut[0].per_group;
  __syncthreads();  // the epilogue's staging overwrites longs
  const int total = long_strips + (G - n_long) * p.cut[1].per_group;
  const int rounds = (total + npairs - 1) / npairs;
  auto strip_of = [&](int r) { return r * npairs + ((r & 1) ? npairs - 1 - pair : pair); };
  const int my_rounds = rounds > 0 && strip_of(rounds - 1) >= total ? rounds - 1 : rounds;  // the last may be short
  // Strips are decoded 32 rounds at a time, one by each lane of a role's warp,
  // and read back by shuffles: decoding alone cost a role's thread 1000 to 1500
  // cycles, as long as half a tile's MMAs.
  struct Strip {
    int rows, row0, prow0, m0, n0, len, g_which;  // prow0: in h, dg, du; len: tiles; g * 8 + open * 4 + which
  };
  // which: 0 dWd [H, I], 1 dWg [I, H], 2 dWu [I, H]; open: the group's last step
  // reaches rows after the last group.
  const int end = row_start[G];
  auto decode = [&](int r) {
    Strip t = {};
    if (r >= my_rounds) return t;
    int at = strip_of(r);
    const bool is_long = at < long_strips;
    const DwParams::Cut& c = p.cut[is_long ? 0 : 1];
    if (!is_long) at -= long_strips;
    const int slot = div_by(at, c.per_group, c.r_group);
    const int g = order[slot + (is_long ? 0 : n_long)];
    at -= slot * c.per_group;
    const int which = at < c.nd ? 0 : (at < c.nd + c.ng ? 1 : 2);
    at -= which == 0 ? 0 : (which == 1 ? c.nd : c.nd + c.ng);
    const int parts = which == 0 ? c.parts_d : c.parts_g, len = which == 0 ? c.len_d : c.len_g;
    const int row = div_by(at, parts, which == 0 ? c.r_d : c.r_g), n_tile = (at - row * parts) * len;
    const int n_tiles = ((which == 0 ? p.I : p.H) + 255) / 256;
    const int n = row_start[g + 1] - row_start[g];
    const int open = n > 0 && end < p.k.rows && row_start[g] + pad16(n) > end ? 4 : 0;
    t = {n > 0 ? n : 0, row_start[g], row_start[g] - row_start[0] + pad_extra[g], row * 256, n_tile * 256,
         n_tiles - n_tile < len ? n_tiles - n_tile : len, g * 8 + open + which};
    return t;
  };
  auto at_round = [&](int v, int r) { return __shfl_sync(0xFFFFFFFFu, v, r & 31); };
  // A stage with `left` rows of the group from its first row on needs clearing
  // when the group ends inside one of its steps.
  auto ragged = [&](int left, bool open) { return (careful || open) && left < kBK && (left & 15) != 0; };

  if (warp == 0 || warp == 6) {
    // ------------------------------------------------------------ producers
    // The whole warp walks the loop in step; one elected lane issues. A once per
    // strip, B once per tile.
    const int ab = warp == 0 ? 0 : 1;
    Ring rg;
    bool ok = true;
    Strip mine = {};
    for (int r = 0; ok && r < my_rounds; ++r) {
      if ((r & 31) == 0) mine = decode(r + lane);
      const int nrows = at_round(mine.rows, r), g_which = at_round(mine.g_which, r), which = g_which & 3;
      const bool open = (g_which & 4) != 0;
      // A: dy (rows as given), dg, du; B: h, then a (rows as given).
      const int row0 = at_round((ab == 0) == (which == 0) ? mine.row0 : mine.prow0, r);
      const int tiles = ab == 0 ? 1 : at_round(mine.len, r);
      const int x0 = at_round(ab == 0 ? mine.m0 : mine.n0, r) + (int)rank * 128;
      const CUtensorMap* maps = ab == 0 ? (which == 0 ? m.dy : (which == 1 ? m.dg : m.du)) : (which == 0 ? m.h : m.a);
      for (int t = 0; ok && t < tiles; ++t) {
        const int x = x0 + t * 256;
        int krow = row0;
        for (int left = nrows; left > 0; left -= kBK, krow += kBK) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(empty_bar(ab, rg.s), rg.ph ^ 1u, abort_flag, p.k.status,
                                                         MOE_DEV_TIMEOUT_PRODUCER, p.k.limit_ns))) {
            ok = false;
            break;
          }
          const int low = left <= 16 ? 2 : (left <= 32 ? 1 : 0);  // box height 64 >> low
          const CUtensorMap* map = maps + low;
          const uint32_t dst = (ab == 0 ? base_u32 : b_ring) + rg.s * kHalfBytes;
          const bool own = ragged(left, open);  // completes on this CTA's tail barrier
          const uint32_t full = full_bar(ab, rg.s);
          const uint32_t bar = own ? tail_bar(ab, rg.s) : (rank == 0 ? full : mapa_shared(full, 0));
          if (elect_one()) {
            if (own) {
              mbar_arrive_expect_tx(bar, (uint32_t)kHalfBytes >> low);
            } else if (rank == 0) {  // both CTAs' bytes (the other's may land first)
              mbar_arrive_expect_tx(bar, 2u * ((uint32_t)kHalfBytes >> low));
              mbar_arrive(bar);
            }
            tma_load_2d_pair(dst, map, bar, x, krow);
            tma_load_2d_pair(dst + kChunk, map, bar, x + 64, krow);
          }
          __syncwarp();
          rg.next(NS);
        }
      }
    }
    if (!ok) {  // let copies already issued land before the CTA leaves: 5 ms
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 5000000ull) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop in step (warp-uniform descriptors); one
    // elected lane issues.
    if (rank == 0) {
      constexpr uint32_t kIdesc = idesc_bf16_f32(256, 256) | 1u << 15 | 1u << 16;
      constexpr uint32_t kStep = 2048 >> 4;  // 16 rows
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
        return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, p.k.status, MOE_DEV_TIMEOUT_MMA,
                                                         p.k.limit_ns)) != 0;
      };
      Ring ra, rb;
      bool ok = true, issued = false;
      Strip mine = {};
      int tile = 0;
      for (int r = 0; ok && r < my_rounds; ++r) {
        if ((r & 31) == 0) mine = decode(r + lane);
        const int nrows = at_round(mine.rows, r), len = at_round(mine.len, r);
        const bool open = (at_round(mine.g_which, r) & 4) != 0;
        const Ring strip = ra;  // where the strip's A starts
        for (int t = 0; ok && t < len; ++t, ++tile) {
          const int acc = tile & 1;
          const uint32_t ap = (uint32_t)(tile >> 1) & 1u;
          if (!wait_all(tempty_bar(acc), ap ^ 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc * 256);
          ra = strip;
          uint32_t accumulate = 0;
          for (int left = nrows; left > 0; left -= kBK) {
            const uint64_t da = sw128_mnmajor_desc(base_u32 + ra.s * kHalfBytes);
            const uint64_t db = sw128_mnmajor_desc(b_ring + rb.s * kHalfBytes);
            if ((t == 0 && !wait_all(full_bar(0, ra.s), ra.ph)) || !wait_all(full_bar(1, rb.s), rb.ph)) {
              ok = false;
              break;
            }
            if (ragged(left, open)) {  // the other CTA's cleared rows
              if (t == 0) mbar_acquire_cluster(full_bar(0, ra.s), ra.ph);
              mbar_acquire_cluster(full_bar(1, rb.s), rb.ph);
            }
            tc_fence_after();
            if (elect_one()) {
              if (left >= kBK) {
                umma_bf16_pair(d, da, db, kIdesc, accumulate);
#pragma unroll
                for (int k = 1; k < kBK / 16; ++k) umma_bf16_pair(d, da + k * kStep, db + k * kStep, kIdesc, 1u);
              } else {
                const int steps = (left + 15) >> 4;
                for (int k = 0; k < steps; ++k)
                  umma_bf16_pair(d, da + (uint64_t)k * kStep, db + (uint64_t)k * kStep, kIdesc,
                                 accumulate | (k ? 1u : 0u));
              }
              umma_commit_pair_mc(empty_bar(1, rb.s), kPairMask);
              if (t == len - 1) umma_commit_pair_mc(empty_bar(0, ra.s), kPairMask);
            }
            __syncwarp();
            accumulate = 1u;
            issued = true;
            ra.next(NS);
            rb.next(NS);
          }
          if (!ok) break;
          if (elect_one()) umma_commit_pair_mc(tfull_bar(acc), kPairMask);
          __syncwarp();
        }
      }
      if (!ok && issued && lane == 0) {  // every issued MMA is done before TMEM is freed
        umma_commit_pair(drain_bar);
        drain_wait(drain_bar, 0, 200000000ull);
      }
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------ clearing
    // A ragged stage of a ring, once this CTA's copies of it have landed: clear
    // the rows from the group's end to the step's end, and hand the stage to
    // the leader. A stage's tail barrier has one phase per ragged use.
    Ring rg[2];
    uint32_t phase[2] = {0, 0};
    Strip mine = {};
    bool ok = true;
    auto pass = [&](int ab, int nrows, bool open) {  // one tile's stages of a ring
      for (int left = nrows; ok && left > 0; left -= kBK) {
        const int st = rg[ab].s;
        if (ragged(left, open)) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(tail_bar(ab, st), (phase[ab] >> st) & 1u, abort_flag,
                                                         p.k.status, MOE_DEV_TIMEOUT_MMA, p.k.limit_ns));
          if (!ok) break;
          phase[ab] ^= 1u << st;
          // Eight lanes clear one 128-byte row (a row's swizzle stays inside it).
          uint8_t* at = base + (ab * NS + st) * kHalfBytes + (lane & 7) * 16;
          for (int i = left + (lane >> 3); i < ((left + 15) & ~15); i += 4) {
            *reinterpret_cast<uint4*>(at + i * 128) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(at + kChunk + i * 128) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) mbar_arrive(full_bar(ab, st));
            else mbar_arrive_remote_release(mapa_shared(full_bar(ab, st), 0));
          }
        }
        rg[ab].next(NS);
      }
    };
    if (careful || end < p.k.rows)
      for (int r = 0; ok && r < my_rounds; ++r) {
        if ((r & 31) == 0) mine = decode(r + lane);
        const int nrows = at_round(mine.rows, r), len = at_round(mine.len, r);
        const bool open = (at_round(mine.g_which, r) & 4) != 0;
        pass(0, nrows, open);
        for (int t = 0; t < len; ++t) pass(1, nrows, open);
      }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;             // this warp may access TMEM lanes 32q .. 32q+31
    const int half = warp > 6 ? 1 : 0;  // its 128 columns
    uint8_t* stg = epi_stage + (half * 4 + q) * 4096;
    Strip mine = {};
    int tile = 0, ok = 1;
    for (int r = 0; ok && r < my_rounds; ++r) {
      if ((r & 31) == 0) mine = decode(r + lane);
      const int which = at_round(mine.g_which, r) & 3, g = at_round(mine.g_which, r) >> 3;
      const int m0 = at_round(mine.m0, r) + (int)rank * 128 + q * 32, len = at_round(mine.len, r);
      int n0 = at_round(mine.n0, r) + half * 128;
      const bool empty = at_round(mine.rows, r) == 0;
      for (int t = 0; t < len; ++t, ++tile, n0 += 256) {
        const int acc = tile & 1;
        const uint32_t ap = (uint32_t)(tile >> 1) & 1u;
        if (lane == 0)
          ok = mbar_wait_bounded(tfull_bar(acc), ap, abort_flag, p.k.status, MOE_DEV_TIMEOUT_EPILOGUE, p.k.limit_ns) ? 1 : 0;
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256 + half * 128);
        // 32 x 64 blocks through the warp's buffer, which is free again as soon
        // as it has been read. (By TMA from that buffer a block's store kept it
        // busy for as long as a short tile's whole MMAs: 2048 tokens, 8 of 64
        // experts, H = 2048, I = 768, uneven loads 199 us against 167. Stores
        // straight from the accumulators' lanes are 32 lines per instruction,
        // and the queue they form delays the loads.) H and I are multiples of
        // 64, so a block is all inside the group's matrix or all outside.
        const int M = which == 0 ? p.H : p.I, N = which == 0 ? p.I : p.H;
        if (m0 < M) {
#pragma unroll 1
          for (int c = 0; c < 128 && n0 + c < N; c += 64) {
            // Four rows of 128 bytes per instruction, first out of L2 again: DX
            // still needs the weights that are there.
            __nv_bfloat16* at = p.dw[which] + ((size_t)g * M + m0 + (lane >> 3)) * N + n0 + c + (lane & 7) * 8;
            if (empty) {
#pragma unroll
              for (int j = 0; j < 8; ++j) __stcs(reinterpret_cast<uint4*>(at + (size_t)(4 * j) * N), make_uint4(0, 0, 0, 0));
            } else {
              stage_bf16_block(tb + c, stg, lane);
              __syncwarp();
              uint4 v[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int row = 4 * j + (lane >> 3);
                v[j] = *reinterpret_cast<const uint4*>(stg + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
              }
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 8; ++j) __stcs(reinterpret_cast<uint4*>(at + (size_t)(4 * j) * N), v[j]);
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

}  // namespace

cudaError_t gemm_grad_dw_prepare_device() {
  return cudaFuncSetAttribute(grouped_weight_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
}

cudaError_t launch_grouped_weight_grad(const GroupedGradArgs& a, int dx_pairs, cudaStream_t s) {
  const int G = a.offsets ? a.G : 1, H = a.H, I = a.I;
  const uint64_t R = a.rows, P = padded_rows(a.rows, G);
  DwMaps m = {};
  for (int i = 0; i < 3; ++i) {
    const uint32_t box = 64u >> i;
    if (!make_tmap_bf16(&m.dy[i], a.dy, H, R, box) || !make_tmap_bf16(&m.dg[i], a.dg, I, P, box) ||
        !make_tmap_bf16(&m.du[i], a.du, I, P, box) || !make_tmap_bf16(&m.h[i], a.h, I, P, box) ||
        !make_tmap_bf16(&m.a[i], a.a, H, R, box))
      return cudaErrorInvalidValue;
  }
  DwParams p = {};
  p.k.offsets = a.offsets;
  p.k.G = G;
  p.k.rows = a.rows;
  p.k.status = a.status;
  p.k.limit_ns = a.wait_limit_ns;
  p.H = H;
  p.I = I;
  void* dw[] = {a.dw_down, a.dw_gate, a.dw_up};
  for (int i = 0; i < 3; ++i) p.dw[i] = static_cast<__nv_bfloat16*>(dw[i]);
  p.stages = ring_stages(G);
  p.odd = a.odd;
  p.chain = a.chain;
  p.last = a.da == nullptr;
  auto recip = [](int d) { return d > 1 ? (uint32_t)((1ull << 32) / (uint32_t)d) : 0xFFFFFFFFu; };
  const int tiles_h = (H + 255) / 256, tiles_i = (I + 255) / 256;
  auto cut = [&](int most) {
    DwParams::Cut c = {};
    c.parts_d = (tiles_i + most - 1) / most;
    c.parts_g = (tiles_h + most - 1) / most;
    c.len_d = (tiles_i + c.parts_d - 1) / c.parts_d;
    c.len_g = (tiles_h + c.parts_g - 1) / c.parts_g;
    c.nd = tiles_h * c.parts_d;
    c.ng = tiles_i * c.parts_g;
    c.per_group = c.nd + 2 * c.ng;
    c.r_group = recip(c.per_group);
    c.r_d = recip(c.parts_d);
    c.r_g = recip(c.parts_g);
    return c;
  };
  const long long max_pairs = a.num_sms / 2;
  p.cut[0] = cut(1);
  int most = 4;
  while (most > 1 && (long long)G * cut(most).per_group < 8 * max_pairs) most >>= 1;
  p.cut[1] = cut(most);
  const long long tiles = (long long)G * p.cut[0].per_group;
  int pairs = (int)(tiles < max_pairs ? tiles : max_pairs);
  // DX, which may run beside this launch, starts where a pair is free. Leave it
  // its pairs, if that costs few more rounds of short tiles (about 1 us each; DX
  // would otherwise start 8 us later at 128 tokens, 2 of 8 experts, H = 1024, I =
  // 512: 2.1 us of the pass's 38.9, with the two in the other order).
  const long long strips = (long long)G * p.cut[1].per_group, spare = max_pairs - dx_pairs;
  auto rounds = [&](long long n) { return (strips + n - 1) / n; };
  if (spare > 0 && spare < pairs && rounds(spare) <= rounds(pairs) + (a.rows <= 256ll * G ? 4 : 0)) pairs = (int)spare;
  if (pairs < 1) return cudaErrorInvalidValue;
  return launch_dependent(grouped_weight_grad_kernel, 2 * pairs, kThreads, smem_bytes(G, p.stages), s, true, /*cluster=*/2, m,
                          p);
}

}  // namespace moe
