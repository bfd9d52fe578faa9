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
// and du are rounded to bf16 once, as the tensor cores read them.
//
// One kernel, three modes. Persistent, one CTA per SM, tiles of 128 x 256 fp32
// accumulators double-buffered in TMEM (512 columns), K in steps of 64 through
// a ring of 48 KB stages written by TMA:
//   warp 0      TMA producer (one thread); modes with more than three boxes per
//               stage split them with warp 6;
//   warp 1      TMEM allocation and tcgen05.mma (M = 128, N = 256, K = 16);
//   warps 2..5  epilogue, 32 accumulator rows each.
//
// Operands. The forward's weights are K-major for the forward products; three
// of the four products here reduce over another axis, so their operands are
// read MN-major from the same row-major tensors, with no transposed copy: a
// box of 64 columns x 64 rows lands as 64 rows (the reduction axis) of 128
// swizzled bytes, the tensor cores' MN-major operand layout, and the
// instruction descriptor's transpose bit is set.
//   mode  A (128 rows of M)              B (256 rows of N)           reduction
//   Q     dy rows, K-major               Wd columns, MN-major        H
//   GU    a rows, K-major                Wg | Wu rows, K-major       H
//   DX    dg rows, then du rows, K-major Wg, then Wu columns, MN     I, twice
// The weight gradients (gemm_grad_dw.cu) reduce over the rows.
//
// Every wait is bounded; on expiry the CTA records an error code in the status
// word, drains its in-flight copies and MMAs, frees TMEM and exits.
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

constexpr int kBK = 64;           // reduction elements per stage
constexpr int kMaxGroups = 1024;
constexpr int kMaxSmem = 232448;  // 227 KB dynamic shared memory per CTA

template <int MODE>
struct GradGeo {
  static constexpr bool B_MN = MODE != kGU;
  static constexpr int A_BYTES = 128 * 128;  // 16 KB
  static constexpr int B_BYTES = 256 * 128;  // 32 KB
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // Warp 6 is a second producer where a stage has more than three boxes.
  static constexpr int THREADS = MODE == kGU ? 192 : 224;
  static constexpr int TABLE_BYTES = 3 * (kMaxGroups + 8) * 4;  // tile, row and padded row starts
  static constexpr int BAR_BYTES = 512;
  static constexpr int EPI_WARP = 4096;  // one warp's staging block: 32 rows of 128 bytes
  static constexpr int EPI_BYTES = 4 * EPI_WARP;
  static constexpr int EXTRA = 1024 + TABLE_BYTES + BAR_BYTES + EPI_BYTES;
  static constexpr int S = (kMaxSmem - EXTRA) / STAGE_BYTES;
  static constexpr int RING_BYTES = S * STAGE_BYTES;
  static constexpr int SMEM = EXTRA + RING_BYTES;
  static constexpr int NBARS = 2 * S + 5;
  static constexpr int TILE_N = MODE == kGU ? 128 : 256;  // output columns per tile
  static_assert(S >= 4, "ring too shallow");
  static_assert(NBARS * 8 + 8 <= BAR_BYTES, "barrier area");
  static_assert(SMEM <= kMaxSmem, "shared memory budget");
};

struct GradParams {
  KParams k;              // offsets, G, rows, status, limit_ns; N = output columns
  int H, I;
  int num_kb;             // stages per tile (Q, GU: H / 64; DX: 2 I / 64)
  float* q;               // [rows, I]
  __nv_bfloat16 *h, *dg, *du;  // [prows, I], padded (padded_rows)
  int prows;
  int* odd;               // set where gate or q is not finite
  __nv_bfloat16* da;      // [rows, H]
};

// A warp's block of 32 rows x 32 bf16 columns (lane = row, its 32 values packed
// in w) to global memory, the first `nr` rows: staged as 64-byte rows (16-byte
// chunk j of row r at chunk j ^ (r / 2 % 4)), then eight rows per store
// instruction, four lanes to a row.
__device__ __forceinline__ void store_block32(const uint32_t (&w)[16], uint8_t* stg, int lane, int nr,
                                              __nv_bfloat16* dst, size_t pitch) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(stg + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  __syncwarp();
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int r = it * 8 + (lane >> 2), j = lane & 3;
    if (r < nr)
      *reinterpret_cast<uint4*>(dst + r * pitch + j * 8) =
          *reinterpret_cast<const uint4*>(stg + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
  }
}

// The staged block's first `nr` rows to rows row0.. of a row-major bf16 or
// fp32 matrix whose rows are `pitch` bytes long, at byte `col` (a block that
// ends inside it: a TMA box would also write the next group's rows).
__device__ __forceinline__ void copy_staged_rows(const uint8_t* stg, int lane, int nr, uint8_t* base, size_t row0,
                                                 size_t pitch, size_t col) {
  __syncwarp();
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int r = it * 4 + (lane >> 3), j = lane & 7;
    if (r < nr)
      *reinterpret_cast<uint4*>(base + (row0 + r) * pitch + col + j * 16) =
          *reinterpret_cast<const uint4*>(stg + r * 128 + ((j ^ (r & 7)) << 4));
  }
  __syncwarp();
}

// Epilogue of one 128 x TILE_N tile by one warp (32 accumulator rows).
template <int MODE>
__device__ __forceinline__ void grad_epilogue(const GradParams& p, const TileInfo& ti, int pad0, uint32_t tb, int q,
                                              int lane, uint8_t* stg, const CUtensorMap* map_out) {
  const int r0 = ti.tt * 128 + q * 32;  // the warp's first row in the group
  const int nr = ti.nrows - r0;         // rows of the group from there on
  if (nr <= 0) return;                  // (r0 % 16 == 0: no padding here either)
  if (MODE == kGU) {
    // q comes in coalesced (four rows of 128 bytes per load instruction), one
    // block of 32 columns ahead, and goes through the staging buffer to the
    // lane that holds the row's accumulators.
    const size_t row = (size_t)ti.row0 + r0;
    // h, dg, du: the group's rows and the zero rows that fill its last step.
    const size_t prow = (size_t)pad0 + r0;
    const bool live = lane < nr;
    int np = pad16(ti.nrows) - r0;
    if ((long long)prow + np > p.prows) np = (int)(p.prows - (long long)prow);  // decreasing offsets
    bool odd = false;
    const int c0 = ti.wt * 128;
    const int ncol = p.I - c0 < 128 ? p.I - c0 : 128;  // a multiple of 64
    float4 nq[8];
    auto load_q = [&](int c) {
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int r = it * 4 + (lane >> 3);
        nq[it] = r < nr ? *reinterpret_cast<const float4*>(p.q + (row + r) * p.I + c0 + c + (lane & 7) * 4)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    load_q(0);
#pragma unroll 1
    for (int c = 0; c < ncol; c += 32) {
      __syncwarp();
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int r = it * 4 + (lane >> 3);
        *reinterpret_cast<float4*>(stg + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) = nq[it];
      }
      __syncwarp();
      float qv[32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 t = *reinterpret_cast<const float4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4));
        qv[4 * j] = t.x;
        qv[4 * j + 1] = t.y;
        qv[4 * j + 2] = t.z;
        qv[4 * j + 3] = t.w;
      }
      if (c + 32 < ncol) load_q(c + 32);
      uint32_t g[32], u[32];
      tmem_ld_32x32b_x32(tb + c, g);
      tmem_ld_32x32b_x32(tb + 128 + c, u);
      tmem_ld_wait();
      // An infinity or NaN in the row of a or of dy leaves none of its gate
      // values, or of its q values, finite.
      odd = odd || !(fabsf(__uint_as_float(g[0])) <= 3.402823466e38f) || !(fabsf(qv[0]) <= 3.402823466e38f);
      uint32_t ph[16], pg[16], pu[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float hv[2], gv[2], uv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float gt = __uint_as_float(g[2 * j + i]), up = __uint_as_float(u[2 * j + i]), qq = qv[2 * j + i];
          const float sg = __fdividef(1.0f, 1.0f + __expf(-gt));
          const float act = gt * sg;
          hv[i] = act * up;
          uv[i] = qq * act;
          gv[i] = qq * up * sg * fmaf(gt, 1.0f - sg, 1.0f);
        }
        ph[j] = live ? pack_bf16(hv[0], hv[1]) : 0u;
        pg[j] = live ? pack_bf16(gv[0], gv[1]) : 0u;
        pu[j] = live ? pack_bf16(uv[0], uv[1]) : 0u;
      }
      const size_t at = prow * p.I + c0 + c;
      store_block32(ph, stg, lane, np, p.h + at, p.I);
      store_block32(pg, stg + 2048, lane, np, p.dg + at, p.I);
      store_block32(pu, stg, lane, np, p.du + at, p.I);
    }
    if (odd && live) *p.odd = 1;
  } else if (MODE == kQ) {
    const size_t row = (size_t)ti.row0 + r0;
#pragma unroll 1
    for (int c = 0; c < 256; c += 32) {
      const int col = ti.wt * 256 + c;
      if (col >= p.I) break;
      uint32_t v[32];
      tmem_ld_32x32b_x32(tb + c, v);
      tmem_ld_wait();
      if (lane == 0) bulk_wait_group_read0();
      __syncwarp();
      uint8_t* srow = stg + lane * 128;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(srow + ((j ^ (lane & 7)) << 4)) =
            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      if (nr >= 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(map_out, smem_u32(stg), col, (int)row);
          bulk_commit_group();
        }
      } else {
        copy_staged_rows(stg, lane, nr, reinterpret_cast<uint8_t*>(p.q), row, (size_t)p.I * 4, (size_t)col * 4);
      }
    }
  } else {  // DX
    const size_t row = (size_t)ti.row0 + r0;
#pragma unroll 1
    for (int c = 0; c < 256; c += 64) {
      const int col = ti.wt * 256 + c;
      if (col >= p.H) break;
      stage_bf16_block(tb + c, stg, lane);
      if (nr >= 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(map_out, smem_u32(stg), col, (int)row);
          bulk_commit_group();
        }
      } else {
        copy_staged_rows(stg, lane, nr, reinterpret_cast<uint8_t*>(p.da), row, (size_t)p.H * 2, (size_t)col * 2);
      }
    }
  }
}

// Operand and output maps. Q: a = dy, b0 = Wd, out = q. GU: a = a, b0 / b1 =
// Wg / Wu. DX: a = dg, a2 = du, b0 / b1 = Wg / Wu, out = da.
struct GradMaps {
  CUtensorMap a, a2, b0, b1, out;
};
template <int MODE>
__global__ void __launch_bounds__(GradGeo<MODE>::THREADS, 1)
    grouped_grad_kernel(const __grid_constant__ GradMaps m, const GradParams p) {
  using Gm = GradGeo<MODE>;
  constexpr int NS = Gm::S;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
  uint8_t* base = smem_raw + pad;
  const uint32_t base_u32 = raw_addr + pad;
  // Shared memory: ring | epilogue staging | tables | barriers.
  uint8_t* epi_stage = base + Gm::RING_BYTES;
  int32_t* tile_start = reinterpret_cast<int32_t*>(epi_stage + Gm::EPI_BYTES);
  int32_t* row_start = tile_start + kMaxGroups + 8;
  int32_t* pad_start = row_start + kMaxGroups + 8;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi_stage + Gm::EPI_BYTES + Gm::TABLE_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Gm::NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (NS + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * NS + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * NS + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * NS + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.k.G;
  allow_next_launch();

  // ---- row starts; tile_start[g] = tiles of groups before g.
  fill_row_start(p.k, row_start, threadIdx.x, Gm::THREADS);
  const int n_wt = (p.k.N + Gm::TILE_N - 1) / Gm::TILE_N;
  for (int g = threadIdx.x; g < G; g += Gm::THREADS) {
    int r0, nr;
    group_rows(p.k, g, r0, nr);
    tile_start[g] = n_wt * ((nr + 127) / 128);
    pad_start[g] = pad16(nr);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  __syncthreads();
  if (warp == 0) scan_warp(tile_start, G, lane);
  if (MODE != kQ && warp == 2) scan_warp(pad_start, G, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Up to here nothing was read that the launch before this one writes (its
  // blocks may still be running: programmatic dependent launch).
  wait_for_previous_launch();
  if (MODE == kQ && blockIdx.x == 0 && threadIdx.x == 0) *p.odd = 0;
  const uint32_t tmem_base = *tmem_slot;
  const int total = tile_start[G];

  if (warp == 0 || warp == 6) {
    // ------------------------------------------------------------ producers
    // Boxes of a stage: A, then B's in order. Warp 0 arms the stage's barrier
    // with all its bytes and issues the first; the others issue the rest (a
    // transaction may land before it is expected). A box costs its thread about
    // 100 to 150 cycles, a stage's MMAs take 512.
    if (lane == 0) {
      const bool first = warp == 0;
      Ring rg;
      Armed armed;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
        const TileInfo ti = decode_tile_s<128>(G, tile_start, row_start, tile);
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait_bounded(empty_bar(rg.s), rg.ph ^ 1u, abort_flag, p.k.status, MOE_DEV_TIMEOUT_PRODUCER,
                                 p.k.limit_ns)) {
            ok = false;
            break;
          }
          const uint32_t fb = full_bar(rg.s);
          const uint32_t sa = base_u32 + rg.s * Gm::STAGE_BYTES, sb = sa + Gm::A_BYTES;
          if (first) mbar_arrive_expect_tx(fb, Gm::STAGE_BYTES);
          if constexpr (MODE == kGU) {
            tma_load_2d(sa, &m.a, fb, kb * kBK, ti.row0 + ti.tt * 128);
            tma_load_2d(sb, &m.b0, fb, kb * kBK, ti.g * p.I + ti.wt * 128);
            tma_load_2d(sb + Gm::A_BYTES, &m.b1, fb, kb * kBK, ti.g * p.I + ti.wt * 128);
          } else {
            // DX: the first half of the stages is dg Wg, the second du Wu.
            const int half = p.num_kb >> 1;
            const bool second = MODE == kDX && kb >= half;
            const int kx = (second ? kb - half : kb) * kBK;
            const CUtensorMap* mb = second ? &m.b1 : &m.b0;
            const int krow = ti.g * (MODE == kQ ? p.H : p.I) + kx;
            if (first) {
              tma_load_2d(sa, second ? &m.a2 : &m.a, fb, kx, (MODE == kDX ? pad_start[ti.g] : ti.row0) + ti.tt * 128);
              tma_load_2d(sb, mb, fb, ti.wt * 256, krow);
            } else {
#pragma unroll
              for (int j = 1; j < 4; ++j) tma_load_2d(sb + j * kChunk, mb, fb, ti.wt * 256 + j * 64, krow);
            }
          }
          armed.mark(rg);
          rg.next(NS);
        }
      }
      if (!ok) {  // let copies already issued land before the CTA exits
        for (int s = 0; s < NS; ++s)
          if (armed.mask & (1u << s)) drain_wait(full_bar(s), (armed.phase >> s) & 1u, 100000000ull);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop in step, polls included, so that tile, stage
    // and descriptor values are warp-uniform (the tensor core instructions take
    // uniform registers: 290 cycles to issue a stage, against 360 from one
    // diverged lane); one elected lane issues.
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, 256) | (Gm::B_MN ? 1u << 16 : 0u);
    constexpr uint32_t kStepA = 32 >> 4, kStepB = Gm::B_MN ? 2048 >> 4 : 32 >> 4;
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
      return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, p.k.status, MOE_DEV_TIMEOUT_MMA,
                                                       p.k.limit_ns)) != 0;
    };
    Ring rg;
    bool ok = true, issued = false;
    int local = 0;
    for (int tile = blockIdx.x; ok && tile < total; tile += gridDim.x, ++local) {
      const int acc = local & 1;
      const uint32_t ap = (uint32_t)(local >> 1) & 1u;
      if (!wait_all(tempty_bar(acc), ap ^ 1u)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(acc * 256);
      for (int kb = 0; kb < p.num_kb; ++kb) {
        const uint32_t sa = base_u32 + rg.s * Gm::STAGE_BYTES, sb = sa + Gm::A_BYTES;
        const uint64_t da = sw128_kmajor_desc(sa);
        const uint64_t db = Gm::B_MN ? sw128_mnmajor_desc(sb) : sw128_kmajor_desc(sb);
        if (!wait_all(full_bar(rg.s), rg.ph)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          umma_bf16(d, da, db, kIdesc, kb ? 1u : 0u);
#pragma unroll
          for (int k = 1; k < kBK / 16; ++k) umma_bf16(d, da + k * kStepA, db + k * kStepB, kIdesc, 1u);
          umma_commit(empty_bar(rg.s));
        }
        __syncwarp();
        issued = true;
        rg.next(NS);
      }
      if (!ok) break;
      if (elect_one()) umma_commit(tfull_bar(acc));
      __syncwarp();
    }
    if (!ok && issued && lane == 0) {  // wait for every issued MMA before TMEM is freed
      umma_commit(drain_bar);
      drain_wait(drain_bar, 0, 100000000ull);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // this warp may access TMEM lanes 32q .. 32q+31
    uint8_t* stg = epi_stage + q * Gm::EPI_WARP;
    int local = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x, ++local) {
      const int acc = local & 1;
      const uint32_t ap = (uint32_t)(local >> 1) & 1u;
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait_bounded(tfull_bar(acc), ap, abort_flag, p.k.status, MOE_DEV_TIMEOUT_EPILOGUE, p.k.limit_ns) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256);
      const TileInfo ti = decode_tile_s<128>(G, tile_start, row_start, tile);
      grad_epilogue<MODE>(p, ti, pad_start[ti.g], tb, q, lane, stg, &m.out);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(acc));
    }
    if (lane == 0) bulk_wait_group0();  // this warp's bulk stores are complete
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int MODE>
cudaError_t run_mode(const GradMaps& m, const GradParams& p, long long max_tiles, int num_sms, cudaStream_t s) {
  using Gm = GradGeo<MODE>;
  if (max_tiles <= 0) return cudaSuccess;
  const int grid = (int)(max_tiles < num_sms ? max_tiles : num_sms);
  // Q starts after everything before it; the others' prologues may overlap the
  // end of the launch before them (its offsets were there before Q).
  return launch_dependent(grouped_grad_kernel<MODE>, grid, Gm::THREADS, Gm::SMEM, s, MODE != kQ, /*cluster=*/1, m, p);
}

template <int MODE>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(grouped_grad_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              GradGeo<MODE>::SMEM);
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
  p.da = static_cast<__nv_bfloat16*>(a.da);
  const uint64_t R = a.rows, GI = (uint64_t)G * I, GH = (uint64_t)G * H;
  const long long row_tiles = (a.rows + 127) / 128 + (long long)G;  // at most: one ragged tile per group
  auto ceil_div = [](long long v, long long d) { return (v + d - 1) / d; };
  cudaError_t e = cudaSuccess;
  bool maps = true;
  {
    GradMaps m = {};
    maps = make_tmap_bf16(&m.a, a.dy, H, R, 128) && make_tmap_bf16(&m.b0, a.w_down, I, GH, 64) &&
           make_tmap_f32_store(&m.out, a.q, I, R);
    if (!maps) return cudaErrorInvalidValue;
    p.k.N = I;
    p.num_kb = H / kBK;
    e = run_mode<kQ>(m, p, row_tiles * ceil_div(I, 256), a.num_sms, s);
  }
  if (e == cudaSuccess) {
    GradMaps m = {};
    maps = make_tmap_bf16(&m.a, a.a, H, R, 128) && make_tmap_bf16(&m.b0, a.w_gate, H, GI, 128) &&
           make_tmap_bf16(&m.b1, a.w_up, H, GI, 128);
    if (!maps) return cudaErrorInvalidValue;
    p.k.N = I;
    p.num_kb = H / kBK;
    e = run_mode<kGU>(m, p, row_tiles * ceil_div(I, 128), a.num_sms, s);
  }
  if (e == cudaSuccess && a.da) {
    GradMaps m = {};
    const uint64_t P = p.prows;
    maps = make_tmap_bf16(&m.a, a.dg, I, P, 128) && make_tmap_bf16(&m.a2, a.du, I, P, 128) &&
           make_tmap_bf16(&m.b0, a.w_gate, H, GI, 64) && make_tmap_bf16(&m.b1, a.w_up, H, GI, 64) &&
           make_tmap_bf16(&m.out, a.da, H, R, 32);
    if (!maps) return cudaErrorInvalidValue;
    p.k.N = H;
    p.num_kb = 2 * (I / kBK);
    e = run_mode<kDX>(m, p, row_tiles * ceil_div(H, 256), a.num_sms, s);
  }
  if (e == cudaSuccess && want_dw) e = launch_grouped_weight_grad(a, s);
  return e;
}

}  // namespace moe
