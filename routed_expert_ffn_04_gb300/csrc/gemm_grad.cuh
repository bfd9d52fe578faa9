// Building blocks shared by the kernels of the expert products' gradient
// (gemm_grad.cu, gemm_grad_dw.cu).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "gemm_sched.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kChunk = 64 * 128;  // an MN-major box: 64 rows of 128 bytes

// Shared-memory descriptor of an MN-major operand: chunks of 64 columns (128
// swizzled bytes) by 64 rows of the reduction axis, `kChunk` bytes apart;
// groups of 8 rows 1024 bytes apart. A step of 16 rows is 2048 bytes.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);  // [0,14)  start address >> 4
  d |= (uint64_t)(kChunk >> 4) << 16;            // [16,30) leading byte offset: next 64 columns
  d |= (uint64_t)(1024 >> 4) << 32;              // [32,46) stride byte offset: next 8 rows
  d |= (uint64_t)1 << 46;                        // [46,48) descriptor version (tcgen05)
  d |= (uint64_t)2 << 61;                        // [61,64) layout: 128-byte swizzle
  return d;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t is = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

// n / d for n, d < 2^31 with r = floor(2^32 / d): the estimate is at most one low.
__device__ __forceinline__ int div_by(int n, int d, uint32_t r) {
  int q = (int)__umulhi((uint32_t)n, r);
  if (n - q * d >= d) ++q;
  return q;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A copy into this CTA that completes on a barrier of either CTA of the pair
// (`bar` from mapa_shared, or this CTA's own).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// h, dg and du keep a group's rows together with zero rows up to the next
// multiple of 16, the tensor cores' step along the rows: row r of group g is
// row pad_start[g] + r of them. The rows they need for at most `rows` rows in G
// groups:
__host__ __device__ inline long long padded_rows(int rows, int G) { return (long long)rows + 15ll * G; }
__device__ __forceinline__ int pad16(int n) { return (n + 15) & ~15; }

// fill_row_start for launches that may begin before the one that writes the
// offsets has ended: coherent loads, which stay behind the wait (launch.cuh).
__device__ __forceinline__ void fill_row_start_coherent(const KParams& p, int32_t* row_start, int tid, int nthreads) {
  for (int g = tid; g <= p.G; g += nthreads) {
    const int v = p.offsets ? __ldcg(p.offsets + g) : (g == 0 ? 0 : p.rows);
    row_start[g] = v < 0 ? 0 : (v > p.rows ? p.rows : v);
  }
}

// v[0..G-1] to their exclusive sums, v[G] the total, by one warp.
__device__ __forceinline__ void scan_warp(int32_t* v, int G, int lane) {
  const int per = (G + 31) / 32;
  const int b = lane * per < G ? lane * per : G;
  const int e = (b + per < G) ? b + per : G;
  int local = 0;
  for (int g = b; g < e; ++g) local += v[g];
  int incl = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += u;
  }
  int run = incl - local;
  for (int g = b; g < e; ++g) {
    const int c = v[g];
    v[g] = run;
    run += c;
  }
  if (lane == 31) v[G] = incl;
}

// A warp's block of 32 rows x 64 bf16 columns (lane = row, TMEM columns taddr
// .. taddr + 63) into its staging buffer, 128-byte rows, 16-byte chunk j of row
// r at chunk j ^ (r % 8).
__device__ __forceinline__ void stage_bf16_block(uint32_t taddr, uint8_t* stg, int lane) {
  uint32_t v[32], u[32];
  tmem_ld_32x32b_x32(taddr, v);
  tmem_ld_32x32b_x32(taddr + 32, u);
  tmem_ld_wait();
  uint8_t* row = stg + lane * 128;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4], x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
      x[i] = pack_bf16(__uint_as_float(u[8 * j + 2 * i]), __uint_as_float(u[8 * j + 2 * i + 1]));
    }
    *reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + (((j + 4) ^ (lane & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
  }
}

}  // namespace moe
