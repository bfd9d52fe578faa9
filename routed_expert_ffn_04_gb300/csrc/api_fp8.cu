// C-ABI entry points of the products in E4M3 with one fp32 scale per block of
// 128: argument checks (kernels in gemm_fp8.cu and fp8_quant.cu).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe.h"
#include "fp8.cuh"
#include "internal.h"

using namespace moe;

namespace {

moe_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

template <typename... P>
bool all_aligned(P... p) {
  return (ptr_aligned16(p) && ...);
}

bool type_ok(int t) { return t == MOE_FLOAT_BF16 || t == MOE_FLOAT_F32; }
size_t size_of(int t) { return t == MOE_FLOAT_F32 ? 4 : 2; }

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// Whether an output overlaps an input or the other output.
template <int N>
bool clash(const Span& out, const Span& out2, const Span (&in)[N]) {
  if (overlap(out, out2)) return true;
  for (const Span& s : in)
    if (overlap(out, s) || overlap(out2, s)) return true;
  return false;
}

// Groups, rows, and the two sizes of a product's weights.
bool shape_ok(int G, int rows, int a, int b, const int32_t* offsets) {
  return G > 0 && G <= 1024 && rows >= 0 && rows <= kFp8MostRows && a > 0 && b > 0 && a % 16 == 0 && b % 16 == 0 && a <= 65536 && b <= 65536 &&
         (long long)rows * (a > b ? a : b) < (1ll << 40) && (offsets || G == 1);
}
size_t squares(int a, int b) { return (size_t)fp8_blocks(a) * fp8_blocks(b); }

Fp8GemmArgs base_args(moe_handle_t h, int G, const int32_t* offsets, int rows, int N, int K) {
  Fp8GemmArgs g = {};
  g.G = G;
  g.offsets = offsets;
  g.rows = rows;
  g.N = N;
  g.K = K;
  g.num_sms = g.device_sms = handle_num_sms(h);
  g.status = handle_status_word(h);
  g.wait_limit_ns = handle_wait_limit_ns(h);
  return g;
}

}  // namespace

extern "C" {

MOE_API moe_status_t moe_quantize_fp8(moe_handle_t h, const void* x, moe_float_t x_type, int64_t batch, int rows,
                                      int cols, int squares_, uint8_t* q, float* scale, moe_stream_t stream) {
  if (!type_ok(x_type) || batch < 0 || rows < 0 || cols <= 0 || cols % 16) return MOE_ERR_INVALID_ARG;
  if (rows > kFp8MostRows || cols > kFp8MostRows || batch > (1ll << 31) || (rows && batch * rows > (1ll << 40) / cols)) return MOE_ERR_INVALID_ARG;
  const int64_t all = batch * rows;
  if (squares_ && batch * fp8_blocks(rows) * fp8_blocks(cols) >= (1ll << 31)) return MOE_ERR_INVALID_ARG;
  if (all > 0 && (!x || !q || !scale)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(x, q, scale)) return MOE_ERR_INVALID_ARG;
  const size_t n = (size_t)all * cols;
  const size_t blocks = squares_ ? (size_t)batch * squares(rows, cols) : (size_t)all * fp8_blocks(cols);
  const Span in[] = {{x, n * size_of(x_type)}};
  if (clash({q, n}, {scale, blocks * 4}, in)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = bind_handle(h);
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = x_type == MOE_FLOAT_F32;
  return status_of(squares_ ? launch_fp8_quantize_squares(x, f32, batch, rows, cols, q, scale, s)
                            : launch_fp8_quantize_rows(x, f32, all, cols, q, scale, s));
}

MOE_API moe_status_t moe_fp8_padded_rows(int rows, int num_groups, int64_t* padded) {
  if (!padded || rows < 0 || rows > kFp8MostRows || num_groups <= 0 || num_groups > 1024) return MOE_ERR_INVALID_ARG;
  *padded = fp8_padded_rows(rows, num_groups);
  return MOE_OK;
}

MOE_API moe_status_t moe_quantize_fp8_columns(moe_handle_t h, const void* x, moe_float_t x_type, int num_groups,
                                              int rows, int cols, const int32_t* offsets, uint8_t* q, float* scale,
                                              moe_stream_t stream) {
  if (!type_ok(x_type) || !shape_ok(num_groups, rows, cols, cols, offsets)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !q || !scale)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(x, offsets, q, scale)) return MOE_ERR_INVALID_ARG;
  const size_t padded = (size_t)fp8_padded_rows(rows, num_groups);
  const Span in[] = {{x, (size_t)rows * cols * size_of(x_type)}, {offsets, 4 * ((size_t)num_groups + 1)}};
  if (clash({q, padded * cols}, {scale, padded / 128 * cols * 4}, in)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = bind_handle(h);
  if (st != MOE_OK) return st;
  return status_of(launch_fp8_quantize_columns(x, x_type == MOE_FLOAT_F32, rows, cols, offsets, num_groups, q, scale,
                                               static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status_t moe_grouped_gemm_fp8(moe_handle_t h, int num_groups, int rows, int N, int K, int transposed,
                                          const uint8_t* a, const float* a_scale, const int32_t* offsets,
                                          const uint8_t* w, const float* w_scale, moe_float_t out_type, void* out,
                                          moe_stream_t stream) {
  if (!type_ok(out_type) || !shape_ok(num_groups, rows, N, K, offsets)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!a || !a_scale || !w || !w_scale || !out)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(a, a_scale, offsets, w, w_scale, out)) return MOE_ERR_INVALID_ARG;
  const Span in[] = {{a, (size_t)rows * K}, {a_scale, (size_t)rows * fp8_blocks(K) * 4}, {offsets, 4 * ((size_t)num_groups + 1)},
                     {w, (size_t)num_groups * N * K}, {w_scale, num_groups * squares(N, K) * 4}};
  if (clash({out, (size_t)rows * N * size_of(out_type)}, {nullptr, 0}, in)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = bind_handle(h);
  if (st != MOE_OK) return st;
  Fp8GemmArgs g = base_args(h, num_groups, offsets, rows, N, K);
  g.a = a;
  g.a_scale = a_scale;
  g.w0 = w;
  g.s0 = w_scale;
  g.out = out;
  g.out_f32 = out_type == MOE_FLOAT_F32;
  return status_of(launch_gemm_fp8(g, transposed ? kFp8Transposed : kFp8Forward, static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status_t moe_grouped_gate_up_fp8(moe_handle_t h, int num_groups, int rows, int H, int I, const uint8_t* a,
                                             const float* a_scale, const int32_t* offsets, const uint8_t* w_gate,
                                             const float* s_gate, const uint8_t* w_up, const float* s_up, uint8_t* q,
                                             float* scale, moe_stream_t stream) {
  if (!shape_ok(num_groups, rows, H, I, offsets)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!a || !a_scale || !w_gate || !s_gate || !w_up || !s_up || !q || !scale)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(a, a_scale, offsets, w_gate, s_gate, w_up, s_up, q, scale)) return MOE_ERR_INVALID_ARG;
  const size_t w_bytes = (size_t)num_groups * H * I, s_bytes = num_groups * squares(H, I) * 4;
  const Span in[] = {{a, (size_t)rows * H}, {a_scale, (size_t)rows * fp8_blocks(H) * 4}, {offsets, 4 * ((size_t)num_groups + 1)},
                     {w_gate, w_bytes}, {w_up, w_bytes}, {s_gate, s_bytes}, {s_up, s_bytes}};
  if (clash({q, (size_t)rows * I}, {scale, (size_t)rows * fp8_blocks(I) * 4}, in)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = bind_handle(h);
  if (st != MOE_OK) return st;
  Fp8GemmArgs g = base_args(h, num_groups, offsets, rows, I, H);
  g.a = a;
  g.a_scale = a_scale;
  g.w0 = w_gate;
  g.s0 = s_gate;
  g.w1 = w_up;
  g.s1 = s_up;
  g.out = q;
  g.out_scale = scale;
  return status_of(launch_gemm_fp8(g, kFp8GateUp, static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status_t moe_grouped_weight_grad_fp8(moe_handle_t h, int num_groups, int rows, int N, int K,
                                                 const uint8_t* dy, const float* dy_scale, const uint8_t* a,
                                                 const float* a_scale, const int32_t* offsets, moe_float_t out_type,
                                                 void* dw, moe_stream_t stream) {
  if (!type_ok(out_type) || !shape_ok(num_groups, rows, N, K, offsets)) return MOE_ERR_INVALID_ARG;
  if (!dy || !dy_scale || !a || !a_scale || !dw) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(dy, dy_scale, a, a_scale, offsets, dw)) return MOE_ERR_INVALID_ARG;
  const size_t padded = (size_t)fp8_padded_rows(rows, num_groups);
  const Span in[] = {{dy, padded * N}, {dy_scale, padded / 128 * N * 4}, {a, padded * K}, {a_scale, padded / 128 * K * 4},
                     {offsets, 4 * ((size_t)num_groups + 1)}};
  if (clash({dw, (size_t)num_groups * N * K * size_of(out_type)}, {nullptr, 0}, in)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = bind_handle(h);
  if (st != MOE_OK) return st;
  Fp8GemmArgs g = base_args(h, num_groups, offsets, rows, N, K);
  g.a = dy;
  g.a_scale = dy_scale;
  g.w0 = a;
  g.s0 = a_scale;
  g.out = dw;
  g.out_f32 = out_type == MOE_FLOAT_F32;
  return status_of(launch_gemm_fp8(g, kFp8WeightGrad, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
