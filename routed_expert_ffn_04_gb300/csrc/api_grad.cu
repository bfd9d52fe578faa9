// C-ABI entry points around the layer and of its gradient: argument checks and
// workspace carving (kernels in norm.cu, dispatch_grad.cu and gemm_grad.cu).
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdint>

#include "../../include/moe.h"
#include "internal.h"

using namespace moe;

namespace {

constexpr int kMaxNormCols = 16384;

moe_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

template <typename... P>
bool all_aligned(P... p) {
  return (ptr_aligned16(p) && ...);
}

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

bool norm_shape_ok(int64_t rows, int H, int res_type) {
  return rows >= 0 && rows < (1ll << 31) && H >= 1 && H <= kMaxNormCols &&
         (res_type == MOE_RES_BF16 || res_type == MOE_RES_F32);
}

// Enough for either residual type.
size_t norm_grad_ws(int64_t rows, int H) {
  const int a = norm_grad_blocks(rows, H, false), b = norm_grad_blocks(rows, H, true);
  return align_up((size_t)(a > b ? a : b) * H * 4 + 1, 256);
}

// moe_grouped_swiglu_backward workspace: a flag and two words (256 bytes), q fp32, then h, dgate and dup
// bf16 with each group's rows padded to a multiple of 16.
struct GradWs {
  size_t q, h, dg, du, total;
};
GradWs grad_ws(int rows, int G, int I) {
  const size_t n = (size_t)rows * I, np = ((size_t)rows + 15 * (size_t)G) * I;
  GradWs L;
  L.q = 256;
  L.h = L.q + align_up(n * 4 + 1, 256);
  L.dg = L.h + align_up(np * 2 + 1, 256);
  L.du = L.dg + align_up(np * 2 + 1, 256);
  L.total = L.du + align_up(np * 2 + 1, 256);
  return L;
}

// A number that no other call has, in this process or (nearly surely) in one
// that used the same memory before.
uint64_t next_call() {
  static std::atomic<uint64_t> n{(uint64_t)std::chrono::system_clock::now().time_since_epoch().count() | 1};
  return n.fetch_add(1, std::memory_order_relaxed);
}

bool grad_shape_ok(int num_groups, int rows, int H, int I) {
  return num_groups > 0 && num_groups <= 1024 && rows >= 0 && H > 0 && I > 0 && H % 64 == 0 && I % 64 == 0 &&
         H <= 65536 && I <= 65536 && (long long)rows * (H > I ? H : I) < (1ll << 40);
}

}  // namespace

extern "C" {

MOE_API moe_status_t moe_add_rmsnorm(moe_handle_t h, int64_t rows, int H, moe_residual_t res_type, const void* x,
                                     const void* residual, const void* weight, float eps, void* h_out, void* out,
                                     uint8_t* q, uint8_t* q_scale, float* rstd, moe_stream_t stream) {
  if (!norm_shape_ok(rows, H, res_type)) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_scale != nullptr) || (q && H % 32)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !weight || (!out && !q))) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(x, residual, weight, h_out, out, q, q_scale, rstd)) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = bind_handle(h);
  if (st != MOE_OK) return st;
  NormArgs a = {rows, H, x, residual, weight, eps, h_out, out, q, q_scale, rstd, res_type == MOE_RES_F32};
  return status_of(launch_add_rmsnorm(a, static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status_t moe_add_rmsnorm_backward_workspace_size(int64_t rows, int H, size_t* bytes) {
  if (!bytes || !norm_shape_ok(rows, H, MOE_RES_BF16)) return MOE_ERR_INVALID_ARG;
  *bytes = norm_grad_ws(rows, H);
  return MOE_OK;
}

MOE_API moe_status_t moe_add_rmsnorm_backward(moe_handle_t h, int64_t rows, int H, moe_residual_t res_type,
                                              const void* dout, const void* dh_in, const void* h_res,
                                              const void* weight, const float* rstd, void* dh, void* dx,
                                              float* dweight, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!norm_shape_ok(rows, H, res_type)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!dout || !h_res || !weight || !rstd || !dh)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(dout, dh_in, h_res, weight, rstd, dh, dx, dweight, ws)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && dweight && !ws) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && dweight && ws_bytes < norm_grad_ws(rows, H)) return MOE_ERR_WORKSPACE;
  const moe_status_t st = bind_handle(h);
  if (st != MOE_OK) return st;
  NormGradArgs a = {rows, H, dout, dh_in, h_res, weight, rstd, dh, dx, dweight, static_cast<float*>(ws),
                    res_type == MOE_RES_F32};
  return status_of(launch_add_rmsnorm_backward(a, static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status_t moe_combine_backward(moe_handle_t h, const moe_config_t* cfg, const void* dout,
                                          const float* y_perm, const float* topk_w, const int32_t* flat_to_perm,
                                          const int32_t* topk_idx, const float* logits, void* dy_perm,
                                          float* dtopk_w, float* dlogits, moe_stream_t stream) {
  moe_status_t st = check_config(cfg);
  if (st != MOE_OK) return st;
  const int given = (topk_idx != nullptr) + (logits != nullptr) + (dlogits != nullptr);
  if (given != 0 && given != 3) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!dout || !y_perm || !topk_w || !flat_to_perm || !dy_perm || !dtopk_w)) return MOE_ERR_INVALID_ARG;
  if (dlogits && dlogits == logits) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(dout, y_perm, topk_w, flat_to_perm, topk_idx, logits, dy_perm, dtopk_w, dlogits))
    return MOE_ERR_INVALID_ARG;
  if ((st = bind_handle(h)) != MOE_OK) return st;
  CombineGradArgs a = {};
  a.T = cfg->T;
  a.K = cfg->K;
  a.H = cfg->H;
  a.E = cfg->E;
  a.scaling = cfg->scaling;
  a.route_norm = cfg->route_norm;
  a.dout = dout;
  a.y_perm = y_perm;
  a.topk_w = topk_w;
  a.flat_to_perm = flat_to_perm;
  a.topk_idx = topk_idx;
  a.logits = logits;
  a.dy_perm = dy_perm;
  a.dtopk_w = dtopk_w;
  a.dlogits = dlogits;
  a.num_sms = handle_num_sms(h);
  a.status = handle_status_word(h);
  return status_of(launch_combine_backward(a, static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status_t moe_route_backward(moe_handle_t h, const moe_config_t* cfg, const float* logits,
                                        const int32_t* topk_idx, const float* dtopk_w, float* dlogits,
                                        moe_stream_t stream) {
  moe_status_t st = check_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!logits || !topk_idx || !dtopk_w || !dlogits || dlogits == logits || dlogits == dtopk_w))
    return MOE_ERR_INVALID_ARG;
  if (!all_aligned(logits, topk_idx, dtopk_w, dlogits)) return MOE_ERR_INVALID_ARG;
  if ((st = bind_handle(h)) != MOE_OK) return st;
  return status_of(launch_route_backward(logits, topk_idx, dtopk_w, cfg->T, cfg->E, cfg->K, cfg->scaling,
                                         cfg->route_norm, dlogits, handle_status_word(h),
                                         static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status_t moe_permute_backward(moe_handle_t h, const moe_config_t* cfg, const void* dx_perm,
                                          const int32_t* flat_to_perm, const void* dx_add, void* dx,
                                          moe_stream_t stream) {
  moe_status_t st = check_config(cfg);
  if (st != MOE_OK) return st;
  if (cfg->T > 0 && (!dx_perm || !flat_to_perm || !dx || dx == dx_perm)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(dx_perm, flat_to_perm, dx_add, dx)) return MOE_ERR_INVALID_ARG;
  if ((st = bind_handle(h)) != MOE_OK) return st;
  return status_of(launch_permute_backward(dx_perm, flat_to_perm, cfg->T, cfg->K, cfg->H, dx_add, dx,
                                           handle_status_word(h), static_cast<cudaStream_t>(stream)));
}

MOE_API moe_status_t moe_grouped_gemm_backward_workspace_size(int rows, int num_groups, int H, int I,
                                                                moe_dtype_t dtype, size_t* bytes) {
  if (!bytes || !grad_shape_ok(num_groups, rows, H, I)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16) return is_mx_dtype(dtype) ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  *bytes = grad_ws(rows, num_groups, I).total;
  return MOE_OK;
}

MOE_API moe_status_t moe_grouped_swiglu_backward(moe_handle_t h, int num_groups, int rows, int H, int I,
                                                 moe_dtype_t dtype, const void* a, const void* dy,
                                                 const int32_t* offsets, const void* w_gate, const void* w_up,
                                                 const void* w_down, void* da, void* dw_gate, void* dw_up,
                                                 void* dw_down, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!grad_shape_ok(num_groups, rows, H, I)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16) return is_mx_dtype(dtype) ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  if (offsets == nullptr && num_groups != 1) return MOE_ERR_INVALID_ARG;
  const int dws = (dw_gate != nullptr) + (dw_up != nullptr) + (dw_down != nullptr);
  if ((dws != 0 && dws != 3) || (rows > 0 && dws == 0 && !da)) return MOE_ERR_INVALID_ARG;
  if (!w_gate || !w_up || !w_down || !ws || (rows > 0 && (!a || !dy))) return MOE_ERR_INVALID_ARG;
  if (!all_aligned(a, dy, offsets, w_gate, w_up, w_down, da, dw_gate, dw_up, dw_down, ws)) return MOE_ERR_INVALID_ARG;
  const GradWs L = grad_ws(rows, num_groups, I);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  // da is written while the weight gradients still read a and dy.
  const size_t row_bytes = (size_t)rows * H * 2, w_bytes = (size_t)num_groups * H * I * 2;
  const Span written[] = {{da, row_bytes}, {dw_gate, w_bytes}, {dw_up, w_bytes}, {dw_down, w_bytes}, {ws, L.total}};
  const Span read[] = {{a, row_bytes},       {dy, row_bytes},   {offsets, 4 * ((size_t)num_groups + 1)},
                       {w_gate, w_bytes}, {w_up, w_bytes}, {w_down, w_bytes}};
  for (const Span& w : written) {
    for (const Span& r : read)
      if (overlap(w, r)) return MOE_ERR_INVALID_ARG;
    for (const Span& o : written)
      if (&o != &w && overlap(w, o)) return MOE_ERR_INVALID_ARG;
  }
  const moe_status_t st = bind_handle(h);
  if (st != MOE_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(ws);
  GroupedGradArgs g = {};
  g.G = num_groups;
  g.offsets = offsets;
  g.rows = rows;
  g.H = H;
  g.I = I;
  g.a = a;
  g.dy = dy;
  g.w_gate = w_gate;
  g.w_up = w_up;
  g.w_down = w_down;
  g.odd = reinterpret_cast<int*>(w);
  g.chain = {reinterpret_cast<uint64_t*>(w + 64), reinterpret_cast<uint64_t*>(w + 128), next_call()};
  g.q = reinterpret_cast<float*>(w + L.q);
  g.h = w + L.h;
  g.dg = w + L.dg;
  g.du = w + L.du;
  g.da = da;
  g.dw_gate = dw_gate;
  g.dw_up = dw_up;
  g.dw_down = dw_down;
  g.num_sms = handle_num_sms(h);
  g.status = handle_status_word(h);
  g.wait_limit_ns = handle_wait_limit_ns(h);
  return status_of(launch_grouped_swiglu_backward(g, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
