// E4M3 values with one fp32 scale per block of 128: the rule by which every
// kernel that writes them makes a block's scale and codes.
//   scale = max(amax / 448, 2^-126)      code = E4M3(v / scale), to nearest even, saturating
// The floor keeps 1 / scale finite; an all-zero block has it, with codes 0. A
// block with an infinity or NaN gets that as its scale and the code NaN for
// every value, so what it stands for is NaN throughout.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

namespace moe {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;
constexpr float kFp8LeastScale = 1.17549435e-38f;  // 2^-126

__host__ __device__ inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// |v| as an integer that orders as |v| does, NaN above infinity, so that a
// maximum over a block keeps a NaN.
__device__ __forceinline__ uint32_t fp8_abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) / kFp8Max;
  return s < kFp8LeastScale ? kFp8LeastScale : s;  // a NaN stays
}

__device__ __forceinline__ uint32_t fp8_pack2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  return fp8_pack2(a, b) | fp8_pack2(c, d) << 16;
}
// v / scale rounded once to fp32, as the division is, by one Newton step on the
// quotient (P. Markstein, 1990): with inv = 1 / scale rounded to nearest, y0 = v
// inv is within an ulp and y0 + inv (v - y0 scale) rounds to the quotient. The
// two extra instructions replace a division per value (about ten).
struct Fp8Block {
  float scale, inv;
  __device__ __forceinline__ explicit Fp8Block(float s) : scale(s), inv(1.0f / s) {}
  __device__ __forceinline__ Fp8Block(float s, float i) : scale(s), inv(i) {}
  __device__ __forceinline__ float over(float v) const {
    const float y0 = v * inv;
    return fmaf(fmaf(-y0, scale, v), inv, y0);
  }
  __device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) const {
    return fp8_pack4(over(a), over(b), over(c), over(d));
  }
};

}  // namespace moe
