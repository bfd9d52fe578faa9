// E4M3 values with one fp32 scale per block of 128: the rule by which every
// kernel that writes them makes a block's scale and codes.
//   scale = max(amax / 448, 2^-126)      code = E4M3(v / scale), to nearest even, saturating
// The floor keeps 1 / scale finite; an all-zero block has it, with codes 0. A
// block with an infinity or NaN gets that as its scale and the code NaN for
// every value, so what it stands for is NaN throughout.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

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
// inv is off by up to 1.5 ulp, and y0 + inv (v - y0 scale) is the rounded quotient.
// Tried for every mantissa of the scale and values up to three steps of fp32 to
// either side of each border between two codes: equal, as long as the remainder v -
// y0 scale has all of its bits, which scales below about 2^-93 do not leave it (a
// remainder of 2^-149's size is lost, and at 2^-120 every fiftieth of such values took
// the neighbouring code). Below 2^-80 value and scale are therefore multiplied by 2^64
// first, which changes nothing else. The steps replace a division per value (about ten
// instructions).
constexpr uint32_t kFp8LeastBits = 1u << 23, kFp8SmallBits = (127u - 80) << 23;  // 2^-126, 2^-80
constexpr float kFp8Lift = 1.84467441e19f;                                       // 2^64
struct Fp8Block {
  float scale, inv;
  __device__ __forceinline__ explicit Fp8Block(float s) : scale(s), inv(1.0f / s) {}
  __device__ __forceinline__ Fp8Block(float s, float i) : scale(s), inv(i) {}
  // In (2^-126, 2^-80): the least scale is a power of two, whose quotients are exact.
  __device__ __forceinline__ bool small() const {
    return __float_as_uint(scale) - (kFp8LeastBits + 1) < kFp8SmallBits - (kFp8LeastBits + 1);
  }
  // SMALL: any scale, each lifted by itself; else none that is small.
  template <bool SMALL>
  __device__ __forceinline__ float over(float v) const {
    const float lift = SMALL && small() ? kFp8Lift : 1.0f;
    const float u = v * lift, s = scale * lift, i = SMALL && small() ? inv * (1.0f / kFp8Lift) : inv, y0 = u * i;
    return fmaf(fmaf(-y0, s, u), i, y0);
  }
  template <bool SMALL>
  __device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) const {
    return fp8_pack4(over<SMALL>(a), over<SMALL>(b), over<SMALL>(c), over<SMALL>(d));
  }
};
// work(whether scales may be small): one branch around a thread's codes.
template <typename W>
__device__ __forceinline__ void fp8_by_size(bool small, W&& work) {
  if (small) work(std::true_type{});
  else work(std::false_type{});
}

}  // namespace moe
