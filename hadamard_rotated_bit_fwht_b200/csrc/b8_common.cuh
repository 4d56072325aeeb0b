// b8_common.cuh -- device helpers of the block-scaled 8-bit cache.  Nothing
// here is part of the C ABI.
#pragma once

#include "b8_internal.cuh"
#include "decode_common.cuh"

namespace kvq {
namespace b8 {


__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// physical block of column `col` of sequence b; -1 if the column lies outside
// the table or its entry outside [0, num_blocks)
__device__ __forceinline__ int64_t block_of(const kvq_b8_cache &c, int b, int col) {
  if (col < 0 || col >= c.max_blocks_per_seq) return -1;
  const int p = __ldg(c.block_table + (int64_t)b * c.max_blocks_per_seq + col);
  return p < 0 || p >= c.num_blocks ? -1 : p;
}

// amax below 2^-100 counts as 0: 1 / scale stays finite, and such values
// vanish beside any other.  An infinity or a NaN makes it NaN, and with it every
// value of the block.
__device__ __forceinline__ float scale_of(float amax) {
  if (amax - amax != 0.f) return __int_as_float(0x7fc00000);
  return amax < 0x1p-100f ? 0.f : __fdiv_rn(amax, 127.f);
}
__device__ __forceinline__ float inverse(float scale) {
  return scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
}

// rint(x) of 4 values as packed bytes.  The sum with 1.5 * 2^23 rounds to the
// nearest even integer and leaves it in the low byte.  No clamp is needed:
// scale >= RN(amax / 127) and |x| <= amax give |x * RN(1 / scale)| <= 127 (1 +
// 2^-22), which rounds to 127, and old codes shrink.  Blocks of a NaN scale get
// codes without a meaning.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  constexpr float kMagic = 12582912.f;
  auto one = [](float x) { return __float_as_uint(__fadd_rn(x, kMagic)); };
  return __byte_perm(__byte_perm(one(a), one(b), 0x0040), __byte_perm(one(c), one(d), 0x0040),
                     0x5410);
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  return make_uint2(encode4(__fmul_rn(x[0], inv), __fmul_rn(x[1], inv), __fmul_rn(x[2], inv),
                            __fmul_rn(x[3], inv)),
                    encode4(__fmul_rn(x[4], inv), __fmul_rn(x[5], inv), __fmul_rn(x[6], inv),
                            __fmul_rn(x[7], inv)));
}

// rint(x * inv) of 4 values by packed products and sums (mul2_rn_p0 keeps them
// apart; a row's codes after a rotation take longer this way: 166 against 160 us
// for the prompts of b8_quant.cu)
__device__ __forceinline__ uint32_t scaled4(float2 a, float2 b, float inv) {
  const float2 f = make_float2(inv, inv), magic = make_float2(12582912.f, 12582912.f);
  a = add2_rn(mul2_rn_p0(a, f), magic), b = add2_rn(mul2_rn_p0(b, f), magic);
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}

// the 4 codes of a word as exact fp32 values: byte + 128 in the mantissa of
// 2^23, less 2^23 + 128
__device__ __forceinline__ void codes4(uint32_t w, float2 &a, float2 &b) {
  const uint32_t f = w ^ 0x80808080u;
  const float2 bias = make_float2(-8388736.f, -8388736.f);
  auto one = [&](uint32_t sel) { return __uint_as_float(__byte_perm(f, 0x4B000000u, sel)); };
  a = add2_rn(make_float2(one(0x7440), one(0x7441)), bias);
  b = add2_rn(make_float2(one(0x7442), one(0x7443)), bias);
}
__device__ __forceinline__ void decode4(uint32_t w, float scale, float2 &a, float2 &b) {
  const float2 f = make_float2(scale, scale);
  codes4(w, a, b);
  a = mul2(a, f), b = mul2(b, f);
}
__device__ __forceinline__ void decode4(uint32_t w, float scale, float *out) {
  float2 a, b;
  decode4(w, scale, a, b);
  out[0] = a.x, out[1] = a.y, out[2] = b.x, out[3] = b.y;
}
// rint(code * ratio) of 4 codes
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  float2 a, b;
  codes4(w, a, b);
  return scaled4(a, b, ratio);
}

}  // namespace b8
}  // namespace kvq
