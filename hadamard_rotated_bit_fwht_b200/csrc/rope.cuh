// rope.cuh -- rotary positions: the angle of a pair, and the rotation of the
// 16-element pieces that the rope and append kernels work in.  Nothing here is
// part of the C ABI.
#pragma once

#include <cuda_bf16.h>

#include "b8_internal.cuh"

namespace kvq {
namespace rope {

// Angles are counted in 2^-64 turns, modulo one turn: an integer product with
// the position wraps exactly, however far the position.  turn_rate turns
// radians per position into that unit (fp64: w / 2 pi has a relative error of
// 2^-52, so the angle is off by 2^-52 of the turns made).
__device__ __forceinline__ uint64_t turn_rate(double w) {
  const double f = w * 0.15915494309189533577;
  return (uint64_t)__double2ll_rn((f - rint(f)) * 0x1p63) << 1;
}
// A position as the multiplier of two rates and the factor's sign for sines.
struct Pos {
  uint32_t u;
  float cf, sf;  // factors on cosine and sine
};
__device__ __forceinline__ Pos position(int pos, float factor) {
  return {pos < 0 ? 0u - (uint32_t)pos : (uint32_t)pos, factor, pos < 0 ? -factor : factor};
}
// cos t and sin t of two pairs, times the factors.  The leading 32 bits of each
// angle are cut into a quadrant and a rest of at most an eighth of a turn (30
// bits, rounded to fp32: at most 2^-25 of pi / 4); Taylor's series on the rest
// up to x^9 and x^10 leave 1.8e-9 and 1.1e-10 there.  CUDA's sincospif took two
// thirds of the append kernel's instructions.
__device__ __forceinline__ void turn2(const Pos &p, uint64_t r0, uint64_t r1, float2 &c, float2 &s) {
  uint32_t quad[2];
  float2 x;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint64_t r = i ? r1 : r0;
    const uint32_t hi = __umulhi((uint32_t)r, p.u) + (uint32_t)(r >> 32) * p.u;
    quad[i] = (hi + 0x20000000u) >> 30;
    (i ? x.y : x.x) = (float)(int)(hi - (quad[i] << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  }
  const float2 q = mul2(x, x);
  auto k = [](float v) { return make_float2(v, v); };
  float2 sn = __ffma2_rn(q, k(2.75573192e-6f), k(-1.98412698e-4f));
  float2 cn = __ffma2_rn(q, k(-2.75573192e-7f), k(2.48015873e-5f));
  cn = __ffma2_rn(q, cn, k(-1.38888889e-3f));
  sn = __ffma2_rn(q, sn, k(8.33333333e-3f));
  cn = __ffma2_rn(q, cn, k(4.16666667e-2f));
  sn = __ffma2_rn(q, sn, k(-1.66666667e-1f));
  cn = __ffma2_rn(q, cn, k(-0.5f));
  sn = __ffma2_rn(mul2(q, x), sn, x);
  cn = __ffma2_rn(q, cn, k(1.f));
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const float a = i ? cn.y : cn.x, b = i ? sn.y : sn.x;
    const bool odd = quad[i] & 1;
    // quadrants 0 .. 3: (c, s), (-s, c), (-c, -s), (s, -c)
    const uint32_t cs = ((quad[i] + 1) & 2) << 30, ss = (quad[i] & 2) << 30;
    (i ? c.y : c.x) = __uint_as_float(__float_as_uint(odd ? b : a) ^ cs) * p.cf;
    (i ? s.y : s.x) = __uint_as_float(__float_as_uint(odd ? a : b) ^ ss) * p.sf;
  }
}

// 8 consecutive elements in fp32, in registers; 16-byte aligned addresses
template <bool BF16>
struct Raw8 {
  uint4 r[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ void load8(const void *base, int64_t elem, Raw8<BF16> &x) {
  if (BF16) {
    x.r[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + elem);
  } else {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + elem);
    x.r[0] = p[0];
    x.r[BF16 ? 0 : 1] = p[1];
  }
}
template <bool BF16>
__device__ __forceinline__ void widen8(const Raw8<BF16> &x, float (&v)[8]) {
  if (BF16) {
    const uint32_t w[4] = {x.r[0].x, x.r[0].y, x.r[0].z, x.r[0].w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint4 u = x.r[BF16 ? 0 : i];
      v[4 * i] = __uint_as_float(u.x), v[4 * i + 1] = __uint_as_float(u.y);
      v[4 * i + 2] = __uint_as_float(u.z), v[4 * i + 3] = __uint_as_float(u.w);
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void *base, int64_t elem, const float (&v)[8]) {
  if (BF16) {
    uint4 u;
    uint32_t *w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + elem) = u;
  } else {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + elem);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// A head of D dims falls into D / 16 pieces of two 8-element groups that hold
// whole pairs: piece j < rot / 16 of the rotated dims holds pairs 8j .. 8j + 7
// (groups at 8j and rot / 2 + 8j, or 16j and 16j + 8 when interleaved), the
// others dims 16j .. 16j + 15.
struct Piece {
  int a, b;  // first dim of each group
  int pair;  // first pair, -1 if not rotated
};
__device__ __forceinline__ Piece piece(int j, int rot, int interleaved) {
  Piece p;
  const bool turned = j < rot / 16;
  const bool halves = turned && !interleaved;
  p.a = halves ? 8 * j : 16 * j;
  p.b = halves ? rot / 2 + 8 * j : 16 * j + 8;
  p.pair = turned ? 8 * j : -1;
  return p;
}
// rotate a piece in place; cs[i] = (cos, sin) of pair i of the piece.  Products
// and sums are rounded one by one, as the plain formula does: what is quantized
// next then falls on the same side of a code's border.
__device__ __forceinline__ void rotate_pair(float &a, float &b, float2 cs) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
  b = __fadd_rn(__fmul_rn(y, cs.x), __fmul_rn(x, cs.y));
}
__device__ __forceinline__ void rotate_piece(float (&u)[8], float (&v)[8], const float2 *cs,
                                             int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      rotate_pair(u[2 * i], u[2 * i + 1], cs[i]);
      rotate_pair(v[2 * i], v[2 * i + 1], cs[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) rotate_pair(u[i], v[i], cs[i]);
  }
}

}  // namespace rope
}  // namespace kvq
