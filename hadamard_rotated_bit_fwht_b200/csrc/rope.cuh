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
// cos t and sin t, times factor.  The leading 32 bits of the angle become
// half turns in [-1, 1) in fp32, whose rounding moves the angle by at most
// 2^-25 half turns, 9.4e-8 radians: the size of fp32's own rounding of the
// products that follow.
__device__ __forceinline__ float2 turn(int pos, uint64_t rate, float factor) {
  const int hi = (int)((rate * (uint64_t)(int64_t)pos) >> 32);
  float s, c;
  sincospif((float)hi * 0x1p-31f, &s, &c);
  return make_float2(c * factor, s * factor);
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
// rotate a piece in place; cs[i] = (cos, sin) of pair i of the piece
__device__ __forceinline__ void rotate_piece(float (&u)[8], float (&v)[8], const float2 *cs,
                                             int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float a = u[2 * i], b = u[2 * i + 1];
      u[2 * i] = a * cs[i].x - b * cs[i].y;
      u[2 * i + 1] = b * cs[i].x + a * cs[i].y;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = a * cs[4 + i].x - b * cs[4 + i].y;
      v[2 * i + 1] = b * cs[4 + i].x + a * cs[4 + i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float a = u[i], b = v[i];
      u[i] = a * cs[i].x - b * cs[i].y;
      v[i] = b * cs[i].x + a * cs[i].y;
    }
  }
}

}  // namespace rope
}  // namespace kvq
