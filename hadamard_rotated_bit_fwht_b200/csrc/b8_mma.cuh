// b8_mma.cuh -- the warp-level products over tiles of the block-scaled 8-bit
// cache that the attention and mass kernels share.  Nothing here is part of
// the C ABI.
//
// S = q K^T runs on the integer tensor path (m16n8k32, s8 x s8 -> s32): the K
// codes are B fragments as they lie in memory, nothing is converted.  A query
// row is scaled by 127 * 2^14 / max|q|, rounded to integers n and split exactly
// into int8 digits n = 2^14 H + 2^7 M + L (|M|, |L| <= 64), so its elements are
// off by at most 2^-22 of the row's largest; fp32 queries get a fourth digit,
// 2^-29.  Accumulators start at the bits
// of 1.5 * 2^23: each exact integer sum (below 2^22 for 256 dims) is an fp32
// after one subtraction.
// O^T = V^T P^T runs on the fp16 path (m16n8k16, fp32 accumulation): codes are
// exact in fp16.
//
// A dot product does not depend on the order of its terms, so dims are assigned
// to the fragments in the order in which a thread finds them:
//   S (A = q, B = K): k step 2 blk + s of lane (g, tg) holds dims 64 blk +
//     16 tg + 8 s + {0 .. 3} and {4 .. 7} of token g;
//   O^T (A = V^T, B = P^T): a transposing ldmatrix over pairs of codes gives
//     lane (g, tg) dims 16 c + 2 g and + 1 of tokens 2 tg and 2 tg + 1: rows g
//     and g + 8 of m tile c.  P^T is the accumulator of S as it stands.
#pragma once

#include <cuda_fp16.h>

#include "b8_common.cuh"
#include "decode_common.cuh"

namespace kvq {
namespace b8 {

using dec::ex2;
using dec::mma16816;
using dec::pack_f16x2;
using dec::smem_u32;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kTok = 16;  // tokens of a warp's tile; every block holds whole tiles

// Byte offset of 16-byte chunk `ch` of row r in a staged tile of D-byte rows.
// Chunks of a 128-byte line are permuted so that the eight lanes of one
// shared-memory phase hit different ones: in the K product they read four
// chunks of rows 2p and 2p + 1, a V matrix is one chunk of eight rows.
template <int D>
__device__ __forceinline__ int k_off(int r, int ch) {
  return r * D + 16 * (D == 64 ? ch : ch ^ (4 * (r & 1)));
}
template <int D>
__device__ __forceinline__ int v_off(int r, int ch) {
  return r * D + 16 * (ch ^ (D == 64 ? (r >> 1) & 3 : r & 7));
}

// bytes (sel & 0xf, (sel >> 8) & 0xf) of a sign-flipped word as two exact
// halves: (1024 + c + 128) - 1152
__device__ __forceinline__ uint32_t pair_h2(uint32_t flipped, uint32_t sel) {
  const uint32_t h = __byte_perm(flipped, 0x64646464u, sel);
  const __half2 r =
      __hsub2(*reinterpret_cast<const __half2 *>(&h), __float2half2_rn(1152.f));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// 4 codes of one token -> B fragment of a k step of the K product
__device__ __forceinline__ void k_frag(uint32_t w, uint32_t &b0, uint32_t &b1) {
  const uint32_t f = w ^ 0x80808080u;
  b0 = pair_h2(f, 0x4140);
  b1 = pair_h2(f, 0x4342);
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Power of two that brings amax (>= 0) into [2^13, 2^14); 1 for 0 and
// non-finite values.
__device__ __forceinline__ float query_scale(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23);  // biased exponent
  if (e == 0 || e == 255) return e == 0 && amax > 0.f ? 0x1p126f : 1.f;
  return __uint_as_float((uint32_t)min(max(127 + 13 - (e - 127), 1), 253) << 23);
}

// d = A(s8, 16 x 32, row) * B(s8, 32 x 8, col) + d
__device__ __forceinline__ void imma(uint32_t (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// accumulators begin as the bits of 1.5 * 2^23 and end as an exact fp32
constexpr uint32_t kMagicBits = 0x4B400000u;
__device__ __forceinline__ float isum(uint32_t acc) { return __uint_as_float(acc) - 12582912.f; }

// The queries of a row tile in fragment order: for each k step (D / 32) and
// level 32 lanes x 16 bytes (a0 .. a3).  16 rows: a level a digit.  8 rows: one
// fragment holds the first digit in rows 0 .. 7 and the second in rows 8 .. 15,
// the other the third and (BF16: zeros) the fourth.
template <int D, int R, bool BF16>
struct QTile {
  static constexpr int kLevels = R == 8 ? 2 : BF16 ? 3 : 4;
  static constexpr int kWords = D / 32 * kLevels * 128;
  static constexpr int kBytes = kWords * 4;
};

// digits of dims d0 .. d0 + 3 of row r into the fragment image
template <int D, int R, bool BF16>
__device__ __forceinline__ void q_store(uint32_t *img, int r, int d0, const float (&x)[4]) {
  constexpr int kDigits = BF16 ? 3 : 4;
  uint32_t dig[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    int n = __float2int_rn(x[i]);
#pragma unroll
    for (int v = 0; v < kDigits; v++) {
      const int s = 7 * (kDigits - 1 - v);
      const int h = s ? (n + (1 << s >> 1)) >> s : n;
      n -= h << s;
      dig[v] |= (uint32_t)(h & 255) << (8 * i);
    }
  }
  const int blk = d0 >> 6, tg = (d0 >> 4) & 3, s = (d0 >> 3) & 1, half = (d0 >> 2) & 1;
  constexpr int kL = QTile<D, R, BF16>::kLevels;
  const int g = r & 7;
  uint32_t *at = img + ((2 * blk + s) * kL * 32 + 4 * g + tg) * 4 + 2 * half;
  if (R == 8) {  // a0, a2: row g; a1, a3: row g + 8
    at[0] = dig[0];
    at[1] = dig[1];
    at[128] = dig[2];
    at[129] = dig[3];
  } else {
#pragma unroll
    for (int v = 0; v < kDigits; v++) at[128 * v + (r >> 3)] = dig[v];
  }
}

// The fp16 form for 16 rows of bf16 queries, exact down to 2^-38 of a row's
// largest: for each k step (D / 16) 32 lanes x 16 bytes (a0 .. a3).  Step 4 blk
// + w of lane (g, tg) holds dims 64 blk + 16 tg + 4 w + {0, 1} and {2, 3}, as
// k_frag takes them from the codes.
template <int D>
struct HTile {
  static constexpr int kWords = D / 16 * 128;
};
template <int D>
__device__ __forceinline__ void q_store_half(uint32_t *img, int r, int d0, const float (&x)[4]) {
  const int blk = d0 >> 6, tg = (d0 >> 4) & 3, w = (d0 >> 2) & 3;
  uint32_t *at = img + ((4 * blk + w) * 32 + 4 * (r & 7) + tg) * 4 + (r >> 3);
  at[0] = pack_f16x2(x[0], x[1]);
  at[2] = pack_f16x2(x[2], x[3]);
}

// Raw score of row g + 8 h, column e of an accumulator set s[level][4]: the
// digits' exact sums with their weights.
template <int R, bool BF16>
__device__ __forceinline__ float score(const uint32_t (*s)[4], int h, int e) {
  const float d0 = isum(s[0][2 * h + e]);
  const float d1 = isum(R == 8 ? s[0][2 + e] : s[1][2 * h + e]);
  const float d2 = isum(R == 8 ? s[1][e] : s[2][2 * h + e]);
  const float hi = fmaf(d0, 16384.f, fmaf(d1, 128.f, d2));
  if (BF16) return hi;
  return fmaf(hi, 128.f, isum(R == 8 ? s[1][2 + e] : s[BF16 ? 2 : 3][2 * h + e]));
}

// Fill the images (a row tile after the other) for `rows` rows from row0 on of a
// (sequence, kv head), where row = query * group + head; rows at or past n_rows
// are zero.  inv[r] gets the factor that turns an integer product into a score
// in log2 units.  Each warp takes rows warp, warp + n_warps, ...
// HALF: fp16 images for many rows over the same K fragments (q_store_half).
template <int D, int R, bool BF16, bool HALF = false>
__device__ __forceinline__ void stage_queries(const B8Queries &Q, int q0, int kvh, int row0,
                                              int rows, int n_rows, int warp, int n_warps, int lane,
                                              uint32_t *img, float *inv) {
  constexpr int kPer = D / 128 > 0 ? D / 128 : 1;  // 4-dim groups of a lane
#pragma unroll 4
  for (int r = warp; r < rows; r += n_warps) {
    const int row = row0 + r;
    const bool live = row < n_rows;
    const int i = live ? row / Q.group : 0, j = live ? row - i * Q.group : 0;
    const int64_t at = (int64_t)(q0 + i) * Q.token_stride +
                       (int64_t)(kvh * Q.group + j) * Q.head_stride;
    float x[kPer][4];
    float m = 0.f;
#pragma unroll
    for (int p = 0; p < kPer; p++) {
      const int d0 = 4 * (lane + 32 * p);
      x[p][0] = x[p][1] = x[p][2] = x[p][3] = 0.f;
      if (live && d0 < D) {
        if (BF16) {
          const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(Q.q) + at + d0));
          x[p][0] = bf16lo(u.x), x[p][1] = bf16hi(u.x), x[p][2] = bf16lo(u.y), x[p][3] = bf16hi(u.y);
        } else {
          const float4 u = __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(Q.q) + at + d0));
          x[p][0] = u.x, x[p][1] = u.y, x[p][2] = u.z, x[p][3] = u.w;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; e++) m = fmax_nan(m, fabsf(x[p][e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    // rows of values below 2^-100 score 0 beside any cache; a row with an
    // infinity or NaN scores NaN
    const bool tiny = m < 0x1p-100f;
    const float f = HALF ? query_scale(m) : tiny ? 0.f : __fdiv_rn(BF16 ? 2080768.f : 266338304.f, m);
#pragma unroll
    for (int p = 0; p < kPer; p++) {
      const int d0 = 4 * (lane + 32 * p);
#pragma unroll
      for (int e = 0; e < 4; e++) x[p][e] *= f;
      if (d0 >= D) continue;
      if (HALF)
        q_store_half<D>(img + r / 16 * HTile<D>::kWords, r % 16, d0, x[p]);
      else
        q_store<D, R, BF16>(img + r / R * QTile<D, R, BF16>::kWords, r % R, d0, x[p]);
    }
    if (lane == 0) inv[r] = tiny ? 0.f : m - m == 0.f ? __fdiv_rn(Q.scale * kLog2e, f) : m - m;
  }
}

// first query row and number of query tokens of sequence b; a range that
// leaves [0, total_q) or is longer than max_q counts as none
__device__ __forceinline__ int query_range(const B8Queries &Q, int b, int &q0) {
  if (Q.cu_q == nullptr) {
    q0 = b;
    return b < Q.total_q ? 1 : 0;
  }
  q0 = __ldcg(Q.cu_q + b);
  const int64_t n = (int64_t)__ldcg(Q.cu_q + b + 1) - q0;
  if (q0 < 0 || n <= 0 || n > Q.max_q || q0 + n > Q.total_q) return 0;
  return (int)n;
}

__device__ __forceinline__ int seq_len(const B8Queries &Q, const kvq_b8_cache &c, int b) {
  const int64_t cap = (int64_t)c.max_blocks_per_seq * c.block_size;
  return (int)min((int64_t)min(max(__ldcg(Q.seq_lens + b), 0), Q.max_seq_len), cap);
}

}  // namespace b8
}  // namespace kvq
