// b8_mma.cuh -- the warp-level products over tiles of the block-scaled 8-bit
// cache that the attention and mass kernels share.  Nothing here is part of
// the C ABI.
//
// Codes are integers of at most 8 bits, exact in fp16, so both products run on
// the fp16 tensor path (m16n8k16, fp32 accumulation).  Queries are scaled by a
// power of two that brings the row's largest magnitude to [2^13, 2^14): a bf16
// query is then exact in fp16 down to 2^-38 of that maximum, an fp32 query is
// split into hi + lo, 22 bits.
//
// A dot product does not depend on the order of its terms, so dims and tokens
// are assigned to the fragments in the order in which a thread finds them in
// 16-byte pieces of a row; no transpose or ldmatrix is needed:
//   S = q K^T (A = q, B = K): k step 4 blk + w of lane (g, tg) holds dims
//     64 blk + 16 tg + 4 w + {0, 1} and {2, 3} of token g;
//   O^T = V^T P^T (A = V^T, B = P^T): rows g and g + 8 of m tile j are dims
//     16 g + 2 j and 16 g + 2 j + 1 (of each 128; 8 g + 2 j for D = 64), so a
//     lane takes 16 consecutive dims of its tokens 2 tg, 2 tg + 1, 2 tg + 8,
//     2 tg + 9, and P^T is the accumulator of S as it stands.
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

// Byte offset of 16-byte chunk `ch` of row r in a staged tile of D-byte rows.
// Chunks of a 128-byte line are permuted so that the eight lanes of one
// shared-memory phase hit different chunks: in the K product they read four
// chunks of rows 2p and 2p + 1, in the V product two chunks of rows i, i + 2,
// i + 4, i + 6.
template <int D>
__device__ __forceinline__ int k_off(int r, int ch) {
  return r * D + 16 * (D == 64 ? ch : ch ^ (4 * (r & 1)));
}
template <int D>
__device__ __forceinline__ int v_off(int r, int ch) {
  const int at = r * (D / 16) + ch;  // chunk of the tile
  return 16 * (at ^ (2 * ((r >> 1) & 3)));
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

// The queries of a row tile in fragment order.  For each k step (D / 16) and
// level (1: fp16, or hi; 2: lo) 32 lanes x 16 bytes (a0..a3).  With 8 rows and
// two levels the low part takes rows 8..15 of the one fragment.
template <int D, int R, bool HILO>
struct QTile {
  static constexpr int kLevels = HILO && R == 16 ? 2 : 1;
  static constexpr int kWords = D / 16 * kLevels * 128;
  static constexpr int kBytes = kWords * 4;
};

// elements 4 x of one row (fp32, scaled) into the fragment image: dims d0 ..
// d0 + 3 of row r
template <int D, int R, bool HILO>
__device__ __forceinline__ void q_store(uint32_t *img, int r, int d0, const float (&x)[4]) {
  const int blk = d0 >> 6, tg = (d0 >> 4) & 3, w = (d0 >> 2) & 3, ks = 4 * blk + w;
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int i = 0; i < 2; i++) dec::split_hilo(make_float2(x[2 * i], x[2 * i + 1]), hi[i], lo[i]);
  const int g = r & 7, half = r >> 3;  // a0, a2: rows g; a1, a3: rows g + 8
  constexpr int kL = QTile<D, R, HILO>::kLevels;
  uint32_t *at = img + (ks * kL * 32 + 4 * g + tg) * 4;
  at[half] = hi[0];
  at[2 + half] = hi[1];
  if (R == 8) {
    at[1] = HILO ? lo[0] : 0u;
    at[3] = HILO ? lo[1] : 0u;
  } else if (HILO) {
    at[128 + half] = lo[0];
    at[128 + 2 + half] = lo[1];
  }
}

// Fill the image for rows row0 .. row0 + R - 1 of a (sequence, kv head), where
// row = query * group + head; rows at or past n_rows are zero.  inv[r] gets the
// factor that turns a raw product into a score: scale / query_scale.  Each warp
// takes rows warp, warp + kWarps, ...
template <int D, int R, bool HILO>
__device__ __forceinline__ void stage_queries(const B8Queries &Q, int q0, int kvh, int row0,
                                              int n_rows, int warp, int n_warps, int lane,
                                              uint32_t *img, float *inv) {
  constexpr int kPer = D / 128 > 0 ? D / 128 : 1;  // 4-dim groups of a lane
  for (int r = warp; r < R; r += n_warps) {
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
        if (HILO) {
          const float4 u = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(Q.q) + at + d0));
          x[p][0] = u.x, x[p][1] = u.y, x[p][2] = u.z, x[p][3] = u.w;
        } else {
          const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(Q.q) + at + d0));
          x[p][0] = bf16lo(u.x), x[p][1] = bf16hi(u.x), x[p][2] = bf16lo(u.y), x[p][3] = bf16hi(u.y);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; e++) m = fmax_nan(m, fabsf(x[p][e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float f = query_scale(m);
#pragma unroll
    for (int p = 0; p < kPer; p++) {
      const int d0 = 4 * (lane + 32 * p);
#pragma unroll
      for (int e = 0; e < 4; e++) x[p][e] *= f;
      if (d0 < D) q_store<D, R, HILO>(img, r, d0, x[p]);
    }
    // scale / f in log2 units; f is a power of two, so the quotient is exact
    if (lane == 0) inv[r] = __fdiv_rn(Q.scale * kLog2e, f);
  }
}

// first query row and number of query tokens of sequence b; a range that
// leaves [0, total_q) or is longer than max_q counts as none
__device__ __forceinline__ int query_range(const B8Queries &Q, int b, int &q0) {
  if (Q.cu_q == nullptr) {
    q0 = b;
    return b < Q.total_q ? 1 : 0;
  }
  q0 = __ldg(Q.cu_q + b);
  const int64_t n = (int64_t)__ldg(Q.cu_q + b + 1) - q0;
  if (q0 < 0 || n <= 0 || n > Q.max_q || q0 + n > Q.total_q) return 0;
  return (int)n;
}

__device__ __forceinline__ int seq_len(const B8Queries &Q, const kvq_b8_cache &c, int b) {
  const int64_t cap = (int64_t)c.max_blocks_per_seq * c.block_size;
  return (int)min((int64_t)min(max(__ldg(Q.seq_lens + b), 0), Q.max_seq_len), cap);
}

}  // namespace b8
}  // namespace kvq
