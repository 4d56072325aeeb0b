// b8_quant.cu -- append to and read back from the block-scaled 8-bit cache
// (kvq_b8_append, kvq_b8_gather).
//
// Per (block, kv head) of K or V: scale = max(amax / 127, old), codes
// rint(x / scale).  One CTA owns one block of one head, so the scale, the new
// codes and the rescaled older codes have one writer and nothing depends on
// an order.  The new rows are read once: all of them are copied to shared
// memory at once, and between the maximum and the rounding their rotated fp32
// values wait there, over what they came from (a thread handles its own 16
// elements throughout).  Blocks too large for that (more than kKeep bytes) are
// read and rotated a second time.
//
// Prompts of 8 sequences (197 thousand rows of 256 dims of K and of V, bf16, K
// rotated, blocks of 64): append 109 us, 303 MB; issue slots 63 % used, the
// angles a third of them (49 us at a plain copy's rate).  Read back: 51 us, 5.9
// TB/s, two thirds of it stores.  One token in each of 64 sequences: 5.5 us and
// 4.4 us, launches and chains of dependent loads.
#include "b8_common.cuh"
#include "rope.cuh"

namespace kvq {
namespace {

using namespace rope;

constexpr int kThreads = 256;
constexpr int kKeep = 64 * 1024;  // fp32 bytes of a block's new rows, three CTAs an SM
constexpr int kAhead = 2;         // pieces whose loads are in flight together

// grid: (touched block of the sequence + cols * (2 * sequence + is_v), kv head)
template <bool BF16, bool KEEP>
__global__ void __launch_bounds__(kThreads, 3)
    b8_append_kernel(kvq_b8_cache c, kvq_heads k, kvq_heads v, int t_new, int cols,
                     const int32_t *__restrict__ start_pos, const int32_t *__restrict__ new_lens,
                     kvq_rope_spec spec, const int32_t *__restrict__ rope_pos,
                     uint32_t *__restrict__ err) {
  __shared__ float warp_max[kThreads / 32];
  const int unit = blockIdx.x / cols, b = unit >> 1, h = blockIdx.y;
  const bool is_v = unit & 1;
  const int start = __ldg(start_pos + b);
  const int n_new = new_lens ? min(max(__ldg(new_lens + b), 0), t_new) : t_new;
  const int bs = c.block_size, D = c.head_dim;
  // positions in 64 bits: start + n_new may pass 2^31
  const int64_t end = min((int64_t)start + n_new, (int64_t)c.max_blocks_per_seq * bs);
  const int64_t first = max(start, 0);
  const int64_t col = first / bs + (blockIdx.x - unit * cols);
  const int64_t lo = max(first, col * bs), hi = min(end, (col + 1) * bs);
  if (lo >= hi) return;
  const int64_t slot = b8::block_of(c, b, (int)col);
  if (slot < 0) return;
  const kvq_heads &src = is_v ? v : k;
  int8_t *codes = (is_v ? c.v_codes : c.k_codes) + (slot * c.num_kv_heads + h) * bs * D;
  float *scale_at = (is_v ? c.v_scales : c.k_scales) + slot * c.num_kv_heads + h;
  if (!in_bounds(slot, slot + 1, c.num_blocks, err)) return;
  const int r0 = (int)(lo - col * bs);       // first new row of the block
  const float old = start > col * bs ? *scale_at : 0.f;
  const int pieces = D / 16, items = (int)(hi - lo) * pieces;
  const bool turned = !is_v && spec.d_inv_freq != nullptr;
  const int rot = turned ? spec.rot_dim : 0;

  // blockDim is a multiple of the pieces of a row: a thread's pieces are the
  // same dims of different rows
  const Piece p = piece(threadIdx.x & (pieces - 1), rot, spec.interleaved);
  const int row_shift = __ffs(pieces) - 1;
  const int64_t tok0 = (int64_t)b * t_new + (lo - start);
  extern __shared__ float4 kept[];  // [piece of the thread][4][thread]
  if (KEEP) {
    int n = 0;
    for (int it = threadIdx.x; it < items; it += blockDim.x, n++) {
      const int64_t at = (tok0 + (it >> row_shift)) * src.token_stride + h * src.head_stride;
      const uint32_t to = dec::smem_u32(kept + (size_t)n * 4 * blockDim.x + threadIdx.x);
      constexpr int kEach = BF16 ? 1 : 2;  // 16-byte chunks of 8 elements
      const char *base = static_cast<const char *>(src.data);
#pragma unroll
      for (int k = 0; k < 2 * kEach; k++)
        b8::cp_async16(to + k * 16 * blockDim.x,
                       base + (at + (k < kEach ? p.a : p.b)) * (BF16 ? 2 : 4) + 16 * (k % kEach));
    }
    b8::cp_commit();
  }
  uint64_t rate[8];
  if (p.pair >= 0) {
#pragma unroll
    for (int e = 0; e < 8; e++) rate[e] = turn_rate(__ldg(spec.d_inv_freq + p.pair + e));
  }
  auto turned_piece = [&](int row, const Raw8<BF16> &ra, const Raw8<BF16> &rb, float (&x)[8],
                          float (&y)[8]) {
    widen8<BF16>(ra, x);
    widen8<BF16>(rb, y);
    if (p.pair >= 0) {
      const int pos = rope_pos ? __ldg(rope_pos + tok0 + row) : (int)(lo + row);
      const Pos at = position(pos, spec.factor);
      float2 cs[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float2 cc, ss;
        turn2(at, rate[e], rate[e + 1], cc, ss);
        cs[e] = make_float2(cc.x, ss.x);
        cs[e + 1] = make_float2(cc.y, ss.y);
      }
      rotate_piece(x, y, cs, spec.interleaved);
    }
  };
  auto put = [&](const float (&x)[8], const float (&y)[8], int row, float inv) {
    int8_t *at = codes + (int64_t)(r0 + row) * D;
    *reinterpret_cast<uint2 *>(at + p.a) = b8::encode8(x, inv);
    *reinterpret_cast<uint2 *>(at + p.b) = b8::encode8(y, inv);
  };
  // every piece of the thread, kAhead at a time: f(row, x, y)
  auto each = [&](auto f) {
    for (int it = threadIdx.x; it < items; it += kAhead * blockDim.x) {
      Raw8<BF16> ra[kAhead], rb[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; k++) {
        const int row = (it + k * (int)blockDim.x) >> row_shift;
        if (it + k * (int)blockDim.x < items) {
          const int64_t at = (tok0 + row) * src.token_stride + h * src.head_stride;
          load8<BF16>(src.data, at + p.a, ra[k]);
          load8<BF16>(src.data, at + p.b, rb[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; k++) {
        const int row = (it + k * (int)blockDim.x) >> row_shift;
        if (it + k * (int)blockDim.x < items) {
          float x[8], y[8];
          turned_piece(row, ra[k], rb[k], x, y);
          f(row, x, y);
        }
      }
    }
  };
  float amax = 0.f;
  auto raise = [&](const float (&x)[8], const float (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e++) amax = fmax_nan(amax, fmax_nan(fabsf(x[e]), fabsf(y[e])));
  };
  if (KEEP) {
    b8::cp_wait<0>();
    int n = 0;
    for (int it = threadIdx.x; it < items; it += blockDim.x, n++) {
      float4 *at = kept + (size_t)n * 4 * blockDim.x + threadIdx.x;
      Raw8<BF16> ra, rb;
      constexpr int kEach = BF16 ? 1 : 2;
#pragma unroll
      for (int k = 0; k < kEach; k++) {
        ra.r[k] = *reinterpret_cast<const uint4 *>(at + k * blockDim.x);
        rb.r[k] = *reinterpret_cast<const uint4 *>(at + (kEach + k) * blockDim.x);
      }
      float x[8], y[8];
      turned_piece(it >> row_shift, ra, rb, x, y);
      raise(x, y);
      at[0] = make_float4(x[0], x[1], x[2], x[3]);
      at[blockDim.x] = make_float4(x[4], x[5], x[6], x[7]);
      at[2 * blockDim.x] = make_float4(y[0], y[1], y[2], y[3]);
      at[3 * blockDim.x] = make_float4(y[4], y[5], y[6], y[7]);
    }
  } else {
    each([&](int, const float (&x)[8], const float (&y)[8]) { raise(x, y); });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; w++) amax = fmax_nan(amax, warp_max[w]);
  const float scale = fmax_nan(b8::scale_of(amax), old);
  const float inv = b8::inverse(scale);

  if (KEEP) {
    int n = 0;
    for (int it = threadIdx.x; it < items; it += blockDim.x, n++) {
      const float4 *at = kept + (size_t)n * 4 * blockDim.x + threadIdx.x;
      const float4 u0 = at[0], u1 = at[blockDim.x], v0 = at[2 * blockDim.x], v1 = at[3 * blockDim.x];
      const float x[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
      const float y[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      put(x, y, it >> row_shift, inv);
    }
  } else {
    each([&](int row, const float (&x)[8], const float (&y)[8]) { put(x, y, row, inv); });
  }
  // the block's earlier rows follow a scale that grew
  if (old > 0.f && scale > old) {
    const float ratio = __fdiv_rn(old, scale);
    for (int it = threadIdx.x; it < r0 * pieces; it += blockDim.x) {
      uint4 *at = reinterpret_cast<uint4 *>(codes) + it;
      uint4 w = *at;
      w.x = b8::rescale4(w.x, ratio), w.y = b8::rescale4(w.y, ratio);
      w.z = b8::rescale4(w.z, ratio), w.w = b8::rescale4(w.w, ratio);
      *at = w;
    }
  }
  if (threadIdx.x == 0) *scale_at = scale;
}

// 32 bytes to `at`; wide: it is 32-byte aligned
__device__ __forceinline__ void store32(void *at, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4 *p = static_cast<uint4 *>(at);
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// 16 codes as values at element `elem`
template <bool BF16>
__device__ __forceinline__ void decode16(void *base, int64_t elem, const uint4 &codes, float scale,
                                         bool wide) {
  float x[16];
  b8::decode4(codes.x, scale, x), b8::decode4(codes.y, scale, x + 4);
  b8::decode4(codes.z, scale, x + 8), b8::decode4(codes.w, scale, x + 12);
  uint32_t w[8];
  if (BF16) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    store32(static_cast<uint16_t *>(base) + elem, w, wide);
  } else {
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int i = 0; i < 8; i++) w[i] = __float_as_uint(x[8 * h + i]);
      store32(static_cast<float *>(base) + elem + 8 * h, w, wide);
    }
  }
}

// grid: (run of 256 pieces of a sequence's rows, sequence).  A piece is 16
// elements of K and of V, stored 32 bytes at a time where the outputs are
// aligned to that: 134 MB of codes to 268 MB of bf16 take 60 us, two 16-byte
// stores a piece 78.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads)
    b8_gather_kernel(kvq_b8_cache c, uint32_t total, int count,
                     const int32_t *__restrict__ first, const int32_t *__restrict__ ends,
                     void *__restrict__ k_out, void *__restrict__ v_out, bool wide,
                     uint32_t *__restrict__ err) {
  constexpr uint32_t kPieces = D / 16;
  const int b = blockIdx.y;
  const uint32_t hkv = c.num_kv_heads;
  const int shift = __ffs(c.block_size) - 1;
  const int64_t t0 = __ldg(first + b);
  const int64_t cap = min((int64_t)__ldg(ends + b), (int64_t)c.max_blocks_per_seq * c.block_size);
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const uint32_t row = i / kPieces, tok = row / hkv, h = row - tok * hkv;
  const int64_t t = t0 + tok;
  int64_t slot = -1;
  if (t >= 0 && t < cap) slot = b8::block_of(c, b, (int)(t >> shift));
  uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
  float ks = 0.f, vs = 0.f;
  if (slot >= 0 && in_bounds(slot, slot + 1, c.num_blocks, err)) {
    const int64_t sh = slot * hkv + h;
    const int64_t at = ((sh << shift) + (t & (c.block_size - 1))) * D + 16 * (i % kPieces);
    kw = __ldg(reinterpret_cast<const uint4 *>(c.k_codes + at));
    vw = __ldg(reinterpret_cast<const uint4 *>(c.v_codes + at));
    ks = __ldg(c.k_scales + sh);
    vs = __ldg(c.v_scales + sh);
  }
  const int64_t to = ((int64_t)b * total + i) * 16;
  decode16<BF16>(k_out, to, kw, ks, wide);
  decode16<BF16>(v_out, to, vw, vs, wide);
}

}  // namespace

template <bool BF16, bool KEEP>
static cudaError_t append(const kvq_b8_cache &c, const kvq_heads &k, const kvq_heads &v, dim3 grid,
                          int threads, int smem, int cols, int t_new,
                          const int32_t *start_pos, const int32_t *new_lens,
                          const kvq_rope_spec &spec, const int32_t *rope_pos, cudaStream_t s) {
  // (48 KB hold the kernel's own few bytes too)
  if (smem > 32 * 1024) {
    const cudaError_t e = allow_smem<b8_append_kernel<BF16, KEEP>>(kKeep);
    if (e != cudaSuccess) return e;
  }
  b8_append_kernel<BF16, KEEP><<<grid, threads, smem, s>>>(c, k, v, t_new, cols, start_pos, new_lens, spec, rope_pos,
                                device_error_word());
  return cudaGetLastError();
}

cudaError_t launch_b8_append(const kvq_b8_cache &c, const kvq_heads &k, const kvq_heads &v,
                             int bf16, int batch, int t_new, const int32_t *start_pos,
                             const int32_t *new_lens, const kvq_rope_spec &spec,
                             const int32_t *rope_pos, cudaStream_t s) {
  const int cols = (int)min(((int64_t)t_new + c.block_size - 2) / c.block_size + 1,
                            (int64_t)c.max_blocks_per_seq);
  const int items = min(t_new, c.block_size) * (c.head_dim / 16);
  int threads = 32;
  while (threads < kThreads && threads < items) threads *= 2;
  const dim3 grid((unsigned)cols * 2u * batch, c.num_kv_heads);
  // 64 bytes a piece, whole rounds of the threads
  const int64_t bytes = (int64_t)(items + threads - 1) / threads * threads * 64;
  const bool keep = bytes <= kKeep;
  auto *f = bf16 ? (keep ? append<true, true> : append<true, false>)
                 : (keep ? append<false, true> : append<false, false>);
  return f(c, k, v, grid, threads, keep ? (int)bytes : 0, cols, t_new, start_pos, new_lens, spec,
           rope_pos, s);
}

template <bool BF16, int D>
static void gather(const kvq_b8_cache &c, int batch, const int32_t *first, const int32_t *ends,
                   int count, void *k_out, void *v_out, cudaStream_t s) {
  const uint32_t total = (uint32_t)count * c.num_kv_heads * (D / 16);
  const bool wide = (reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) % 32 == 0;
  const dim3 grid((total + kThreads - 1) / kThreads, batch);
  b8_gather_kernel<BF16, D><<<grid, kThreads, 0, s>>>(c, total, count, first, ends, k_out, v_out, wide,
                                                      device_error_word());
}

cudaError_t launch_b8_gather(const kvq_b8_cache &c, int batch, const int32_t *first,
                             const int32_t *ends, int count, int bf16, void *k_out, void *v_out,
                             cudaStream_t s) {
  auto *f = c.head_dim == 64    ? (bf16 ? gather<true, 64> : gather<false, 64>)
            : c.head_dim == 128 ? (bf16 ? gather<true, 128> : gather<false, 128>)
                                : (bf16 ? gather<true, 256> : gather<false, 256>);
  f(c, batch, first, ends, count, k_out, v_out, s);
  return cudaGetLastError();
}

}  // namespace kvq
