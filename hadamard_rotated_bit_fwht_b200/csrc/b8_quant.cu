// b8_quant.cu -- append to and read back from the block-scaled 8-bit cache
// (kvq_b8_append, kvq_b8_gather).
//
// Per (block, kv head) of K or V: scale = max(amax / 127, old), codes
// rint(x / scale).  One CTA owns one block of one head, so the scale, the new
// codes and the rescaled older codes have one writer and nothing depends on
// an order.  The new rows are read once and kept in registers between the
// maximum and the rounding; blocks too large for that (more than kItems
// 16-element pieces a thread) are read a second time, from L2.
#include "b8_common.cuh"
#include "rope.cuh"

namespace kvq {
namespace {

using namespace rope;

constexpr int kThreads = 256;
constexpr int kItems = 4;  // pieces of 16 elements a thread keeps

// grid: (touched block of the sequence + cols * (2 * sequence + is_v), kv head)
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
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

  auto fetch = [&](int it, float (&x)[8], float (&y)[8], int &row, Piece &p) {
    row = it / pieces;
    p = piece(it - row * pieces, rot, spec.interleaved);
    const int64_t tok = (int64_t)b * t_new + (lo - start) + row;
    const int64_t at = tok * src.token_stride + h * src.head_stride;
    Raw8<BF16> ra, rb;
    load8<BF16>(src.data, at + p.a, ra);
    load8<BF16>(src.data, at + p.b, rb);
    widen8<BF16>(ra, x);
    widen8<BF16>(rb, y);
    if (p.pair >= 0) {
      const int pos = rope_pos ? __ldg(rope_pos + tok) : (int)(lo + row);
      float2 cs[8];
#pragma unroll
      for (int e = 0; e < 8; e++) cs[e] = turn(pos, __ldg(spec.d_inv_freq + p.pair + e), spec.factor);
      rotate_piece(x, y, cs, spec.interleaved);
    }
  };

  const bool keep = items <= kItems * (int)blockDim.x;
  float xs[kItems][8], ys[kItems][8];
  float amax = 0.f;
  if (keep) {
#pragma unroll
    for (int i = 0; i < kItems; i++) {
      const int it = threadIdx.x + i * blockDim.x;
      if (it < items) {
        int row;
        Piece p;
        fetch(it, xs[i], ys[i], row, p);
#pragma unroll
        for (int e = 0; e < 8; e++) amax = fmaxf(amax, fmaxf(fabsf(xs[i][e]), fabsf(ys[i][e])));
      }
    }
  } else {
    for (int it = threadIdx.x; it < items; it += blockDim.x) {
      int row;
      Piece p;
      float x[8], y[8];
      fetch(it, x, y, row, p);
#pragma unroll
      for (int e = 0; e < 8; e++) amax = fmaxf(amax, fmaxf(fabsf(x[e]), fabsf(y[e])));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; w++) amax = fmaxf(amax, warp_max[w]);
  const float scale = fmaxf(b8::scale_of(amax), old);
  const float inv = b8::inverse(scale);

  auto put = [&](const float (&x)[8], const float (&y)[8], int row, const Piece &p) {
    int8_t *at = codes + (int64_t)(r0 + row) * D;
    *reinterpret_cast<uint2 *>(at + p.a) = b8::encode8(x, inv);
    *reinterpret_cast<uint2 *>(at + p.b) = b8::encode8(y, inv);
  };
  if (keep) {
#pragma unroll
    for (int i = 0; i < kItems; i++) {
      const int it = threadIdx.x + i * blockDim.x;
      if (it < items) {
        const int row = it / pieces;
        put(xs[i], ys[i], row, piece(it - row * pieces, rot, spec.interleaved));
      }
    }
  } else {
    for (int it = threadIdx.x; it < items; it += blockDim.x) {
      int row;
      Piece p;
      float x[8], y[8];
      fetch(it, x, y, row, p);
      put(x, y, row, p);
    }
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

// grid-stride over 16-element pieces of the output; adjacent threads take
// adjacent 16-byte code chunks
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    b8_gather_kernel(kvq_b8_cache c, int64_t total, int count,
                     const int32_t *__restrict__ first, const int32_t *__restrict__ ends,
                     void *__restrict__ k_out, void *__restrict__ v_out,
                     uint32_t *__restrict__ err) {
  const int pieces = c.head_dim / 16;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / pieces;
    const int j = (int)(i - row * pieces);
    const int64_t bt = row / c.num_kv_heads;
    const int h = (int)(row - bt * c.num_kv_heads);
    const int b = (int)(bt / count);
    const int64_t t = (int64_t)__ldg(first + b) + (bt - (int64_t)b * count);
    int64_t slot = -1;
    if (t >= 0 && t < __ldg(ends + b) && t < (int64_t)c.max_blocks_per_seq * c.block_size)
      slot = b8::block_of(c, b, (int)(t / c.block_size));
    if (slot >= 0 && !in_bounds(slot, slot + 1, c.num_blocks, err)) slot = -1;
    const int64_t sh = slot * c.num_kv_heads + h;
    const int64_t at = (sh * c.block_size + t % c.block_size) * c.head_dim + 16 * j;
    const int64_t to = row * c.head_dim + 16 * j;
#pragma unroll
    for (int w = 0; w < 2; w++) {
      float x[8] = {}, y[8] = {};
      if (slot >= 0) {
        const uint4 u = *reinterpret_cast<const uint4 *>((w ? c.v_codes : c.k_codes) + at);
        const float s = (w ? c.v_scales : c.k_scales)[sh];
        b8::decode4(u.x, s, x), b8::decode4(u.y, s, x + 4);
        b8::decode4(u.z, s, y), b8::decode4(u.w, s, y + 4);
      }
      void *out = w ? v_out : k_out;
      store8<BF16>(out, to, x);
      store8<BF16>(out, to + 8, y);
    }
  }
}

}  // namespace

cudaError_t launch_b8_append(const kvq_b8_cache &c, const kvq_heads &k, const kvq_heads &v,
                             int bf16, int batch, int t_new, const int32_t *start_pos,
                             const int32_t *new_lens, const kvq_rope_spec &spec,
                             const int32_t *rope_pos, cudaStream_t s) {
  const int cols = min((t_new + c.block_size - 2) / c.block_size + 1, c.max_blocks_per_seq);
  const int items = min(t_new, c.block_size) * (c.head_dim / 16);
  int threads = 32;
  while (threads < kThreads && threads < items) threads *= 2;
  const dim3 grid((unsigned)cols * 2u * batch, c.num_kv_heads);
  uint32_t *err = device_error_word();
  if (bf16)
    b8_append_kernel<true><<<grid, threads, 0, s>>>(c, k, v, t_new, cols, start_pos, new_lens, spec,
                                                    rope_pos, err);
  else
    b8_append_kernel<false><<<grid, threads, 0, s>>>(c, k, v, t_new, cols, start_pos, new_lens, spec,
                                                     rope_pos, err);
  return cudaGetLastError();
}

cudaError_t launch_b8_gather(const kvq_b8_cache &c, int batch, const int32_t *first,
                             const int32_t *ends, int count, int bf16, void *k_out, void *v_out,
                             cudaStream_t s) {
  const int64_t total = (int64_t)batch * count * c.num_kv_heads * (c.head_dim / 16);
  const int64_t want = (total + kThreads - 1) / kThreads;
  const int ctas = (int)min(want, (int64_t)kNumSMs * 8);
  uint32_t *err = device_error_word();
  if (bf16)
    b8_gather_kernel<true><<<ctas, kThreads, 0, s>>>(c, total, count, first, ends, k_out, v_out, err);
  else
    b8_gather_kernel<false><<<ctas, kThreads, 0, s>>>(c, total, count, first, ends, k_out, v_out, err);
  return cudaGetLastError();
}

}  // namespace kvq
