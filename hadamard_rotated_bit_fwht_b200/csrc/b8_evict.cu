// b8_evict.cu -- eviction from the block-scaled 8-bit cache (kvq_b8_evict):
// each (sequence, kv head) keeps its first `sinks` tokens, its last `recent`
// and the heaviest of the others by accumulated weight, ties to the lowest
// index; the kept rows are quantized again, block by block, into other blocks.
//
// Selection: one CTA per (sequence, kv head) finds the k-th largest weight by
// a radix select over order-preserving 32-bit keys (digits of 11, 11 and 10
// bits, counted in shared memory), then walks the tokens in order and writes
// the kept indices where a prefix sum puts them.  Requantization: one CTA per
// kept block of a head and plane; rows are held in registers between the
// block's maximum and the rounding, so kept codes are read once.  Bound: HBM.
#include "b8_common.cuh"

namespace kvq {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kWarps = kSelThreads / 32;
constexpr int kBins = 2048;

struct EvictArgs {
  kvq_b8_cache src, dst;
  int batch, max_seq_len, keep, recent, sinks;
  const int32_t *seq_lens;
  const float *mass;
  int64_t mass_stride;
  int32_t *new_lens, *kept;
  float *mass_out;
  int64_t mass_out_stride;
  uint32_t *err;
};

// larger float, larger key; +0 and -0 alike, NaN above everything
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int evict_len(const EvictArgs &a, int b) {
  const int64_t cap = (int64_t)a.src.max_blocks_per_seq * a.src.block_size;
  return (int)min((int64_t)min(max(__ldg(a.seq_lens + b), 0), a.max_seq_len), cap);
}

// grid: kv head + heads * sequence
__global__ void __launch_bounds__(kSelThreads) b8_select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int bins[kBins];
  __shared__ int wsum[2][kWarps];
  __shared__ int found[2];  // digit, elements above it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x, b = unit / a.src.num_kv_heads;
  const int n = evict_len(a, b);
  const int m = min(n, a.keep);
  const float *w = a.mass + (int64_t)unit * a.mass_stride;
  int32_t *kept = a.kept + (int64_t)unit * a.keep;
  float *mout = a.mass_out + (int64_t)unit * a.mass_out_stride;
  if (unit - b * a.src.num_kv_heads == 0 && tid == 0) a.new_lens[b] = m;
  for (int64_t i = m + tid; i < a.mass_out_stride; i += kSelThreads) mout[i] = 0.f;
  for (int i = m + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  if (n <= a.keep) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i, mout[i] = w[i];
    return;
  }
  const int lo = a.sinks, hi = n - a.recent;  // the tokens that compete
  const int k = m - a.sinks - a.recent;       // how many of them stay, < hi - lo

  // the k-th largest key `prefix`, and how many of its equals stay
  uint32_t prefix = 0, mask = 0;
  int need = k;
  if (k > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; pass++) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int nb = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < nb; i += kSelThreads) bins[i] = 0;
      __syncthreads();
#pragma unroll 8
      for (int i = lo + tid; i < hi; i += kSelThreads) {
        const uint32_t key = order_key(w[i]);
        if ((key & mask) == prefix) atomicAdd(&bins[key >> shift & (nb - 1)], 1);
      }
      __syncthreads();
      // elements in bins above each: thread t owns the bins of rank 2 t and
      // 2 t + 1 from the top (one bin in the last pass)
      const int per = nb / kSelThreads;
      const int top = nb - 1 - tid * per;
      const int c0 = bins[top], c1 = per == 2 ? bins[top - 1] : 0;
      int incl = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) wsum[0][warp] = incl;
      __syncthreads();
      int above = incl - c0 - c1;
      for (int i = 0; i < warp; i++) above += wsum[0][i];
      if (above < need && need <= above + c0) found[0] = top, found[1] = above;
      if (above + c0 < need && need <= above + c0 + c1) found[0] = top - 1, found[1] = above + c0;
      __syncthreads();
      prefix |= (uint32_t)found[0] << shift;
      mask |= (uint32_t)(nb - 1) << shift;
      need -= found[1];
      __syncthreads();
    }
  }
  // in order: warp v takes a run of tokens, 32 at a time
  const int run = (n + kWarps * 32 - 1) / (kWarps * 32) * 32;
  const int r0 = min(n, warp * run), r1 = min(n, r0 + run);
  auto kind = [&](int i) {  // 2: kept, 1: equal to the border, 0: dropped
    if (i >= r1) return 0;
    if (i < lo || i >= hi) return 2;
    if (k == 0) return 0;
    const uint32_t key = order_key(w[i]);
    return key > prefix ? 2 : key == prefix ? 1 : 0;
  };
  int over = 0, equal = 0;
#pragma unroll 4
  for (int i = r0; i < r1; i += 32) {
    const int x = kind(i + lane);
    over += __popc(__ballot_sync(0xffffffffu, x == 2));
    equal += __popc(__ballot_sync(0xffffffffu, x == 1));
  }
  if (lane == 0) wsum[0][warp] = over, wsum[1][warp] = equal;
  __syncthreads();
  over = equal = 0;
  for (int i = 0; i < warp; i++) over += wsum[0][i], equal += wsum[1][i];
  const uint32_t below = (1u << lane) - 1;
#pragma unroll 4
  for (int i = r0; i < r1; i += 32) {
    const int x = kind(i + lane);
    const uint32_t o = __ballot_sync(0xffffffffu, x == 2), e = __ballot_sync(0xffffffffu, x == 1);
    const int eq = equal + __popc(e & below);  // equals before this token
    const int at = over + __popc(o & below) + min(eq, need);
    if (x == 2 || (x == 1 && eq < need)) {
      kept[at] = i + lane;
      mout[at] = w[i + lane];
    }
    over += __popc(o);
    equal += __popc(e);
  }
}

constexpr int kItems = 4;  // 16-code pieces a thread holds

// grid: plane (K, V) + 2 * (kept block + cols * (kv head + heads * sequence))
template <int kMost>
__global__ void __launch_bounds__(kMost) b8_requant_kernel(const __grid_constant__ EvictArgs a, int cols) {
  __shared__ float warp_max[32];
  int u = blockIdx.x;
  const bool is_v = u & 1;
  u >>= 1;
  const int col = u % cols;
  u /= cols;  // (sequence, kv head)
  const int hkv = a.src.num_kv_heads, h = u % hkv, b = u / hkv;
  const int bs = a.dst.block_size, D = a.dst.head_dim;
  const int rows = min(bs, min(evict_len(a, b), a.keep) - col * bs);
  if (rows <= 0) return;
  const int64_t to = b8::block_of(a.dst, b, col);
  if (to < 0 || !in_bounds(to, to + 1, a.dst.num_blocks, a.err)) return;
  const int32_t *kept = a.kept + (int64_t)u * a.keep + (int64_t)col * bs;
  const int8_t *codes = is_v ? a.src.v_codes : a.src.k_codes;
  const float *scales = is_v ? a.src.v_scales : a.src.k_scales;
  const int pieces = D / 16, items = rows * pieces;
  uint4 raw[kItems];
  float sc[kItems];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kItems; i++) {
    const int it = threadIdx.x + i * blockDim.x;
    raw[i] = make_uint4(0, 0, 0, 0);
    sc[i] = 0.f;
    if (it < items) {
      const int r = it / pieces, t = kept[r];
      const int64_t slot = b8::block_of(a.src, b, t / a.src.block_size);
      if (slot >= 0 && in_bounds(slot, slot + 1, a.src.num_blocks, a.err)) {
        const int64_t sh = slot * hkv + h;
        raw[i] = *reinterpret_cast<const uint4 *>(
            codes + (sh * a.src.block_size + t % a.src.block_size) * D + 16 * (it - r * pieces));
        sc[i] = scales[sh];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kItems; i++) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float x[4];
      b8::decode4(w[j], sc[i], x);
#pragma unroll
      for (int e = 0; e < 4; e++) amax = fmaxf(amax, fabsf(x[e]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < (int)blockDim.x / 32; w++) amax = fmaxf(amax, warp_max[w]);
  const float scale = b8::scale_of(amax), inv = b8::inverse(scale);
  const int64_t dh = to * hkv + h;
  int8_t *out = (is_v ? a.dst.v_codes : a.dst.k_codes) + dh * bs * D;
#pragma unroll
  for (int i = 0; i < kItems; i++) {
    const int it = threadIdx.x + i * blockDim.x;
    if (it < items) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        float x[4];
        b8::decode4(w[j], sc[i], x);
        o[j] = b8::encode4(__fmul_rn(x[0], inv), __fmul_rn(x[1], inv), __fmul_rn(x[2], inv),
                           __fmul_rn(x[3], inv));
      }
      *reinterpret_cast<uint4 *>(out + 16 * (int64_t)it) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (threadIdx.x == 0) (is_v ? a.dst.v_scales : a.dst.k_scales)[dh] = scale;
}

}  // namespace

cudaError_t launch_b8_evict(const kvq_b8_cache &src, const kvq_b8_cache &dst, int batch,
                            const int32_t *seq_lens, int max_seq_len, const float *mass,
                            int64_t mass_stride, int keep, int recent, int sinks,
                            int32_t *new_lens, int32_t *kept, float *mass_out,
                            int64_t mass_out_stride, cudaStream_t s) {
  const EvictArgs a = {src,  dst,         batch,    max_seq_len, keep,     recent,          sinks, seq_lens,
                       mass, mass_stride, new_lens, kept,        mass_out, mass_out_stride, device_error_word()};
  b8_select_kernel<<<batch * src.num_kv_heads, kSelThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int cols = (min(keep, max_seq_len) + dst.block_size - 1) / dst.block_size;
  if (cols == 0) return cudaSuccess;
  const int items = dst.block_size * (dst.head_dim / 16);
  int threads = 32;
  while (threads < 256 && threads < items) threads *= 2;
  while (threads * kItems < items) threads *= 2;
  const unsigned ctas = (unsigned)(2LL * cols * batch * src.num_kv_heads);
  // blocks above 1024 pieces want up to 1024 threads, whose 64 registers each
  // would spill: two instances
  if (threads <= 256)
    b8_requant_kernel<256><<<ctas, threads, 0, s>>>(a, cols);
  else
    b8_requant_kernel<1024><<<ctas, threads, 0, s>>>(a, cols);
  return cudaGetLastError();
}

}  // namespace kvq
