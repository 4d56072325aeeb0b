// b8_evict.cu -- eviction from the block-scaled 8-bit cache (kvq_b8_evict):
// each (sequence, kv head) keeps its first `sinks` tokens, its last `recent`
// and the heaviest of the others by accumulated weight, ties to the lowest
// index; the kept rows are quantized again, block by block, into other blocks.
//
// Selection: one CTA per (sequence, kv head) finds the k-th largest weight by
// a radix select over order-preserving 32-bit keys (digits of 11, 11 and 10
// bits, counted in shared memory), then walks the tokens in order and writes
// the kept indices where a prefix sum puts them.  Requantization: a warp
// or a CTA per kept block of a head; rows are held in registers between the
// block's maximum and the rounding, so kept codes are read once.  Bound: HBM.
// 16 sequences of 12000 to 16384 tokens to 4096, 8 kv heads, D 128: selection 20
// us (up to 64 KB of weights a CTA, five walks; instructions), requantization 66 us for 268 MB,
// 4.1 TB/s, packed fp32 (72 us by single instructions, 8 a code: both products
// are rounded as an append's).  With the read back 156 us; 158 if the walks ask
// for each key whether it lies in shared memory.
#include <type_traits>

#include "b8_common.cuh"
#include "b8_internal.cuh"

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
__global__ void __launch_bounds__(kSelThreads)
    b8_select_kernel(const __grid_constant__ EvictArgs a, int cached) {
  extern __shared__ uint32_t keys[];  // of the first `cached` tokens
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

  const int nc = min(n, cached);
#pragma unroll 8
  for (int i = tid; i < nc; i += kSelThreads) keys[i] = order_key(w[i]);
  __syncthreads();
  // all: every key lies in shared memory
  auto select = [&](auto all) {
    auto key_of = [&](int i) { return decltype(all)::value || i < nc ? keys[i] : order_key(w[i]); };

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
          const uint32_t key = key_of(i);
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
        // the warps before this one (as many as a warp has lanes)
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[0][lane] : 0);
        const int above = before + incl - c0 - c1;
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
    // is token i kept for certain; does it equal the border
    auto kind = [&](int i, bool &over, bool &equal) {
      const uint32_t key = i < r1 ? key_of(i) : 0u;
      const bool free = i >= lo && i < hi;
      over = i < r1 && (!free || (k > 0 && key > prefix));
      equal = i < r1 && free && k > 0 && key == prefix;
    };
    int over = 0, equal = 0;
#pragma unroll 4
    for (int i = r0 + lane; i < r1; i += 32) {
      bool o, e;
      kind(i, o, e);
      over += o;
      equal += e;
    }
    over = __reduce_add_sync(0xffffffffu, over);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) wsum[0][warp] = over, wsum[1][warp] = equal;
    __syncthreads();
    over = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[0][lane] : 0);
    equal = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[1][lane] : 0);
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 4
    for (int i = r0; i < r1; i += 32) {
      bool is_over, is_equal;
      kind(i + lane, is_over, is_equal);
      const uint32_t o = __ballot_sync(0xffffffffu, is_over), e = __ballot_sync(0xffffffffu, is_equal);
      const int eq = equal + __popc(e & below);  // equals before this token
      const int at = over + __popc(o & below) + min(eq, need);
      if (is_over || (is_equal && eq < need)) {
        kept[at] = i + lane;
        mout[at] = w[i + lane];
      }
      over += __popc(o);
      equal += __popc(e);
    }
  };
  if (n <= nc)
    select(std::true_type());
  else
    select(std::false_type());
}

// A block of a head is 1 to 16 runs of 4 KB a plane; one warp holds its run of
// K and V (8 16-byte pieces a lane and plane) in registers between the block's
// maximum and the rounding.  Warps walk many blocks: while the codes of one are
// on their way, the scales and table entries of the next one's rows and the
// kept indices of the one after are too (a row or two a lane), so that the
// chain index -> block -> scale costs no time of its own.
constexpr int kItems = 8;

// two bytes of w as signed 16-bit values (a selector's high bit repeats the
// byte's sign, which __byte_perm does not offer)
template <uint32_t kSel>
__device__ __forceinline__ uint32_t sext2(uint32_t w) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(kSel));
  return r;
}

// Blocks of one run: a warp each.  Larger ones: a CTA of `runs` warps each.
// unit: kept block + cols * (kv head + heads * sequence)
template <int D>
__global__ void __launch_bounds__(512)
    b8_requant_kernel(const __grid_constant__ EvictArgs a, int cols, int runs, int64_t units) {
  __shared__ float warp_max[2][2][16];
  constexpr int kPieces = D / 16, kRows = 4096 / D, kMine = (kRows + 31) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int run = runs > 1 ? warp : 0, r0 = run * kRows;
  const int64_t stride = runs > 1 ? gridDim.x : (int64_t)gridDim.x * (blockDim.x / 32);
  int64_t unit = runs > 1 ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / 32) + warp;
  const int hkv = a.src.num_kv_heads;
  const int bs = a.dst.block_size, sbs = a.src.block_size, shift = __ffs(sbs) - 1;

  // kept index of the lane's row i of a unit's run, -1 if there is none
  auto load_kept = [&](int64_t u, int (&t)[kMine]) {
#pragma unroll
    for (int i = 0; i < kMine; i++) t[i] = -1;
    if (u >= units) return;
    const int64_t bh = u / cols;
    const int row0 = (int)(u - bh * cols) * bs + r0;
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      const int r = lane + 32 * i;
      // entries behind the last kept token are -1
      if (r < kRows && r0 + r < bs && row0 + r < a.keep) t[i] = __ldcg(a.kept + bh * a.keep + row0 + r);
    }
  };
  // its block and, on lane 0, the block that the unit goes to
  auto load_slots = [&](int64_t u, const int (&t)[kMine], int (&slot)[kMine], int &to) {
    to = -1;
    if (u >= units) return;
    const int64_t bh = u / cols;
    const int b = (int)(bh / hkv);
#pragma unroll
    for (int i = 0; i < kMine; i++)
      slot[i] = t[i] < 0 ? -1 : (int)b8::block_of(a.src, b, t[i] >> shift);
    to = (int)b8::block_of(a.dst, b, (int)(u - bh * cols));
  };
  int t[kMine], slot[kMine], to;
  load_kept(unit, t);
  load_slots(unit, t, slot, to);
  int t2[kMine];
  load_kept(unit + stride, t2);
  int parity = 0;
  for (; unit < units; unit += stride, parity ^= 1) {
    const int64_t bh = unit / cols;
    const int h = (int)(bh % hkv);
    int64_t src[kMine];
    float ks[kMine], vs[kMine];
#pragma unroll
    for (int i = 0; i < kMine; i++) {
      src[i] = -1;
      ks[i] = vs[i] = 0.f;
      if (slot[i] >= 0 && in_bounds(slot[i], slot[i] + 1, a.src.num_blocks, a.err)) {
        const int64_t sh = (int64_t)slot[i] * hkv + h;
        src[i] = ((sh << shift) + (t[i] & (sbs - 1))) * D;
        ks[i] = a.src.k_scales[sh];
        vs[i] = a.src.v_scales[sh];
      }
    }
    const int dst = to;
    // rows of the run that are kept (an unmapped source stores zeros)
    uint32_t has[kMine];
#pragma unroll
    for (int i = 0; i < kMine; i++) has[i] = __ballot_sync(0xffffffffu, t[i] >= 0);
    uint4 raw[2][kItems];
#pragma unroll
    for (int i = 0; i < kItems; i++) {
      // row of the run; whether it is one of the lanes' first or second rows
      // goes by i alone
      const int r = (lane + 32 * i) / kPieces;
      const int64_t at = __shfl_sync(0xffffffffu, src[32 * i / kPieces / 32], r & 31);
      raw[0][i] = raw[1][i] = make_uint4(0, 0, 0, 0);
      if (at >= 0) {
        raw[0][i] = *reinterpret_cast<const uint4 *>(a.src.k_codes + at + 16 * (lane % kPieces));
        raw[1][i] = *reinterpret_cast<const uint4 *>(a.src.v_codes + at + 16 * (lane % kPieces));
      }
    }
    // the next units' indices
#pragma unroll
    for (int i = 0; i < kMine; i++) t[i] = t2[i];
    load_slots(unit + stride, t, slot, to);
    load_kept(unit + 2 * stride, t2);

    float amax[2] = {0.f, 0.f};
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
      for (int i = 0; i < kItems; i++) {
        const float sc = __shfl_sync(0xffffffffu, (p ? vs : ks)[32 * i / kPieces / 32],
                                     (lane + 32 * i) / kPieces & 31);
        const uint32_t w[4] = {raw[p][i].x, raw[p][i].y, raw[p][i].z, raw[p][i].w};
        // the largest magnitude of the codes (rounding keeps the order), over
        // their even and odd bytes as pairs of 16 bits
        uint32_t top = 0, low = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t even = sext2<0xA280>(w[j]), odd = sext2<0xB391>(w[j]);
          top = __vimax3_s16x2(top, even, odd);
          low = __vimin3_s16x2(low, even, odd);
        }
        const int hi = max((int)(int16_t)top, (int)top >> 16);
        const int lo = min((int)(int16_t)low, (int)low >> 16);
        const int m = max(hi, -lo);
        amax[p] = fmax_nan(amax[p], __fmul_rn((float)m, sc));
      }
#pragma unroll
    for (int p = 0; p < 2; p++)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        amax[p] = fmax_nan(amax[p], __shfl_xor_sync(0xffffffffu, amax[p], o));
    if (runs > 1) {
      // two sets, so that one barrier a unit is enough
      if (lane == 0) warp_max[parity][0][warp] = amax[0], warp_max[parity][1][warp] = amax[1];
      __syncthreads();
      for (int w = 0; w < runs; w++) {
        amax[0] = fmax_nan(amax[0], warp_max[parity][0][w]);
        amax[1] = fmax_nan(amax[1], warp_max[parity][1][w]);
      }
    }
    // a block without kept tokens, or one that is not mapped, is left alone
    const int first = (int)(unit - bh * cols) * bs;
    const bool store = dst >= 0 && first < min(evict_len(a, (int)(bh / hkv)), a.keep) &&
                       in_bounds(dst, (int64_t)dst + 1, a.dst.num_blocks, a.err);
    if (!store) continue;
    const int64_t dh = (int64_t)dst * hkv + h;
#pragma unroll
    for (int p = 0; p < 2; p++) {
      const float scale = b8::scale_of(amax[p]), inv = b8::inverse(scale);
      int8_t *out = (p ? a.dst.v_codes : a.dst.k_codes) + (dh * bs + r0) * D;
#pragma unroll
      for (int i = 0; i < kItems; i++) {
        const int r = (lane + 32 * i) / kPieces;
        const float sc =
            __shfl_sync(0xffffffffu, (p ? vs : ks)[32 * i / kPieces / 32], r & 31);
        const uint32_t w[4] = {raw[p][i].x, raw[p][i].y, raw[p][i].z, raw[p][i].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          float2 x, y;
          b8::decode4(w[j], sc, x, y);
          o[j] = b8::scaled4(x, y, inv);
        }
        if (has[32 * i / kPieces / 32] >> (r & 31) & 1)
          *reinterpret_cast<uint4 *>(out + 16 * (lane + 32 * i)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (lane == 0 && run == 0) (p ? a.dst.v_scales : a.dst.k_scales)[dh] = scale;
    }
  }
}

}  // namespace

cudaError_t launch_b8_evict(const kvq_b8_cache &src, const kvq_b8_cache &dst, int batch,
                            const int32_t *seq_lens, int max_seq_len, const float *mass,
                            int64_t mass_stride, int keep, int recent, int sinks,
                            int32_t *new_lens, int32_t *kept, float *mass_out,
                            int64_t mass_out_stride, cudaStream_t s) {
  const EvictArgs a = {src,  dst,         batch,    max_seq_len, keep,     recent,          sinks, seq_lens,
                       mass, mass_stride, new_lens, kept,        mass_out, mass_out_stride, device_error_word()};
  // keys of up to 48 K tokens stay in shared memory between the passes
  const int cached = min(max_seq_len, 49152);
  cudaError_t e = allow_smem<b8_select_kernel>(49152 * 4);
  if (e != cudaSuccess) return e;
  b8_select_kernel<<<batch * src.num_kv_heads, kSelThreads, cached * 4, s>>>(a, cached);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int cols = (min(keep, max_seq_len) + dst.block_size - 1) / dst.block_size;
  if (cols == 0) return cudaSuccess;
  const int64_t units = (int64_t)cols * batch * src.num_kv_heads;
  const int runs = max(1, dst.block_size * dst.head_dim / 4096);
  const int threads = runs > 1 ? 32 * runs : 128;
  // 16 warps an SM hold 128 KB of codes
  const int64_t resident = (int64_t)kNumSMs * max(1, 512 / threads);
  const unsigned ctas = (unsigned)min(runs > 1 ? units : (units + 3) / 4, resident);
  switch (dst.head_dim) {
    case 64: b8_requant_kernel<64><<<ctas, threads, 0, s>>>(a, cols, runs, units); break;
    case 128: b8_requant_kernel<128><<<ctas, threads, 0, s>>>(a, cols, runs, units); break;
    default: b8_requant_kernel<256><<<ctas, threads, 0, s>>>(a, cols, runs, units); break;
  }
  return cudaGetLastError();
}

}  // namespace kvq
