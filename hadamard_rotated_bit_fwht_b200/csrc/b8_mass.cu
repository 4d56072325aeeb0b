// b8_mass.cu -- accumulated attention weight of the block-scaled 8-bit cache
// (kvq_b8_attn_mass): mass[b][h][t] += sum over the rows (query, head of the
// group) that attend to token t of exp(score - lse).
//
// One CTA takes a range of tokens of a (sequence, kv head); a warp takes
// kTiles 16-token tiles at a time, converts their K codes to fp16 fragments
// once and runs every row over them, so each token has one owner: no atomics,
// and the sum's order depends on the sizes alone.  Rows come in chunks staged
// in shared memory (once if one chunk holds them all).  Bound for a few rows:
// the K codes from HBM.
#include "b8_mma.cuh"

namespace kvq {
namespace {

using namespace b8;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

template <int D, bool HILO>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;   // 16-token tiles of a warp's step
  static constexpr int kTileBytes = kTok * D;
  static constexpr int kStageBytes = kTiles * (kTileBytes + 16);  // + k_scale
  static constexpr int kStages = 2;  // 64 KB in flight per SM
  static constexpr int kChunk = 64;  // rows staged at once
  using Q = QTile<D, 16, HILO>;
  static constexpr int kOffQ = kWarps * kStages * kStageBytes;
  static constexpr int kOffInv = kOffQ + kChunk / 16 * Q::kBytes;
  static constexpr int kOffLse = kOffInv + kChunk * 4;
  static constexpr int kOffLim = kOffLse + kChunk * 4;
  static constexpr int kSmem = kOffLim + kChunk * 4;
  static constexpr int kCtas = D == 256 && HILO ? 1 : 2;
  static_assert((kSmem + 1024) * kCtas <= 228 * 1024, "shared memory per SM");
};

struct MassArgs {
  kvq_b8_cache c;
  B8Queries q;
  const float *lse;
  float *mass;
  int64_t mass_stride;
  int ranges, range_tokens;
  uint32_t *err;
};

// grid: range + ranges * (kv head + heads * sequence)
template <int D, bool HILO>
__global__ void __launch_bounds__(kThreads, Cfg<D, HILO>::kCtas)
    b8_mass_kernel(const __grid_constant__ MassArgs a) {
  using C = Cfg<D, HILO>;
  constexpr int kKs = D / 16, kL = C::Q::kLevels, kT = C::kTiles;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tg = lane & 3;
  const kvq_b8_cache &c = a.c;
  int u = blockIdx.x;
  const int range = u % a.ranges;
  u /= a.ranges;
  const int kvh = u % c.num_kv_heads, b = u / c.num_kv_heads;
  int q0;
  const int nq = query_range(a.q, b, q0);
  const int n_rows = nq * a.q.group;
  const int len = seq_len(a.q, c, b);
  const int t0 = range * a.range_tokens, t1 = min(len, t0 + a.range_tokens);
  if (n_rows == 0 || t0 >= t1) return;

  uint32_t *qimg = reinterpret_cast<uint32_t *>(smem + C::kOffQ);
  float *inv_s = reinterpret_cast<float *>(smem + C::kOffInv);
  float *lse_s = reinterpret_cast<float *>(smem + C::kOffLse);
  int *lim_s = reinterpret_cast<int *>(smem + C::kOffLim);

  // step it of this warp: tiles first + it * 8 * kT + {0 .. kT - 1}
  const int first = t0 / kTok + warp * kT, end = (t1 + kTok - 1) / kTok;
  const int n_steps = (end - t0 / kTok + kWarps * kT - 1) / (kWarps * kT);  // of the CTA
  uint8_t *ring = smem + warp * C::kStages * C::kStageBytes;
  const int per_block = c.block_size / kTok;
  const int32_t *table = c.block_table + (int64_t)b * c.max_blocks_per_seq;
  int page_base = 0, page[kT];
  auto load_pages = [&](int base) {
    page_base = base;
#pragma unroll
    for (int k = 0; k < kT; k++) {
      const int tile = first + (base + lane) * kWarps * kT + k;
      page[k] = tile < end ? __ldg(table + tile / per_block) : -1;
      if (page[k] >= c.num_blocks) page[k] = -1;
    }
  };
  uint32_t live = 0;  // bit kT * stage + k
  auto issue = [&](int it) {
    const int st = it % C::kStages;
    if (it < n_steps) {
      if (it >= page_base + 32) load_pages(it);
#pragma unroll
      for (int k = 0; k < kT; k++) {
        const int slot = __shfl_sync(0xffffffffu, page[k], it - page_base);
        const int tile = first + it * kWarps * kT + k;
        const uint32_t bit = 1u << (kT * st + k);
        const bool mapped = slot >= 0 && in_bounds(slot, slot + 1, c.num_blocks, a.err);
        live = mapped ? live | bit : live & ~bit;
        if (mapped) {
          const int64_t sh = (int64_t)slot * c.num_kv_heads + kvh;
          const int8_t *src = c.k_codes + (sh * c.block_size + tile % per_block * kTok) * D;
          const uint32_t dst =
              smem_u32(ring + st * C::kStageBytes + k * (C::kTileBytes + 16));
#pragma unroll
          for (int i = 0; i < C::kTileBytes / 512; i++) {
            const int ch = lane + 32 * i;
            cp_async16(dst + k_off<D>(ch / (D / 16), ch % (D / 16)), src + 16 * ch);
          }
          if (lane == 0) cp_async4(dst + C::kTileBytes, c.k_scales + sh);
        }
      }
    }
    cp_commit();
  };
  load_pages(0);
#pragma unroll
  for (int i = 0; i < C::kStages - 1; i++) issue(i);

  const int n_chunks = (n_rows + C::kChunk - 1) / C::kChunk;
  auto stage_chunk = [&](int row0) {
    const int tiles = (min(C::kChunk, n_rows - row0) + 15) / 16;
    for (int t = 0; t < tiles; t++)
      stage_queries<D, 16, HILO>(a.q, q0, kvh, row0 + 16 * t, n_rows, warp, kWarps, lane,
                                 qimg + t * C::Q::kWords, inv_s + 16 * t);
    for (int r = tid; r < 16 * tiles; r += kThreads) {
      const int row = row0 + r;
      float x = INFINITY;  // exp2(s - inf): nothing
      int lim = 0;
      if (row < n_rows) {
        const int i = row / a.q.group;
        const int64_t at = (int64_t)(q0 + i) * a.q.num_heads + kvh * a.q.group + row - i * a.q.group;
        x = __ldg(a.lse + at) * kLog2e;
        if (x == -INFINITY) x = INFINITY;
        lim = max(0, len - nq + i + 1);
      }
      lse_s[r] = x;
      lim_s[r] = lim;
    }
  };
  if (n_chunks == 1) {
    stage_chunk(0);
    __syncthreads();
  }

  float *out = a.mass + ((int64_t)b * c.num_kv_heads + kvh) * a.mass_stride;
  for (int it = 0; it < n_steps; it++) {
    cp_wait<C::kStages - 2>();
    __syncwarp();
    issue(it + C::kStages - 1);
    const int st = it % C::kStages;
    const uint32_t on = live >> (kT * st) & ((1u << kT) - 1);
    const int tok = (first + it * kWarps * kT) * kTok;
    uint32_t kf[kT * 2][kKs][2];
    float ksc[kT];
    if (on) {
#pragma unroll
      for (int k = 0; k < kT; k++) {
        const uint8_t *kt = ring + st * C::kStageBytes + k * (C::kTileBytes + 16);
        ksc[k] = on >> k & 1 ? *reinterpret_cast<const float *>(kt + C::kTileBytes) : 0.f;
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
          for (int blk = 0; blk < D / 64; blk++) {
            const uint4 w = *reinterpret_cast<const uint4 *>(kt + k_off<D>(8 * n + g, 4 * blk + tg));
#pragma unroll
            for (int i = 0; i < 4; i++)
              k_frag(word(w, i), kf[2 * k + n][4 * blk + i][0], kf[2 * k + n][4 * blk + i][1]);
          }
      }
    }
    float sum[kT * 2][2];
#pragma unroll
    for (int n = 0; n < kT * 2; n++) sum[n][0] = sum[n][1] = 0.f;
    for (int ch = 0; ch < n_chunks; ch++) {
      const int row0 = ch * C::kChunk;
      if (n_chunks > 1) {
        // rows that see none of the CTA's tokens of this step
        const int i_last = (min(row0 + C::kChunk, n_rows) - 1) / a.q.group;
        if (len - nq + i_last + 1 <= (t0 / kTok + it * kWarps * kT) * kTok) continue;
        __syncthreads();
        stage_chunk(row0);
        __syncthreads();
      }
      if (!on) continue;
      const int tiles = (min(C::kChunk, n_rows - row0) + 15) / 16;
      for (int t = 0; t < tiles; t++) {
        // limits grow with the row; rows past the end have limit 0
        const int last = min(row0 + 16 * t + 16, n_rows) - row0 - 1;
        if (lim_s[last] <= tok) continue;
        const uint32_t *img = qimg + t * C::Q::kWords;
        float s[kT * 2][4];
#pragma unroll
        for (int n = 0; n < kT * 2; n++)
#pragma unroll
          for (int e = 0; e < 4; e++) s[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < kKs; ks++) {
#pragma unroll
          for (int v = 0; v < kL; v++) {
            const uint4 qa = *reinterpret_cast<const uint4 *>(img + ((ks * kL + v) * 32 + lane) * 4);
#pragma unroll
            for (int n = 0; n < kT * 2; n++) mma16816(s[n], qa, kf[n][ks][0], kf[n][ks][1]);
          }
        }
        const float l0 = lse_s[16 * t + g], l1 = lse_s[16 * t + g + 8];
        const float i0 = inv_s[16 * t + g], i1 = inv_s[16 * t + g + 8];
        const int m0 = lim_s[16 * t + g], m1 = lim_s[16 * t + g + 8];
        const bool cut = tok + kT * kTok > lim_s[16 * t] || last != 16 * t + 15;
#pragma unroll
        for (int n = 0; n < kT * 2; n++) {
          const float f0 = i0 * ksc[n >> 1], f1 = i1 * ksc[n >> 1];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float p0 = ex2(s[n][e] * f0 - l0), p1 = ex2(s[n][2 + e] * f1 - l1);
            if (cut) {
              const int at = tok + 8 * n + 2 * tg + e;
              p0 = at < m0 ? p0 : 0.f;
              p1 = at < m1 ? p1 : 0.f;
            }
            sum[n][e] += p0 + p1;
          }
        }
      }
    }
    if (!on) continue;
#pragma unroll
    for (int n = 0; n < kT * 2; n++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum[n][e] += __shfl_xor_sync(0xffffffffu, sum[n][e], o);
        const int at = tok + 8 * n + 2 * tg + e;
        // one lane of the eight that hold the sum writes it
        if (g == n && at < t1 && (on >> (n >> 1) & 1)) out[at] += sum[n][e];
      }
  }
  cp_wait<0>();
}

template <int D, bool HILO>
cudaError_t launch(const MassArgs &a, cudaStream_t s) {
  using C = Cfg<D, HILO>;
  auto *k = b8_mass_kernel<D, HILO>;
  const cudaError_t e =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  k<<<(unsigned)((int64_t)a.q.batch * a.c.num_kv_heads * a.ranges), kThreads, C::kSmem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_b8_mass(const kvq_b8_cache &c, const B8Queries &q, const float *lse,
                           float *mass, int64_t mass_stride, cudaStream_t s) {
  MassArgs a = {c, q, lse, mass, mass_stride, 1, 0, device_error_word()};
  const int64_t len =
      max((int64_t)1, min((int64_t)q.max_seq_len, (int64_t)c.max_blocks_per_seq * c.block_size));
  const int64_t granule = kWarps * kTok * (c.head_dim == 256 ? 1 : 2);
  const int64_t units = (int64_t)q.batch * c.num_kv_heads;
  const int64_t most = (len + granule - 1) / granule;
  const int64_t resident = kNumSMs * 2;
  int64_t want = max((resident + units - 1) / units, min((4 * resident + units - 1) / units, (len + 2047) / 2048));
  want = max((int64_t)1, min(want, most));
  a.range_tokens = (int)(((len + want - 1) / want + granule - 1) / granule * granule);
  a.ranges = (int)((len + a.range_tokens - 1) / a.range_tokens);
  switch (c.head_dim) {
    case 64: return q.bf16 ? launch<64, false>(a, s) : launch<64, true>(a, s);
    case 128: return q.bf16 ? launch<128, false>(a, s) : launch<128, true>(a, s);
    default: return q.bf16 ? launch<256, false>(a, s) : launch<256, true>(a, s);
  }
}

}  // namespace kvq
