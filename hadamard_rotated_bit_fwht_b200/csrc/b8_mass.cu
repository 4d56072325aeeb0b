// b8_mass.cu -- accumulated attention weight of the block-scaled 8-bit cache
// (kvq_b8_attn_mass): mass[b][h][t] += sum over the rows (query, head of the
// group) that attend to token t of exp(score - lse).
//
// One CTA takes a range of tokens of a (sequence, kv head); a warp takes
// kTiles 16-token tiles at a time and runs every row over them, so each token
// has one owner, and the sum's order depends on the sizes alone.  Rows come in
// chunks of up to kChunk staged in shared memory; every chunk walks the CTA's
// tokens, which then come from L2.  Bound for a few rows: the K codes from HBM.
// 32 sequences of 2048 to 16384 tokens, 8 kv heads, D 128, one query each: 70
// us, 4.6 TB/s (71 % of a plain copy; issue slots 51 % used, uneven ends).  The
// last 32 queries of 4 prompts (128 rows): 35 us, a fourth of it the staging of
// the rows, the rest latency at 16 warps an SM (40 us with 16 tokens a step, whose
// query fragments are read from shared memory twice as often).
#include "b8_mma.cuh"

namespace kvq {
namespace {

using namespace b8;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

template <int D, int R, bool BF16>
struct Cfg {
  // many bf16 rows: fp16 products, K codes converted once for all of them
  static constexpr bool kHalf = R == 16 && BF16;
  // 16-token tiles of a warp's step
  static constexpr int kTiles = D == 256 || (R == 16 && !kHalf) ? 1 : 2;
  static constexpr int kTileBytes = kTok * D;
  static constexpr int kStageBytes = kTiles * (kTileBytes + 16);  // + k_scale
  static constexpr int kStages = kHalf && kTiles == 2 ? 2 : 3;  // 64 to 128 KB in flight an SM
  static constexpr int kChunk = R == 8 ? 8 : 128;   // rows staged at once
  static constexpr int kQWords = kHalf ? HTile<D>::kWords : QTile<D, R, BF16>::kWords;
  static constexpr int kOffInv = kWarps * kStages * kStageBytes;
  static constexpr int kOffLse = kOffInv + kChunk * 4;
  static constexpr int kOffLim = kOffLse + kChunk * 4;
  static constexpr int kOffQ = kOffLim + kChunk * 4;  // last: as many row tiles as there are
  static constexpr int smem(int row_tiles) { return kOffQ + row_tiles * kQWords * 4; }
  static_assert(smem(kChunk / R) <= 227 * 1024, "shared memory per CTA");
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
template <int D, int R, bool BF16>
__global__ void __launch_bounds__(kThreads, 2)
    b8_mass_kernel(const __grid_constant__ MassArgs a) {
  using C = Cfg<D, R, BF16>;
  constexpr int kKs = D / 32, kL = QTile<D, R, BF16>::kLevels, kT = C::kTiles;
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
  // (the last range may end past 2^31)
  const int t0 = range * a.range_tokens, t1 = (int)min((int64_t)len, (int64_t)t0 + a.range_tokens);
  if (n_rows == 0 || t0 >= t1) return;

  uint32_t *qimg = reinterpret_cast<uint32_t *>(smem + C::kOffQ);
  float *inv_s = reinterpret_cast<float *>(smem + C::kOffInv);
  float *lse_s = reinterpret_cast<float *>(smem + C::kOffLse);
  int *lim_s = reinterpret_cast<int *>(smem + C::kOffLim);

  // step it of this warp: tiles first + it * 8 * kT + {0 .. kT - 1}
  const int first = t0 / kTok + warp * kT;
  int end = 0, n_steps = 0;  // of the chunk at hand
  uint8_t *ring = smem + warp * C::kStages * C::kStageBytes;
  const int per_block = c.block_size / kTok, pb_shift = __ffs(per_block) - 1;
  const int32_t *table = c.block_table + (int64_t)b * c.max_blocks_per_seq;
  int page_base = 0, page[kT];
  auto load_pages = [&](int base) {
    page_base = base;
#pragma unroll
    for (int k = 0; k < kT; k++) {
      const int tile = first + (base + lane) * kWarps * kT + k;
      page[k] = tile < end ? __ldg(table + (tile >> pb_shift)) : -1;
      if (page[k] >= c.num_blocks) page[k] = -1;
    }
  };
  uint32_t live = 0;  // bit kT * stage + k
  constexpr int kStep = 512 / D;  // rows that a warp's 16-byte chunks cover
  const int kr = lane / (D / 16), kc = lane % (D / 16);
  auto issue = [&](int it, int st) {
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
          const int8_t *src = c.k_codes + (sh * c.block_size + (tile & (per_block - 1)) * kTok) * D + 16 * lane;
          const uint32_t dst =
              smem_u32(ring + st * C::kStageBytes + k * (C::kTileBytes + 16));
#pragma unroll
          for (int i = 0; i < C::kTileBytes / 512; i++)
            cp_async16(dst + k_off<D>(kr + i * kStep, kc), src + 512 * i);
          if (lane == 0) cp_async4(dst + C::kTileBytes, c.k_scales + sh);
        }
      }
    }
    cp_commit();
  };
  const int n_chunks = (n_rows + C::kChunk - 1) / C::kChunk;
  auto stage_chunk = [&](int row0) {
    const int tiles = (min(C::kChunk, n_rows - row0) + R - 1) / R;
    stage_queries<D, R, BF16, C::kHalf>(a.q, q0, kvh, row0, R * tiles, n_rows, warp, kWarps, lane, qimg, inv_s);
    for (int r = tid; r < R * tiles; r += kThreads) {
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
  float *out = a.mass + ((int64_t)b * c.num_kv_heads + kvh) * a.mass_stride;
  for (int ch = 0; ch < n_chunks; ch++) {
    const int row0 = ch * C::kChunk;
    // tokens that some row of the chunk sees
    const int i_last = (min(row0 + C::kChunk, n_rows) - 1) / a.q.group;
    const int tc = min(t1, len - nq + i_last + 1);
    if (tc <= t0) continue;
    end = (tc + kTok - 1) / kTok;
    n_steps = (end - first + kWarps * kT - 1) / (kWarps * kT);
    load_pages(0);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; i++) issue(i, i);
    if (ch > 0) __syncthreads();
    stage_chunk(row0);
    __syncthreads();
    const int tiles = (min(C::kChunk, n_rows - row0) + R - 1) / R;
    for (int it = 0, st = 0; it < n_steps; it++, st = st + 1 == C::kStages ? 0 : st + 1) {
      cp_wait<C::kStages - 2>();
      __syncwarp();
      issue(it + C::kStages - 1, st == 0 ? C::kStages - 1 : st - 1);
      const uint32_t on = live >> (kT * st) & ((1u << kT) - 1);
      const int tok = (first + it * kWarps * kT) * kTok;
      uint4 kf[C::kHalf ? 1 : kT * 2][C::kHalf ? 1 : D / 64];       // codes
      uint32_t kh[C::kHalf ? kT * 2 : 1][C::kHalf ? D / 16 : 1][2];  // or halves
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
              if constexpr (C::kHalf) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                  k_frag(word(w, i), kh[2 * k + n][4 * blk + i][0], kh[2 * k + n][4 * blk + i][1]);
              } else {
                kf[2 * k + n][blk] = w;
              }
            }
        }
      }
      float sum[kT * 4];  // token 8 (i / 2) + 2 tg + (i & 1)
#pragma unroll
      for (int i = 0; i < kT * 4; i++) sum[i] = 0.f;
      if (!on) continue;
      for (int t = 0; t < tiles; t++) {
        // limits grow with the row
        const int last = min(row0 + R * t + R, n_rows) - row0 - 1;
        if (lim_s[last] <= tok) continue;
        const uint32_t *img = qimg + t * C::kQWords;
        constexpr int kHalf = R / 8;  // rows g, and g + 8
        float lse[kHalf], inv[kHalf];
        int lim[kHalf];
#pragma unroll
        for (int h = 0; h < kHalf; h++) {
          lse[h] = lse_s[R * t + g + 8 * h];
          inv[h] = inv_s[R * t + g + 8 * h];
          lim[h] = lim_s[R * t + g + 8 * h];
        }
        const bool cut = tok + kT * kTok > lim_s[R * t];
        // two 8-token blocks at a time
#pragma unroll
        for (int k = 0; k < kT; k++) {
          uint32_t s[2][kL][4];
          float sh[2][4];
          if constexpr (C::kHalf) {
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
              for (int e = 0; e < 4; e++) sh[n][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ks++) {
              const uint4 qa = *reinterpret_cast<const uint4 *>(img + (ks * 32 + lane) * 4);
#pragma unroll
              for (int n = 0; n < 2; n++)
                mma16816(sh[n], qa, kh[2 * k + n][ks][0], kh[2 * k + n][ks][1]);
            }
          } else {
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
              for (int v = 0; v < kL; v++)
#pragma unroll
                for (int e = 0; e < 4; e++) s[n][v][e] = kMagicBits;
#pragma unroll
            for (int ks = 0; ks < kKs; ks++) {
#pragma unroll
              for (int v = 0; v < kL; v++) {
                const uint4 qa = *reinterpret_cast<const uint4 *>(img + ((ks * kL + v) * 32 + lane) * 4);
#pragma unroll
                for (int n = 0; n < 2; n++) {
                  const uint4 &w = kf[2 * k + n][ks >> 1];
                  imma(s[n][v], qa, ks & 1 ? w.z : w.x, ks & 1 ? w.w : w.y);
                }
              }
            }
          }
#pragma unroll
          for (int n = 0; n < 2; n++)
#pragma unroll
            for (int h = 0; h < kHalf; h++)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                float x;
                if constexpr (C::kHalf)
                  x = sh[n][2 * h + e];
                else
                  x = score<R, BF16>(s[n], h, e);
                x *= inv[h] * ksc[k];
                float p = ex2(x - lse[h]);
                if (cut && tok + 16 * k + 8 * n + 2 * tg + e >= lim[h]) p = 0.f;
                sum[4 * k + 2 * n + e] += p;
              }
        }
      }
      // sums over the 8 lanes of a column, halving what each lane carries: lanes
      // end with value (lane / 4) mod kT * 4
      int mine = 0;
#pragma unroll
      for (int o = 16, w = kT * 2; o >= 4; o >>= 1, w >>= 1) {
        const bool up = lane & o;
        if (w >= 1) {
#pragma unroll
          for (int i = 0; i < w; i++) {
            const float give = up ? sum[i] : sum[i + w], keep = up ? sum[i + w] : sum[i];
            sum[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
          mine += up ? w : 0;
        } else {
          sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
        }
      }
      // kT == 1: lanes 4 apart hold the same value
      const int at = tok + 8 * (mine >> 1) + 2 * tg + (mine & 1);
      // the token has this one writer, so the reduction at L2 (which nobody waits
      // for) adds in a fixed order
      if ((kT == 2 || !(lane & 4)) && at < tc && (on >> (mine >> 2) & 1)) atomicAdd(out + at, sum[0]);
    }
    cp_wait<0>();
    __syncwarp();
  }
}

template <int D, int R, bool BF16>
cudaError_t launch(const MassArgs &a, cudaStream_t s) {
  using C = Cfg<D, R, BF16>;
  const int64_t rows = min((int64_t)C::kChunk, (int64_t)a.q.max_q * a.q.group);
  const int smem = C::smem((int)(rows + R - 1) / R);
  const cudaError_t e = allow_smem<b8_mass_kernel<D, R, BF16>>(C::smem(C::kChunk / R));
  if (e != cudaSuccess) return e;
  const unsigned ctas = (unsigned)((int64_t)a.q.batch * a.c.num_kv_heads * a.ranges);
  b8_mass_kernel<D, R, BF16><<<ctas, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t by_rows(const MassArgs &a, cudaStream_t s) {
  if ((int64_t)a.q.max_q * a.q.group <= 8)
    return a.q.bf16 ? launch<D, 8, true>(a, s) : launch<D, 8, false>(a, s);
  return a.q.bf16 ? launch<D, 16, true>(a, s) : launch<D, 16, false>(a, s);
}

}  // namespace

cudaError_t launch_b8_mass(const kvq_b8_cache &c, const B8Queries &q, const float *lse,
                           float *mass, int64_t mass_stride, cudaStream_t s) {
  MassArgs a = {c, q, lse, mass, mass_stride, 1, 0, device_error_word()};
  const int64_t len =
      max((int64_t)1, min((int64_t)q.max_seq_len, (int64_t)c.max_blocks_per_seq * c.block_size));
  const bool few = (int64_t)q.max_q * q.group <= 8;
  const int64_t granule = kWarps * kTok * (c.head_dim == 256 || (!few && !q.bf16) ? 1 : 2);
  const int64_t units = (int64_t)q.batch * c.num_kv_heads;
  const int64_t most = (len + granule - 1) / granule;
  const int64_t resident = kNumSMs * 2;
  // few rows: about four CTAs for each that the card holds, of at least 2048
  // tokens where that fills it once; many: the card once, as every CTA stages
  // the rows
  // (whose lengths differ: half as many again)
  int64_t want = 3 * resident / (2 * units);
  if (few)
    want = max((resident + units - 1) / units, min((4 * resident + units - 1) / units, (len + 2047) / 2048));
  want = max((int64_t)1, min(want, most));
  a.range_tokens = (int)(((len + want - 1) / want + granule - 1) / granule * granule);
  a.ranges = (int)((len + a.range_tokens - 1) / a.range_tokens);
  switch (c.head_dim) {
    case 64: return by_rows<64>(a, s);
    case 128: return by_rows<128>(a, s);
    default: return by_rows<256>(a, s);
  }
}

}  // namespace kvq
