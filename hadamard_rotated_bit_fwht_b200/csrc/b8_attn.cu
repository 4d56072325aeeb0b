// b8_attn.cu -- attention over the block-scaled 8-bit cache (kvq_b8_attn):
// out = softmax(scale q K^T + causal mask) V, ragged queries.
//
// The rows of a (sequence, kv head) are its (query, head of the group) pairs,
// query-major.  One CTA takes one tile of R = 8 or 16 rows and one range of
// tokens; its 8 warps take 16-token tiles in turn, each with its own softmax
// state (m, l, O), staged by cp.async into a ring that only this warp reads
// (no CTA barrier inside the loop).  The states are merged once at the end.  Up
// to 8 ranges form a cluster, which shares a sequence's real length evenly and
// merges through distributed shared memory; more are merged by a second kernel.
// Bound for a few rows: the codes from HBM, read once.  131072 tokens of 4 kv
// heads, D 256: 55 us, 4.9 TB/s (75 % of a plain copy); 32 sequences of 2048 to
// 16384 tokens, 8 kv heads, D 128: 119 us, 5.0 TB/s; 777 tokens: 6.6 us.  An even
// share of all tokens for each CTA was 3 % faster on the second and 40 % slower
// on short batches: not taken.
//   * Scores are kept in log2 units in fp32; m follows the row maximum with a
//     slack of 8 (p up to 2^8), so O is rarely rescaled.
//   * P enters the second product as p * v_scale in fp16 (bf16 output) or as
//     fp16 hi + lo (fp32 output), in units of 2^mv / 64 where mv follows the
//     row's maximum of score + log2(v_scale) as m does that of the scores: at
//     most 2^14, and fp16's range counts down from the row's own largest p *
//     v_scale, whatever scales its other tokens have.  l sums the unrounded p.
//     m and mv are integers, so factors between them are powers of two.
#include <cuda_bf16.h>

#include "b8_attn.cuh"
#include "b8_mma.cuh"

namespace kvq {
namespace {

using namespace b8;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kEmpty = -1e30f;  // running maximum before any token
constexpr float kSlack = 8.f;

// HILO: fp32 output, probabilities as fp16 hi + lo
template <int D, int R, bool HILO>
struct Cfg {
  static constexpr int kTileBytes = kTok * D;           // K or V of a warp's tile
  static constexpr int kStageBytes = 2 * kTileBytes + 16;  // + k_scale, v_scale
  static constexpr int kCtas = D == 256 || R == 16 ? 1 : 2;  // resident per SM
  // 128 KB of tiles in flight or landing per SM
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? (kCtas == 2 ? 3 : 5) : (kCtas == 2 ? 5 : 9);
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  // after the ring: queries, their factors and their token limits
  static constexpr int kOffQ = kRing;
  static constexpr int kOffInv = kOffQ + QTile<D, R, !HILO>::kBytes;
  static constexpr int kOffLim = kOffInv + R * 4;
  static constexpr int kSmem = kOffLim + R * 4;
  // the merge reuses the ring: per warp R x (D + 4) of O, then m, l and mv
  static constexpr int kRow = D + 4;
  static constexpr int kOffM = kWarps * R * kRow * 4;
  // in a cluster: this CTA's merged record, read by the others
  static constexpr int kOffRec = (kOffM + kWarps * 3 * R * 4 + 15) / 16 * 16;
  static_assert(kOffRec + R * kRow * 4 <= kRing, "merge fits the ring");
  static_assert(kSmem * kCtas <= 227 * 1024, "shared memory per SM");
};

// ---- clusters
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// this shared-memory address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int D, bool HILO>
__device__ __forceinline__ void store_out(void *out, int64_t at, float4 v) {
  if (HILO) {
    *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = v;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t *>(&a);
    u.y = *reinterpret_cast<const uint32_t *>(&b);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) = u;
  }
}

// grid: split + splits * (row tile + row_tiles * (kv head + heads * sequence))
template <int D, int R, bool HILO>
__global__ void __launch_bounds__(kThreads, Cfg<D, R, HILO>::kCtas)
    b8_attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<D, R, HILO>;
  constexpr int kNb = R / 8;       // n blocks of the second product
  constexpr int kMt = D / 16;      // m tiles of the second product
  constexpr int kKs = D / 32;      // k steps of the first product
  constexpr int kL = QTile<D, R, !HILO>::kLevels;
  dec::grid_dependency_wait();
  // short calls let the next kernel's launch overlap
  if (a.p.cluster) dec::launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tg = lane & 3;
  const kvq_b8_cache &c = a.c;

  int u = blockIdx.x;
  const int split = u % a.p.splits;
  u /= a.p.splits;
  const int rt = u % a.p.row_tiles;
  u /= a.p.row_tiles;
  const int kvh = u % c.num_kv_heads, b = u / c.num_kv_heads;

  int q0;
  const int nq = query_range(a.q, b, q0);
  const int n_rows = nq * a.q.group, row0 = rt * R;
  if (row0 >= n_rows) return;
  const int len = seq_len(a.q, c, b);
  // query i attends to tokens below len - nq + i + 1
  const int i_last = (min(row0 + R, n_rows) - 1) / a.q.group;
  const int hi_lim = max(0, len - nq + i_last + 1);
  const int lo_lim = max(0, len - nq + row0 / a.q.group + 1);
  // a cluster's CTAs share the tokens that there are, in whole rounds of tiles
  const int share = a.p.cluster ? (hi_lim + a.p.splits * kWarps * kTok - 1) / (a.p.splits * kWarps * kTok) *
                                      kWarps * kTok
                                : a.p.split_tokens;
  const int t0 = (int)min((int64_t)split * share, (int64_t)hi_lim);
  const int t1 = (int)min((int64_t)hi_lim, (int64_t)t0 + share);
  if (t0 >= t1 && split > 0 && !a.p.cluster) return;  // the combine kernel knows

  uint32_t *qimg = reinterpret_cast<uint32_t *>(smem + C::kOffQ);
  float *inv_s = reinterpret_cast<float *>(smem + C::kOffInv);
  int *lim_s = reinterpret_cast<int *>(smem + C::kOffLim);

  // ---- staging of this warp's tiles: tile w of the range goes to warp w % 8
  const int first = t0 / kTok + warp;
  const int n_tiles = t1 > t0 ? max(0, ((t1 + kTok - 1) / kTok - first + kWarps - 1) / kWarps) : 0;
  uint8_t *ring = smem + warp * C::kStages * C::kStageBytes;
  const int per_block = c.block_size / kTok, pb_shift = __ffs(per_block) - 1;
  const int32_t *table = c.block_table + (int64_t)b * c.max_blocks_per_seq;
  // lane l holds the block of tile page_base + l
  int page_base = 0, page = -1;
  auto load_pages = [&](int base) {
    page_base = base;
    const int col = (first + (base + lane) * kWarps) >> pb_shift;
    page = base + lane < n_tiles && col < c.max_blocks_per_seq ? __ldcg(table + col) : -1;
    if (page >= c.num_blocks) page = -1;
  };
  uint32_t live = 0;  // bit s: the tile in stage s is mapped
  // 16-byte chunk lane + 32 i of a tile is chunk kc of row kr + i * kStep
  constexpr int kStep = 512 / D;
  const int kr = lane / (D / 16), kc = lane % (D / 16);
  auto issue = [&](int it, int st) {
    if (it < n_tiles) {
      if (it >= page_base + 32) load_pages(it);
      const int slot = __shfl_sync(0xffffffffu, page, it - page_base);
      const int tile = first + it * kWarps;
      const bool mapped = slot >= 0 && in_bounds(slot, slot + 1, c.num_blocks, a.err);
      live = mapped ? live | (1u << st) : live & ~(1u << st);
      if (mapped) {
        const int64_t sh = (int64_t)slot * c.num_kv_heads + kvh;
        const int64_t off = (sh * c.block_size + (tile & (per_block - 1)) * kTok) * D + 16 * lane;
        const uint32_t dst = smem_u32(ring + st * C::kStageBytes);
        const int8_t *ksrc = c.k_codes + off, *vsrc = c.v_codes + off;
#pragma unroll
        for (int i = 0; i < C::kTileBytes / 512; i++) {
          cp_async16(dst + k_off<D>(kr + i * kStep, kc), ksrc + 512 * i);
          cp_async16(dst + C::kTileBytes + v_off<D>(kr + i * kStep, kc), vsrc + 512 * i);
        }
        if (lane < 2)
          cp_async4(dst + 2 * C::kTileBytes + 4 * lane, (lane ? c.v_scales : c.k_scales) + sh);
      }
    }
    cp_commit();
  };
  if (n_tiles > 0) load_pages(0);
#pragma unroll
  for (int i = 0; i < C::kStages - 1; i++) issue(i, i);

  stage_queries<D, R, !HILO>(a.q, q0, kvh, row0, R, n_rows, warp, kWarps, lane, qimg, inv_s);
  if (tid < R) lim_s[tid] = row0 + tid < n_rows ? max(0, len - nq + (row0 + tid) / a.q.group + 1) : 0;
  __syncthreads();
  const float inv0 = inv_s[g], inv1 = R == 16 ? inv_s[R == 16 ? g + 8 : g] : 0.f;
  const int lim0 = lim_s[g], lim1 = R == 16 ? lim_s[R == 16 ? g + 8 : g] : 0;
  const bool whole = row0 + R <= n_rows;

  constexpr bool kQRegs = R == 8 && D <= 128;
  uint4 qr[kQRegs ? kKs * kL : 1];
  if (kQRegs) {
#pragma unroll
    for (int i = 0; i < kKs * kL; i++)
      qr[kQRegs ? i : 0] = *reinterpret_cast<const uint4 *>(qimg + (i * 32 + lane) * 4);
  }

  float o[kMt][kNb][4];
#pragma unroll
  for (int j = 0; j < kMt; j++)
#pragma unroll
    for (int n = 0; n < kNb; n++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[j][n][e] = 0.f;
  // vinv: 64 * 2^(m - mv)
  float m[kNb], l[kNb], mv[kNb], vinv[kNb];
#pragma unroll
  for (int n = 0; n < kNb; n++) m[n] = mv[n] = kEmpty, l[n] = 0.f, vinv[n] = 1.f;
  // rows of the V matrices that this lane addresses
  const int v_row = (lane & 7) + (lane & 8), v_ch = lane >> 4;

  for (int it = 0, st = 0; it < n_tiles; it++, st = st + 1 == C::kStages ? 0 : st + 1) {
    cp_wait<C::kStages - 2>();
    __syncwarp();
    issue(it + C::kStages - 1, st == 0 ? C::kStages - 1 : st - 1);
    if (!(live >> st & 1)) continue;
    const uint8_t *kt = ring + st * C::kStageBytes;
    const uint32_t vt = smem_u32(kt + C::kTileBytes);
    const float2 kv = *reinterpret_cast<const float2 *>(kt + 2 * C::kTileBytes);  // scales
    const int tok = (first + it * kWarps) * kTok;

    // S: rows g (0, 1) and g + 8 (2, 3), tokens 8 n + 2 tg, + 1, of each level
    uint32_t s[2][kL][4];
#pragma unroll
    for (int n = 0; n < 2; n++)
#pragma unroll
      for (int v = 0; v < kL; v++)
#pragma unroll
        for (int e = 0; e < 4; e++) s[n][v][e] = kMagicBits;
#pragma unroll
    for (int blk = 0; blk < D / 64; blk++) {
      uint4 kw[2];
#pragma unroll
      for (int n = 0; n < 2; n++)
        kw[n] = *reinterpret_cast<const uint4 *>(kt + k_off<D>(8 * n + g, 4 * blk + tg));
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int ks = 2 * blk + h;
#pragma unroll
        for (int v = 0; v < kL; v++) {
          const uint4 qa = kQRegs ? qr[kQRegs ? ks * kL + v : 0]
                                  : *reinterpret_cast<const uint4 *>(qimg + ((ks * kL + v) * 32 + lane) * 4);
#pragma unroll
          for (int n = 0; n < 2; n++)
            imma(s[n][v], qa, h ? kw[n].z : kw[n].x, h ? kw[n].w : kw[n].y);
        }
      }
    }
    // scores in log2 units, p[row block][token pair]
    float p[kNb][4];
#pragma unroll
    for (int nb = 0; nb < kNb; nb++) {
      const float f = (nb ? inv1 : inv0) * kv.x;
#pragma unroll
      for (int n = 0; n < 2; n++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          p[nb][2 * n + e] = score<R, !HILO>(s[n], nb, e) * f;
        }
    }
    if (tok + kTok > lo_lim || !whole) {
#pragma unroll
      for (int nb = 0; nb < kNb; nb++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (tok + 8 * (e >> 1) + 2 * tg + (e & 1) >= (nb ? lim1 : lim0)) p[nb][e] = -INFINITY;
    }
    // m and mv need not be the maxima: they move once those pass them by kSlack
    const float lv = __log2f(kv.y);  // -inf for a block of zeros
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < kNb; nb++) {
      const float x = fmaxf(fmaxf(p[nb][0], p[nb][1]), fmaxf(p[nb][2], p[nb][3]));
      grow |= x > m[nb] + kSlack || x + lv > mv[nb] + kSlack;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nb = 0; nb < kNb; nb++) {
        float x = fmaxf(fmaxf(p[nb][0], p[nb][1]), fmaxf(p[nb][2], p[nb][3]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const float mn = x > m[nb] + kSlack ? ceilf(x) : m[nb];
        l[nb] *= ex2(m[nb] - mn);
        m[nb] = mn;
        const float vn = x + lv > mv[nb] + kSlack ? ceilf(x + lv) : mv[nb];
        const float al = ex2(mv[nb] - vn);
        mv[nb] = vn;
        // scales down to 2^-107, which an append makes, stay below 2^126
        vinv[nb] = ex2(fminf(fmaxf(mn - vn + 6.f, -126.f), 126.f));
        // this lane's columns of O are rows 2 tg and 2 tg + 1 of the block
        const float a0 = __shfl_sync(0xffffffffu, al, 8 * tg);
        const float a1 = __shfl_sync(0xffffffffu, al, 8 * tg + 4);
#pragma unroll
        for (int j = 0; j < kMt; j++) {
          o[j][nb][0] *= a0, o[j][nb][1] *= a1;
          o[j][nb][2] *= a0, o[j][nb][3] *= a1;
        }
      }
    }
    uint32_t ph[kNb][2], pl[kNb][2];
#pragma unroll
    for (int nb = 0; nb < kNb; nb++) {
      // (finite: a product past 2^127 would meet weights below 2^-113 alone, and
      // 0 * inf would be NaN; rows that see nothing of the tile take nothing of a NaN)
      float vf = kv.y * vinv[nb];
      vf = vf > 0x1p127f ? 0x1p127f : (nb ? lim1 : lim0) > tok ? vf : 0.f;
#pragma unroll
      for (int n = 0; n < 2; n++) {
        const float e0 = ex2(p[nb][2 * n] - m[nb]), e1 = ex2(p[nb][2 * n + 1] - m[nb]);
        l[nb] += e0 + e1;
        const float2 w = make_float2(e0 * vf, e1 * vf);
        if (HILO)
          dec::split_hilo(w, ph[nb][n], pl[nb][n]);
        else
          ph[nb][n] = pack_f16x2(w.x, w.y);
      }
    }
    // O^T += V^T P^T, two m tiles a load
#pragma unroll
    for (int j = 0; j < kMt; j += 2) {
      uint32_t w[4];  // tokens 0 .. 7 and 8 .. 15 of chunk j, then of chunk j + 1
      dec::ldsm_x4_t(vt + v_off<D>(v_row, j + v_ch), w);
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const uint32_t x = w[2 * h] ^ 0x80808080u, y = w[2 * h + 1] ^ 0x80808080u;
        const uint32_t fr[4] = {pair_h2(x, 0x4240), pair_h2(x, 0x4341), pair_h2(y, 0x4240),
                                pair_h2(y, 0x4341)};
#pragma unroll
        for (int nb = 0; nb < kNb; nb++) {
          mma16816(o[j + h][nb], fr, ph[nb][0], ph[nb][1]);
          if (HILO) mma16816(o[j + h][nb], fr, pl[nb][0], pl[nb][1]);
        }
      }
    }
  }
  cp_wait<0>();
#pragma unroll
  for (int nb = 0; nb < kNb; nb++) {
    l[nb] += __shfl_xor_sync(0xffffffffu, l[nb], 1);
    l[nb] += __shfl_xor_sync(0xffffffffu, l[nb], 2);
  }
  __syncthreads();  // every warp is done with its ring

  // ---- merge of the warps' states
  float *mo = reinterpret_cast<float *>(smem) + warp * R * C::kRow;
  float *mm = reinterpret_cast<float *>(smem + C::kOffM);  // [warp][R]
  float *ml = mm + kWarps * R, *mvs = ml + kWarps * R;
#pragma unroll
  for (int nb = 0; nb < kNb; nb++) {
#pragma unroll
    for (int e = 0; e < 2; e++) {
      float *row = mo + (8 * nb + 2 * tg + e) * C::kRow;
#pragma unroll
      for (int j = 0; j < kMt; j++)
        *reinterpret_cast<float2 *>(row + 16 * j + 2 * g) = make_float2(o[j][nb][e], o[j][nb][2 + e]);
    }
    if (tg == 0) {
      mm[warp * R + 8 * nb + g] = m[nb];
      ml[warp * R + 8 * nb + g] = l[nb];
      mvs[warp * R + 8 * nb + g] = mv[nb];
    }
  }
  __syncthreads();
  // warp w: rows w, w + 8
  for (int r = warp; r < R; r += kWarps) {
    const int row = row0 + r;
    if (row >= n_rows) break;
    float M = kEmpty, MV = kEmpty, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) M = fmaxf(M, mm[w * R + r]), MV = fmaxf(MV, mvs[w * R + r]);
    float f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      L += ex2(mm[w * R + r] - M) * ml[w * R + r];
      f[w] = ex2(mvs[w * R + r] - MV);
    }
    const bool direct = a.p.splits == 1;
    // (from units of 2^MV / 64: after the sum, which would lose terms of scales near
    // fp32's lower end)
    const float unit = ex2(MV - M - 6.f);
    const float norm = direct ? (L > 0.f ? __fdiv_rn(1.f, L) : L == 0.f ? 0.f : L) : 1.f;
    const int i = row / a.q.group, head = kvh * a.q.group + row - i * a.q.group;
    const int64_t orow = (int64_t)(q0 + i) * a.q.num_heads + head;
    float *rec = a.p.cluster ? reinterpret_cast<float *>(smem + C::kOffRec) + r * C::kRow
                             : a.ws + ((int64_t)blockIdx.x * R + r) * (D + 4);
    for (int d = 4 * lane; d < D; d += 128) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(smem) +
                                                           (w * R + r) * C::kRow + d);
        acc.x += f[w] * x.x, acc.y += f[w] * x.y, acc.z += f[w] * x.z, acc.w += f[w] * x.w;
      }
      acc.x *= unit, acc.y *= unit, acc.z *= unit, acc.w *= unit;
      acc.x *= norm, acc.y *= norm, acc.z *= norm, acc.w *= norm;
      if (direct)
        store_out<D, HILO>(a.out, orow * D + d, acc);
      else
        *reinterpret_cast<float4 *>(rec + 4 + d) = acc;
    }
    if (lane == 0) {
      if (!direct)
        rec[0] = M, rec[1] = L;
      else if (a.lse != nullptr)
        a.lse[orow] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
    }
  }
  if (!a.p.cluster) return;
  // rows split, split + splits, ... are this CTA's to join; lane s has the
  // state of CTA s
  cluster_sync();
  const uint32_t recs = smem_u32(smem + C::kOffRec);
  for (int r = split + warp * a.p.splits; r < R; r += kWarps * a.p.splits) {
    const int row = row0 + r;
    if (row >= n_rows) break;
    const uint32_t at = recs + r * C::kRow * 4;
    float4 st = make_float4(kEmpty, 0.f, 0.f, 0.f);
    if (lane < a.p.splits) st = ld_cluster4(in_cta(at, lane));
    float M = st.x;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float f = ex2(st.x - M);
    float L = lane < a.p.splits ? f * st.y : 0.f;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    M = __shfl_sync(0xffffffffu, M, 0);
    L = __shfl_sync(0xffffffffu, L, 0);
    const float norm = L > 0.f ? __fdiv_rn(1.f, L) : L == 0.f ? 0.f : L;
    const int i = row / a.q.group;
    const int64_t orow = (int64_t)(q0 + i) * a.q.num_heads + kvh * a.q.group + row - i * a.q.group;
    float4 acc[D / 128 > 0 ? D / 128 : 1];
#pragma unroll
    for (int h = 0; h < (D + 127) / 128; h++) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c8 = 0; c8 < 8; c8++) {
      const float fs = __shfl_sync(0xffffffffu, f, c8);
      if (c8 < a.p.splits) {
#pragma unroll
        for (int h = 0; h < (D + 127) / 128; h++) {
          if (4 * lane + 128 * h >= D) continue;
          const float4 x = ld_cluster4(in_cta(at + 16 + 16 * lane + 512 * h, c8));
          acc[h].x += fs * x.x, acc[h].y += fs * x.y, acc[h].z += fs * x.z, acc[h].w += fs * x.w;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < (D + 127) / 128; h++) {
      const int d = 4 * lane + 128 * h;
      if (d >= D) continue;
      acc[h].x *= norm, acc[h].y *= norm, acc[h].z *= norm, acc[h].w *= norm;
      store_out<D, HILO>(a.out, orow * D + d, acc[h]);
    }
    if (lane == 0 && a.lse != nullptr) a.lse[orow] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
  }
  cluster_sync();  // the others may still read this CTA's record
}

// One CTA per row: merge its splits' records.
// grid: row of the tile + R * (row tile + row_tiles * (kv head + heads * sequence))
template <int D, bool HILO, int kCombine>
__global__ void __launch_bounds__(kCombine) b8_combine_kernel(const __grid_constant__ AttnArgs a) {
  dec::grid_dependency_wait();
  constexpr int kCols = D / 4, kParts = kCombine / kCols;
  __shared__ float part[kParts > 1 ? (kParts - 1) * D : 1];
  __shared__ float red[2][kCombine / 32];
  const int R = a.p.rows, tid = threadIdx.x;
  const int r = blockIdx.x % R;
  const int unit = blockIdx.x / R;
  int u = unit;
  const int rt = u % a.p.row_tiles;
  u /= a.p.row_tiles;
  const int kvh = u % a.c.num_kv_heads, b = u / a.c.num_kv_heads;
  int q0;
  const int nq = query_range(a.q, b, q0);
  const int n_rows = nq * a.q.group, row = rt * R + r;
  if (row >= n_rows) return;
  const int len = seq_len(a.q, a.c, b);
  const int i_last = (min(rt * R + R, n_rows) - 1) / a.q.group;
  const int hi_lim = max(0, len - nq + i_last + 1);
  const int n = (int)max((int64_t)1, ((int64_t)hi_lim + a.p.split_tokens - 1) / a.p.split_tokens);
  const float *rec = a.ws + ((int64_t)unit * a.p.splits * R + r) * (D + 4);
  const int64_t step = (int64_t)R * (D + 4);
  float M = kEmpty;
  for (int s = tid; s < n; s += kCombine) M = fmaxf(M, rec[s * step]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if ((tid & 31) == 0) red[0][tid >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombine / 32; w++) M = fmaxf(M, red[0][w]);
  float L = 0.f;
  for (int s = tid; s < n; s += kCombine) L += ex2(rec[s * step] - M) * rec[s * step + 1];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if ((tid & 31) == 0) red[1][tid >> 5] = L;
  const int col = tid % kCols, pt = tid / kCols;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = pt; s < n; s += kParts) {
    const float f = ex2(rec[s * step] - M);
    const float4 x = *reinterpret_cast<const float4 *>(rec + s * step + 4 + 4 * col);
    acc.x += f * x.x, acc.y += f * x.y, acc.z += f * x.z, acc.w += f * x.w;
  }
  if (kParts > 1 && pt > 0)
    *reinterpret_cast<float4 *>(part + (pt - 1) * D + 4 * col) = acc;
  __syncthreads();
  if (pt > 0) return;
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kCombine / 32; w++) L += red[1][w];
#pragma unroll
  for (int i = 0; i < kParts - 1; i++) {
    const float4 x = *reinterpret_cast<const float4 *>(part + i * D + 4 * col);
    acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
  }
  const float norm = L > 0.f ? __fdiv_rn(1.f, L) : L == 0.f ? 0.f : L;
  acc.x *= norm, acc.y *= norm, acc.z *= norm, acc.w *= norm;
  const int i = row / a.q.group;
  const int64_t orow = (int64_t)(q0 + i) * a.q.num_heads + kvh * a.q.group + row - i * a.q.group;
  store_out<D, HILO>(a.out, orow * D + 4 * col, acc);
  if (tid == 0 && a.lse != nullptr) a.lse[orow] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
}

template <int D, int R, bool HILO>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
  using C = Cfg<D, R, HILO>;
  const cudaError_t e = allow_smem<b8_attn_kernel<D, R, HILO>>(C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.q.batch * a.c.num_kv_heads * a.p.row_tiles;
  // (a short decode among others: 6.6 us a call instead of 8.2)
  return launch_early(b8_attn_kernel<D, R, HILO>, dim3((unsigned)(units * a.p.splits)), kThreads,
                      C::kSmem, s, a.p.cluster ? a.p.splits : 1, a);
}

template <int D, bool HILO, int kCombine>
cudaError_t combine(const AttnArgs &a, cudaStream_t s) {
  const int64_t units = (int64_t)a.q.batch * a.c.num_kv_heads * a.p.row_tiles;
  return launch_early(b8_combine_kernel<D, HILO, kCombine>, dim3((unsigned)(units * a.p.rows)),
                      kCombine, 0, s, 1, a);
}

template <int D>
cudaError_t by_rows(const AttnArgs &a, cudaStream_t s) {
  cudaError_t e;
  if (a.p.prefill)
    e = launch_b8_prefill(a, s);
  else if (a.p.rows == 8)
    e = a.q.bf16 ? launch<D, 8, false>(a, s) : launch<D, 8, true>(a, s);
  else
    e = a.q.bf16 ? launch<D, 16, false>(a, s) : launch<D, 16, true>(a, s);
  if (e != cudaSuccess || a.p.prefill || a.p.splits == 1 || a.p.cluster) return e;
  // few rows of many splits want more threads a row
  if (a.p.splits > 8) return a.q.bf16 ? combine<D, false, 512>(a, s) : combine<D, true, 512>(a, s);
  return a.q.bf16 ? combine<D, false, 128>(a, s) : combine<D, true, 128>(a, s);
}



}  // namespace

B8Plan plan_b8_attn(const kvq_b8_cache &c, int bf16, int group, int batch, int max_q,
                    int max_seq_len) {
  B8Plan p;
  const int64_t rows = (int64_t)max_q * group;
  const int64_t cap = (int64_t)c.max_blocks_per_seq * c.block_size;
  const int64_t len = max((int64_t)1, min((int64_t)max_seq_len, cap));
  p.cluster = 0;
  // The many-row kernel costs a tile of 256 rows whatever it holds, this file's
  // one of 16: 16 sequences of 4096 tokens, 8 kv heads, D = 128, 32 rows 114 us
  // against 96, 48 rows 114 against 139.  Where there is less to do, its longer
  // set-up counts: one such sequence 25 us against 18 at 64 rows, 25 against 27
  // at 128.
  const int64_t tiles16 = (int64_t)batch * c.num_kv_heads * ((rows + 15) / 16);
  p.prefill = bf16 && (rows >= 128 || (rows >= 48 && tiles16 * len >= 400000));
  p.rows = p.prefill ? b8_prefill_rows(c.head_dim) : rows <= 8 ? 8 : 16;
  p.row_tiles = (int)((rows + p.rows - 1) / p.rows);
  const int64_t units = (int64_t)batch * c.num_kv_heads * p.row_tiles;
  p.splits = 1, p.split_tokens = 0;
  if (p.prefill) return p;  // cut on the device
  const int resident = kNumSMs * (c.head_dim == 256 || p.rows == 16 ? 1 : 2);
  const int64_t full = (resident + units - 1) / units;  // splits that fill the card once
  const int64_t granule = kWarps * kTok;
  const int64_t most = (len + granule - 1) / granule;
  // clusters where all of them fit the card at once and a CTA's share is short:
  // they save the second kernel, but the CTAs of one all wait for its slowest
  // (118 us by two kernels against 130 by clusters of 8 for 32 sequences of
  // 2048 to 16384 tokens and 8 kv heads; 11.1 against 9.8 for one of 777)
  const int64_t in_cluster = min(min((int64_t)8, most), resident / units);
  p.cluster = in_cluster > 1 && len <= in_cluster * 2048;
  int64_t want;
  if (p.cluster) {
    want = in_cluster;
  } else if (batch == 1) {
    // one length: whole waves of equal splits, as few as fill the card
    want = max((int64_t)1, resident / units);
  } else {
    // lengths differ: about four CTAs for each that the card holds at once, of
    // at least 16 tiles a warp where that leaves one CTA for each
    want = min((4 * (int64_t)resident + units - 1) / units, max(full, (len + 2047) / 2048));
  }
  want = max((int64_t)1, min(want, (len + granule - 1) / granule));
  int64_t tokens = (len + want - 1) / want;
  tokens = (tokens + granule - 1) / granule * granule;
  p.split_tokens = (int)tokens;
  p.splits = (int)((len + tokens - 1) / tokens);
  p.cluster = p.cluster && p.splits > 1;
  return p;
}

size_t b8_attn_workspace_bytes(const kvq_b8_cache &c, int batch, const B8Plan &p) {
  if (p.prefill) return b8_prefill_workspace(c.head_dim);
  if (p.splits == 1 || p.cluster) return 0;
  return (size_t)batch * c.num_kv_heads * p.row_tiles * p.splits * p.rows * (c.head_dim + 4) * 4;
}

cudaError_t launch_b8_attn(const kvq_b8_cache &c, const B8Queries &q, const B8Plan &p, void *out,
                           float *lse, float *ws, cudaStream_t s) {
  const AttnArgs a = {c, q, p, out, lse, ws, device_error_word(), wait_poll_limit()};
  switch (c.head_dim) {
    case 64: return by_rows<64>(a, s);
    case 128: return by_rows<128>(a, s);
    default: return by_rows<256>(a, s);
  }
}

}  // namespace kvq
