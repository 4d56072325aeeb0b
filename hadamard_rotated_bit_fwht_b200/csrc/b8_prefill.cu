// b8_prefill.cu -- many-row attention over the block-scaled 8-bit cache
// (kvq_b8_attn with bf16 queries): both products on the fifth-generation
// tensor cores, accumulators in tensor memory.
//
// A CTA takes kNT tiles of 128 rows (query, head of the group) of one
// (sequence, kv head) and a range of tokens, kBN at a time.  Roles:
//   softmax  one warpgroup per row tile, one row per thread: scores come from
//            tensor memory, probabilities go back there as fp16 over them;
//   convert  four warps: int8 codes from global memory to exact fp16 tiles in
//            the 128-byte swizzle, K row by row (dims contiguous) and V in the
//            same image, read by the second product with its dims as rows;
//   issue    one thread: S(i) = Q K^T, O += P(i) V, two score buffers, so that
//            one item's softmax runs beside the other's products (a warpgroup of
//            its own for the split of the registers).
// Scores are scaled after the product: a row's factor is its thread's, a
// block's scale one of 8 group constants of the tile.  The V scale joins the
// exponent: p' = 2^(s + log2 v_scale - ve), where ve follows the row's maximum of
// that sum less 6 (p' up to 2^6, and 2^14 with a slack of 8, so that O is rarely
// rescaled by its softmax threads): fp16's range counts down from the row's own
// largest p * v_scale.  O is in units of 2^ve, and so is l, which sums p' of each
// 16-token group divided by v_scale (and 2^20, to stay far from fp32's ends).  V
// scales 2^-97 and more below the largest so far count as that: fp32 would lose
// their p' from l.
// Bound: the chain scores -> softmax -> products of a row tile; two tiles take
// turns on the tensor pipe.  4 prompts of 572 to 778 queries, 32 heads on 8 kv
// heads, D 128, 6516 to 8075 tokens: 387 us, 792 TFLOP/s (48 % of a cuBLAS bf16
// product).  A tile's 16 products take about 2000 cycles from the first to the
// last where their operations are 1024, V's layout (dims as rows or as columns)
// aside; descriptors by constant steps, the wait for V in front of that for the
// probabilities and no masks for rows of no query brought 410 to 383 (units of the
// largest V scale that a CTA had met saved 4 us of 387, and lost rows on blocks of
// far smaller ones).  At 410 it
// took as long without exp2, or without the stores of P; 354 with next to no
// softmax, 383 with half of the score products, 379 without the conversion.
// Tiles of 64 tokens with two score buffers a row tile took 660 us (their
// products cost as much as those of 128), P in halves 560.
#include <cuda_bf16.h>

#include "b8_attn.cuh"
#include "b8_mma.cuh"

namespace kvq {
namespace {

using namespace b8;
using dec::mbar_arrive;
using dec::mbar_init;

template <int D>
struct PCfg {
  static constexpr int kNT = D == 256 ? 1 : 2;    // row tiles
  static constexpr int kBN = D == 256 ? 64 : 128; // tokens of a tile
  static constexpr int kGroups = kBN / 16;
  static constexpr int kRows = 128 * kNT;
  static constexpr int kSoft = 128 * kNT;
  // softmax warpgroups, the converting one, and one whose first warp issues
  static constexpr int kThreads = kSoft + 128 + 128;
  // registers a thread (kNT == 2): a softmax thread holds a whole row of scores.
  // Launched with 128 each; 256 x 184 + 128 x 96 + 128 x 48 = 512 x 128.
  static constexpr int kRegsSoft = 184, kRegsConvert = 96, kRegsIssue = 48;
  static constexpr int kQTileBytes = 128 * D * 2;
  static constexpr int kKVBytes = kBN * D * 2;
  static constexpr int kInfo = 4;                 // slots of group constants
  static constexpr int kOffK = kNT * kQTileBytes;
  static constexpr int kOffV = kOffK + 2 * kKVBytes;
  static constexpr int kOffInfo = kOffV + 2 * kKVBytes;
  // k scale, log2 of the V scale, its inverse / 2^20; largest and smallest log2
  static constexpr int kInfoFloats = 3 * 8 + 4;
  static constexpr int kOffBar = kOffInfo + kInfo * kInfoFloats * 4;
  // k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2],
  // o_done[2], info_full[4], drain, all_done[2]
  static constexpr int kBars = 21;
  static constexpr int kOffMisc = kOffBar + kBars * 8;  // abort flag, tensor memory base
  static constexpr int kUsed = kOffMisc + 16 + 1024;    // 1024: alignment
  // one CTA per SM (it takes all of tensor memory)
  static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static constexpr int kColO = 0, kColS = kNT * D;
  static_assert(kColS + 2 * kBN <= 512, "tensor memory columns");
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

// ---- tcgen05
__device__ __forceinline__ void t5_alloc(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void t5_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void t5_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void t5_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void t5_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void t5_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void t5_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// 32 columns of this thread's lane
__device__ __forceinline__ void t5_ld32(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]),
        "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr));
}
// The loads are asynchronous: their registers hold nothing before this wait.
// It takes them as operands, so that no use moves in front of it.
__device__ __forceinline__ void t5_wait_ld(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
        "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
        "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]),
        "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]),
        "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
      :
      : "memory");
}
// further loads of the same wait
__device__ __forceinline__ void after_wait(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]),
                   "+f"(v[i + 5]), "+f"(v[i + 6]), "+f"(v[i + 7]));
}
__device__ __forceinline__ void t5_ld16(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void t5_wait_ld(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
        "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
        "+f"(v[14]), "+f"(v[15])
      :
      : "memory");
}
__device__ __forceinline__ void t5_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void t5_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void t5_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major operands: rows
// of 64 halves, groups of 8 rows `stride` bytes apart.  MN-major ones: 64
// halves of the M or N extent per 128-byte row, groups of 8 k rows `stride`
// bytes apart, further 64 of M or N `lead` bytes away.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// fp16 operands, fp32 accumulator, M = 128
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool b_mn_major) {
  return 1u << 4 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}

// 16 codes -> 16 exact halves
__device__ __forceinline__ void widen16(const uint4 &w, uint4 (&h)[2]) {
  k_frag(w.x, h[0].x, h[0].y);
  k_frag(w.y, h[0].z, h[0].w);
  k_frag(w.z, h[1].x, h[1].y);
  k_frag(w.w, h[1].z, h[1].w);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// the largest score of the first `left` tokens of a 16-token group (all of them
// unless cut); in: the group's constants
__device__ __forceinline__ float group_max(float *x, const float *in, float inv, bool cut,
                                           int left) {
  if (cut) {
    // unseen tokens repeat the first one
#pragma unroll
    for (int e = 1; e < 16; e++) x[e] = e < left ? x[e] : x[0];
  }
  float g0 = max3(x[0], x[1], x[2]), g1 = max3(x[3], x[4], x[5]);
  g0 = max3(g0, x[6], x[7]);
  g1 = max3(g1, x[8], x[9]);
  g0 = max3(g0, x[10], x[11]);
  g1 = max3(g1, x[12], x[13]);
  g0 = max3(g0, x[14], x[15]);
  // unmapped groups have a log2 scale of -inf
  const float y = fmaxf(g0, g1) * (inv * in[0]);
  return in[8] == -INFINITY || (cut && left <= 0) ? -INFINITY : y;
}
// a group of scores -> p' as fp16 at `to`; l grows by p' / v_scale / 2^20.
// CUT: only the first `left` tokens are seen.
template <bool CUT>
__device__ __forceinline__ void group_exp(const float *s, const float *in, float inv, float ve,
                                          int left, float &l, uint32_t to) {
  const float f = inv * in[0], c = in[8] - ve;
  const float2 f2 = make_float2(f, f), c2 = make_float2(c, c);
  float2 p[8];
#pragma unroll
  for (int e = 0; e < 8; e++) p[e] = __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), f2, c2);
#pragma unroll
  for (int e = 0; e < 8; e++) p[e] = make_float2(ex2(p[e].x), ex2(p[e].y));
  if (CUT) {
#pragma unroll
    for (int e = 0; e < 8; e++) {
      p[e].x = 2 * e < left ? p[e].x : 0.f;
      p[e].y = 2 * e + 1 < left ? p[e].y : 0.f;
    }
  }
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; e++) w[e] = pack_f16x2(p[e].x, p[e].y);
  t5_st8(to, w);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1)
#pragma unroll
    for (int e = 0; e < o; e++) p[e] = add2(p[e], p[e + o]);
  if (!CUT || left > 0) l = fmaf(p[0].x + p[0].y, in[16], l);
}

// ---- work
// A CTA per unit (row tile of a sequence and kv head), the longest sequences
// first, in whole waves of the card's SMs; the units of the last, partial wave
// (all of them where there are fewer units than SMs) are cut along their tokens
// into as many pieces as fill it, and a second kernel joins those.  Without the
// cut a prompt chunk of 336 units ended on 40 SMs: 491 us.  Lengths live on the
// device, so each CTA finds its unit: it ranks the sequences and counts their
// row tiles.
constexpr int kLeast = 4;  // tiles of a piece
struct Job {
  int b, kvh, rt;      // b < 0: nothing to do
  int piece, pieces;   // of the unit's tokens (some may be empty)
  int tail;            // index among the cut units, -1 if not one
};
// behind the records of the pieces (at most one an SM): what each cut unit is
__device__ __forceinline__ int4 *metas(const AttnArgs &a, int rows, int dim) {
  return reinterpret_cast<int4 *>(a.ws + (int64_t)kNumSMs * rows * (dim + 4));
}
template <class C>
__device__ Job find_job(const AttnArgs &a) {
  __shared__ int ids[C::kThreads], tiles[C::kThreads];  // sequences by rank, their row tiles
  const int tid = threadIdx.x, batch = a.q.batch, hkv = a.c.num_kv_heads;
  Job j = {-1, 0, 0, 0, 1, -1};
  int4 *meta = metas(a, C::kRows, a.c.head_dim);
  if (batch > C::kThreads) {  // as they come, uncut
    int u = blockIdx.x;
    if (u == 0 && tid < kNumSMs) meta[tid].x = -1;
    j.kvh = u % hkv;
    u /= hkv;
    j.rt = a.p.row_tiles - 1 - u % a.p.row_tiles;
    u /= a.p.row_tiles;
    j.b = u < batch ? u : -1;
    return j;
  }
  if (tid < batch) {
    const int mine = seq_len(a.q, a.c, tid);
    int rank = 0, q0;
    for (int o = 0; o < batch; o++) {
      const int l = seq_len(a.q, a.c, o);
      rank += l > mine || (l == mine && o < tid);
    }
    ids[rank] = tid;
    tiles[rank] = (query_range(a.q, tid, q0) * a.q.group + C::kRows - 1) / C::kRows;
  }
  __syncthreads();
  int units = 0;
  for (int s = 0; s < batch; s++) units += tiles[s] * hkv;
  const int whole = units / kNumSMs * kNumSMs, rest = units - whole;
  const int pieces = rest ? kNumSMs / rest : 1;
  if (blockIdx.x == 0 && tid < kNumSMs && (tid >= rest || pieces == 1)) meta[tid].x = -1;
  int u = blockIdx.x;
  if (u >= whole) {
    u -= whole;
    if (pieces > 1) {
      j.tail = u / pieces;
      j.piece = u % pieces;
      j.pieces = pieces;
      u = j.tail;
    }
    u += whole;
  }
  for (int s = 0; s < batch; s++) {
    const int n = tiles[s] * hkv;
    if (u < n) {
      j.b = ids[s];
      j.rt = tiles[s] - 1 - u / hkv;
      j.kvh = u % hkv;
      break;
    }
    u -= n;
  }
  return j;
}

// One warp per row of the cut units: join the pieces' records.
// grid: 8 rows + rows / 8 * cut unit
template <int D>
__global__ void __launch_bounds__(256) b8_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int kRows = PCfg<D>::kRows;
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x / (kRows / 8);
  const int r = blockIdx.x % (kRows / 8) * 8 + (threadIdx.x >> 5);
  dec::grid_dependency_wait();
  const int4 m = metas(a, kRows, D)[unit];
  if (m.x < 0) return;
  int q0;
  const int n_rows = query_range(a.q, m.x, q0) * a.q.group, row = m.z * kRows + r;
  if (row >= n_rows) return;
  const int n = m.w & 0xffff, slots = m.w >> 16;
  const float *rec = a.ws + ((int64_t)unit * slots * kRows + r) * (D + 4);
  constexpr int64_t kStep = (int64_t)kRows * (D + 4);
  // lane l: states of pieces l, l + 32, ... (at most kNumSMs)
  constexpr int kMost = (kNumSMs + 31) / 32;
  float pm[kMost], pl[kMost];
  float M = -1e30f, L = 0.f;
#pragma unroll
  for (int i = 0; i < kMost; i++) {
    const int s = lane + 32 * i;
    const float2 x = s < n ? *reinterpret_cast<const float2 *>(rec + s * kStep) : make_float2(-1e30f, 0.f);
    pm[i] = x.x, pl[i] = x.y;
    M = fmaxf(M, x.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
  for (int i = 0; i < kMost; i++) {
    pm[i] = ex2(pm[i] - M);
    L += pm[i] * pl[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  constexpr int kPer = D / 128 > 0 ? D / 128 : 1;
  float4 acc[kPer];
#pragma unroll
  for (int h = 0; h < kPer; h++) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kMost; i++) {
#pragma unroll 8
    for (int s = 32 * i; s < min(n, 32 * i + 32); s++) {
      const float f = __shfl_sync(0xffffffffu, pm[i], s & 31);
#pragma unroll
      for (int h = 0; h < kPer; h++) {
        if (4 * lane + 128 * h >= D) continue;
        const float4 x = *reinterpret_cast<const float4 *>(rec + s * kStep + 4 + 4 * lane + 128 * h);
        acc[h].x += f * x.x, acc[h].y += f * x.y, acc[h].z += f * x.z, acc[h].w += f * x.w;
      }
    }
  }
  const float norm = L > 0.f ? __fdiv_rn(1.f, L) : L == 0.f ? 0.f : L;
  const int i = row / a.q.group;
  const int64_t orow = (int64_t)(q0 + i) * a.q.num_heads + m.y * a.q.group + row - i * a.q.group;
#pragma unroll
  for (int h = 0; h < kPer; h++) {
    const int d = 4 * lane + 128 * h;
    if (d >= D) continue;
    const __nv_bfloat162 u = __floats2bfloat162_rn(acc[h].x * norm, acc[h].y * norm);
    const __nv_bfloat162 v = __floats2bfloat162_rn(acc[h].z * norm, acc[h].w * norm);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + orow * D + d) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
  }
  if (lane == 0 && a.lse != nullptr) a.lse[orow] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
}

template <int D>
__global__ void __launch_bounds__(PCfg<D>::kThreads, 1)
    b8_prefill_kernel(const __grid_constant__ AttnArgs a) {
  using C = PCfg<D>;
  constexpr int kBN = C::kBN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const kvq_b8_cache &c = a.c;

  const Job job = find_job<C>(a);
  if (job.b < 0) return;
  const int b = job.b, kvh = job.kvh, rt = job.rt;
  int q0;
  const int nq = query_range(a.q, b, q0);
  const int n_rows = nq * a.q.group, row0 = rt * C::kRows;
  if (row0 >= n_rows) return;
  const int len = seq_len(a.q, c, b);
  const int i_last = (min(row0 + C::kRows, n_rows) - 1) / a.q.group;
  const int hi_lim = max(0, len - nq + i_last + 1);
  const int all_tiles = (hi_lim + kBN - 1) / kBN;
  const int per = max(kLeast, (all_tiles + job.pieces - 1) / job.pieces);
  const int pieces = max(1, (all_tiles + per - 1) / per);  // that hold work
  if (job.piece >= pieces) return;
  if (job.tail >= 0 && job.piece == 0 && tid == 0)
    metas(a, C::kRows, D)[job.tail] = make_int4(pieces > 1 ? b : -1, kvh, rt, job.pieces << 16 | pieces);
  const int t0 = job.piece * per * kBN;
  const int t1 = (int)min((int64_t)hi_lim, (int64_t)t0 + (int64_t)per * kBN);  // (past 2^31)
  const int nt = C::kNT == 2 && n_rows - row0 > 128 ? 2 : 1;
  const int n_tiles = t1 > t0 ? (t1 - t0 + kBN - 1) / kBN : 0;
  const int n_items = n_tiles * nt;

  const uint32_t base = smem_u32(smem);
  const uint32_t bars = base + C::kOffBar;
  const uint32_t k_full = bars, k_empty = bars + 16, v_full = bars + 32, v_empty = bars + 48,
                 s_full = bars + 64, p_full = bars + 80, o_done = bars + 96, info_full = bars + 112,
                 drain = bars + 144, all_done = bars + 152;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc);
  uint32_t *tmem_at = reinterpret_cast<uint32_t *>(smem + C::kOffMisc + 4);
  float *info = reinterpret_cast<float *>(smem + C::kOffInfo);
  constexpr int kIssueWarp = C::kSoft / 32 + 4;
  if (tid == 0) {
    for (int i = 0; i < 2; i++) {
      mbar_init(k_full + 8 * i, 128);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, 128);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 128);
      mbar_init(o_done + 8 * i, 1);
      mbar_init(all_done + 8 * i, 1);
    }
    for (int i = 0; i < C::kInfo; i++) mbar_init(info_full + 8 * i, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssueWarp) t5_alloc(base + C::kOffMisc + 4, 512);

  // bounded wait; false once any thread of the CTA has given up
  auto wait1 = [&](uint32_t bar, uint32_t parity) {
    if (dec::mbar_wait(bar, parity, abort_flag, a.polls)) return true;
    *abort_flag = 1;
    dec::report(a.err, KVQ_DEVERR_WAIT_TIMEOUT);
    return false;
  };
  // the same for a whole warp: one answer for all lanes
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait1(bar, parity)) != 0;
  };

  // ---- queries: a thread brings its row into [2^13, 2^14) by a power of two
  // and stores it as fp16
  const int wg = warp >> 2;  // row tile of a softmax warp
  const int r = tid & 127;
  const int row = row0 + wg * 128 + r;
  const bool soft = tid < C::kSoft && wg < nt;
  const bool live = soft && row < n_rows;
  const int qi = live ? row / a.q.group : 0;
  const int head = kvh * a.q.group + (live ? row - qi * a.q.group : 0);
  float inv = 0.f;
  if (soft) {
    const uint4 *src = reinterpret_cast<const uint4 *>(
        static_cast<const uint16_t *>(a.q.q) + (int64_t)(q0 + qi) * a.q.token_stride +
        (int64_t)head * a.q.head_stride);
    float m = 0.f;
#pragma unroll 8
    for (int ch = 0; ch < D / 8; ch++) {
      const uint4 w = live ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; e++)
        m = fmax_nan(m, fmax_nan(fabsf(bf16lo(ww[e])), fabsf(bf16hi(ww[e]))));
    }
    // the sign of the scale goes into q, so that scores grow with products
    const float f = copysignf(query_scale(m), a.q.scale);
    inv = __fdiv_rn(a.q.scale * kLog2e, f);
    uint8_t *dst = smem + wg * C::kQTileBytes + r * 128;
#pragma unroll 8
    for (int ch = 0; ch < D / 8; ch++) {
      const uint4 w = live ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
      uint4 h;
      h.x = pack_f16x2(bf16lo(w.x) * f, bf16hi(w.x) * f);
      h.y = pack_f16x2(bf16lo(w.y) * f, bf16hi(w.y) * f);
      h.z = pack_f16x2(bf16lo(w.z) * f, bf16hi(w.z) * f);
      h.w = pack_f16x2(bf16lo(w.w) * f, bf16hi(w.w) * f);
      *reinterpret_cast<uint4 *>(dst + (ch >> 3) * (128 * 128) + (((ch & 7) ^ (r & 7)) << 4)) = h;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  t5_before();
  __syncthreads();
  t5_after();
  const uint32_t tmem = *tmem_at;
  // (every warp takes its share, idle ones too)
  if (warp < C::kSoft / 32) {
    if constexpr (C::kNT == 2)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoft));
    if (soft) {
    // ---------------------------------------------------------- softmax
    // (rows of no query: all tokens, so that they cost their warp no masks)
    const int lim = live ? max(0, len - nq + qi + 1) : 1 << 30;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // 32 lanes a warp
    const uint32_t o_at = lanes + C::kColO + wg * D;
    float ve = -1e30f, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_tiles; j++) {
      const int i = j * nt + wg, buf = i & 1;
      const uint32_t s_at = lanes + C::kColS + buf * kBN;
      if (!wait(info_full + 8 * (j & 3), (j >> 2) & 1) || !wait(s_full + 8 * buf, (i >> 1) & 1)) {
        ok = false;
        break;
      }
      t5_after();
      const float *in = info + (j & 3) * C::kInfoFloats;
      const int tok = t0 + j * kBN;
      const bool cut = __any_sync(0xffffffffu, tok + kBN > lim);
      // row maximum
      float mx = -INFINITY;
      float s[kBN / 32][32];
#pragma unroll
      for (int ch = 0; ch < kBN / 32; ch++) t5_ld32(s_at + 32 * ch, s[ch]);
      t5_wait_ld(s[0]);
#pragma unroll
      for (int ch = 1; ch < kBN / 32; ch++) after_wait(s[ch]);
#pragma unroll
      for (int gr = 0; gr < C::kGroups; gr++)
        mx = fmaxf(mx, group_max(s[gr / 2] + 16 * (gr & 1), in + gr, inv, cut, lim - tok - 16 * gr));
      // (with the tile's largest V scale in the place of each group's: a bound)
      if (__any_sync(0xffffffffu, mx > ve + 14.f - in[24])) {
        // the bound serves where the tile's V scales are no more than 4 apart (a
        // maximum over the groups every time: 398 us instead of 387)
        float mvx = mx + in[24];
        if (!(in[24] - in[25] <= 2.f)) {
          mvx = -INFINITY;
#pragma unroll 1
          for (int gr = 0; gr < C::kGroups; gr++) {
            float x[16];
            t5_ld16(s_at + 16 * gr, x);
            t5_wait_ld(x);
            mvx = fmaxf(mvx, in[8 + gr] + group_max(x, in + gr, inv, cut, lim - tok - 16 * gr));
          }
        }
        // an integer, so that f is a power of two
        const float vn = mvx > ve + 14.f ? ceilf(mvx) - 6.f : ve;
        const float f = ex2(ve - vn);
        l *= f;
        ve = vn;
        if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
          if (!wait(o_done + 8 * wg, (j - 1) & 1)) {
            ok = false;
            break;
          }
          t5_after();
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ch++) {
            float o[32];
            t5_ld32(o_at + 32 * ch, o);
            t5_wait_ld(o);
#pragma unroll
            for (int h = 0; h < 2; h++) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; e++) w[e] = __float_as_uint(o[16 * h + e] * f);
              t5_st16(o_at + 32 * ch + 16 * h, w);
            }
          }
        }
      }
      // probabilities, over the scores that were read
      if (!cut) {
#pragma unroll
        for (int gr = 0; gr < C::kGroups; gr++)
          group_exp<false>(s[gr / 2] + 16 * (gr & 1), in + gr, inv, ve, 0, l, s_at + 8 * gr);
      } else {
        // the tiles at the end of a row's tokens: group_max has changed the
        // scores, so they are read again
#pragma unroll 1
        for (int gr = 0; gr < C::kGroups; gr++) {
          float x[16];
          t5_ld16(s_at + 16 * gr, x);
          t5_wait_ld(x);
          group_exp<true>(x, in + gr, inv, ve, lim - tok - 16 * gr, l, s_at + 8 * gr);
        }
      }
      t5_wait_st();
      t5_before();
      mbar_arrive(p_full + 8 * buf);
    }
    // ---- result
    // (a barrier of its own: a wait tells a phase from the next one only, and at
    // this point o_done may be one, two or three phases on)
    if (ok && n_tiles > 0) ok = wait(all_done + 8 * wg, 0);
    t5_after();
    const bool direct = pieces == 1;
    const float nan = __int_as_float(0x7fc00000);
    // a record holds l in [1, 2) and O for it
    const float e = l > 0.f ? floorf(log2f(l)) : 0.f;
    float norm = direct ? 0x1p-20f / l : ex2(-20.f - e);
    if (!(l > 0.f)) norm = l;
    float m = ve + 20.f + e;
    if (!direct) l *= ex2(-e);
    if (!ok) norm = m = l = nan;
    const int64_t orow = (int64_t)(q0 + qi) * a.q.num_heads + head;
    float *rec = a.ws + (((int64_t)job.tail * job.pieces + job.piece) * C::kRows + wg * 128 + r) * (D + 4);
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ch++) {
      float o[32];
      __syncwarp();
      if (n_tiles > 0) {
        t5_ld32(o_at + 32 * ch, o);
        t5_wait_ld(o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; e++) o[e] = 0.f;
      }
      if (!live) continue;
#pragma unroll
      for (int e = 0; e < 32; e++) o[e] = norm == 0.f ? 0.f : o[e] * norm;
      if (direct) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + orow * D + 32 * ch);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          uint4 w;
          uint32_t *x = &w.x;
#pragma unroll
          for (int h = 0; h < 4; h++) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(o[8 * e + 2 * h], o[8 * e + 2 * h + 1]);
            x[h] = *reinterpret_cast<const uint32_t *>(&y);
          }
          dst[e] = w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
          *reinterpret_cast<float4 *>(rec + 4 + 32 * ch + 4 * e) =
              make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    }
    if (live) {
      if (!direct)
        rec[0] = m, rec[1] = l;
      else if (a.lse != nullptr)
        a.lse[orow] = l == 0.f ? -INFINITY : kLn2 * (ve + 20.f + log2f(l));
    }
    }
  } else if (warp < kIssueWarp) {
    if constexpr (C::kNT == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsConvert));
    // ---------------------------------------------------------- convert
    constexpr int kPer = kBN * D / 16 / 128;  // 16-code pieces a thread has of a tile
    const int ct = tid - C::kSoft;
    const int32_t *table = c.block_table + (int64_t)b * c.max_blocks_per_seq;
    const int bs = c.block_size, shift = __ffs(bs) - 1;
    // lane l: block of 16-token group l % kGroups of tile j, -1 if unmapped or
    // past the range
    auto slots_of = [&](int j) {
      int p = -1;
      if (j >= n_tiles) return p;
      const int t = t0 + j * kBN + (lane % C::kGroups) * 16;
      if (t < t1) {
        p = __ldg(table + (t >> shift));
        if (p < 0 || p >= c.num_blocks || !in_bounds(p, p + 1, c.num_blocks, a.err)) p = -1;
      }
      return p;
    };
    // piece i of a thread is token 32 (i % kTr) + ct / 4, dims 64 (i / kTr) +
    // 16 (ct % 4) .. + 15; a tile's pieces stay in registers from their load to
    // their conversion one tile later (staged in shared memory they would take
    // a third of its bandwidth, which the products need)
    constexpr int kTr = kBN / 32;
    const int r4 = ct >> 2, c4 = ct & 3;
    auto copy = [&](const int8_t *codes, int j, int slots, uint4 (&x)[kPer]) {
      // first code of the lane's group; groups without a block take block 0's
      // codes, which meet probabilities of 0 (a choice between a load and a zero
      // would wait for the load right here)
      int64_t off = 0;
      if (slots >= 0) {
        const int t = t0 + j * kBN + (lane % C::kGroups) * 16;
        off = ((((int64_t)slots * c.num_kv_heads + kvh) << shift) + (t & (bs - 1))) * D;
      }
#pragma unroll
      for (int i = 0; i < kTr; i++) {
        const int tr = 32 * i + r4;
        const int64_t o = __shfl_sync(0xffffffffu, off, tr >> 4);
        const uint4 *src = reinterpret_cast<const uint4 *>(codes + o + (tr & 15) * D + 16 * c4);
#pragma unroll
        for (int pl = 0; pl < D / 64; pl++)
          x[pl * kTr + i] = __ldg(src + 4 * pl);
      }
    };
    auto put = [&](uint8_t *dst, const uint4 (&x)[kPer]) {
#pragma unroll
      for (int i = 0; i < kPer; i++) {
        const int tr = 32 * (i % kTr) + r4;
        uint4 h[2];
        widen16(x[i], h);
        uint8_t *at = dst + (i / kTr) * (kBN * 128) + tr * 128;
        *reinterpret_cast<uint4 *>(at + (((2 * c4) ^ (tr & 7)) << 4)) = h[0];
        *reinterpret_cast<uint4 *>(at + (((2 * c4 + 1) ^ (tr & 7)) << 4)) = h[1];
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    };
    uint4 kx[kPer], vx[kPer];
    float most = -INFINITY;  // log2 of the largest V scale so far
    int slots = slots_of(0), next = slots_of(1);
    copy(c.k_codes, 0, slots, kx);
    copy(c.v_codes, 0, slots, vx);
    auto scales_of = [&](int slots, float &ks, float &vs) {
      ks = vs = 0.f;
      if (warp == C::kSoft / 32 && slots >= 0) {
        ks = __ldg(c.k_scales + (int64_t)slots * c.num_kv_heads + kvh);
        vs = __ldg(c.v_scales + (int64_t)slots * c.num_kv_heads + kvh);
      }
    };
    float ks, vs;
    scales_of(slots, ks, vs);
    for (int j = 0; j < n_tiles; j++) {
      const int st = j & 1;
      const int after = slots_of(j + 2);
      if (warp == C::kSoft / 32) {
        // the tile's group constants; slot j % 4 was last read for tile j - 4,
        // whose second product was waited for before V of tile j - 2 was stored
        // infinite and NaN scales spoil the scores, and so do those whose share of l
        // would vanish (their sums leave fp32's range before long)
        const bool fine = vs < 0x1p105f;
        float lv = fine ? log2f(vs) : 0.f;
        float hi = slots >= 0 ? lv : -INFINITY, lo;
#pragma unroll
        for (int o = 1; o < C::kGroups; o <<= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        most = fmaxf(most, hi);
        // (an append makes no scale below 2^-107 but 0)
        lv = fmaxf(lv, fmaxf(most - 97.f, -108.f));
        hi = slots >= 0 ? lv : -INFINITY, lo = slots >= 0 ? lv : INFINITY;
#pragma unroll
        for (int o = 1; o < C::kGroups; o <<= 1) {
          hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
          lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        }
        float *in = info + (j & 3) * C::kInfoFloats;
        if (lane < C::kGroups) {
          in[lane] = fine ? ks : __int_as_float(0x7fc00000);
          in[8 + lane] = slots >= 0 ? lv : -INFINITY;
          in[16 + lane] = slots >= 0 ? ex2(-20.f - lv) : 0.f;
          if (lane == 0) in[24] = hi, in[25] = lo;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(info_full + 8 * (j & 3));
      }
      if (j >= 2 && !wait(k_empty + 8 * st, ((j - 2) >> 1) & 1)) break;
      put(smem + C::kOffK + st * C::kKVBytes, kx);
      mbar_arrive(k_full + 8 * st);
      copy(c.k_codes, j + 1, next, kx);
      scales_of(next, ks, vs);
      if (j >= 2 && !wait(v_empty + 8 * st, ((j - 2) >> 1) & 1)) break;
      put(smem + C::kOffV + st * C::kKVBytes, vx);
      mbar_arrive(v_full + 8 * st);
      copy(c.v_codes, j + 1, next, vx);
      slots = next;
      next = after;
    }
  } else {
    if constexpr (C::kNT == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsIssue));
    if (warp == kIssueWarp && lane == 0) {
    // ---------------------------------------------------------- issue
    constexpr uint32_t kIdS = instr_desc(kBN, false), kIdO = instr_desc(D, true);
    bool ok = true;
    // descriptors of the operands' first pieces; a piece `bytes` on adds bytes / 16
    const uint64_t q0d = smem_desc(base, 16, 1024), k0d = smem_desc(base + C::kOffK, 16, 1024),
                   v0d = smem_desc(base + C::kOffV, kBN * 128, 1024);
    auto issue_s = [&](int i) {
      const int j = nt == 2 ? i >> 1 : i, t = i - j * nt, st = j & 1;
      if (t == 0) ok = wait1(k_full + 8 * st, (j >> 1) & 1);
      if (!ok) return;
      t5_after();
      const uint32_t d = tmem + C::kColS + (i & 1) * kBN;
      const uint64_t qd = q0d + (t ? C::kQTileBytes / 16 : 0), kd = k0d + (st ? C::kKVBytes / 16 : 0);
#pragma unroll
      for (int ks = 0; ks < D / 16; ks++)
        t5_mma_ss(d, qd + ((ks >> 2) * (128 * 128) + (ks & 3) * 32) / 16,
                  kd + ((ks >> 2) * (kBN * 128) + (ks & 3) * 32) / 16, kIdS, ks > 0);
      t5_commit(s_full + 8 * (i & 1));
      if (t == nt - 1) t5_commit(k_empty + 8 * st);
    };
    for (int i = 0; i < min(2, n_items) && ok; i++) issue_s(i);
    for (int i = 0; i < n_items && ok; i++) {
      const int j = nt == 2 ? i >> 1 : i, t = i - j * nt, st = j & 1;
      // V first: it has long been there when the probabilities come
      if (t == 0) ok = wait1(v_full + 8 * st, (j >> 1) & 1);
      ok = ok && wait1(p_full + 8 * (i & 1), (i >> 1) & 1);
      if (!ok) break;
      t5_after();
      const uint32_t p = tmem + C::kColS + (i & 1) * kBN;
      const uint64_t vd = v0d + (st ? C::kKVBytes / 16 : 0);
#pragma unroll
      for (int ks = 0; ks < kBN / 16; ks++)
        t5_mma_ts(tmem + C::kColO + t * D, p + 8 * ks, vd + ks * (2048 / 16), kIdO, j > 0 || ks > 0);
      t5_commit((j == n_tiles - 1 ? all_done : o_done) + 8 * t);
      if (t == nt - 1) t5_commit(v_empty + 8 * st);
      if (i + 2 < n_items) issue_s(i + 2);
    }
    // Products end before tensor memory is given back and the CTA leaves, whoever
    // gave up: a softmax warp may have done so after the last product's issue.  (A
    // bounded wait, like every other.  It covers the commits to k_empty and v_empty
    // that nobody waits for, too.)
    t5_commit(drain);
    for (int n = 0; n < (1 << 20) && !dec::mbar_try(drain, 0); n++) {
    }
    }
  }
  __syncwarp();
  t5_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    t5_after();
    t5_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
  using C = PCfg<D>;
  cudaError_t e = allow_smem<b8_prefill_kernel<D>>(C::kSmem);
  if (e != cudaSuccess) return e;
  // the units that there may be, and the pieces that the last ones are cut into
  const int64_t units = (int64_t)a.q.batch * a.c.num_kv_heads * a.p.row_tiles;
  b8_prefill_kernel<D><<<(unsigned)(units + kNumSMs), C::kThreads, C::kSmem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kNumSMs * C::kRows / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, b8_join_kernel<D>, a);
}

}  // namespace

int b8_prefill_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }
size_t b8_prefill_workspace(int head_dim) {
  return (size_t)kNumSMs * (b8_prefill_rows(head_dim) * (head_dim + 4) * 4 + sizeof(int4));
}

cudaError_t launch_b8_prefill(const AttnArgs &a, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch<64>(a, s);
    case 128: return launch<128>(a, s);
    default: return launch<256>(a, s);
  }
}

}  // namespace kvq
