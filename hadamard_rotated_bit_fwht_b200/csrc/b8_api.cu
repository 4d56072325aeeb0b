// b8_api.cu -- the extern "C" entry points of the rotary positions and of the
// block-scaled 8-bit cache: host-side argument validation and dispatch.
#include <math.h>
#include <stdlib.h>

#include "b8_internal.cuh"

using namespace kvq;

namespace {

cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }

kvq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// do the ranges of na and nb 4-byte values share one
bool overlap(const void *a, __int128 na, const void *b, __int128 nb) {
  const __int128 x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * nb && y < x + 4 * na;
}

bool good_dtype(kvq_dtype t) { return t == KVQ_F32 || t == KVQ_BF16; }

kvq_status check_heads(const kvq_heads *x) {
  if (!x || !x->data || !aligned(x->data, 16) || x->num_heads < 1) return KVQ_ERR_INVALID_ARG;
  if (x->token_stride % 8 || x->head_stride % 8) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

kvq_status check_rope(const kvq_rope_spec *r, int head_dim) {
  if (!r || !r->d_inv_freq || !aligned(r->d_inv_freq, 8) || !isfinite(r->factor))
    return KVQ_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim > head_dim) return KVQ_ERR_INVALID_ARG;
  return r->rot_dim % 16 ? KVQ_ERR_UNSUPPORTED : KVQ_OK;
}

kvq_status check_b8(const kvq_b8_cache *c) {
  if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !c->block_table)
    return KVQ_ERR_INVALID_ARG;
  if (c->num_kv_heads < 1 || c->head_dim < 1 || c->block_size < 1 || c->num_blocks < 1 ||
      c->num_seqs < 1 || c->max_blocks_per_seq < 1)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16)) return KVQ_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  const int bs = c->block_size;
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128 && bs != 256) return KVQ_ERR_UNSUPPORTED;
  // grid rows, 32-bit row coordinates of the code planes and 32-bit positions (of tiles
  // that end past the last token too)
  if (c->num_kv_heads > 65535 || (int64_t)c->num_blocks * c->num_kv_heads * bs >= (1LL << 31) ||
      (int64_t)c->max_blocks_per_seq * bs >= (1LL << 31) - 4096)
    return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

kvq_status check_queries(const kvq_b8_cache &c, const kvq_b8_queries *q, B8Queries &out) {
  if (!q || !good_dtype(q->dtype) || q->batch < 0 || q->total_q < 0 || q->max_q < 0 ||
      q->max_seq_len < 0 || q->batch > c.num_seqs || !isfinite(q->scale))
    return KVQ_ERR_INVALID_ARG;
  if (!q->d_cu_q && q->total_q != q->batch) return KVQ_ERR_INVALID_ARG;
  if (q->batch > 0 && q->total_q > 0) {
    const kvq_status st = check_heads(&q->q);
    if (st != KVQ_OK) return st;
    if (!q->d_seq_lens || q->q.num_heads % c.num_kv_heads) return KVQ_ERR_INVALID_ARG;
  }
  out.q = q->q.data;
  out.token_stride = q->q.token_stride;
  out.head_stride = q->q.head_stride;
  out.bf16 = q->dtype == KVQ_BF16;
  out.num_heads = q->q.num_heads;
  out.group = q->q.num_heads / c.num_kv_heads;
  out.batch = q->batch;
  out.total_q = q->total_q;
  out.max_q = q->d_cu_q ? q->max_q : 1;
  out.cu_q = q->d_cu_q;
  out.seq_lens = q->d_seq_lens;
  out.max_seq_len = q->max_seq_len;
  out.scale = q->scale;
  return KVQ_OK;
}

// (sequence, head, row tile, split) units are counted in 31 bits, and so are
// their rows
bool plan_fits(const kvq_b8_cache &c, int batch, const B8Plan &p) {
  return (int64_t)batch * c.num_kv_heads * p.row_tiles < (1LL << 31) / ((int64_t)p.splits * p.rows);
}

}  // namespace

extern "C" {

kvq_status kvq_rope_frequencies(int32_t rot_dim, double base, kvq_rope_scaling kind, double scale,
                                double trained_len, double beta_fast, double beta_slow,
                                double *inv_freq, float *factor) {
  if (rot_dim < 2 || rot_dim % 2 || !(base > 0) || !isfinite(base) || !(scale >= 1) ||
      !isfinite(scale) || !inv_freq || !factor)
    return KVQ_ERR_INVALID_ARG;
  if (kind < KVQ_ROPE_NONE || kind > KVQ_ROPE_YARN) return KVQ_ERR_INVALID_ARG;
  if (kind == KVQ_ROPE_YARN &&
      (!(trained_len > 0) || !isfinite(trained_len) || !(beta_fast > beta_slow) ||
       !isfinite(beta_fast) || !isfinite(beta_slow)))
    return KVQ_ERR_INVALID_ARG;
  // one pair alone has exponent 0: any base gives the same frequency
  if (kind == KVQ_ROPE_NTK && rot_dim > 2) base *= pow(scale, (double)rot_dim / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; i++) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (kind == KVQ_ROPE_LINEAR) f /= scale;
    if (kind == KVQ_ROPE_YARN) {
      const double turns = trained_len * f / 6.283185307179586477;
      const double ramp = fmin(fmax((turns - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0);
      f = f / scale * (1.0 - ramp) + f * ramp;
    }
    inv_freq[i] = f;
  }
  *factor = kind == KVQ_ROPE_YARN ? (float)(0.1 * log(scale) + 1.0) : 1.f;
  return KVQ_OK;
}

kvq_status kvq_rope(const kvq_rope_spec *spec, kvq_dtype dtype, int32_t head_dim,
                    int32_t num_tokens, const int32_t *d_positions, int32_t inverse,
                    const kvq_heads *q, const kvq_heads *q_out, const kvq_heads *k,
                    const kvq_heads *k_out, void *stream) {
  if (num_tokens < 0 || head_dim < 1 || !good_dtype(dtype)) return KVQ_ERR_INVALID_ARG;
  kvq_status st = check_rope(spec, head_dim);
  if (st != KVQ_OK) return st;
  if (head_dim % 16 || head_dim > 512) return KVQ_ERR_UNSUPPORTED;
  if (!k != !k_out) return KVQ_ERR_INVALID_ARG;
  if (num_tokens == 0) return KVQ_OK;
  if (!d_positions) return KVQ_ERR_INVALID_ARG;
  const kvq_heads *views[4] = {q, q_out, k, k_out};
  for (int i = 0; i < (k ? 4 : 2); i++)
    if ((st = check_heads(views[i])) != KVQ_OK) return st;
  for (int i = 0; i < (k ? 4 : 2); i += 2) {
    const kvq_heads *a = views[i], *b = views[i + 1];
    if (a->num_heads != b->num_heads) return KVQ_ERR_INVALID_ARG;
    // heads of an output that share elements (of a broadcast view) would be rotated
    // more than once, or race
    const int64_t ts = llabs(b->token_stride), hs = llabs(b->head_stride);
    if ((num_tokens > 1 && ts < head_dim) || (b->num_heads > 1 && hs < head_dim) ||
        (num_tokens > 1 && b->num_heads > 1 && ts == hs))
      return KVQ_ERR_INVALID_ARG;
    // in place means the very same view
    if (a->data == b->data &&
        (a->token_stride != b->token_stride || a->head_stride != b->head_stride))
      return KVQ_ERR_INVALID_ARG;
  }
  // pieces of one CTA's tokens are counted in 32 bits
  if (((int64_t)q->num_heads + (k ? k->num_heads : 0)) * (head_dim / 16) >= (1LL << 28))
    return KVQ_ERR_UNSUPPORTED;
  const kvq_heads none = {nullptr, 0, 0, 0};
  return from_cuda(launch_rope(*spec, dtype == KVQ_BF16, head_dim, num_tokens, d_positions,
                               inverse != 0, *q, *q_out, k ? *k : none, k ? *k_out : none,
                               as_stream(stream)));
}

kvq_status kvq_b8_append(const kvq_b8_cache *cache, const kvq_heads *k, const kvq_heads *v,
                         kvq_dtype dtype, int32_t batch, int32_t t_new,
                         const int32_t *d_start_pos, const int32_t *d_new_lens,
                         const kvq_rope_spec *rope, const int32_t *d_rope_pos, void *stream) {
  kvq_status st = check_b8(cache);
  if (st != KVQ_OK) return st;
  if (batch < 0 || t_new < 0 || !good_dtype(dtype) || batch > cache->num_seqs)
    return KVQ_ERR_INVALID_ARG;
  if (rope && (st = check_rope(rope, cache->head_dim)) != KVQ_OK) return st;
  if (batch == 0 || t_new == 0) return KVQ_OK;
  if (!d_start_pos) return KVQ_ERR_INVALID_ARG;
  if ((st = check_heads(k)) != KVQ_OK || (st = check_heads(v)) != KVQ_OK) return st;
  if (k->num_heads != cache->num_kv_heads || v->num_heads != cache->num_kv_heads)
    return KVQ_ERR_INVALID_ARG;
  // one CTA per (sequence, touched block, K or V)
  if (2LL * batch * (t_new / cache->block_size + 2) >= (1LL << 31)) return KVQ_ERR_UNSUPPORTED;
  const kvq_rope_spec none = {nullptr, 0, 0, 1.f};
  return from_cuda(launch_b8_append(*cache, *k, *v, dtype == KVQ_BF16, batch, t_new, d_start_pos,
                                    d_new_lens, rope ? *rope : none, d_rope_pos,
                                    as_stream(stream)));
}

kvq_status kvq_b8_gather(const kvq_b8_cache *cache, int32_t batch, const int32_t *d_first,
                         const int32_t *d_ends, int32_t count, kvq_dtype dtype, void *k_out,
                         void *v_out, void *stream) {
  kvq_status st = check_b8(cache);
  if (st != KVQ_OK) return st;
  if (batch < 0 || count < 0 || !good_dtype(dtype) || batch > cache->num_seqs)
    return KVQ_ERR_INVALID_ARG;
  if (batch == 0 || count == 0) return KVQ_OK;
  if (!d_first || !d_ends || !k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16))
    return KVQ_ERR_INVALID_ARG;
  // 8-element pieces of a sequence in 32 bits, sequences on a grid axis
  if ((int64_t)count * cache->num_kv_heads * (cache->head_dim / 8) >= (1LL << 31) || batch > 65535)
    return KVQ_ERR_UNSUPPORTED;
  return from_cuda(launch_b8_gather(*cache, batch, d_first, d_ends, count, dtype == KVQ_BF16,
                                    k_out, v_out, as_stream(stream)));
}

size_t kvq_b8_attn_workspace(const kvq_b8_cache *cache, kvq_dtype dtype, int32_t num_q_heads,
                             int32_t batch, int32_t max_q, int32_t max_seq_len) {
  if (check_b8(cache) != KVQ_OK || !good_dtype(dtype) || num_q_heads < 1 || num_q_heads % cache->num_kv_heads ||
      batch < 1 || max_q < 1 || max_seq_len < 0)
    return 0;
  const int group = num_q_heads / cache->num_kv_heads;
  if ((int64_t)max_q * group >= (1LL << 31) - 256) return 0;
  return b8_attn_workspace_bytes(*cache, batch,
                                 plan_b8_attn(*cache, dtype == KVQ_BF16, group, batch, max_q, max_seq_len));
}

kvq_status kvq_b8_attn(const kvq_b8_cache *cache, const kvq_b8_queries *queries, void *out,
                       float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  kvq_status st = check_b8(cache);
  if (st != KVQ_OK) return st;
  B8Queries q;
  if ((st = check_queries(*cache, queries, q)) != KVQ_OK) return st;
  if (q.batch == 0 || q.total_q == 0 || q.max_q == 0) return KVQ_OK;
  if (!out || !aligned(out, 16)) return KVQ_ERR_INVALID_ARG;
  if ((int64_t)q.max_q * q.group >= (1LL << 31) - 256) return KVQ_ERR_UNSUPPORTED;
  const B8Plan p = plan_b8_attn(*cache, q.bf16, q.group, q.batch, q.max_q, q.max_seq_len);
  if (!plan_fits(*cache, q.batch, p)) return KVQ_ERR_UNSUPPORTED;
  const size_t need = b8_attn_workspace_bytes(*cache, q.batch, p);
  if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return KVQ_ERR_WORKSPACE;
  // other CTAs may still read the queries when one writes its rows
  if (out == q.q) return KVQ_ERR_INVALID_ARG;
  return from_cuda(launch_b8_attn(*cache, q, p, out, lse, static_cast<float *>(workspace),
                                  as_stream(stream)));
}

kvq_status kvq_b8_attn_mass(const kvq_b8_cache *cache, const kvq_b8_queries *queries,
                            const float *lse, float *mass, int64_t mass_stride, void *stream) {
  kvq_status st = check_b8(cache);
  if (st != KVQ_OK) return st;
  B8Queries q;
  if ((st = check_queries(*cache, queries, q)) != KVQ_OK) return st;
  if (q.batch == 0 || q.total_q == 0 || q.max_q == 0 || q.max_seq_len == 0) return KVQ_OK;
  if (!lse || !mass || mass_stride < q.max_seq_len) return KVQ_ERR_INVALID_ARG;
  // row and CTA indices of 32 bits (a CTA takes at least 128 tokens)
  if ((int64_t)q.max_q * q.group >= (1LL << 31) - 64 ||
      (int64_t)q.batch * cache->num_kv_heads >= (1LL << 31) / (q.max_seq_len / 128 + 1))
    return KVQ_ERR_UNSUPPORTED;
  return from_cuda(launch_b8_mass(*cache, q, lse, mass, mass_stride, as_stream(stream)));
}

kvq_status kvq_b8_evict(const kvq_b8_cache *src, const kvq_b8_cache *dst, int32_t batch,
                        const int32_t *d_seq_lens, int32_t max_seq_len, const float *mass,
                        int64_t mass_stride, int32_t keep, int32_t recent, int32_t sinks,
                        int32_t *new_lens, int32_t *kept, float *mass_out,
                        int64_t mass_out_stride, void *stream) {
  kvq_status st;
  if ((st = check_b8(src)) != KVQ_OK || (st = check_b8(dst)) != KVQ_OK) return st;
  if (batch < 0 || batch > src->num_seqs || batch > dst->num_seqs || max_seq_len < 0 || keep < 1 ||
      recent < 0 || sinks < 0 || (int64_t)recent + sinks > keep)
    return KVQ_ERR_INVALID_ARG;
  if (src->num_kv_heads != dst->num_kv_heads || src->head_dim != dst->head_dim ||
      keep > (int64_t)dst->max_blocks_per_seq * dst->block_size)
    return KVQ_ERR_INVALID_ARG;
  if (batch == 0) return KVQ_OK;
  if (!d_seq_lens || (!mass && max_seq_len > 0) || !new_lens || !kept || !mass_out ||
      mass_stride < max_seq_len || mass_out_stride < keep)
    return KVQ_ERR_INVALID_ARG;
  // the same table over the same planes: every block would be read and written
  if (src->block_table == dst->block_table &&
      (src->k_codes == dst->k_codes || src->v_codes == dst->v_codes ||
       src->k_scales == dst->k_scales || src->v_scales == dst->v_scales))
    return KVQ_ERR_INVALID_ARG;
  // outputs are no inputs, nor each other: some CTAs have written before others read
  const __int128 rows = (__int128)batch * src->num_kv_heads;
  const struct {
    const void *at;
    __int128 n;
  } out[3] = {{new_lens, batch}, {kept, rows * keep}, {mass_out, rows * mass_out_stride}};
  for (int i = 0; i < 3; i++) {
    if (overlap(out[i].at, out[i].n, d_seq_lens, batch)) return KVQ_ERR_INVALID_ARG;
    if (max_seq_len > 0 &&
        overlap(out[i].at, out[i].n, mass, (rows - 1) * mass_stride + max_seq_len))
      return KVQ_ERR_INVALID_ARG;
    for (int j = 0; j < i; j++)
      if (overlap(out[i].at, out[i].n, out[j].at, out[j].n)) return KVQ_ERR_INVALID_ARG;
  }
  if (2LL * batch * src->num_kv_heads >= (1LL << 31) / (keep / dst->block_size + 1))
    return KVQ_ERR_UNSUPPORTED;
  return from_cuda(launch_b8_evict(*src, *dst, batch, d_seq_lens, max_seq_len, mass, mass_stride,
                                   keep, recent, sinks, new_lens, kept, mass_out, mass_out_stride,
                                   as_stream(stream)));
}

}  // extern "C"
