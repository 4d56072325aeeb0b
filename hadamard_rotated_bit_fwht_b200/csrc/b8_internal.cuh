// b8_internal.cuh -- launchers of the rotary positions and of the block-scaled
// 8-bit cache.  Nothing here is part of the C ABI.
#pragma once

#include "kvq_internal.cuh"

#include <atomic>

namespace kvq {

// Let kernel f use up to `bytes` of dynamic shared memory: asked of the driver
// once per kernel and device (each instance of the template has its own set).
template <auto f>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch that may begin while the kernel before it on the stream ends; cluster:
// CTAs of a cluster (1: none).  Every thread of f starts with
// dec::grid_dependency_wait(): it waits until that kernel is done and its writes
// are visible, so stream order is kept and only the launch itself overlaps.  What
// such kernels read they read past L1 (__ldcg, cp.async.cg) or with plain loads, not
// through the read-only path, whose data must not change while a grid exists.  Block
// scales come through L1 (cp.async.ca, as 4 bytes must): a kernel that writes them
// has to end before its dependents may begin, as those here do.
template <class... P, class... A>
cudaError_t launch_early(void (*f)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                         int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, f, P(args)...);
}

// q, k: heads to rotate (k.num_heads 0: none); spec.d_inv_freq set
cudaError_t launch_rope(const kvq_rope_spec &spec, int bf16, int head_dim, int num_tokens,
                        const int32_t *positions, int inverse, const kvq_heads &q,
                        const kvq_heads &q_out, const kvq_heads &k, const kvq_heads &k_out,
                        cudaStream_t s);
// spec.d_inv_freq nullptr: K is stored as it comes
cudaError_t launch_b8_append(const kvq_b8_cache &c, const kvq_heads &k, const kvq_heads &v,
                             int bf16, int batch, int t_new, const int32_t *start_pos,
                             const int32_t *new_lens, const kvq_rope_spec &spec,
                             const int32_t *rope_pos, cudaStream_t s);
cudaError_t launch_b8_gather(const kvq_b8_cache &c, int batch, const int32_t *first,
                             const int32_t *ends, int count, int bf16, void *k_out, void *v_out,
                             cudaStream_t s);

// The queries of an attention or mass call: sequence b's are rows cu_q[b] ..
// cu_q[b + 1] - 1 (cu_q nullptr: row b).
struct B8Queries {
  const void *q;
  int64_t token_stride, head_stride;  // elements
  int bf16, num_heads, group;         // group = num_heads / kv heads
  int batch, total_q, max_q;
  const int32_t *cu_q, *seq_lens;
  int max_seq_len;  // lengths are clamped to [0, max_seq_len]
  float scale;
};
// How a call is cut: `row_tiles` tiles of `rows` (head, query) rows for each
// (sequence, kv head), each over `splits` ranges of `split_tokens` tokens.
struct B8Plan {
  int rows, row_tiles, splits, split_tokens;
  int prefill;  // 1: the many-row kernel
  int cluster;  // 1: the splits of a unit are one cluster
};
B8Plan plan_b8_attn(const kvq_b8_cache &c, int bf16, int group, int batch, int max_q,
                    int max_seq_len);
size_t b8_attn_workspace_bytes(const kvq_b8_cache &c, int batch, const B8Plan &p);
// out: q's dtype [total_q][num_heads][D]; lse: [total_q][num_heads] or nullptr
cudaError_t launch_b8_attn(const kvq_b8_cache &c, const B8Queries &q, const B8Plan &p, void *out,
                           float *lse, float *ws, cudaStream_t s);
// mass: [batch][kv heads][mass_stride]
cudaError_t launch_b8_mass(const kvq_b8_cache &c, const B8Queries &q, const float *lse,
                           float *mass, int64_t mass_stride, cudaStream_t s);

// kept: [batch][kv heads][keep], mass_out: [batch][kv heads][mass_out_stride]
cudaError_t launch_b8_evict(const kvq_b8_cache &src, const kvq_b8_cache &dst, int batch,
                            const int32_t *seq_lens, int max_seq_len, const float *mass,
                            int64_t mass_stride, int keep, int recent, int sinks,
                            int32_t *new_lens, int32_t *kept, float *mass_out,
                            int64_t mass_out_stride, cudaStream_t s);

}  // namespace kvq
