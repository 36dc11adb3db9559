// chunk_attention.cu -- attention of a ragged chunk's rows over the paged cache: the 16-bit
// cache's forms of the kernel in chunk_attention.cuh.
#include "chunk_attention.cuh"

namespace dflash {

int chunk_attention_num_segments(const dflash_geom &g, int B, int n_rows, int window) {
  return segments_of(g, B, n_rows, window);
}
size_t chunk_attention_workspace_bytes(const dflash_geom &g, int B, int n_rows, int S) {
  return workspace_of(g, B, n_rows, S);
}

cudaError_t launch_chunk_attention(const dflash_geom &g, int B, int layer, int n_rows,
                                   const void *q, int64_t q_stride, const void *pool,
                                   const int32_t *tbl, const int32_t *cu, const int32_t *ctx,
                                   const int32_t *kv, int32_t window, const float *sinks,
                                   float scale, int mask_mode, int S, void *ws, void *out,
                                   int64_t out_stride, int32_t *st, cudaStream_t s) {
  return launch_attention<false>(g, B, layer, n_rows, q, q_stride, pool, nullptr, tbl, cu, ctx, kv,
                                 window, sinks, scale, mask_mode, S, ws, out, out_stride, st, s);
}

}  // namespace dflash
