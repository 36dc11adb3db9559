// chunk_attention.cu -- attention of a ragged chunk's rows over the paged
// cache: any number of rows per request, causal or bidirectional, sliding
// window, sinks.
//
// Mathematics: softmax with one pass over the keys, a running maximum and sum
// (fp32); the sink starts the sum as a logit without a value.
#include <math.h>

#include "dflash_internal.cuh"
#include "sm100_ptx.cuh"

namespace dflash {
namespace {

struct ChunkAttnParams {
  int B, n_rows, hq, nkv, G, hd, layer, NP, P, M, window, mask_mode;
  float scale;
  const uint16_t *q, *pool;
  int64_t qs, os;
  const int32_t *tbl, *cu, *ctx, *kv;
  const float *sinks;
  uint16_t *out;
  int32_t *st;
};

// One warp per (row, head); a lane holds hd / 32 dims.
template <int HD>
__global__ void __launch_bounds__(128) chunk_attn_rows_kernel(const ChunkAttnParams p) {
  constexpr int E = HD / 32;
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / p.hq), h = static_cast<int>(w % p.hq);
  if (t >= p.n_rows) return;
  int lo = 0, hi = p.B - 1;  // the last request whose first row is <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int r = lo, a = p.cu[r], b = p.cu[r + 1];
  if (t < a || t >= b) return;
  const int c = p.ctx[r];
  if (a < 0 || b > p.n_rows || c < 0) {
    if (lane == 0) raise_status(p.st, DFLASH_DEV_BAD_ROWS);
    return;
  }
  int kv = p.kv[r];
  const int cap = p.M * p.P;
  if (kv < 0 || kv > cap) {
    if (lane == 0) raise_status(p.st, DFLASH_DEV_KV_LEN_RANGE);
    kv = kv < 0 ? 0 : cap;
  }
  const int pos = c + (t - a);
  const int last = p.mask_mode == DFLASH_MASK_CAUSAL_TAIL ? min(pos, kv - 1) : kv - 1;
  const int first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float qv[E], acc[E];
  const uint16_t *q = p.q + t * p.qs + static_cast<int64_t>(h) * HD + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = bf16_to_f32(q[e]) * p.scale;
    acc[e] = 0.f;
  }
  float m = p.sinks ? p.sinks[h] : -INFINITY, l = p.sinks ? 1.f : 0.f;
  for (int j = first; j <= last; ++j) {
    const int page = p.tbl[static_cast<int64_t>(r) * p.M + j / p.P];
    if (page < 0 || page >= p.NP) {
      if (lane == 0) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
      continue;
    }
    const size_t row = ((static_cast<size_t>(p.layer) * p.NP + page) * 2 * p.nkv + h / p.G) * p.P +
                       j % p.P;
    const uint16_t *k = p.pool + row * HD + lane * E;
    const uint16_t *v = k + static_cast<size_t>(p.nkv) * p.P * HD;
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) d += qv[e] * bf16_to_f32(k[e]);
    d = warp_sum(d);
    const float mn = fmaxf(m, d);
    const float sc = m == -INFINITY ? 0.f : __expf(m - mn), w1 = __expf(d - mn);
    l = l * sc + w1;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * sc + w1 * bf16_to_f32(v[e]);
    m = mn;
  }
  uint16_t *o = p.out + t * p.os + static_cast<int64_t>(h) * HD + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = f32_to_bf16_rn(l > 0.f ? acc[e] / l : 0.f);
}

}  // namespace

int chunk_attention_num_segments(const dflash_geom &g, int B, int n_rows) {
  (void)g;
  (void)B;
  (void)n_rows;
  return 1;
}

size_t chunk_attention_workspace_bytes(const dflash_geom &g, int B, int n_rows, int S) {
  (void)g;
  (void)B;
  (void)n_rows;
  (void)S;
  return 0;
}

cudaError_t launch_chunk_attention(const dflash_geom &g, int B, int layer, int n_rows,
                                   const void *q, int64_t q_stride, const void *pool,
                                   const int32_t *tbl, const int32_t *cu, const int32_t *ctx,
                                   const int32_t *kv, int32_t window, const float *sinks,
                                   float scale, int mask_mode, int S, void *ws, void *out,
                                   int64_t out_stride, int32_t *st, cudaStream_t s) {
  (void)S;
  (void)ws;
  ChunkAttnParams p;
  p.B = B;
  p.n_rows = n_rows;
  p.hq = g.hq;
  p.nkv = g.nkv;
  p.G = g.hq / g.nkv;
  p.hd = g.head_dim;
  p.layer = layer;
  p.NP = g.num_pool_pages;
  p.P = g.page_size;
  p.M = g.max_pages;
  p.window = window;
  p.mask_mode = mask_mode;
  p.scale = scale;
  p.q = static_cast<const uint16_t *>(q);
  p.pool = static_cast<const uint16_t *>(pool);
  p.qs = q_stride;
  p.os = out_stride;
  p.tbl = tbl;
  p.cu = cu;
  p.ctx = ctx;
  p.kv = kv;
  p.sinks = sinks;
  p.out = static_cast<uint16_t *>(out);
  p.st = st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(n_rows) * g.hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return g.head_dim == 64 ? cudaLaunchKernelEx(&cfg, chunk_attn_rows_kernel<64>, p)
                          : cudaLaunchKernelEx(&cfg, chunk_attn_rows_kernel<128>, p);
}

}  // namespace dflash
