// chunk_attention8.cu -- attention of a ragged chunk's rows over a cache held in 8 bits.
//
// One pass over a row's keys with a running maximum and sum (fp32).
#include "cache8.cuh"
#include "dflash_internal.cuh"
#include "sm100_ptx.cuh"

namespace dflash {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct Attn8Params {
  Cache8 cache;
  int B, n_rows, hq, nkv, M, window, mask_mode;
  float scale_log2;
  const uint16_t *q;
  int64_t qs, os;
  const int32_t *tbl, *cu, *ctx, *kv;
  const float *sinks;
  uint16_t *out;
  int32_t *st;
};

// One warp for a row and a head, HD / 32 dims a lane.
template <int HD>
__global__ void __launch_bounds__(128) chunk_attn8_kernel(const Attn8Params p) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / p.hq), h = static_cast<int>(w % p.hq);
  if (t >= p.n_rows) return;
  int r = 0, n = p.B;  // the last request whose first row is <= t
  while (n > 1) {
    const int half = n / 2;
    if (p.cu[r + half] <= t) {
      r += half;
      n -= half;
    } else {
      n = half;
    }
  }
  const bool report = lane == 0 && h == 0;
  const int a = p.cu[r], b = p.cu[r + 1], c = p.ctx[r];
  if (a < 0 || b < a || b > p.n_rows || c < 0 || c > INT32_MAX - p.n_rows) {
    if (report) raise_status(p.st, DFLASH_DEV_BAD_ROWS);
    return;
  }
  if (t < a || t >= b) return;
  int kv = p.kv[r];
  const int cap = p.M * p.cache.P;
  if (kv < 0 || kv > cap) {
    if (report) raise_status(p.st, DFLASH_DEV_KV_LEN_RANGE);
    kv = kv < 0 ? 0 : cap;
  }
  const int pos = c + t - a, kvh = h / (p.hq / p.nkv);
  const int hi = p.mask_mode == DFLASH_MASK_CAUSAL_TAIL ? min(pos, kv - 1) : kv - 1;
  float q[E], acc[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e)
    q[e] = bf16_to_f32(p.q[t * p.qs + h * HD + lane * E + e]) * p.scale_log2;
  for (int j = p.window > 0 ? max(0, pos - p.window + 1) : 0; j <= hi; ++j) {
    const int pg = p.tbl[static_cast<int64_t>(r) * p.M + j / p.cache.P], sl = j % p.cache.P;
    if (pg < 0 || pg >= p.cache.NP) {
      if (report) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
      continue;
    }
    const uint8_t *k = p.cache.code(pg, 0, kvh, sl) + lane * E;
    const uint8_t *v = p.cache.code(pg, 1, kvh, sl) + lane * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * e4m3_values(k[e]).x;
    s = warp_sum(s) * scale8_value(*p.cache.scale(pg, 0, kvh, sl));
    const float mn = fmaxf(m, s), old = m == -INFINITY ? 0.f : ptx::ex2(m - mn),
                x = ptx::ex2(s - mn), vs = scale8_value(*p.cache.scale(pg, 1, kvh, sl));
    l = l * old + x;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * old + x * (e4m3_values(v[e]).x * vs);
    m = mn;
  }
  float gain = 0.f;
  if (m != -INFINITY) {
    const float sk = p.sinks ? p.sinks[h] * kLog2e : -INFINITY, top = fmaxf(m, sk);
    gain = ptx::ex2(m - top) / (l * ptx::ex2(m - top) + ptx::ex2(sk - top));
  }
  for (int e = 0; e < E; ++e)
    p.out[t * p.os + h * HD + lane * E + e] = f32_to_bf16_rn(gain != 0.f ? acc[e] * gain : 0.f);
}

}  // namespace

int chunk_attention8_num_segments(const dflash_geom &, int, int, int) { return 1; }
size_t chunk_attention8_workspace_bytes(const dflash_geom &, int, int, int) { return 0; }

cudaError_t launch_chunk_attention8(const dflash_geom &g, int B, int layer, int n_rows,
                                    const void *q, int64_t q_stride, const dflash_cache8 &cache,
                                    const int32_t *tbl, const int32_t *cu, const int32_t *ctx,
                                    const int32_t *kv, int32_t window, const float *sinks,
                                    float scale, int mask_mode, int, void *, void *out,
                                    int64_t out_stride, int32_t *st, cudaStream_t s) {
  Attn8Params p = {};
  p.cache = cache8_of(g, cache, layer);
  p.B = B;
  p.n_rows = n_rows;
  p.hq = g.hq;
  p.nkv = g.nkv;
  p.M = g.max_pages;
  p.window = window;
  p.mask_mode = mask_mode;
  p.scale_log2 = scale * kLog2e;
  p.q = static_cast<const uint16_t *>(q);
  p.qs = q_stride;
  p.os = out_stride;
  p.tbl = tbl;
  p.cu = cu;
  p.ctx = ctx;
  p.kv = kv;
  p.sinks = sinks;
  p.out = static_cast<uint16_t *>(out);
  p.st = st;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(n_rows) * g.hq + 3) / 4);
  if (g.head_dim == 64)
    chunk_attn8_kernel<64><<<grid, 128, 0, s>>>(p);
  else
    chunk_attn8_kernel<128><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace dflash
