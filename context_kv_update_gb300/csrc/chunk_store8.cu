// chunk_store8.cu -- a ragged chunk's rows into a cache held in 8 bits, and rows of that cache
// read back.
//
// Mathematics: k is normed and turned as in the 16-bit store (fp32), then a block's exponent
// comes from the largest magnitude of its rows by the bits of that number (no logarithm: the
// smallest e with a <= 448 * 2^e), so x * 2^-e is exact and each value is rounded once.
#include "cache8.cuh"
#include "chunk_turn.cuh"
#include "dflash_internal.cuh"

namespace dflash {
namespace {

struct Store8Params {
  Cache8 cache;
  int n_rows, rot, layout;
  float eps, mag;
  const uint16_t *k, *v;
  int64_t ks, vs;
  const uint16_t *gk;
  const int32_t *pos, *page, *slot;
  int32_t *st;
};

// Row t's block, counted over all pages of the pool, or -1 where it has none.
__device__ __forceinline__ int64_t block_of(const Store8Params &p, int t, bool report) {
  if (p.pos[t] < 0 || p.page[t] < 0) return -1;
  const int pg = p.page[t], sl = p.slot[t];
  if (pg >= p.cache.NP || sl < 0 || sl >= p.cache.P) {
    if (report) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
    return -1;
  }
  return static_cast<int64_t>(pg) * (p.cache.P / p.cache.block) + sl / p.cache.block;
}

// One CTA for a row that is the first of its block's, a head, K or V.
__global__ void __launch_bounds__(128)
    chunk_store8_kernel(const Store8Params p, const __grid_constant__ TurnFreqs tf) {
  __shared__ float s_max[4];
  const int t0 = blockIdx.x, h = blockIdx.y, kv = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hd = p.cache.hd, block = p.cache.block;
  const int64_t b = block_of(p, t0, threadIdx.x == 0 && h == 0 && kv == 0);
  if (b < 0 || (t0 > 0 && block_of(p, t0 - 1, false) == b)) return;
  int n = 1;
  uint64_t written = 1ull << (p.slot[t0] % block);
  while (t0 + n < p.n_rows && block_of(p, t0 + n, false) == b) {
    if (n == block) {  // more rows than slots
      if (threadIdx.x == 0) raise_status(p.st, DFLASH_DEV_BAD_ROWS);
      break;
    }
    written |= 1ull << (p.slot[t0 + n++] % block);
  }
  const int half = p.rot / 2;
  auto norm = [&](const uint16_t *x) {
    if (kv || !p.gk) return 1.f;
    float ss = 0.f;
    for (int d = lane; d < hd; d += 32) ss += bf16_to_f32(x[d]) * bf16_to_f32(x[d]);
    return rsqrtf(warp_sum(ss) / static_cast<float>(hd) + p.eps);
  };
  auto value = [&](const uint16_t *x, float inv, int pos, int d) {
    auto one = [&](int e) {
      const float f = bf16_to_f32(x[e]);
      return kv || !p.gk ? f : f * inv * bf16_to_f32(p.gk[e]);
    };
    if (kv || d >= p.rot) return one(d);
    const bool halves = p.layout == DFLASH_ROPE_HALF;
    const int j = halves ? (d < half ? d : d - half) : d / 2;
    const bool first = halves ? d < half : d % 2 == 0;
    const float2 cs = turn_cos_sin(pos, tf.f[j], p.mag);
    const float a = one(halves ? j : 2 * j), c = one(halves ? j + half : 2 * j + 1);
    return first ? a * cs.x - c * cs.y : c * cs.x + a * cs.y;
  };
  auto row = [&](int i) {
    return (kv ? p.v + (t0 + i) * p.vs : p.k + (t0 + i) * p.ks) + static_cast<int64_t>(h) * hd;
  };
  float most = 0.f;
  for (int i = warp; i < n; i += 4) {
    const float inv = norm(row(i));
    for (int d = lane; d < hd; d += 32) {
      const float f = fabsf(value(row(i), inv, p.pos[t0 + i], d));
      if (f < INFINITY) most = fmaxf(most, f);
    }
  }
  most = warp_max(most);
  if (lane == 0) s_max[warp] = most;
  __syncthreads();
  most = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  int e = scale8_exponent(most);
  const int page = p.page[t0], slot0 = p.slot[t0] / block * block;
  uint8_t *scale = p.cache.scale(page, kv, h, slot0);
  if (!(written & 1)) {  // the block goes on
    const int before = static_cast<int>(*scale) - 127;
    e = max(e, before);
    if (e != before) {
      const float shift = before - e < -149 ? 0.f : exp2_int(before - e);
      for (int s = warp; s < block; s += 4) {
        if ((written >> s) & 1) continue;
        uint8_t *c = p.cache.code(page, kv, h, slot0 + s);
        for (int d = lane; d < hd; d += 32)
          c[d] = static_cast<uint8_t>(e4m3_pair(e4m3_values(c[d]).x * shift, 0.f));
      }
    }
  }
  const float down = exp2_int(-e);
  for (int i = warp; i < n; i += 4) {
    const float inv = norm(row(i));
    uint8_t *c = p.cache.code(page, kv, h, p.slot[t0 + i]);
    for (int d = lane; d < hd; d += 32) {
      const float f = value(row(i), inv, p.pos[t0 + i], d);
      c[d] = fabsf(f) < INFINITY ? static_cast<uint8_t>(e4m3_pair(f * down, 0.f)) : 0x7f;
    }
  }
  __syncthreads();  // every thread has read the scale
  if (threadIdx.x == 0) *scale = static_cast<uint8_t>(e + 127);
}

struct Read8Params {
  Cache8 cache;
  int n_rows;
  const int32_t *page, *slot;
  uint16_t *out[2];
  int64_t stride[2];
  int32_t *st;
};

// One CTA for a row; a thread a value.
__global__ void __launch_bounds__(256) chunk_read8_kernel(const Read8Params p) {
  const int t = blockIdx.x, pg = p.page[t], sl = p.slot[t];
  if (pg < 0) return;
  if (pg >= p.cache.NP || sl < 0 || sl >= p.cache.P) {
    if (threadIdx.x == 0) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
    return;
  }
  for (int kv = 0; kv < 2; ++kv) {
    if (!p.out[kv]) continue;
    for (int i = threadIdx.x; i < p.cache.nkv * p.cache.hd; i += blockDim.x) {
      const int h = i / p.cache.hd;
      const float f = e4m3_values(p.cache.code(pg, kv, h, sl)[i - h * p.cache.hd]).x *
                      scale8_value(*p.cache.scale(pg, kv, h, sl));
      p.out[kv][t * p.stride[kv] + i] = f32_to_bf16_rn(f);
    }
  }
}

}  // namespace

cudaError_t launch_chunk_rope_store8(const dflash_geom &g, int layer, int n_rows,
                                     const dflash_rope_spec &rope, const void *q, int64_t q_stride,
                                     const void *k, int64_t k_stride, const void *v,
                                     int64_t v_stride, const void *gamma_q, const void *gamma_k,
                                     const int32_t *pos, const int32_t *page, const int32_t *slot,
                                     void *q_out, int64_t q_out_stride, const dflash_cache8 &cache,
                                     int32_t *st, cudaStream_t s) {
  if (q) {
    const cudaError_t e = launch_chunk_rope_store(
        g, layer, n_rows, rope, q, q_stride, nullptr, 0, nullptr, 0, gamma_q, nullptr, pos, nullptr,
        nullptr, q_out, q_out_stride, nullptr, st, s);
    if (e != cudaSuccess || !k) return e;
  }
  const TurnTable &table = turn_table(rope, g.rope_theta);
  Store8Params p = {};
  p.cache = cache8_of(g, cache, layer);
  p.n_rows = n_rows;
  p.rot = rope.rot_dim;
  p.layout = rope.layout;
  p.eps = static_cast<float>(g.eps_k);
  p.mag = table.mag;
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.ks = k_stride;
  p.vs = v_stride;
  p.gk = static_cast<const uint16_t *>(gamma_k);
  p.pos = pos;
  p.page = page;
  p.slot = slot;
  p.st = st;
  chunk_store8_kernel<<<dim3(n_rows, g.nkv, 2), 128, 0, s>>>(p, table.tf);
  return cudaGetLastError();
}

cudaError_t launch_chunk_read8(const dflash_geom &g, int layer, int n_rows,
                               const dflash_cache8 &cache, const int32_t *page,
                               const int32_t *slot, void *k_out, int64_t k_stride, void *v_out,
                               int64_t v_stride, int32_t *st, cudaStream_t s) {
  Read8Params p = {cache8_of(g, cache, layer), n_rows, page, slot,
                   {static_cast<uint16_t *>(k_out), static_cast<uint16_t *>(v_out)},
                   {k_stride, v_stride}, st};
  chunk_read8_kernel<<<n_rows, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace dflash
