// chunk_rope.cu -- per-head RMSNorm, rotary positions and the paged store of a
// ragged chunk's q, k and v rows.
//
// Mathematics: pair j of a head turns by the angle p * f_j.  The angle is kept
// in turns as 64-bit fixed point, (p * round(f_j / (2 pi) * 2^64)) mod 2^64:
// one integer product reduces it exactly, whatever the position, where a float
// product would lose the low bits; its top 32 bits go to sincospi.  Norm and
// rotation are fp32, rounded to bf16 once at the store (nearest even).
#include <cmath>

#include "dflash_internal.cuh"
#include "sm100_ptx.cuh"

namespace dflash {
namespace {

struct TurnFreqs {
  uint64_t f[kMaxHeadDim / 2];  // turns per position, 2^64 to a turn
};

struct RopeStoreParams {
  int n_rows, hq, nkv, hd, rot, layout, P, NP, layer;
  float eps, mag;
  const uint16_t *q, *k, *v;
  int64_t qs, ks, vs, qos;
  const uint16_t *gq, *gk;
  const int32_t *pos, *page, *slot;
  uint16_t *q_out, *pool;
  int32_t *st;
};

// cos and sin (times the magnitude) of position p at f turns per position.
__device__ __forceinline__ float2 turn_cos_sin(int p, uint64_t f, float mag) {
  const uint64_t t = static_cast<uint64_t>(static_cast<uint32_t>(p)) * f;
  float s, c;  // top 32 bits: a signed fraction of half a turn in units of 2^-31
  sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * mag, s * mag);
}

// Where the K (kv = 0) or V row of head h goes, or nullptr.
__device__ __forceinline__ uint16_t *pool_row(const RopeStoreParams &p, int pg, int sl, int kv,
                                              int h) {
  return p.pool +
         ((((static_cast<size_t>(p.layer) * p.NP + pg) * 2 + kv) * p.nkv + h) * p.P + sl) * p.hd;
}

// One warp per (row, head of q, k or v), a pair or a value per lane.
__global__ void __launch_bounds__(256)
    chunk_rope_kernel(const RopeStoreParams p, const TurnFreqs tf) {
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int pos = p.pos[t];
  if (pos < 0) return;
  int pg = -1, sl = 0;
  if (p.k) {  // queries alone: page and slot may be null
    pg = p.page[t];
    sl = p.slot[t];
  }
  bool stored = pg >= 0;
  if (stored && (pg >= p.NP || sl < 0 || sl >= p.P)) {
    if (threadIdx.x == 0) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
    stored = false;
  }
  const int heads = p.hq + 2 * p.nkv, half = p.rot / 2;
  for (int h = threadIdx.x >> 5; h < heads; h += blockDim.x >> 5) {
    const int kind = h < p.hq ? 0 : (h < p.hq + p.nkv ? 1 : 2);  // q, k, v
    if (kind == 0 ? p.q == nullptr : !stored) continue;
    const int hh = kind == 0 ? h : (kind == 1 ? h - p.hq : h - p.hq - p.nkv);
    const uint16_t *src = kind == 0 ? p.q + t * p.qs : (kind == 1 ? p.k + t * p.ks : p.v + t * p.vs);
    src += static_cast<int64_t>(hh) * p.hd;
    uint16_t *dst = kind == 0 ? p.q_out + t * p.qos + static_cast<int64_t>(hh) * p.hd
                              : pool_row(p, pg, sl, kind - 1, hh);
    if (kind == 2) {
      for (int d = lane; d < p.hd; d += 32) dst[d] = src[d];
      continue;
    }
    const uint16_t *gamma = kind == 0 ? p.gq : p.gk;
    float inv = 1.f;
    if (gamma) {
      float ss = 0.f;
      for (int d = lane; d < p.hd; d += 32) {
        const float x = bf16_to_f32(src[d]);
        ss += x * x;
      }
      inv = rsqrtf(warp_sum(ss) / static_cast<float>(p.hd) + p.eps);
    }
    auto value = [&](int d) {
      const float x = bf16_to_f32(src[d]);
      return gamma ? x * inv * bf16_to_f32(gamma[d]) : x;
    };
    for (int j = lane; j < half; j += 32) {
      const int da = p.layout == DFLASH_ROPE_HALF ? j : 2 * j;
      const int db = p.layout == DFLASH_ROPE_HALF ? j + half : 2 * j + 1;
      const float2 cs = turn_cos_sin(pos, tf.f[j], p.mag);
      const float a = value(da), b = value(db);
      dst[da] = f32_to_bf16_rn(a * cs.x - b * cs.y);
      dst[db] = f32_to_bf16_rn(b * cs.x + a * cs.y);
    }
    for (int d = p.rot + lane; d < p.hd; d += 32) dst[d] = f32_to_bf16_rn(value(d));
  }
}

// Turns per position of every pair, and the factor on cos and sin.
void fill_turn_freqs(TurnFreqs *tf, float *mag, const dflash_rope_spec &r, int rot, double theta) {
  const double two_pi = 6.283185307179586476925286766559;
  double j0 = 0.0, j1 = 0.0;
  *mag = 1.f;
  if (r.scaling == DFLASH_ROPE_YARN) {
    const double per = rot / (2.0 * std::log(theta));
    j0 = std::fmax(std::floor(per * std::log(r.trained_ctx / (two_pi * r.beta_fast))), 0.0);
    j1 = std::fmin(std::ceil(per * std::log(r.trained_ctx / (two_pi * r.beta_slow))), rot - 1.0);
    *mag = static_cast<float>(r.magnitude > 0.0 ? r.magnitude : 0.1 * std::log(r.factor) + 1.0);
  }
  for (int j = 0; j < rot / 2; ++j) {
    double f = std::pow(theta, -2.0 * j / rot);
    if (r.scaling == DFLASH_ROPE_LINEAR) f /= r.factor;
    if (r.scaling == DFLASH_ROPE_YARN) {
      const double u = std::fmin(std::fmax((j - j0) / std::fmax(j1 - j0, 1e-3), 0.0), 1.0);
      f = f / r.factor * u + f * (1.0 - u);
    }
    const double turns = f / two_pi;
    // the fraction of a turn; 2^64 times it is an integer below 2^64 (a
    // double's 53 bits)
    tf->f[j] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
  }
}

}  // namespace

cudaError_t launch_chunk_rope_store(const dflash_geom &g, int layer, int n_rows,
                                    const dflash_rope_spec &rope, const void *q, int64_t q_stride,
                                    const void *k, int64_t k_stride, const void *v,
                                    int64_t v_stride, const void *gamma_q, const void *gamma_k,
                                    const int32_t *pos, const int32_t *page, const int32_t *slot,
                                    void *q_out, int64_t q_out_stride, void *pool, int32_t *st,
                                    cudaStream_t s) {
  RopeStoreParams p;
  p.n_rows = n_rows;
  p.hq = g.hq;
  p.nkv = g.nkv;
  p.hd = g.head_dim;
  p.rot = rope.rot_dim;
  p.layout = rope.layout;
  p.P = g.page_size;
  p.NP = g.num_pool_pages;
  p.layer = layer;
  p.eps = static_cast<float>(g.eps_k);
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.qs = q_stride;
  p.ks = k_stride;
  p.vs = v_stride;
  p.qos = q_out_stride;
  p.gq = static_cast<const uint16_t *>(gamma_q);
  p.gk = static_cast<const uint16_t *>(gamma_k);
  p.pos = pos;
  p.page = page;
  p.slot = slot;
  p.q_out = static_cast<uint16_t *>(q_out);
  p.pool = static_cast<uint16_t *>(pool);
  p.st = st;
  TurnFreqs tf = {};
  fill_turn_freqs(&tf, &p.mag, rope, p.rot, g.rope_theta);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(n_rows);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_rope_kernel, p, tf);
}

}  // namespace dflash
