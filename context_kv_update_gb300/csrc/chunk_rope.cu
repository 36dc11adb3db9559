// chunk_rope.cu -- per-head RMSNorm, rotary positions and the paged store of a
// ragged chunk's q, k and v rows.
//
// Mathematics: pair j of a head turns by the angle p * f_j.  The angle is kept
// in turns as 64-bit fixed point, (p * round(f_j / (2 pi) * 2^64)) mod 2^64:
// one integer product reduces it exactly, whatever the position, where a float
// product would lose the low bits; its top 32 bits go to sincospi.  Norm and
// rotation are fp32, rounded to bf16 once at the store (nearest even).
#include <cmath>
#include <cstring>

#include "dflash_internal.cuh"
#include "sm100_ptx.cuh"

namespace dflash {
namespace {

struct TurnFreqs {
  uint64_t f[kMaxHeadDim / 2];  // turns per position, 2^64 to a turn
};

struct RopeStoreParams {
  int n_rows, hq, nkv, hd, rot, layout, P, NP, layer;
  int rows, lph;  // rows of a CTA, lanes of a head
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

// Row t's page and slot, or page -1 where the row's keys are not stored.
__device__ __forceinline__ int2 row_place(const RopeStoreParams &p, int t, bool report) {
  const int pg = p.page[t], sl = p.slot[t];
  if (pg < 0) return make_int2(-1, 0);
  if (pg >= p.NP || sl < 0 || sl >= p.P) {
    if (report) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
    return make_int2(-1, 0);
  }
  return make_int2(pg, sl);
}

// VW values (8 or 4) as one 16- or 8-byte access.
template <int VW>
struct Chunk;
template <>
struct Chunk<8> {
  uint4 w;
};
template <>
struct Chunk<4> {
  uint2 w;
};
template <int VW>
__device__ __forceinline__ void unpack(const Chunk<VW> &c, float *x) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&c);
#pragma unroll
  for (int e = 0; e < VW / 2; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
template <int VW>
__device__ __forceinline__ Chunk<VW> pack(const float *x) {
  Chunk<VW> c;
  uint32_t *w = reinterpret_cast<uint32_t *>(&c);
#pragma unroll
  for (int e = 0; e < VW / 2; ++e) w[e] = ptx::pack_bf16x2(x[2 * e], x[2 * e + 1]);
  return c;
}

constexpr int kRopeThreads = 256;
constexpr int kMaxRopeRows = 4;  // rows of a CTA

// A unit is two chunks of VW values of one head, held by one thread: in the
// half layout the two chunks that turn together (d, d + rot/2), in the pairs
// layout two neighbouring ones; dims past rot_dim go in neighbouring chunks.
// The `lph` lanes (a power of two) that hold a head add up its norm by
// shuffles.  cos and sin of the CTA's rows are formed once, in shared memory,
// while each thread's first unit is on its way; every byte of q, k and v is
// then read and written once.
template <int VW, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads)
    chunk_rope_kernel(const RopeStoreParams p, const __grid_constant__ TurnFreqs tf) {
  __shared__ float2 s_cs[kMaxRopeRows][kMaxHeadDim / 2];
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int row0 = blockIdx.x * p.rows, rows = min(p.rows, p.n_rows - row0);
  const int half = p.rot >> 1;
  const int u = threadIdx.x & (p.lph - 1), step = kRopeThreads / p.lph;
  const int nq = p.q ? p.hq : 0, heads = nq + (p.k ? p.nkv : 0);  // q heads, then k heads
  const bool halves = p.layout == DFLASH_ROPE_HALF;

  // the unit's chunks: where, and whether they turn
  int d0, d1;
  bool turn0, turn1;
  if (halves) {
    const int nrot = half / VW;
    turn0 = turn1 = u < nrot;
    d0 = turn0 ? VW * u : p.rot + 2 * VW * (u - nrot);
    d1 = turn0 ? d0 + half : d0 + VW;
  } else {
    d0 = 2 * VW * u;
    d1 = d0 + VW;
    turn0 = d0 < p.rot;
    turn1 = d1 < p.rot;
  }
  const bool has0 = d0 < p.hd, has1 = d1 < p.hd;

  struct Item {
    int t, h;  // chunk row, head (q heads, then k heads)
  };
  auto item = [&](int i) {
    const int rr = i / heads;
    return Item{row0 + rr, i - rr * heads};
  };
  auto source = [&](const Item &it) {
    return it.h < nq ? p.q + it.t * p.qs + static_cast<int64_t>(it.h) * p.hd
                     : p.k + it.t * p.ks + static_cast<int64_t>(it.h - nq) * p.hd;
  };
  auto fetch = [&](int i, Chunk<VW> *a, Chunk<VW> *b) {
    *a = Chunk<VW>{};
    *b = Chunk<VW>{};
    if (i >= rows * heads) return;
    const uint16_t *src = source(item(i));
    if (has0) *a = *reinterpret_cast<const Chunk<VW> *>(src + d0);
    if (has1) *b = *reinterpret_cast<const Chunk<VW> *>(src + d1);
  };
  const int first = threadIdx.x / p.lph;
  Chunk<VW> a, b;
  fetch(first, &a, &b);

  for (int i = threadIdx.x; i < rows * half; i += kRopeThreads) {
    const int rr = i / half, j = i - rr * half;
    s_cs[rr][j] = turn_cos_sin(p.pos[row0 + rr], tf.f[j], p.mag);
  }
  __syncthreads();

  // whole warps take every step of the loop: the norm's shuffles need them
  const int items = rows * heads, passes = (items + step - 1) / step;
  for (int n = 0; n < passes; ++n) {
    const int i = first + n * step;
    Chunk<VW> na, nb;
    fetch(i + step, &na, &nb);
    const bool in = i < items;
    const Item it = item(in ? i : 0);
    float x[2 * VW];
    unpack<VW>(a, x);
    unpack<VW>(b, x + VW);
    if constexpr (kNorm) {
      const uint16_t *gamma = it.h < nq ? p.gq : p.gk;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * VW; ++e) ss += x[e] * x[e];
      for (int o = p.lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (gamma) {
        const float inv = rsqrtf(ss / static_cast<float>(p.hd) + p.eps);
        Chunk<VW> g0 = {}, g1 = {};
        if (has0) g0 = *reinterpret_cast<const Chunk<VW> *>(gamma + d0);
        if (has1) g1 = *reinterpret_cast<const Chunk<VW> *>(gamma + d1);
        float gv[2 * VW];
        unpack<VW>(g0, gv);
        unpack<VW>(g1, gv + VW);
#pragma unroll
        for (int e = 0; e < 2 * VW; ++e) x[e] = x[e] * inv * gv[e];
      }
    }
    if (in && has0) {
      const int pos = p.pos[it.t];
      uint16_t *dst = nullptr;
      if (pos >= 0) {
        if (it.h < nq) {
          dst = p.q_out + it.t * p.qos + static_cast<int64_t>(it.h) * p.hd;
        } else {
          const int2 at = row_place(p, it.t, u == 0 && it.h == nq);
          if (at.x >= 0) dst = pool_row(p, at.x, at.y, 0, it.h - nq);
        }
      }
      if (dst) {
        if (turn0) {
          const float2 *cs = s_cs[it.t - row0] + VW * u;
          if (halves) {
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              const float2 w = cs[e];
              const float s = x[e], t = x[VW + e];
              x[e] = s * w.x - t * w.y;
              x[VW + e] = t * w.x + s * w.y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < VW; ++e) {  // pair e: chunk e / (VW / 2)
              if (e >= VW / 2 && !turn1) break;
              const float2 w = cs[e];
              const float s = x[2 * e], t = x[2 * e + 1];
              x[2 * e] = s * w.x - t * w.y;
              x[2 * e + 1] = t * w.x + s * w.y;
            }
          }
        }
        *reinterpret_cast<Chunk<VW> *>(dst + d0) = pack<VW>(x);
        if (has1) *reinterpret_cast<Chunk<VW> *>(dst + d1) = pack<VW>(x + VW);
      }
    }
    a = na;
    b = nb;
  }

  // v rows: copied 16 bytes a thread
  if (p.k) {
    const int vecs = p.hd / 8, per = p.nkv * vecs;
    for (int i = threadIdx.x; i < rows * per; i += kRopeThreads) {
      const int rr = i / per, e = i - rr * per, h = e / vecs, t = row0 + rr;
      if (p.pos[t] < 0) continue;
      const int2 at = row_place(p, t, false);
      if (at.x < 0) continue;
      reinterpret_cast<uint4 *>(pool_row(p, at.x, at.y, 1, h))[e - h * vecs] =
          reinterpret_cast<const uint4 *>(p.v + t * p.vs)[e];
    }
  }
}

// Widths that no 8-byte chunk fits (an odd number of pairs, or of two): one
// warp per (row, head of q, k or v), a pair or a value per lane.
__global__ void __launch_bounds__(256)
    chunk_rope_pairs_kernel(const RopeStoreParams p, const __grid_constant__ TurnFreqs tf) {
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int pos = p.pos[t];
  if (pos < 0) return;
  const int2 at = p.k ? row_place(p, t, threadIdx.x == 0) : make_int2(-1, 0);
  const int heads = p.hq + 2 * p.nkv, half = p.rot / 2;
  for (int h = threadIdx.x >> 5; h < heads; h += blockDim.x >> 5) {
    const int kind = h < p.hq ? 0 : (h < p.hq + p.nkv ? 1 : 2);  // q, k, v
    if (kind == 0 ? p.q == nullptr : at.x < 0) continue;
    const int hh = kind == 0 ? h : (kind == 1 ? h - p.hq : h - p.hq - p.nkv);
    const uint16_t *src = kind == 0 ? p.q + t * p.qs : (kind == 1 ? p.k + t * p.ks : p.v + t * p.vs);
    src += static_cast<int64_t>(hh) * p.hd;
    uint16_t *dst = kind == 0 ? p.q_out + t * p.qos + static_cast<int64_t>(hh) * p.hd
                              : pool_row(p, at.x, at.y, kind - 1, hh);
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
// (The powers of a 128-wide head take the host ~5 us: the launcher keeps the
// thread's last table with the specification it was made from.)
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
  struct Table {
    dflash_rope_spec spec;
    double theta;
    float mag;
    TurnFreqs tf;
  };
  static thread_local Table last = {};  // rot_dim 0: made from nothing yet
  if (std::memcmp(&last.spec, &rope, sizeof(rope)) != 0 || last.theta != g.rope_theta) {
    last.spec = rope;
    last.theta = g.rope_theta;
    fill_turn_freqs(&last.tf, &last.mag, rope, p.rot, g.rope_theta);
  }
  const TurnFreqs &tf = last.tf;
  p.mag = last.mag;
  // the widest chunk (16 or 8 bytes) that no turning pair of chunks is cut by
  const bool halves = p.layout == DFLASH_ROPE_HALF;
  const int unit = halves ? p.rot / 2 : p.rot;  // a whole number of chunks
  const int vw = unit % 8 == 0 ? 8 : (unit % 4 == 0 ? 4 : 0);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(n_rows);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (vw == 0) return cudaLaunchKernelEx(&cfg, chunk_rope_pairs_kernel, p, tf);
  const int units = halves ? p.rot / (2 * vw) + (p.hd - p.rot + 2 * vw - 1) / (2 * vw)
                           : (p.hd + 2 * vw - 1) / (2 * vw);
  p.lph = 1;
  while (p.lph < units) p.lph *= 2;
  p.rows = 1;
  while (p.rows < kMaxRopeRows && n_rows > 8 * device_sm_count() * p.rows) p.rows *= 2;
  cfg.gridDim = dim3((n_rows + p.rows - 1) / p.rows);
  const bool norm = gamma_q || gamma_k;
  if (vw == 8)
    return norm ? cudaLaunchKernelEx(&cfg, chunk_rope_kernel<8, true>, p, tf)
                : cudaLaunchKernelEx(&cfg, chunk_rope_kernel<8, false>, p, tf);
  return norm ? cudaLaunchKernelEx(&cfg, chunk_rope_kernel<4, true>, p, tf)
              : cudaLaunchKernelEx(&cfg, chunk_rope_kernel<4, false>, p, tf);
}

}  // namespace dflash
