// chunk_rope.cu -- per-head RMSNorm, rotary positions and the paged store of a
// ragged chunk's q, k and v rows.
//
// Mathematics: pair j of a head turns by the angle p * f_j.  The angle is kept
// in turns as 64-bit fixed point, (p * round(f_j / (2 pi) * 2^64)) mod 2^64:
// one integer product reduces it exactly, whatever the position, where a float
// product would lose the low bits; its top 32 bits go to sincospi.  Norm and
// rotation are fp32, rounded to bf16 once at the store (nearest even).
//
// Bound by HBM: 8192 rows of 32 + 8 + 8 heads of 128 (201 MB) take 40 us, 5.0 TB/s,
// where a plain copy of as many bytes takes 33; 40000 rows of 24 + 4 + 4 heads of 64
// take 53, 6.2 TB/s (65 with groups of at most four rows); a few rows are bound
// by latency (16 rows: 4 us on the device).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "dflash_internal.cuh"
#include "f32x2.cuh"
#include "sm100_ptx.cuh"

namespace dflash {
namespace {

struct TurnFreqs {
  uint64_t f[kMaxHeadDim / 2];  // turns per position, 2^64 to a turn
};

struct RopeStoreParams {
  int n_rows, hq, nkv, hd, rot, layout, P, NP, layer;
  int rows, lph;   // rows of a CTA, lanes of a head
  int skip_group;  // tests only: of each CTA's groups the one that is not loaded (-1: off)
  float eps, inv_hd, mag;
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
// As pairs of fp32: chunk pairs (2 e, 2 e + 1).
template <int VW>
__device__ __forceinline__ void unpack(const Chunk<VW> &c, float2 *x) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&c);
#pragma unroll
  for (int e = 0; e < VW / 2; ++e)
    x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
}
template <int VW>
__device__ __forceinline__ Chunk<VW> pack(const float2 *x) {
  Chunk<VW> c;
  uint32_t *w = reinterpret_cast<uint32_t *>(&c);
#pragma unroll
  for (int e = 0; e < VW / 2; ++e) w[e] = ptx::pack_bf16x2(x[e].x, x[e].y);
  return c;
}

constexpr int kRopeWarps = 8;    // of a CTA
constexpr int kMaxRopeRows = 8;  // rows of a group, at most: a warp each
constexpr int kRopeSmem = 208 * 1024;

// Bulk copy of `bytes` (a multiple of 16) from global to shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// Rows are brought into shared memory whole, by bulk copies that hold no
// registers, a group of p.rows rows while the group before it is worked on: loads
// that wait in registers kept too few bytes in flight (46.6 us at 8192 rows of 48
// heads), and a CTA for each group spends most of its life waiting (43.7 us; this form
// 40.2).
//
// A unit is two chunks of VW values of one head, held by one lane: in the half
// layout the two chunks that turn together (d, d + rot/2), in the pairs layout
// two neighbouring ones; dims past rot_dim go in neighbouring chunks.  The `lph`
// lanes (a power of two) that hold a head add up its norm by shuffles.  A warp
// walks over heads of one row, so the row's cos and sin, times the norm's gain,
// stay in a lane's registers: out = inv a A + inv b B (two fp32 lanes an
// instruction).
template <int VW, bool kNorm, bool kHalf>
__global__ void __launch_bounds__(32 * kRopeWarps, 2)
    chunk_rope_kernel(const RopeStoreParams p, const __grid_constant__ TurnFreqs tf) {
  extern __shared__ __align__(128) uint8_t rope_smem[];  // [2 stages][rows]: q, k, v heads
  __shared__ __align__(16) float s_turn[kMaxRopeRows][2][kMaxHeadDim / 2];
  __shared__ __align__(8) uint64_t s_bar[2];
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nq = p.q ? p.hq : 0, nk = p.k ? p.nkv : 0;
  const uint32_t head_bytes = 2u * p.hd, row_bytes = (nq + 2 * nk) * head_bytes;
  const int groups = (p.n_rows + p.rows - 1) / p.rows;
  // this warp's row of a group, its share of the row's heads
  const int wpr = kRopeWarps / p.rows, rr = warp / wpr, part = warp - rr * wpr;
  ptx::griddep_launch();
  auto load = [&](int group, int stage, int nth) {  // by thread 0
    if (nth == p.skip_group) return;
    const int r0 = group * p.rows, rows = min(p.rows, p.n_rows - r0);
    const uint32_t bar = ptx::smem_u32(&s_bar[stage]);
    ptx::mbar_arrive_expect_tx(bar, rows * row_bytes);
    for (int i = 0; i < rows; ++i) {
      const int64_t t = r0 + i;
      uint8_t *dst = rope_smem + (stage * p.rows + i) * row_bytes;
      if (nq) bulk_load(dst, p.q + t * p.qs, nq * head_bytes, bar);
      if (nk) {
        bulk_load(dst + nq * head_bytes, p.k + t * p.ks, nk * head_bytes, bar);
        bulk_load(dst + (nq + nk) * head_bytes, p.v + t * p.vs, nk * head_bytes, bar);
      }
    }
  };
  if (threadIdx.x == 0) {
    s_abort = 0;
    ptx::mbar_init(ptx::smem_u32(&s_bar[0]), 1);
    ptx::mbar_init(ptx::smem_u32(&s_bar[1]), 1);
    ptx::fence_mbar_init();
    ptx::griddep_wait();
    load(blockIdx.x, 0, 0);
    if (blockIdx.x + gridDim.x < groups) load(blockIdx.x + gridDim.x, 1, 1);
  }
  ptx::griddep_wait();
  struct Place {
    int pos, page, slot;
  };
  auto place = [&](int group) {  // of this warp's row; pos -1: none
    Place a{-1, -1, 0};
    const int t = group * p.rows + rr;
    if (group < groups && t < p.n_rows) {
      a.pos = p.pos[t];
      if (nk) {
        a.page = p.page[t];
        a.slot = p.slot[t];
      }
    }
    return a;
  };
  Place here = place(blockIdx.x);
  __syncthreads();

  const int half = p.rot >> 1;
  // the lane's unit: its chunks, and whether they turn
  const int u = lane & (p.lph - 1), hl = lane / p.lph, hpw = 32 / p.lph;
  int d0, d1;
  bool turn0, turn1;
  if (kHalf) {
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

  const int64_t head = static_cast<int64_t>(p.P) * p.hd;  // pool values between two heads

  // The whole warp takes every step: the norm's shuffles need it.
  constexpr int kHv = VW / 2;
  auto turned = [&](const uint8_t *src, int heads, const uint16_t *gamma, uint16_t *dst,
                    int64_t dst_step) {
    float2 g[2 * kHv];
#pragma unroll
    for (int e = 0; e < 2 * kHv; ++e) g[e] = make_float2(1.f, 1.f);
    if (kNorm && gamma) {
      if (has0) unpack<VW>(*reinterpret_cast<const Chunk<VW> *>(gamma + d0), g);
      if (has1) unpack<VW>(*reinterpret_cast<const Chunk<VW> *>(gamma + d1), g + kHv);
    }
    // half layout: a = x[e], b = x[kHv + e], two pairs at once; pairs layout: x[e]
    // holds one pair (a, b), turned by (A, C) and, swapped, by (B, D)
    float2 A[2 * kHv], B[2 * kHv];
#pragma unroll
    for (int e = 0; e < 2 * kHv; ++e) {
      if (kHalf) {
        const int i = e % kHv, j = VW * u + 2 * i;
        const float2 c = turn0 ? make_float2(s_turn[rr][0][j], s_turn[rr][0][j + 1])
                               : make_float2(1.f, 1.f);
        const float2 sn = turn0 ? make_float2(s_turn[rr][1][j], s_turn[rr][1][j + 1])
                                : make_float2(0.f, 0.f);
        const float2 other = g[e < kHv ? kHv + i : i];
        A[e] = mul2(c, g[e]);
        B[e] = mul2(sn, other);
        if (e < kHv) B[e] = make_float2(-B[e].x, -B[e].y);
      } else {
        const bool turns = e < kHv ? turn0 : turn1;
        const float c = turns ? s_turn[rr][0][VW * u + e] : 1.f;
        const float sn = turns ? s_turn[rr][1][VW * u + e] : 0.f;
        A[e] = make_float2(c * g[e].x, c * g[e].y);
        B[e] = make_float2(-sn * g[e].y, sn * g[e].x);
      }
    }
    const uint8_t *from = src + (part * hpw + hl) * head_bytes;
    uint16_t *to = dst + (part * hpw + hl) * dst_step;
    const int step = wpr * hpw;
    for (int h = part * hpw + hl; h - hl < heads; h += step) {
      const bool in = h < heads;
      Chunk<VW> a = {}, b = {};
      if (in && has0) a = *reinterpret_cast<const Chunk<VW> *>(from + 2 * d0);
      if (in && has1) b = *reinterpret_cast<const Chunk<VW> *>(from + 2 * d1);
      float2 x[2 * kHv];
      unpack<VW>(a, x);
      unpack<VW>(b, x + kHv);
      float inv = 1.f;
      if (kNorm && gamma) {
        float2 s0 = mul2(x[0], x[0]), s1 = mul2(x[kHv], x[kHv]);
#pragma unroll
        for (int e = 1; e < kHv; ++e) {
          s0 = fma2(x[e], x[e], s0);
          s1 = fma2(x[kHv + e], x[kHv + e], s1);
        }
        float sum = (s0.x + s1.x) + (s0.y + s1.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (o < p.lph) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        inv = rsqrtf(fmaf(sum, p.inv_hd, p.eps));
      }
      if (in) {
        const float2 inv2 = make_float2(inv, inv);
        if (kNorm) {
#pragma unroll
          for (int e = 0; e < 2 * kHv; ++e) x[e] = mul2(x[e], inv2);
        }
        float2 y[2 * kHv];
#pragma unroll
        for (int e = 0; e < 2 * kHv; ++e) {
          const bool turns = kHalf || e < kHv ? turn0 : turn1;
          const float2 other = kHalf ? x[e < kHv ? kHv + e : e - kHv] : make_float2(x[e].y, x[e].x);
          y[e] = mul2(x[e], A[e]);
          if (turns) y[e] = fma2(other, B[e], y[e]);  // nothing of the other one, not even an
        }                                            // infinite one, in dims that do not turn
        if (has0) *reinterpret_cast<Chunk<VW> *>(to + d0) = pack<VW>(y);
        if (has1) *reinterpret_cast<Chunk<VW> *>(to + d1) = pack<VW>(y + kHv);
      }
      from += step * head_bytes;
      to += step * dst_step;
    }
  };

  uint32_t phase = 0u;  // bit s: of stage s
  int stage = 0, nth = 0;
  for (int group = blockIdx.x; group < groups; group += gridDim.x, ++nth) {
    const int t = group * p.rows + rr;
    const Place now = here;
    here = place(group + gridDim.x);
    for (int j = part * 32 + lane; j < half; j += 32 * wpr) {
      const float2 cs = turn_cos_sin(now.pos, tf.f[j], p.mag);
      s_turn[rr][0][j] = cs.x;
      s_turn[rr][1][j] = cs.y;
    }
    ptx::bar_sync(1 + rr, 32 * wpr);  // the warps of this row
    const bool got = __all_sync(
        0xffffffffu, ptx::mbar_wait(ptx::smem_u32(&s_bar[stage]), (phase >> stage) & 1u, &s_abort));
    if (!got && lane == 0) raise_status(p.st, DFLASH_DEV_WAIT_TIMEOUT);
    if (got && now.pos >= 0) {
      const uint8_t *row = rope_smem + (stage * p.rows + rr) * row_bytes;
      if (nq) turned(row, nq, p.gq, p.q_out + t * p.qos, p.hd);
      if (now.page >= p.NP || (now.page >= 0 && (now.slot < 0 || now.slot >= p.P))) {
        if (lane == 0 && part == 0) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
      } else if (now.page >= 0) {
        uint16_t *pool = pool_row(p, now.page, now.slot, 0, 0);
        turned(row + nq * head_bytes, nk, p.gk, pool, head);
        // v: copied 16 bytes a lane
        const int vecs = p.hd / 8, total = nk * vecs;
        const uint4 *v = reinterpret_cast<const uint4 *>(row + (nq + nk) * head_bytes);
        for (int i = part * 32 + lane; i < total; i += 32 * wpr) {
          const int h = i / vecs;
          reinterpret_cast<uint4 *>(pool + (nk + h) * head)[i - h * vecs] = v[i];
        }
      }
    }
    if (__syncthreads_or(!got)) {  // wind down: the copies in flight land before the CTA ends
      for (int i = 0; i < 2 && threadIdx.x == 0; ++i, stage ^= 1) {
        volatile int dummy = 0;
        if (group + i * gridDim.x < groups)
          ptx::mbar_wait(ptx::smem_u32(&s_bar[stage]), (phase >> stage) & 1u, &dummy);
      }
      return;
    }
    // the stage and the angles are free
    if (threadIdx.x == 0 && group + 2 * gridDim.x < groups)
      load(group + 2 * gridDim.x, stage, nth + 2);
    phase ^= 1u << stage;
    stage ^= 1;
  }
}

// Widths that no 8-byte chunk fits (an odd number of pairs, or of two), and rows
// too large for shared memory: one warp per (row, head of q, k or v), a pair or a value per lane.
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
  p.inv_hd = 1.f / static_cast<float>(g.head_dim);
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
  p.skip_group = attention_test_skip_tile_value();
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
  const size_t row_bytes = 2ull * p.hd * ((q ? p.hq : 0) + (k ? 2 * p.nkv : 0));
  const int vw = 2 * row_bytes > kRopeSmem ? 0 : unit % 8 == 0 ? 8 : unit % 4 == 0 ? 4 : 0;
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
  // two CTAs an SM, each with two stages of as many rows as fit, and as leave
  // every CTA a group
  p.rows = 1;
  while (p.rows < kMaxRopeRows && n_rows > 2 * device_sm_count() * p.rows &&
         4 * p.rows * row_bytes <= kRopeSmem / 2)
    p.rows *= 2;
  const int groups = (n_rows + p.rows - 1) / p.rows;
  cfg.gridDim = dim3(std::min(groups, 2 * device_sm_count()));
  cfg.dynamicSmemBytes = 2 * p.rows * row_bytes;
  const bool norm = gamma_q || gamma_k;
  auto launch = [&](auto width, auto with_norm) {
    constexpr int kVW = decltype(width)::value;
    constexpr bool kNorm = decltype(with_norm)::value;
    cudaError_t e = ensure_smem_limit<chunk_rope_kernel<kVW, kNorm, true>>(kRopeSmem);
    if (e == cudaSuccess) e = ensure_smem_limit<chunk_rope_kernel<kVW, kNorm, false>>(kRopeSmem);
    if (e != cudaSuccess) return e;
    return halves ? cudaLaunchKernelEx(&cfg, chunk_rope_kernel<kVW, kNorm, true>, p, tf)
                  : cudaLaunchKernelEx(&cfg, chunk_rope_kernel<kVW, kNorm, false>, p, tf);
  };
  using Wide = std::integral_constant<int, 8>;
  using Narrow = std::integral_constant<int, 4>;
  if (vw == 8) return norm ? launch(Wide{}, std::true_type{}) : launch(Wide{}, std::false_type{});
  return norm ? launch(Narrow{}, std::true_type{}) : launch(Narrow{}, std::false_type{});
}

}  // namespace dflash
