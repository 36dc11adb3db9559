// chunk_store8.cu -- a ragged chunk's rows into a cache held in 8 bits, and rows of that cache
// read back.
//
// Mathematics: k is normed and turned as in the 16-bit store (fp32), then a block's exponent
// comes from the largest magnitude of its rows by the bits of that number (no logarithm: the
// smallest e with a <= 448 * 2^e), so x * 2^-e is exact and each value is rounded once.
#include "cache8.cuh"
#include "chunk_turn.cuh"
#include "dflash_internal.cuh"
#include "f32x2.cuh"
#include "sm100_ptx.cuh"

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

// One CTA for a row that is the first of its block's, a head, K or V: what the kernel below does not
// take.  Simple and slow: each angle is taken four times, and a thread loads a value at once.  8192
// rows of 32 + 8 + 8 heads: 257 us for heads of 128 of which 24 dims turn by halves, 277 for heads of
// 96, 356 for 256 (54 in the kernel below, where 128 turn).
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

// The heads of 64 or 128 that no turning pair of 8-value chunks is cut by: one launch for q, k
// and v.  A row's HD values are held by HD / 16 lanes, two chunks of 8 each: in the half layout
// the two that turn together, in the pairs layout neighbouring ones (as the 16-bit store).
//
// K and V.  A CTA takes the blocks that its window of rows is the first in, for one head of K
// or V; a warp holds kRows rows in registers, so that memory is read once: blocks of that many
// rows are a warp's, each, larger ones all four warps' (they join their largest values).  Every
// (row, pair) of a head is turned once, so its angle is taken where it is needed.
//
// Q.  A CTA takes 16 pieces, each as many heads of a row as a warp holds.
//
// Bound by HBM: 8192 rows of 32 + 8 + 8 heads of 128 are 184 MB with their codes and take 54 us, 3.4
// TB/s: q alone 29 us (134 MB), k and v alone 31 (50 MB, a window of rows a CTA).
constexpr int kQPieces = 16;

struct Store8Fast {
  Store8Params s;
  const uint16_t *q, *gq;
  uint16_t *q_out;
  int64_t qs, qos;
  int hq, window, q_pieces, kv_blocks;  // q_pieces: of a row
};

template <int HD, bool kHalf>
struct Lanes {
  static constexpr int kLanes = HD / 16, kAtOnce = 32 / kLanes;  // of a row; rows of a warp's access
  int d0, d1, pair0;
  bool turn0, turn1;
  __device__ __forceinline__ explicit Lanes(int lane, int rot) {
    const int u = lane % kLanes;
    pair0 = 8 * u;
    if (kHalf) {
      const int nrot = rot / 16;
      turn0 = turn1 = u < nrot;
      d0 = turn0 ? 8 * u : rot + 16 * (u - nrot);
      d1 = turn0 ? d0 + rot / 2 : d0 + 8;
    } else {
      d0 = 16 * u;
      d1 = d0 + 8;
      turn0 = d0 < rot;
      turn1 = d1 < rot;
    }
  }
};

__device__ __forceinline__ void unpack8(const uint4 &v, float *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = ptx::pack_bf16x2(x[2 * e], x[2 * e + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's gains.
struct Gains {
  uint4 g[2] = {};
  bool norm;
  template <class L>
  __device__ __forceinline__ Gains(const uint16_t *gamma, const L &at) : norm(gamma != nullptr) {
    if (norm) {
      g[0] = *reinterpret_cast<const uint4 *>(gamma + at.d0);
      g[1] = *reinterpret_cast<const uint4 *>(gamma + at.d1);
    }
  }
};
// The turns of pairs `first` on.  (Through a generic address: as constants, the lanes' different
// places are read one after another.)
template <int N>
__device__ __forceinline__ void turns_of(const TurnFreqs &tf, int first, bool any, uint64_t (&f)[N]) {
  const uint64_t *from = tf.f + first;
  asm("" : "+l"(from));
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = any ? from[e] : 0;
}
// cos and sin of a key's pairs.  The angle is a fraction of a turn in 32 bits: its nearest quarter
// is taken off exactly, what is left is x, at most pi / 4, and the series of sin x up to x^9 and of
// cos x up to x^10 are off by at most 2^-28 there; with fp32's roundings 2^-23 in all.  (An angle
// off by more changes codes: with the hardware's functions, 2^-21, in the same time, 8192 rows were
// seven times as far from fp32's.  The exact ones take 89 us instead of 53.)  Two pairs an
// instruction.
__device__ __forceinline__ void key_angles(const uint64_t (&f)[8], int pos, float mag,
                                           float (&c)[8], float (&s)[8]) {
  const float2 one = make_float2(1.f, 1.f);
  auto both = [](float v) { return make_float2(v, v); };
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    uint32_t u[2];
    float x0[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t t = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * f[e + i];
      // top 32 bits: a signed fraction of half a turn in units of 2^-31; an eighth of a turn added
      u[i] = static_cast<uint32_t>(t >> 32) + 0x20000000u;
      x0[i] = static_cast<float>(static_cast<int32_t>(u[i] & 0x3fffffffu) - 0x20000000);
    }
    const float2 x = mul2(make_float2(x0[0], x0[1]), both(3.14159265358979f * 0x1p-31f));
    const float2 y = mul2(x, x);
    float2 sn = fma2(y, both(1.f / 362880.f), both(-1.f / 5040.f));
    sn = fma2(sn, y, both(1.f / 120.f));
    sn = fma2(sn, y, both(-1.f / 6.f));
    sn = fma2(mul2(sn, y), x, x);
    float2 cs = fma2(y, both(-1.f / 3628800.f), both(1.f / 40320.f));
    cs = fma2(cs, y, both(-1.f / 720.f));
    cs = fma2(cs, y, both(1.f / 24.f));
    cs = fma2(cs, y, both(-0.5f));
    cs = fma2(cs, y, one);
    sn = mul2(sn, both(mag));
    cs = mul2(cs, both(mag));
    const float a[2] = {sn.x, sn.y}, b[2] = {cs.x, cs.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // the quarters again: u's two top bits
      const bool odd = u[i] & 0x40000000u;
      s[e + i] = __uint_as_float(__float_as_uint(odd ? b[i] : a[i]) ^ (u[i] & 0x80000000u));
      c[e + i] = __uint_as_float(__float_as_uint(odd ? a[i] : b[i]) ^
                                 ((u[i] + 0x40000000u) & 0x80000000u));
    }
  }
}
// cos and sin of a query row's pairs, as in the 16-bit store: the lanes that hold the same
// dims of different heads take some of them each.
template <class L>
__device__ __forceinline__ void query_angles(const uint64_t (&f)[8 / L::kAtOnce], int lane, int pos,
                                             float mag, float (&c)[8], float (&s)[8]) {
  constexpr int kEach = 8 / L::kAtOnce;
  float2 mine[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) mine[e] = turn_cos_sin(pos, f[e], mag);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int from = e / kEach * L::kLanes + lane % L::kLanes;
    c[e] = __shfl_sync(0xffffffffu, mine[e % kEach].x, from);
    s[e] = __shfl_sync(0xffffffffu, mine[e % kEach].y, from);
  }
}
// The norm's factor of a row that kLanes lanes hold.
template <int kLanes>
__device__ __forceinline__ float norm_of(const float (&x)[16], float eps, int hd) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a = fmaf(x[e], x[e], a);
    b = fmaf(x[8 + e], x[8 + e], b);
  }
  a += b;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return rsqrtf(a / static_cast<float>(hd) + eps);
}
template <int kLanes>
__device__ __forceinline__ void norm16(const Gains &k, float eps, int hd, float (&x)[16]) {
  if (!k.norm) return;
  const float inv = norm_of<kLanes>(x, eps, hd);
  float g[16];
  unpack8(k.g[0], g);
  unpack8(k.g[1], g + 8);
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = x[e] * inv * g[e];
}
template <bool kHalf>
__device__ __forceinline__ void turn16(float (&x)[16], const float (&c)[8], const float (&s)[8],
                                       bool turn0, bool turn1) {
  if (kHalf) {
    if (!turn0) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = x[e], b = x[8 + e];
      x[e] = a * c[e] - b * s[e];
      x[8 + e] = b * c[e] + a * s[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!(e < 4 ? turn0 : turn1)) continue;
      const float a = x[2 * e], b = x[2 * e + 1];
      x[2 * e] = a * c[e] - b * s[e];
      x[2 * e + 1] = b * c[e] + a * s[e];
    }
  }
}

template <int HD, bool kHalf>
__device__ __forceinline__ void store_q(const Store8Fast &p, const TurnFreqs &tf, int block) {
  using L = Lanes<HD, kHalf>;
  constexpr int kEach = kQPieces / 4;  // of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const L at(lane, p.s.rot);
  const Gains gains(p.gq, at);
  uint64_t f[8 / L::kAtOnce];
  turns_of(tf, at.pair0 + lane / L::kLanes * (8 / L::kAtOnce), at.turn0, f);
  const int64_t first = static_cast<int64_t>(block) * kQPieces + warp * kEach;
  uint4 v[kEach][2] = {};
  int pos[kEach], row[kEach], head[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t r = (first + i) / p.q_pieces;
    row[i] = static_cast<int>(r < p.s.n_rows ? r : 0);
    head[i] = static_cast<int>(first + i - r * p.q_pieces) * L::kAtOnce + lane / L::kLanes;
    pos[i] = r < p.s.n_rows ? p.s.pos[row[i]] : -1;
    if (head[i] < p.hq && r < p.s.n_rows) {
      const uint16_t *src = p.q + row[i] * p.qs + static_cast<int64_t>(head[i]) * HD;
      v[i][0] = *reinterpret_cast<const uint4 *>(src + at.d0);
      v[i][1] = *reinterpret_cast<const uint4 *>(src + at.d1);
    }
  }
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (pos[i] < 0) continue;  // the whole warp's row
    if (p.s.rot && (i == 0 || pos[i] != pos[i ? i - 1 : 0]))  // uniform
      query_angles<L>(f, lane, pos[i], p.s.mag, c, s);
    float x[16];
    unpack8(v[i][0], x);
    unpack8(v[i][1], x + 8);
    norm16<L::kLanes>(gains, p.s.eps, HD, x);
    turn16<kHalf>(x, c, s, at.turn0, at.turn1);
    if (head[i] < p.hq) {
      uint16_t *dst = p.q_out + row[i] * p.qos + static_cast<int64_t>(head[i]) * HD;
      *reinterpret_cast<uint4 *>(dst + at.d0) = pack8(x);
      *reinterpret_cast<uint4 *>(dst + at.d1) = pack8(x + 8);
    }
  }
}

constexpr int kMostWindow = 64;

template <int HD, bool kHalf>
__global__ void __launch_bounds__(128, 4)
    chunk_store8_fast_kernel(const __grid_constant__ Store8Fast p,
                             const __grid_constant__ TurnFreqs tf) {
  using L = Lanes<HD, kHalf>;
  constexpr int kIters = 4, kRows = kIters * L::kAtOnce;  // rows that a warp holds
  ptx::griddep_launch();
  ptx::griddep_wait();
  if (blockIdx.x >= p.kv_blocks) {
    store_q<HD, kHalf>(p, tf, blockIdx.x - p.kv_blocks);
    return;
  }
  __shared__ int64_t s_block[kMostWindow + 65];  // of rows first - 1 on
  __shared__ float s_most[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Cache8 &cache = p.s.cache;
  const int hk = blockIdx.x % (2 * cache.nkv), kv = hk & 1, h = hk >> 1;
  const int first = blockIdx.x / (2 * cache.nkv) * p.window, block = cache.block;
  const L at(lane, kv ? 0 : p.s.rot);
  const Gains gains(kv ? nullptr : p.s.gk, at);
  uint64_t f[8];
  turns_of(tf, at.pair0, at.turn0, f);
  for (int x = threadIdx.x; x <= p.window + block; x += 128) {
    const int t = first - 1 + x;
    const bool mine = hk == 0 && t >= first && t < first + p.window;  // reports it
    s_block[x] = t >= 0 && t < p.s.n_rows ? block_of(p.s, t, mine) : -1;
  }
  __syncthreads();
  const int sub = lane / L::kLanes;  // the lane's row of kAtOnce
  const uint16_t *src = (kv ? p.s.v : p.s.k) + static_cast<int64_t>(h) * HD;
  const int64_t step = kv ? p.s.vs : p.s.ks;

  // bit i: row i of the window is the first of its block
  auto starts = [&](int i) {
    const bool yes = i < p.window && s_block[1 + i] >= 0 && s_block[i] != s_block[1 + i];
    return __ballot_sync(0xffffffffu, yes);
  };
  uint64_t left = starts(lane) | static_cast<uint64_t>(p.window > 32 ? starts(32 + lane) : 0u) << 32;
  int small = 0;  // runs that are one warp's, so far
  for (; left; left &= left - 1) {
    const int i = __ffsll(static_cast<long long>(left)) - 1;
    const int64_t id = s_block[1 + i];
    // rows of the block: up to the first that is another's
    auto others = [&](int r) {
      return __ballot_sync(0xffffffffu, r <= block && s_block[1 + i + min(r, block)] != id);
    };
    uint32_t end = others(lane + 1);
    int n = end ? __ffs(end) : 33;
    if (!end && (end = others(lane + 33)) != 0) n = 32 + __ffs(end);
    else if (!end) n = 65;
    n = min(n, block + 1);
    if (n > block) {  // more rows than slots
      if (threadIdx.x == 0 && hk == 0) raise_status(p.s.st, DFLASH_DEV_BAD_ROWS);
      n = block;
    }
    const bool together = n > kRows;
    if (!together && (small++ & 3) != warp) continue;
    const int t0 = first + i, page = p.s.page[t0], slot0 = p.s.slot[t0] / block * block;
    uint8_t *scale = cache.scale(page, kv, h, slot0);
    const int before = static_cast<int>(*scale) - 127;
    // this warp's rows: a whole number of kAtOnce
    const int each = together ? ((n + 3) / 4 + L::kAtOnce - 1) / L::kAtOnce * L::kAtOnce : kRows;
    const int r0 = t0 + (together ? warp * each : 0);
    const int rows = max(min(each, t0 + n - r0), 0);
    uint4 v[kIters][2] = {};
    int slot[kIters], pos[kIters];
#pragma unroll
    for (int j = 0; j < kIters; ++j) {
      const int r = j * L::kAtOnce + sub;
      slot[j] = -1;
      pos[j] = 0;
      if (r < rows) {
        const uint16_t *x = src + (r0 + r) * step;
        v[j][0] = *reinterpret_cast<const uint4 *>(x + at.d0);
        v[j][1] = *reinterpret_cast<const uint4 *>(x + at.d1);
        slot[j] = p.s.slot[r0 + r];
        pos[j] = p.s.pos[r0 + r];
      }
    }
    // the slots that the block's rows write: bit s of slot s
    uint64_t written = 0;
    for (int r = lane; r < n; r += 32) written |= 1ull << (p.s.slot[t0 + r] - slot0);
    written = static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(written))) |
              static_cast<uint64_t>(
                  __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(written >> 32)))
                  << 32;
    float y[kIters][16], most = 0.f;
#pragma unroll
    for (int j = 0; j < kIters; ++j) {
      if (j * L::kAtOnce >= rows) {  // the whole warp
#pragma unroll
        for (int e = 0; e < 16; ++e) y[j][e] = 0.f;
        continue;
      }
      unpack8(v[j][0], y[j]);
      unpack8(v[j][1], y[j] + 8);
      norm16<L::kLanes>(gains, p.s.eps, HD, y[j]);
      if (at.turn0 && slot[j] >= 0) {
        float c[8], s[8];
        key_angles(f, pos[j], p.s.mag, c, s);
        turn16<kHalf>(y[j], c, s, at.turn0, at.turn1);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(y[j][e]));  // NaN counts for nothing
    }
    if (__any_sync(0xffffffffu, !(most < INFINITY))) {  // nor do infinities, which become NaN
      most = 0.f;
#pragma unroll
      for (int j = 0; j < kIters; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (fabsf(y[j][e]) < INFINITY) most = fmaxf(most, fabsf(y[j][e]));
          else y[j][e] = NAN;
        }
    }
    most = warp_max(most);
    if (together) {
      if (lane == 0) s_most[warp] = most;
      __syncthreads();
      most = fmaxf(fmaxf(s_most[0], s_most[1]), fmaxf(s_most[2], s_most[3]));
      __syncthreads();
    }
    int e = scale8_exponent(most);
    if (!(written & 1)) {  // the block goes on
      e = max(e, before);
      if (e != before) {
        const float shift = before - e < -149 ? 0.f : exp2_int(before - e);
        const int vecs = block * HD / 16, c16 = HD / 16;
        uint4 *cells = reinterpret_cast<uint4 *>(cache.code(page, kv, h, slot0));
        for (int x = (together ? threadIdx.x : lane); x < vecs; x += together ? 128 : 32) {
          if ((written >> (x / c16)) & 1) continue;
          const uint4 old = cells[x];
          uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float2 lo = e4m3_values(w[b]), hi = e4m3_values(w[b] >> 16);
            w[b] = e4m3_pair(lo.x * shift, lo.y * shift) |
                   e4m3_pair(hi.x * shift, hi.y * shift) << 16;
          }
          cells[x] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    const float down = exp2_int(-e);
#pragma unroll
    for (int j = 0; j < kIters; ++j) {
      if (slot[j] < 0) continue;
      uint32_t w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        w[b] = e4m3_pair(y[j][4 * b] * down, y[j][4 * b + 1] * down) |
               e4m3_pair(y[j][4 * b + 2] * down, y[j][4 * b + 3] * down) << 16;
      uint8_t *cell = cache.code(page, kv, h, slot[j]);
      *reinterpret_cast<uint2 *>(cell + at.d0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2 *>(cell + at.d1) = make_uint2(w[2], w[3]);
    }
    // (every warp has read the scale before the barriers, where there is more than one)
    if (lane == 0 && (!together || warp == 0)) *scale = static_cast<uint8_t>(e + 127);
  }
}

struct Read8Params {
  Cache8 cache;
  int n_rows, rows, vecs, sides;  // rows of a CTA, 16 codes each of a row's K (or V), K and V
  int wide_out;                   // 32-byte aligned rows
  const int32_t *page, *slot;
  uint16_t *out[2];
  int64_t stride[2];
  int32_t *st;
};

// 16 codes a lane, of the same heads' dims in kReadEach rows: all loads before the first is used.
// Bound by HBM: 32768 rows of 8 heads of 128 (202 MB) 38 us, 5.3 TB/s.
constexpr int kReadEach = 2;
__global__ void __launch_bounds__(256, 8)
    chunk_read8_kernel(const __grid_constant__ Read8Params p) {
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int per_row = p.vecs * p.sides, lanes = min(per_row, 256), at_once = 256 / lanes;
  const int mine = threadIdx.x / lanes, head = p.cache.hd / 16;
  const int r1 = min((blockIdx.x + 1) * p.rows, p.n_rows);
  if (mine >= at_once) return;
  for (int y = threadIdx.x - mine * lanes; y < per_row; y += lanes) {
    const int kv = p.sides == 1 ? (p.out[0] ? 0 : 1) : y >= p.vecs;
    const int c = y - (p.sides == 2 && kv ? p.vecs : 0), h = c / head;
    uint16_t *out = p.out[kv] + 16 * c;
    for (int r = blockIdx.x * p.rows + mine; r < r1; r += kReadEach * at_once) {
      uint4 codes[kReadEach];
      uint32_t scale[kReadEach];
      bool here[kReadEach];
#pragma unroll
      for (int i = 0; i < kReadEach; ++i) {
        const int t = r + i * at_once;
        here[i] = false;
        if (t >= r1) continue;
        const int pg = p.page[t], sl = p.slot[t];
        if (pg < 0) continue;
        if (pg >= p.cache.NP || sl < 0 || sl >= p.cache.P) {
          if (y == 0) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
          continue;
        }
        here[i] = true;
        codes[i] =
            __ldcs(reinterpret_cast<const uint4 *>(p.cache.code(pg, kv, h, sl)) + (c - h * head));
        scale[i] = *p.cache.scale(pg, kv, h, sl);
      }
#pragma unroll
      for (int i = 0; i < kReadEach; ++i) {
        if (!here[i]) continue;
        uint16_t *to = out + static_cast<int64_t>(r + i * at_once) * p.stride[kv];
        const float f = scale8_value(scale[i]);
        const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
        uint32_t o[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const float2 v = e4m3_values(w[b >> 1] >> (16 * (b & 1)));
          o[b] = ptx::pack_bf16x2(v.x * f, v.y * f);
        }
        if (p.wide_out) {  // whole sectors
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to),
                       "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]),
                       "r"(o[7])
                       : "memory");
        } else {
          reinterpret_cast<uint4 *>(to)[0] = make_uint4(o[0], o[1], o[2], o[3]);
          reinterpret_cast<uint4 *>(to)[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
  }
}

// A launch that may begin under the end of the one before it.
cudaLaunchConfig_t config(cudaLaunchAttribute *attr, int64_t blocks, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_chunk_rope_store8(const dflash_geom &g, int layer, int n_rows,
                                     const dflash_rope_spec &rope, const void *q, int64_t q_stride,
                                     const void *k, int64_t k_stride, const void *v,
                                     int64_t v_stride, const void *gamma_q, const void *gamma_k,
                                     const int32_t *pos, const int32_t *page, const int32_t *slot,
                                     void *q_out, int64_t q_out_stride, const dflash_cache8 &cache,
                                     int32_t *st, cudaStream_t s) {
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
  const bool halves = rope.layout == DFLASH_ROPE_HALF;
  if ((g.head_dim == 64 || g.head_dim == 128) && rope.rot_dim % (halves ? 16 : 8) == 0) {
    Store8Fast f = {};
    f.s = p;
    f.q = static_cast<const uint16_t *>(q);
    f.gq = static_cast<const uint16_t *>(gamma_q);
    f.q_out = static_cast<uint16_t *>(q_out);
    f.qs = q_stride;
    f.qos = q_out_stride;
    f.hq = g.hq;
    // Rows of a CTA's window: single tokens are a block each, a prompt's rows share one.  Fixed
    // at 16 or 64, us: 64 single tokens 11 and 34 instead of 7.1; 8192 rows of a prompt 66 and 50
    // instead of 54.5 (32 here), 5003 rows of 64-wide heads 22.6 and 12.8 instead of 15.9 (32).
    f.window = 1;
    while (f.window < kMostWindow && n_rows > 256 * f.window) f.window *= 2;
    const int at_once = 512 / g.head_dim;
    f.q_pieces = (g.hq + at_once - 1) / at_once;
    const int64_t kv_blocks =
        k ? static_cast<int64_t>((n_rows + f.window - 1) / f.window) * 2 * g.nkv : 0;
    const int64_t q_blocks =
        q ? (static_cast<int64_t>(n_rows) * f.q_pieces + kQPieces - 1) / kQPieces : 0;
    if (kv_blocks + q_blocks >= (1LL << 31)) return cudaErrorInvalidValue;
    f.kv_blocks = static_cast<int>(kv_blocks);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(attr, kv_blocks + q_blocks, 128, s);
    if (g.head_dim == 64)
      return cudaLaunchKernelEx(&cfg, halves ? chunk_store8_fast_kernel<64, true>
                                             : chunk_store8_fast_kernel<64, false>, f, table.tf);
    return cudaLaunchKernelEx(&cfg, halves ? chunk_store8_fast_kernel<128, true>
                                           : chunk_store8_fast_kernel<128, false>, f, table.tf);
  }
  if (q) {
    const cudaError_t e = launch_chunk_rope_store(
        g, layer, n_rows, rope, q, q_stride, nullptr, 0, nullptr, 0, gamma_q, nullptr, pos, nullptr,
        nullptr, q_out, q_out_stride, nullptr, st, s);
    if (e != cudaSuccess || !k) return e;
  }
  chunk_store8_kernel<<<dim3(n_rows, g.nkv, 2), 128, 0, s>>>(p, table.tf);
  return cudaGetLastError();
}

cudaError_t launch_chunk_read8(const dflash_geom &g, int layer, int n_rows,
                               const dflash_cache8 &cache, const int32_t *page,
                               const int32_t *slot, void *k_out, int64_t k_stride, void *v_out,
                               int64_t v_stride, int32_t *st, cudaStream_t s) {
  Read8Params p = {};
  p.cache = cache8_of(g, cache, layer);
  p.n_rows = n_rows;
  p.vecs = g.nkv * g.head_dim / 16;
  p.sides = (k_out != nullptr) + (v_out != nullptr);
  // Rows of a CTA: a step of its threads', two where that still fills the card (8 CTAs an SM): 32768
  // rows 38.0 us instead of 41; two where it does not would only leave SMs idle.
  const int at_once = std::max(256 / (p.vecs * p.sides), 1) * kReadEach;
  p.rows = at_once * (n_rows > 16LL * at_once * device_sm_count() ? 2 : 1);
  p.page = page;
  p.slot = slot;
  p.out[0] = static_cast<uint16_t *>(k_out);
  p.out[1] = static_cast<uint16_t *>(v_out);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.wide_out = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out) |
                 2 * static_cast<uintptr_t>(k_stride | v_stride)) &
                31u) == 0;
  p.st = st;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(attr, (n_rows + p.rows - 1) / p.rows, 256, s);
  return cudaLaunchKernelEx(&cfg, chunk_read8_kernel, p);
}

}  // namespace dflash
