// chunk8_roles.cuh -- what the kernels of chunk_attention8.cu and chunk_attention8_few.cu share:
// the warps that find the work, look up scales and load tiles, the split of Q, V's widening.
#pragma once

#include "cache8.cuh"
#include "chunk_work.cuh"

namespace dflash {

// Work tiles of 2^shift rows for the kernel of few rows (heads of 128).
constexpr int kLeastFewShift = 4, kMostFewShift = 5;
cudaError_t launch_attn8_few(int shift, const CUtensorMap &tm, const ChunkParams &p,
                             const Cache8 &cache, dim3 grid, cudaStream_t s);

namespace {

constexpr int kThreads = 512;
// Registers: 512 threads launch with 128 each; the softmax groups take more (64 scores, or as many
// results, beside a work's state), the others give them up: 2 x 128 x 184 + 128 x 64 + 128 x 80 =
// 65536.
constexpr int kSoftmaxRegs = 184, kIssueRegs = 64, kWidenRegs = 80;
static_assert(256 * kSoftmaxRegs + 128 * (kIssueRegs + kWidenRegs) <= kThreads * 128, "");
constexpr int kWidenTeam = 4;  // warps that widen a tile of V
constexpr int kMetaBatch = 4, kMetaBatches = 4;  // key tiles looked up at once, of that many more
// P's weights carry 2^7: fp16's smallest steps are further below a row's largest weight then.
// (The reference maximum lags by up to 2^8, and 2^15 is still an fp16 number.)
constexpr float kLift = 7.f;

// What the softmax and the widening warps need to know of a key tile.
struct __align__(16) TileMeta {
  float k[8];     // K's factor of each 16 keys
  uint32_t v[8];  // V's: an fp16 factor, the scale byte << 16, 1 << 24 where the keys are there
  int E;          // the tile's weights times V give units of 2^E
  int far;        // bf16 instead of fp16 (E = 0)
  int bad;        // bits of the 16 keys each that are visible on a page outside the pool, then
                  // (bits 8 to 15) of those whose K has a scale of NaN
  int pad;
};

// D(tmem) (+)= A * B^T of e4m3 operands in shared memory, K = 32 a step.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f8f6f4: format 0 of A and B is e4m3; kind::f16: format 0 is fp16, 1 bf16.
constexpr uint32_t idesc_of(int M, int N, uint32_t format, bool b_mn_major) {
  return (1u << 4) | (format << 7) | (format << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}
constexpr uint32_t kSwizzle64B = 4, kSwizzle32B = 6;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two codes (bits 0-7 and 8-15 of pair) as fp16 numbers.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t pair) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(pair)));
  return r;
}

template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barriers, by their place: rings of K's tiles, of V's, of V's in 16 bits, of scales (full, empty),
// then the softmax groups', Q's, the works'.
template <int kK, int kV, int kW, int kS>
struct Bars {
  static constexpr int kKs = kK, kVs = kV, kWides = kW, kScores = kS;
  static constexpr int kKFull = 0, kKEmpty = kKFull + kKs, kVFull = kKEmpty + kKs,
                       kVEmpty = kVFull + kVs, kWFull = kVEmpty + kVs, kWEmpty = kWFull + kWides,
                       kMFull = kWEmpty + kWides, kMEmpty = kMFull + kMetaBatches,
                       kSFull = kMEmpty + kMetaBatches, kPFull = kSFull + kScores,
                       kODone = kPFull + 2,
                       kQReady = kODone + 2, kQEmpty = kQReady + 1, kDrain = kQEmpty + 1,
                       kWorkFull = kDrain + 1, kWorkRead = kWorkFull + 1, kClaim = kWorkRead + 1,
                       kBarCount = kClaim + 1;
};

// A thread's view of its CTA.
template <class Lay>
struct Cta {
  uint8_t *sm;
  uint32_t sm0;
  int lane;
  volatile int *abort_flag;
  Work *shared_work;
  TileMeta *meta;

  __device__ __forceinline__ uint32_t bar(int i) const {
    return sm0 + Lay::kBars + 8u * static_cast<uint32_t>(i);
  }
  // The CTA's works, one after the other, as in the 16-bit kernel.
  __device__ __forceinline__ Work next_work(uint32_t w) const {
    volatile int dummy = 0;
    Work d = {};
    if (__all_sync(0xffffffffu, chunk_wait<false, 16>(bar(Lay::kWorkFull), w & 1, &dummy)))
      d = shared_work[w & 1];
    else
      *abort_flag = 1;
    return d;
  }
  __device__ __forceinline__ void have_read() const {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(Lay::kWorkRead));
  }
  // Whether the nth use of a ring of n slots may begin: its barrier and phase.
  __device__ __forceinline__ bool reuse(int first, int at, int n) const {
    return at < n || chunk_wait<false>(bar(first + at % n),
                                       static_cast<uint32_t>((at / n - 1) & 1), abort_flag);
  }
  __device__ __forceinline__ bool arrived(int first, int at, int n) const {
    return chunk_wait<false>(bar(first + at % n), static_cast<uint32_t>((at / n) & 1), abort_flag);
  }
  // Waits on up to three barriers at the cost of one: each is polled by lanes of its own.
  struct At {
    uint32_t bar, phase;
  };
  __device__ __forceinline__ At full(int first, int at, int n) const {
    return At{bar(first + at % n), static_cast<uint32_t>((at / n) & 1)};
  }
  template <bool kSpin>
  __device__ __forceinline__ bool wait(At a, At b, At e) const {
    const At x = lane == 1 ? b : lane == 2 ? e : a;
    return __all_sync(0xffffffffu, chunk_wait<kSpin>(x.bar, x.phase, abort_flag));
  }
  // Whether the phase is over, without a wait.
  __device__ __forceinline__ bool passed(int i, uint32_t phase) const {
    return __all_sync(0xffffffffu, ptx::mbar_test(bar(i), phase));
  }
  __device__ __forceinline__ const TileMeta &scales(int batch, int t) const {
    return meta[batch % kMetaBatches * kMetaBatch + t % kMetaBatch];
  }
  // A thread's barriers, before any is used.
  __device__ __forceinline__ void init_bars() const {
    auto init = [&](int first, int n, uint32_t arrivals) {
      for (int i = 0; i < n; ++i) ptx::mbar_init(bar(first + i), arrivals);
    };
    init(Lay::kKFull, Lay::kKs, 1);
    init(Lay::kKEmpty, Lay::kKs, 1);
    init(Lay::kVFull, Lay::kVs, 1);
    init(Lay::kVEmpty, Lay::kVs, kWidenTeam);
    init(Lay::kWFull, Lay::kWides, kWidenTeam);
    init(Lay::kWEmpty, Lay::kWides, 1);
    init(Lay::kMFull, kMetaBatches, 1);
    init(Lay::kMEmpty, kMetaBatches, 8 + Lay::kWideners + 1);  // softmax, widening, issuing warps
    init(Lay::kSFull, Lay::kScores, 1);
    init(Lay::kPFull, 2, 4);  // one arrival per warp of the group
    init(Lay::kODone, 2, 1);
    init(Lay::kQReady, 1, 8);  // the warps that split Q
    init(Lay::kQEmpty, 1, 1);
    init(Lay::kDrain, 1, 1);
    init(Lay::kWorkFull, 1, 1);
    init(Lay::kWorkRead, 1, 11 + Lay::kWideners);  // every other warp
    init(Lay::kClaim, 1, 1);
  }
};

// Scales of a work's key tiles: false where a wait ran out.
template <class Lay>
__device__ __forceinline__ bool look_up_scales(const Cta<Lay> &c, const ChunkParams &p,
                                               const Cache8 &cache, const Work &d, int &batches) {
  const int lane = c.lane;
  // Lane 8 i + g: 16 keys g of tile i of four.  Pages are looked up two batches ahead, scales
  // one.
  const int mine = lane >> 3, g16 = 16 * (lane & 7);
  const int shift = 31 - __clz(cache.block), blocks = cache.P >> shift;
  bool ok = true;
  auto key_of = [&](int t) { return (d.t0 + t + mine) * kKT + g16; };
  auto look = [&](int t) {  // the page, -1 where it is none of the pool, -2 where no key is seen
    const int key = key_of(t);
    if (t + mine >= d.n || key > d.hi_max || key + 15 < d.lo_min) return -2;
    const int page = p.tbl[static_cast<int64_t>(d.r) * p.M + key / cache.P];
    return page >= 0 && page < cache.NP ? page : -1;
  };
  auto fetch = [&](int t, int page) {
    if (page < 0) return 0u;
    const uint8_t *k = cache.scales + cache.head(page, 0, d.kvh) * blocks +
                       (key_of(t) % cache.P >> shift);
    return static_cast<uint32_t>(k[0]) |
           static_cast<uint32_t>(k[static_cast<int64_t>(cache.nkv) * blocks]) << 8;
  };
  constexpr int kNone = 1000;
  int E = -kNone;
  bool far = false, any_bad = false;
  int page = look(0), page1 = look(kMetaBatch);
  uint32_t bytes = fetch(0, page);
  for (int t = 0; ok && t < d.n; t += kMetaBatch) {
    const uint32_t bytes1 = fetch(t + kMetaBatch, page1);
    const int page2 = look(t + 2 * kMetaBatch);
    ok = __all_sync(0xffffffffu, c.reuse(Lay::kMEmpty, batches, kMetaBatches));
    if (!ok) break;
    const uint32_t kb = bytes & 255u, vb = bytes >> 8;
    const bool counts = page >= 0 && vb != 255u;
    int top = counts ? static_cast<int>(vb) - 127 : -kNone,
        low = counts ? static_cast<int>(vb) - 127 : kNone;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    int my_E = 0, my_far = 0;
#pragma unroll
    for (int i = 0; i < kMetaBatch; ++i) {
      const int mx = __shfl_sync(0xffffffffu, top, 8 * i),
                mn = __shfl_sync(0xffffffffu, low, 8 * i);
      // (a little more than it must: the accumulators are scaled whenever it grows)
      const int grown = mx > E ? min(mx + 2, 127) : E;
      far = far || (mn != kNone && mn < grown - 14);
      if (!far) E = grown;
      if (i == mine) {
        my_E = far || E == -kNone ? 0 : E;
        my_far = far;
      }
    }
    const uint32_t bad = __ballot_sync(0xffffffffu, page == -1);
    const uint32_t nans = __ballot_sync(0xffffffffu, page >= 0 && kb == 255u);
    any_bad |= bad != 0;
    TileMeta &m = c.meta[batches % kMetaBatches * kMetaBatch + mine];
    m.k[lane & 7] = page >= 0 ? scale8_value(kb) : 1.f;
    const uint32_t factor =
        vb == 255u ? 0x7fffu : static_cast<uint32_t>(15 + static_cast<int>(vb) - 127 - my_E) << 10;
    m.v[lane & 7] = page >= 0 ? (factor & 0xffffu) | vb << 16 | 1u << 24 : 0u;
    if ((lane & 7) == 0) {
      m.E = my_E;
      m.far = my_far;
      m.bad = static_cast<int>((bad >> (8 * mine) & 255u) | (nans >> (8 * mine) & 255u) << 8);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(c.bar(Lay::kMFull + batches % kMetaBatches));
    ++batches;
    page = page1;
    page1 = page2;
    bytes = bytes1;
  }
  if (any_bad && lane == 0) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
  return ok;
}

// Finds the CTA's works (its own block's, then those of blocks that have not started), and looks
// up their scales: done with one's, while its last tiles are worked on, the warp is free for the
// next.
template <bool kMany, class Lay>
__device__ __forceinline__ void schedule(const Cta<Lay> &c, const ChunkParams &p,
                                         const Cache8 &cache, bool sorted, const int *sort_tiles,
                                         const uint8_t *sort_places) {
  const int lane = c.lane;
  int block = blockIdx.x, seg = blockIdx.z;
  bool have = true, last = !kMany;
  uint32_t claims = 0;
  int batches = 0;  // of scales
  bool ok = true;
  Order order = {};
  if (sorted) order = read_order(p, lane, sort_tiles, sort_places);
  for (uint32_t w = 0;; ++w) {
    Work d = {};
    while (true) {
      if (have) {
        d = sorted ? describe_sorted(p, order, block, seg, Lay::kShift)
                   : describe(p, block, seg, Lay::kShift, lane);
        have = false;
        if (d.nrow > 0) break;
      }
      if (last) break;
      const uint32_t answer = c.sm0 + Lay::kAnswer;
      if (lane == 0) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive_expect_tx(c.bar(Lay::kClaim), 16);
        claim_block(answer, c.bar(Lay::kClaim));
      }
      __syncwarp();
      volatile int dummy = 0;
      const bool told =
          __all_sync(0xffffffffu, chunk_wait<false, 4>(c.bar(Lay::kClaim), claims & 1, &dummy));
      if (!told) *c.abort_flag = 1;  // a block may be lost: reported
      have = told && claimed_block(answer, &block, &seg);
      __syncwarp();
      ++claims;
      last = !have;  // none left: not to be asked again
    }
    if (lane == 0) {
      c.shared_work[w & 1] = d;
      ptx::mbar_arrive(c.bar(Lay::kWorkFull));
    }
    __syncwarp();
    if (d.nrow == 0) break;
    if (d.n > 0 && ok) ok = look_up_scales(c, p, cache, d, batches);
    if (!kMany) break;
    volatile int dummy = 0;
    if (!__all_sync(0xffffffffu, chunk_wait<false, 4>(c.bar(Lay::kWorkRead), w & 1, &dummy)) ||
        *c.abort_flag)
      last = true;
  }
}

// A place in a ring of N slots and the phase of its next use, for a barrier that a use waits on
// before (kBefore: the slot is free) or after it (its contents are there).
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase;
  __device__ __forceinline__ explicit Ring(bool before) : phase(before ? 1u : 0u) {}
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// Loads K's (kV false) or V's tiles.  A load takes its warp some 700 cycles with a dozen others
// beside it, half of what a tile may take: a warp for each of the two, and what can be is
// worked out once for many tiles.
template <bool kMany, bool kV, class Lay>
__device__ __forceinline__ void load_tiles(const Cta<Lay> &c, const ChunkParams &p,
                                           const CUtensorMap &tm) {
  const int lane = c.lane;
  // A lane a box (page rows).  Boxes without a visible key and pages outside the pool are not
  // loaded.  The next work is claimed once V's loads come to the last kAhead tiles.
  constexpr int kAhead = 3, kSlots = kV ? Lay::kVs : Lay::kKs;
  constexpr int kEmpty = kV ? Lay::kVEmpty : Lay::kKEmpty, kFull = kV ? Lay::kVFull : Lay::kKFull;
  const int shift = 31 - __clz(kKT / p.box_rows), boxes = 1 << shift, per = 32 >> shift;
  const uint32_t box_bytes = p.box_rows * Lay::kHD;
  Ring<kSlots> ring(true);
  int loaded = 0;
  bool ok = true;
  for (uint32_t w = 0; w == 0 || kMany; ++w) {
    const Work d = c.next_work(w);
    if (!kV || d.nrow == 0 || d.n == 0 || !ok) {
      c.have_read();
      if (d.nrow == 0) break;
      if (d.n == 0 || !ok) continue;
    }
    const int n = d.n;
    const uint64_t pol =
        d.total <= (1 << Lay::kShift) ? ptx::policy_evict_first() : ptx::policy_evict_normal();
    // Pages of 32 boxes at once, a lookup ahead of the one in use.  Lane boxes * i + b: the pool's
    // row where box b of tile t + i begins, -1 where it is not loaded.
    auto look = [&](int t) {
      int row = -1;
      t += lane >> shift;
      if (t < n) {
        const int key0 = (d.t0 + t) * kKT + (lane & (boxes - 1)) * p.box_rows;
        if (key0 <= d.hi_max && key0 + p.box_rows > d.lo_min) {
          const int place = key0 / p.P, page = p.tbl[static_cast<int64_t>(d.r) * p.M + place];
          if (page >= 0 && page < p.NP)
            row = static_cast<int>(
                (((static_cast<int64_t>(p.layer) * p.NP + page) * 2 + kV) * p.nkv + d.kvh) * p.P +
                key0 - place * p.P);
        }
      }
      return row;
    };
    int rows = look(0), ahead = look(per), next = per;
    for (int t = 0; t < n; ++t) {
      if (kV && t == max(n - kAhead, 0)) c.have_read();
      if (t == next) {
        rows = ahead;
        next += per;
        ahead = look(next);
      }
      int row = __shfl_sync(0xffffffffu, rows, ((t << shift) + lane) & 31);
      if (lane >= boxes) row = -1;
      if (ok) {
        int bar = kEmpty + ring.slot;
        uint32_t phase = ring.phase;
        bool used = true;
        if (!kV && Lay::kFew) {  // the scores are done: the barrier that tells the softmax
          const int before = loaded - kSlots;
          used = before >= 0;
          bar = Lay::kSFull + (before & 3);
          phase = before >> 2 & 1;
        }
        ok = !used ||
             __all_sync(0xffffffffu, chunk_wait<false>(c.bar(bar), phase, c.abort_flag));
      }
      if (!ok) continue;
      const bool skip = !kV && t == p.skip_tile;
      const uint32_t bar = c.bar(kFull + ring.slot);
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, row >= 0)) * box_bytes;
      if (lane == 0 && !skip) ptx::mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (row >= 0 && !skip)
        ptx::tma_load_2d_hint(c.sm0 + (kV ? Lay::kV : Lay::kK) + ring.slot * Lay::kTile +
                                  lane * box_bytes,
                              &tm, 0, row, bar, pol);
      ring.next();
      ++loaded;
    }
  }
  if (*c.abort_flag && lane == 0) {  // wind down: the last copies land before the CTA ends
    volatile int dummy = 0;
    for (int i = max(loaded - kSlots, 0); i < loaded; ++i)
      chunk_wait<false>(c.bar(kFull + i % kSlots), static_cast<uint32_t>((i / kSlots) & 1), &dummy);
  }
}

// N values of a row that eight lanes hold, as hi + lo (four codes a word) times 2^e.
template <int N>
__device__ __forceinline__ int split_q(const uint4 (&x)[N / 8], uint32_t (&hi)[N / 4],
                                       uint32_t (&lo)[N / 4]) {
  constexpr int kWords = N / 2;
  uint32_t v[kWords];
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    v[4 * i] = x[i].x;
    v[4 * i + 1] = x[i].y;
    v[4 * i + 2] = x[i].z;
    v[4 * i + 3] = x[i].w;
  }
  // the largest magnitude, on the numbers' bits, two at a time
  auto largest = [&] {
    uint32_t two = 0u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) two = __vmaxu2(two, v[i] & 0x7fff7fffu);
    uint32_t most = max(two & 0xffffu, two >> 16);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    return most;
  };
  uint32_t most = largest();
  uint32_t lost[kWords / 4] = {};  // bits of the numbers that are not finite: NaN, and no size
  const bool finite = __all_sync(0xffffffffu, most < 0x7f80u);
  if (!finite) {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((v[i] >> (16 * h) & 0x7fffu) >= 0x7f80u) {
          lost[i / 4] |= 1u << (2 * (i % 4) + h);
          v[i] &= h ? 0xffffu : 0xffff0000u;
        }
    most = largest();
  }
  const int e = scale8_exponent(__uint_as_float(most << 16));
  const float down = exp2_int(-e);
#pragma unroll
  for (int i = 0; i < kWords; i += 2) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w = v[i + j];
      const float2 a = mul2(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)),
                            make_float2(down, down));
      h[j] = e4m3_pair(a.x, a.y);
      const float2 back = e4m3_values(h[j]);
      l[j] = e4m3_pair(a.x - back.x, a.y - back.y);
    }
    hi[i / 2] = h[0] | h[1] << 16;
    lo[i / 2] = l[0] | l[1] << 16;
  }
  if (!finite) {
#pragma unroll
    for (int i = 0; i < kWords / 2; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lost[i / 2] >> (4 * (i & 1) + k) & 1u) hi[i] |= 0x7fu << (8 * k);
  }
  return e;
}

// Part u of eight of a work's row of Q (zeros past the work's rows); tok0: the first row's token.
template <int HD>
__device__ __forceinline__ void fetch_row(const ChunkParams &p, const Work &d, int tok0, int row,
                                          int u, uint4 (&x)[HD / 64]) {
#pragma unroll
  for (int i = 0; i < HD / 64; ++i) x[i] = make_uint4(0, 0, 0, 0);
  if (row >= d.nrow) return;
  const int f = d.row0 - tok0 * p.G + row;
  const int tok = p.G == 1 ? f : static_cast<int>(__umulhi(f, p.g_inv));
  const uint16_t *src = p.q + (d.a + tok0 + tok) * p.qs +
                        static_cast<int64_t>(d.kvh * p.G + f - tok * p.G) * HD + u * (HD / 8);
#pragma unroll
  for (int i = 0; i < HD / 64; ++i) x[i] = reinterpret_cast<const uint4 *>(src)[i];
}

// A work's rows of Q, split by eight warps: eight lanes a row, 32 rows at once and the loads of 128
// in flight.  store(row, u, hi, lo, e) takes a lane's part u of a row.  `loads` works before this
// one had their Q here.
template <class Lay, class Store>
__device__ __forceinline__ bool split_rows(const Cta<Lay> &c, const ChunkParams &p, const Work d,
                                           uint32_t loads, Store store) {
  constexpr int HD = Lay::kHD, kLoads = HD / 64, kAhead = 4;
  const int lane = c.lane, warp = threadIdx.x >> 5, tok0 = d.row0 / p.G, u = lane & 7;
  uint4 x[kAhead][kLoads];
  int row = 4 * warp + (lane >> 3);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch_row<HD>(p, d, tok0, row + 32 * i, u, x[i]);
  // the last scores of the work before are done
  if (loads > 0 && !__all_sync(0xffffffffu, chunk_wait<false>(c.bar(Lay::kQEmpty), (loads - 1) & 1,
                                                              c.abort_flag)))
    return false;
#pragma unroll 1
  for (; row - (lane >> 3) < d.nrow; row += 32) {
    uint32_t hi[2 * kLoads], lo[2 * kLoads];
    const int e = split_q<8 * kLoads>(x[0], hi, lo);
    if (row < d.nrow) store(row, u, hi, lo, e);
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i)
#pragma unroll
      for (int k = 0; k < kLoads; ++k) x[i][k] = x[i + 1][k];
    fetch_row<HD>(p, d, tok0, row + 32 * kAhead, u, x[kAhead - 1]);
  }
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(c.bar(Lay::kQReady));
  return true;
}

// Widens V's tiles to 16 bits: the calling warp's share of the rows, 32.
template <class Lay>
struct Widener {
  static constexpr int kSub = Lay::kHD / 64, kRows = 128 / kWidenTeam;
  uint32_t from[kSub], to[kSub][2];
  int wr, row8[kSub];  // the warp's first row; the lane's of every eight
  __device__ __forceinline__ Widener(int warp, int lane) : wr(kRows * (warp % kWidenTeam)) {
    // A lane's 16 codes of every eight rows (heads of 64: once; 128: twice).  Eight lanes read and
    // write 16 bytes each of different banks: 64: of rows r and r + 1; 128: of r and r ^ 5, since
    // a row's chunks arrive at their number xor r, and leave at twice it xor r.
#pragma unroll
    for (int e = 0; e < kSub; ++e) {
      const int pair = 2 * e + (lane >> 4), c = (lane & 3) + (Lay::kHD == 64 ? 0 : lane >> 1 & 4);
      row8[e] = Lay::kHD == 64 ? lane >> 2 : lane & 4 ? pair ^ 5 : pair;
      const int row = wr + row8[e];
      from[e] = row * Lay::kHD + (Lay::kHD == 64 ? c ^ (row8[e] >> 1) : c ^ row8[e]) * 16;
      for (int i = 0; i < 2; ++i)
        to[e][i] = (c >> 2) * kChunkBytes + row * 128 + (((2 * (c & 3) + i) ^ row8[e]) << 4);
    }
  }
  __device__ __forceinline__ void tile(const Work &d, int t, const TileMeta &tile,
                                       const uint8_t *src, uint8_t *dst) const {
    const uint32_t v0 = tile.v[wr / 16], v1 = tile.v[wr / 16 + kRows / 16 - 1];
    const int kb = (d.t0 + t) * kKT + wr;
    // Rows that no row of the work sees, and those of pages outside the pool, become zeros:
    // a weight of 0 does not silence a NaN.
    const bool whole = kb >= d.lo_min && kb + kRows - 1 <= d.hi_max && (v0 & v1) >> 24;
    const bool far = tile.far != 0;
    // Short loops: in a long run of instructions that other warps' code has driven out of the
    // cache each takes three cycles or four.
    if (whole && !far) {
      uint32_t f = (v0 & 0xffffu) * 0x10001u;
#pragma unroll 1
      for (int i = 0; i < kRows / 8; ++i) {
        if (i == 2) f = (v1 & 0xffffu) * 0x10001u;
        uint4 x[kSub];
#pragma unroll
        for (int e = 0; e < kSub; ++e)
          x[e] = *reinterpret_cast<const uint4 *>(src + from[e] + i * 8 * Lay::kHD);
#pragma unroll
        for (int e = 0; e < kSub; ++e) {
          const uint32_t c[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
          uint32_t r[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            r[2 * j] = mul_f16x2(e4m3_f16x2(c[j]), f);
            r[2 * j + 1] = mul_f16x2(e4m3_f16x2(c[j] >> 16), f);
          }
          uint8_t *o = dst + i * 1024;
          *reinterpret_cast<uint4 *>(o + to[e][0]) = make_uint4(r[0], r[1], r[2], r[3]);
          *reinterpret_cast<uint4 *>(o + to[e][1]) = make_uint4(r[4], r[5], r[6], r[7]);
        }
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < kRows / 8; ++i) {
        const uint32_t v = i < 2 ? v0 : v1, f = (v & 0xffffu) * 0x10001u;
        const float scale = scale8_value(v >> 16 & 255u);
#pragma unroll
        for (int e = 0; e < kSub; ++e) {
          const int key = kb + row8[e] + i * 8;
          const bool keep = v >> 24 && key >= d.lo_min && key <= d.hi_max;
          const uint4 x = *reinterpret_cast<const uint4 *>(src + from[e] + i * 8 * Lay::kHD);
          const uint32_t c[4] = {x.x, x.y, x.z, x.w};
          uint32_t r[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t pair = c[j >> 1] >> (16 * (j & 1));
            if (far) {
              const float2 value = e4m3_values(pair);
              r[j] = ptx::pack_bf16x2(value.x * scale, value.y * scale);
            } else {
              r[j] = mul_f16x2(e4m3_f16x2(pair), f);
            }
            if (!keep) r[j] = 0;
          }
          uint8_t *o = dst + i * 1024;
          *reinterpret_cast<uint4 *>(o + to[e][0]) = make_uint4(r[0], r[1], r[2], r[3]);
          *reinterpret_cast<uint4 *>(o + to[e][1]) = make_uint4(r[4], r[5], r[6], r[7]);
        }
      }
    }
  }
};

// All V tiles of a work, and its scales handed back: `at` tiles and `batches` of scales so far.
template <class Lay, class Early>
__device__ __forceinline__ bool widen_tiles(const Cta<Lay> &c, const Widener<Lay> &widener,
                                            const Work &d, int &at, int &batches, Early early) {
  // A team takes every kTeams-th tile.
  constexpr int kTeams = Lay::kWideners / kWidenTeam;
  const int team = (threadIdx.x >> 5) / kWidenTeam - 12 / kWidenTeam;
  int left = 0;  // batches handed back
  auto hand_back = [&](int to_batch) {
    __syncwarp();
    for (; left < to_batch; ++left)
      if (c.lane == 0) ptx::mbar_arrive(c.bar(Lay::kMEmpty + (batches + left) % kMetaBatches));
  };
  bool ok = true;
#pragma unroll 1
  for (int t = (at ^ team) & (kTeams - 1); t < d.n; t += kTeams) {
    const int b = batches + t / kMetaBatch, v = at + t, raw = v % Lay::kVs, slot = v % Lay::kWides;
    hand_back(t / kMetaBatch);
    ok = (t % kMetaBatch >= kTeams || c.arrived(Lay::kMFull, b, kMetaBatches)) &&
         c.arrived(Lay::kVFull, v, Lay::kVs) && c.reuse(Lay::kWEmpty, v, Lay::kWides);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    early(t);
    widener.tile(d, t, c.scales(b, t), c.sm + Lay::kV + raw * Lay::kTile,
                 c.sm + Lay::kWide + slot * Lay::kTile16);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (c.lane == 0) {
      ptx::mbar_arrive(c.bar(Lay::kWFull + slot));
      ptx::mbar_arrive(c.bar(Lay::kVEmpty + raw));
    }
  }
  at += d.n;
  const int all = (d.n + kMetaBatch - 1) / kMetaBatch;
  hand_back(all);
  batches += all;
  return ok;
}

// Rows of codes, one key of a head each.
inline cudaError_t code_tensor_map(CUtensorMap *m, const void *codes, uint64_t rows, uint32_t hd,
                            uint32_t box_rows) {
  const EncodeTiled encode = encode_tiled_fn();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {hd, rows}, strides[1] = {hd};
  const cuuint32_t box[2] = {hd, box_rows}, each[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(codes), dims, strides, box,
                each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

}  // namespace
}  // namespace dflash
