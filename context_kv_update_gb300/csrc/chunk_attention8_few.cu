// chunk_attention8_few.cu -- attention over a cache held in 8 bits where a work tile has few rows
// (at most 32 of a token and head; single tokens, short drafts) and the key stream is the work.
//
// The kernel of chunk_attention8.cu with the products turned round: the 128 keys of a tile are
// the rows of both results' operands, S^T = K Q^T and O^T = V^T P^T.  The tensor cores then do
// work for N = 16 or 32 rows instead of 128, K's tile is read from shared memory once for
// both parts of Q, and a softmax thread is a key with N scores: 128 threads share what one warp
// did for all keys of a tile (64 single tokens over up to 8192 keys: 219 us that way).
//
// The maximum over keys now runs across threads, so it is only taken when it is needed: a
// thread weighs its scores with the reference it has, and where one exceeds it by 2^8 (a vote of
// the group), or the accumulator's unit changes, the group takes the tile's maxima and scales
// the accumulators (as a rule with its first tile alone).  A row's sum stays in the threads,
// each its keys', until the end.
//
// What bounds it: a key tile takes the chain of warps about 1400 cycles, HBM 1310 (32 KB at 6.8
// TB/s over 152 SMs); where a work ends and the next begins the stream stops for 4 to 6 us,
// and a launch takes 7 us to its first weights.  64 single tokens over up to 8192 keys, 32 heads of
// 128 over 8: 130 us, 4.8 TB/s; one token over 32768: 23.8 us.
#include "chunk8_roles.cuh"

namespace dflash {
namespace {

// 20 warps: as in chunk_attention8.cu, but eight that split Q and widen V, a team of four a tile
// (all eight on each tile: 141 us instead of 133 for 64 single tokens over up to 8192 keys).  640
// threads launch with 96 registers each: 256 x 128 + 128 x 64 + 256 x 80 = 640 x 96.
constexpr int kFewThreads = 640;
// A row's weights carry 2^4 and may exceed its reference by 2^11 more: fp16 holds 2^15, and its
// smallest step is 2^-28 of the reference's weight.
constexpr float kFewLift = 4.f, kFewLag = 11.f;
constexpr int kFewSoftmaxRegs = 128, kFewIssueRegs = 64, kFewWidenRegs = 80;
static_assert(256 * (kFewSoftmaxRegs + kFewWidenRegs) + 128 * kFewIssueRegs <= kFewThreads * 96,
              "");

template <int N>
struct LayoutFew : Bars<3, N == 16 ? 4 : 3, 3, 4> {
  using B = Bars<3, N == 16 ? 4 : 3, 3, 4>;
  static constexpr int kHD = 128, kShift = N == 16 ? 4 : 5, kWideners = 8;
  static constexpr bool kFew = true;
  static constexpr uint32_t kTile = kKT * kHD, kTile16 = 2 * kTile;
  static constexpr uint32_t kK = 2 * N * 128;  // Q: N rows of hi, N of lo
  static constexpr uint32_t kV = kK + B::kKs * kTile;
  static constexpr uint32_t kWide = kV + B::kVs * kTile;
  static constexpr uint32_t kP = kWide + B::kWides * kTile16;  // a group's: 128 keys of N weights
  static constexpr uint32_t kRowState = kP + 2 * kKT * 2 * N;
  static constexpr uint32_t kMeta = kRowState + (2 * N + 2 * N * 11 + 12) * 4;
  static constexpr uint32_t kSortTiles = kMeta + kMetaBatch * kMetaBatches * sizeof(TileMeta);
  static constexpr uint32_t kPlaces = kSortTiles + 4 * kSorted;
  static constexpr uint32_t kWork = kPlaces + kSorted;
  static constexpr uint32_t kAnswer = kWork + 2 * sizeof(Work);
  static constexpr uint32_t kBars = kAnswer + 16;
  static constexpr uint32_t kWords = kBars + 8 * B::kBarCount;
  static constexpr uint32_t kBytes = 1024 + kWords + 16;
  static_assert(kBytes <= kSmemMax, "");
};

// N columns of this warp's lanes.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[N]) {
  if constexpr (N == 32) {
    ptx::tmem_ld32f_sync(taddr, r);
  } else {
    static_assert(N == 16, "");
    uint32_t v[16];
    ptx::tmem_ld16_sync(taddr, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(v[i]);
  }
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7])
      : "r"(taddr)
      : "memory");
}

// The warp's largest; NaN where all are.
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

template <int N, bool kMany>
__global__ void __launch_bounds__(kFewThreads, 1)
    chunk_attn8_few_kernel(const __grid_constant__ CUtensorMap tm,
                           const __grid_constant__ ChunkParams p,
                           const __grid_constant__ Cache8 cache) {
  using Lay = LayoutFew<N>;
  constexpr int HD = 128, kKs = Lay::kKs, kWides = Lay::kWides;
  // S^T of tile t at 64 (t % 4) (hi's scores, then lo's, as one product), O^T of group g at
  // 256 + 128 g
  constexpr uint32_t kColOut = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~static_cast<uintptr_t>(1023));
  const uint32_t sm0 = ptx::smem_u32(sm);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Lay::kWords);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  float *q_scale = reinterpret_cast<float *>(sm + Lay::kRowState);  // of two works: [2][N]
  int *sort_tiles = reinterpret_cast<int *>(sm + Lay::kSortTiles);
  uint8_t *sort_places = sm + Lay::kPlaces;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Cta<Lay> cta = {sm, sm0, lane, abort_flag, reinterpret_cast<Work *>(sm + Lay::kWork),
                        reinterpret_cast<TileMeta *>(sm + Lay::kMeta)};

  if (threadIdx.x == 0) {
    cta.init_bars();
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tm);
  }
  if (warp == 8) {
    ptx::tmem_alloc(ptx::smem_u32(tslot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tslot;
  ptx::griddep_launch();
  ptx::griddep_wait();

  const bool sorted = kMany && p.B > 1 && p.B <= kSorted;
  if (sorted) sort_requests<false>(p, Lay::kShift, sort_tiles, sort_places);

  if (warp >= 12) {
    regs_less<kFewWidenRegs>();
    // ------------------------------------------------ Q's split, V's widening
    const Widener<Lay> widener(warp, lane);
    int at = 0, batches = 0;  // V tiles and batches of scales so far
    uint32_t loads = 0u;
    bool ok = true;
    // Eight lanes a row; rows past the work's are zeros: their scores exceed no reference.
    static_assert(N <= 4 * Lay::kWideners, "");
    const int row = 4 * (warp - 12) + (lane >> 3), u = lane & 7;
    uint4 q[2];
    auto fetch = [&](const Work &d) { fetch_row<HD>(p, d, d.row0 / p.G, row, u, q); };
    auto split = [&](uint32_t w) {
      uint32_t hi[4], lo[4];
      const int e = split_q<16>(q, hi, lo);
      if (row < N) {
        uint8_t *dst = sm + row * 128 + ((u ^ (row & 7)) << 4);
        *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(dst + N * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (u == 0) q_scale[(w & 1) * N + row] = exp2_int(e);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(cta.bar(Lay::kQReady));
      ++loads;
    };
    enum { kNone, kFetched, kSplit } have = kNone;  // this work's Q
    for (uint32_t w = 0; w == 0 || kMany; ++w) {
      const Work d = cta.next_work(w);
      cta.have_read();
      if (d.nrow == 0) break;
      if (d.n == 0 || !ok) continue;
      if (have == kNone) fetch(d);
      if (have != kSplit) {
        ok = loads == 0 || __all_sync(0xffffffffu, chunk_wait<false>(cta.bar(Lay::kQEmpty),
                                                                     (loads - 1) & 1, abort_flag));
        if (!ok) continue;
        split(w);
      }
      have = kNone;
      // The next work's Q between the last tiles, where it is known by then: fetched, and split
      // once the scores of this work are done.  At the end all would wait for it, 2000 cycles.
      auto early = [&](int t) {
        if (!kMany || have == kSplit || t < d.n - 3) return;
        if (have == kNone && cta.passed(Lay::kWorkFull, (w + 1) & 1)) {
          const Work e = cta.next_work(w + 1);
          if (e.n > 0) {
            fetch(e);
            have = kFetched;
          }
        } else if (have == kFetched && cta.passed(Lay::kQEmpty, (loads - 1) & 1)) {
          split(w + 1);
          have = kSplit;
        }
      };
      ok = widen_tiles(cta, widener, d, at, batches, early);
    }
  } else if (warp >= 8) {
    regs_less<kFewIssueRegs>();
    if (warp == 8) {
      load_tiles<kMany, true>(cta, p, tm);
    } else if (warp == 9) {
      schedule<kMany>(cta, p, cache, sorted, sort_tiles, sort_places);
    } else if (warp == 10) {
      load_tiles<kMany, false>(cta, p, tm);
    } else {
      // ---------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc_of(128, 2 * N, 0, false);
      constexpr uint32_t idesc_f16 = idesc_of(128, N, 0, true) | 1u << 15,  // V^T: dims contiguous
          idesc_bf16 = idesc_of(128, N, 1, true) | 1u << 15;
      // warp-uniform copies
      const uint32_t tm0 = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t base = __shfl_sync(0xffffffffu, sm0, 0);
      const uint64_t dq = ptx::desc_kmajor_sw128(base, 0);
      const uint64_t dk = ptx::desc_kmajor_sw128(base + Lay::kK, 0);
      const uint64_t dv = ptx::smem_desc(base + Lay::kWide, kChunkBytes, 1024, ptx::kSwizzle128B);
      // P: keys of 2 N contiguous bytes
      const uint64_t dp = ptx::smem_desc(base + Lay::kP, kChunkBytes, 16 * N,
                                         N == 32 ? kSwizzle64B : kSwizzle32B);
      using At = typename Cta<Lay>::At;
      int at = 0, batches = 0;  // tiles and batches of scales before this work
      Ring<kKs> keys(false);
      Ring<kWides> wide(false);
      uint32_t handed0 = 0u, handed1 = 0u, loads = 0u;  // phases of p_full and q_ready
      bool ok = true;
      auto wait = [&](At a, At b, At c) {
        const bool got = cta.template wait<true>(a, b, c);
        ptx::tc_fence_after();
        return got;
      };
      auto qk = [&](int t) {  // S^T = K (hi, lo)^T, of the work's tile t: K's slot is free then too
        const int buffer = (at + t) & 3;
        const uint64_t a = dk + ((keys.slot * Lay::kTile) >> 4);
#pragma unroll
        for (int ks = 0; ks < HD / 32; ++ks)
          mma_e4m3(tm0 + 64 * buffer, a + (ks * 32 >> 4), dq + (ks * 32 >> 4), idesc_qk,
                   ks > 0 ? 1u : 0u);
        ptx::mma_commit(cta.bar(Lay::kSFull + buffer));
      };
      auto pv = [&](int g, bool first, uint32_t idesc) {  // O_g^T (+)= V^T P^T: P is free then too
        const uint64_t a = dv + ((wide.slot * Lay::kTile16) >> 4);
        const uint64_t b = dp + ((g * kKT * 2 * N) >> 4);
#pragma unroll
        for (int ks = 0; ks < kKT / 16; ++ks)
          ptx::mma_bf16(tm0 + kColOut + 128 * g, a + ((ks * 2048) >> 4), b + ((ks * 32 * N) >> 4),
                        idesc, (!first || ks > 0) ? 1u : 0u);
        ptx::mma_commit(cta.bar(Lay::kWEmpty + wide.slot));
      };
      for (uint32_t w = 0; w == 0 || kMany; ++w) {
        const Work d = cta.next_work(w);
        const int tiles = __shfl_sync(0xffffffffu, d.n, 0);
        if (ok && tiles > 0) {
          const At q = {cta.bar(Lay::kQReady), loads & 1};
          ok = wait(q, q, q);
          ++loads;
        }
        cta.have_read();  // (after the wait: two works' Q later its phase would be the same again)
        if (d.nrow == 0) break;
        if (!ok || tiles == 0) continue;
        // Scores run four tiles ahead of the weights.
        for (int t = 0; ok && t < min(tiles, 4); ++t) {
          const At k = {cta.bar(Lay::kKFull + keys.slot), keys.phase};
          ok = wait(k, k, k);
          if (ok && elect_one()) {
            qk(t);
            if (t == tiles - 1) ptx::mma_commit(cta.bar(Lay::kQEmpty));
          }
          __syncwarp();
          keys.next();
        }
        for (int t = 0; ok && t < tiles; ++t) {
          const bool more = t + 4 < tiles;
          const int b = batches + t / kMetaBatch, g = t & 1;
          const At v = {cta.bar(Lay::kWFull + wide.slot), wide.phase};
          ok = wait(At{cta.bar(Lay::kPFull + g), (g ? handed1 : handed0) & 1}, v,
                    more ? At{cta.bar(Lay::kKFull + keys.slot), keys.phase} : v);
          if (!ok) break;
          if (g) ++handed1; else ++handed0;
          // (the widening warps and the group that handed P over have seen the tile's scales)
          const uint32_t idesc =
              __shfl_sync(0xffffffffu, cta.scales(b, t).far ? idesc_bf16 : idesc_f16, 0);
          if (elect_one()) {
            pv(g, t < 2, idesc);
            if (more) {
              qk(t + 4);
              if (t + 4 == tiles - 1) ptx::mma_commit(cta.bar(Lay::kQEmpty));
            }
            if (t + 2 >= tiles) ptx::mma_commit(cta.bar(Lay::kODone + g));
          }
          __syncwarp();
          wide.next();
          if (more) keys.next();
          if ((t % kMetaBatch == kMetaBatch - 1 || t == tiles - 1) && lane == 0)
            ptx::mbar_arrive(cta.bar(Lay::kMEmpty + b % kMetaBatches));
        }
        at += tiles;
        batches += (tiles + kMetaBatch - 1) / kMetaBatch;
      }
      if (!ok) {
        if (elect_one()) ptx::mma_commit(cta.bar(Lay::kDrain));
        __syncwarp();
        volatile int dummy = 0;
        chunk_wait<false>(cta.bar(Lay::kDrain), 0u, &dummy);
      }
    }
  } else {
    regs_more<kFewSoftmaxRegs>();
    // ------------------------------------------------ softmax groups: a key a thread
    const int g = warp >> 2, w4 = warp & 3;
    const int tid = threadIdx.x & 127;  // TMEM lane = key of the tile, at the end a dim
    const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
    // a group's rows: lo, hi, factor, what is added to the scores (kFewLift - reference, or 0
    // without one), scaling; the warps' maxima, then sums [4]; reference, the last change of what
    // is added; of both groups: units of the accumulators; rows that moved, and without a reference
    float *rows = q_scale + 2 * N + g * 11 * N;
    int *row_lo = reinterpret_cast<int *>(rows), *row_hi = row_lo + N;
    float *row_f = rows + 2 * N, *row_nm = rows + 3 * N, *row_corr = rows + 4 * N,
          *part = rows + 5 * N, *row_m = rows + 9 * N, *row_delta = rows + 10 * N;
    float *units = q_scale + 2 * N + 22 * N;
    uint32_t *marks = reinterpret_cast<uint32_t *>(units) + 4 + 4 * g;
    int batches = 0;
    int at = 0;  // tiles before this work
    uint32_t loads = 0u, outs0 = 0u, outs1 = 0u;  // of q_ready, o_done
    bool ok = true;
    for (uint32_t wk = 0; wk == 0 || kMany; ++wk) {
      const volatile Work &d = cta.shared_work[wk & 1];
      volatile int dummy = 0;
      int nrow = 0, n = 0;
      if (__all_sync(0xffffffffu,
                     chunk_wait<false, 16>(cta.bar(Lay::kWorkFull), wk & 1, &dummy))) {
        nrow = d.nrow;
        n = d.n;
      } else {
        *abort_flag = 1;
      }
      if (n > 0 && ok) {
        ok = __all_sync(0xffffffffu,
                        chunk_wait<false>(cta.bar(Lay::kQReady), loads & 1, abort_flag));
        ++loads;
      }
      cta.have_read();  // (after the wait, as the issuing warp)
      if (nrow == 0) break;
      const int row0 = d.row0, t0 = d.t0;
      // keys that every row sees
      int all_lo, all_hi, x;
      key_range(p, d.c + row0 / p.G, d.kv, &x, &all_hi);
      key_range(p, d.c + (row0 + nrow - 1) / p.G, d.kv, &all_lo, &x);
      if (tid < N) {
        const bool real = tid < nrow;
        int lo = 0, hi = -1;
        if (real) key_range(p, d.c + (row0 + tid) / p.G, d.kv, &lo, &hi);
        row_lo[tid] = lo;
        row_hi[tid] = hi;
        row_f[tid] = real && ok && n > 0 ? q_scale[(wk & 1) * N + tid] * p.scale_log2 : 0.f;
        row_m[tid] = real ? -INFINITY : 0.f;
        row_nm[tid] = 0.f;
      }
      // (A wait that ran out ends the work for the whole group: its warps meet at barriers below,
      // and a barrier has no limit.)
      ok = !ptx::bar_or(2 + g, 128, !ok);

      float l[N];  // this key's share of the rows' sums
#pragma unroll
      for (int r = 0; r < N; ++r) l[r] = 0.f;
      int E = 0, left = 0;
      bool fresh = true;  // some row has no reference yet
      bool lost = false;  // a wait ran out: the group ends together with the next tile's vote
      // The group's product two tiles before, which read P and wrote O.  (A work's first tiles
      // follow a work whose products are all done.)
      auto product_done = [&](int t) {
        return t < 2 || __all_sync(0xffffffffu, cta.arrived(Lay::kWEmpty, at + t - 2, kWides));
      };
      auto hand_back = [&](int to_batch) {
        __syncwarp();
        for (; left < to_batch; ++left)
          if (lane == 0) ptx::mbar_arrive(cta.bar(Lay::kMEmpty + (batches + left) % kMetaBatches));
      };
      for (int t = g; ok && t < n; t += 2) {
        const int b = batches + t / kMetaBatch;
        hand_back(t / kMetaBatch);
        const int buffer = (at + t) & 3;
        const uint32_t tm_s = tmem + 64 * buffer + lane_off;
        bool got = (t % kMetaBatch >= 2 || cta.arrived(Lay::kMFull, b, kMetaBatches)) &&
                   cta.arrived(Lay::kSFull, at + t, 4);
        got = __all_sync(0xffffffffu, got && !lost);
        ptx::tc_fence_after();
        const TileMeta &tile = cta.scales(b, t);
        const int kb = (t0 + t) * kKT, key = kb + tid;
        const float kf = tile.k[tid >> 4];
        const bool dead = (tile.bad >> (tid >> 4)) & 1;
        const bool cut = !(all_lo <= kb && all_hi >= kb + kKT - 1);
        const bool far = tile.far != 0;
        float y[N] = {};
        if (got) {  // scores, in powers of two, relative to the rows' references (if they have one)
          float low[N];
          tmem_ld<N>(tm_s, y);
          tmem_ld<N>(tm_s + N, low);
          const float2 kf2 = make_float2(kf, kf);
#pragma unroll
          for (int r = 0; r < N; r += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(row_f + r);
            const float4 nm = *reinterpret_cast<const float4 *>(row_nm + r);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const int x = r + e;
              const float2 v =
                  fma2(add2(make_float2(y[x], y[x + 1]), make_float2(low[x], low[x + 1])),
                       mul2(e ? make_float2(f.z, f.w) : make_float2(f.x, f.y), kf2),
                       e ? make_float2(nm.z, nm.w) : make_float2(nm.x, nm.y));
              y[x] = v.x;
              y[x + 1] = v.y;
            }
          }
          if (cut) {
#pragma unroll
            for (int r = 0; r < N; ++r)
              if (key < row_lo[r] || key > row_hi[r]) y[r] = -INFINITY;
          }
          if (dead) {
#pragma unroll
            for (int r = 0; r < N; ++r) y[r] = -INFINITY;
          }
        }
        float top = y[0];
#pragma unroll
        for (int r = 1; r < N; ++r) top = fmaxf(top, y[r]);
        const bool need = !got || tile.E != E || top > kFewLag + kFewLift;
        // (A warp whose wait ran out votes too, and all end together: a barrier has no limit.)
        if (fresh || ptx::bar_or(2 + g, 128, need)) {
          if (ptx::bar_or(2 + g, 128, !got)) {
            ok = false;
            break;
          }
          float most = -INFINITY;  // the rows' largest, of the warp's keys
#pragma unroll
          for (int r = 0; r < N; ++r) {
            const float x = warp_max(y[r]);
            if (lane == r) most = x;
          }
          if (lane < N) part[w4 * N + lane] = most;
          ptx::bar_sync(2 + g, 128);
          const float grown = ptx::ex2(static_cast<float>(E - tile.E));
          if (w4 == 0) {  // a thread a row
            const bool row = tid < N;
            float m = 0.f, now = 0.f;
            if (row) {
              const float before = row_nm[tid], x = fmaxf(fmaxf(part[tid], part[N + tid]),
                                                          fmaxf(part[2 * N + tid],
                                                                part[3 * N + tid])) - before;
              m = now = row_m[tid];
              if (m == -INFINITY || x > m + kFewLag) now = fmaxf(m, x);
              const float nm = tid >= nrow || now == -INFINITY ? 0.f : kFewLift - now;
              row_corr[tid] = m == -INFINITY ? 1.f : ptx::ex2(m - now);
              row_delta[tid] = nm - before;
              row_m[tid] = now;
              row_nm[tid] = nm;
            }
            const uint32_t moved = __ballot_sync(0xffffffffu, row && m != -INFINITY && now != m),
                           none = __ballot_sync(0xffffffffu, row && now == -INFINITY);
            if (lane == 0) {
              marks[0] = moved;
              marks[1] = none;
            }
          }
          ptx::bar_sync(2 + g, 128);
          if (t >= 2) {
#pragma unroll
            for (int r = 0; r < N; r += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(row_corr + r);
              l[r] *= f.x;
              l[r + 1] *= f.y;
              l[r + 2] *= f.z;
              l[r + 3] *= f.w;
            }
            lost |= !product_done(t);
            const uint32_t tm_o = tmem + kColOut + 128 * g + lane_off;
#pragma unroll 1
            for (int c = 0; c < N; c += 16) {
              if (!((marks[0] >> c) & 0xffffu) && tile.E == E) continue;
              uint32_t ov[16];
              ptx::tmem_ld16_sync(tm_o + c, ov);
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(row_corr + c + e);
                const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  ov[e + i] = __float_as_uint(__uint_as_float(ov[e + i]) * (fs[i] * grown));
              }
              ptx::tmem_st16(tm_o + c, ov);
            }
            ptx::tmem_wait_st();
          }
          E = tile.E;
          fresh = marks[1] != 0;
#pragma unroll
          for (int r = 0; r < N; r += 4) {
            const float4 dl = *reinterpret_cast<const float4 *>(row_delta + r);
            y[r] += dl.x;
            y[r + 1] += dl.y;
            y[r + 2] += dl.z;
            y[r + 3] += dl.w;
          }
        }
        uint32_t pk[N / 2];
#pragma unroll
        for (int r = 0; r < N; r += 2) {
          y[r] = ptx::ex2(y[r]);
          y[r + 1] = ptx::ex2(y[r + 1]);
          const float2 sum = add2(make_float2(l[r], l[r + 1]), make_float2(y[r], y[r + 1]));
          l[r] = sum.x;
          l[r + 1] = sum.y;
        }
        if (far) {
#pragma unroll
          for (int r = 0; r < N / 2; ++r) pk[r] = ptx::pack_bf16x2(y[2 * r], y[2 * r + 1]);
        } else {
#pragma unroll
          for (int r = 0; r < N / 2; ++r) pk[r] = pack_f16x2(y[2 * r], y[2 * r + 1]);
        }
        lost |= !product_done(t);
        uint8_t *dst = sm + Lay::kP + (g * kKT + tid) * 2 * N;
        const int swap = N == 32 ? tid >> 1 & 3 : tid >> 2 & 1;
#pragma unroll
        for (int u = 0; u < N / 8; ++u)
          *reinterpret_cast<uint4 *>(dst + ((u ^ swap) << 4)) =
              make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0 && !lost) ptx::mbar_arrive(cta.bar(Lay::kPFull + g));
      }
      at += n;
      ok = ok && !lost;
      const int all = (n + kMetaBatch - 1) / kMetaBatch;
      hand_back(all);
      batches += all;
      // ---------------------------------------------- epilogue
      // (while the last products run: the rows' sums, and each group a thread a row for their
      // factors of the two accumulators and where they are written)
      const bool had0 = n > 0, had1 = n > 1;  // groups with products
#pragma unroll
      for (int o = 16, c = N / 2; o > 0; o >>= 1, c >>= 1) {  // halves the rows a lane holds
        if (c > 0) {
#pragma unroll
          for (int r = 0; r < c; ++r) {
            const float give = lane & o ? l[r] : l[r + c], keep = lane & o ? l[r + c] : l[r];
            l[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        } else {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        }
      }
      if (N == 32 || !(lane & 1)) part[w4 * N + (N == 32 ? lane : lane >> 1)] = l[0];
      if (tid == 0) units[g] = exp2_int(min(max(E, -149), 127));
      ok = !ptx::bar_or(1, 256, !ok);
      float *f0 = row_corr, *f1 = row_delta;
      int64_t *row_at = reinterpret_cast<int64_t *>(row_lo);  // (lo and hi are done with)
      if (tid < N) {
        const float *g0 = q_scale + 2 * N, *g1 = g0 + 11 * N;
        const float m0 = ok ? g0[9 * N + tid] : -INFINITY, m1 = ok ? g1[9 * N + tid] : -INFINITY;
        const float m = fmaxf(m0, m1) - kFewLift;  // weights are relative to this
        const float w0 = m0 == -INFINITY ? 0.f : ptx::ex2(m0 - kFewLift - m),
                    w1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - kFewLift - m);
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int i = 5; i < 9; ++i) {
          sum0 += g0[i * N + tid];
          sum1 += g1[i * N + tid];
        }
        const float sum = sum0 * w0 + sum1 * w1;
        // the row saw a key (where all its scores are NaN it has no reference, and a sum of NaN)
        const bool any = tid < nrow && ok && (m != -INFINITY || sum != 0.f);
        const int flat = row0 + tid, tok = flat / p.G, h = d.kvh * p.G + flat - tok * p.G;
        const int64_t orow = static_cast<int64_t>(d.a) + tok;
        int64_t to = orow * p.os + static_cast<int64_t>(h) * HD;
        float gain = 1.f;
        if (p.S == 1) {
          float top = m, den = sum;
          if (p.sinks && any) {
            const float sk = p.sinks[h] * kLog2e;
            top = fmaxf(m, sk);
            den = sum * ptx::ex2(m - top) + ptx::ex2(sk - top);
          }
          gain = any ? ptx::ex2(m - top) / den : 0.f;
        } else {
          const int64_t at = (orow * p.hq + h) * p.S + d.seg;
          to = any ? at * HD : -1;
          // a partial result of about the size of a value, as in chunk_attention8.cu
          const int e = any ? leading_exponent(sum) : 0;
          gain = exp2_int(-e);
          if (tid < nrow && g == 0) {
            p.ws_m[at] = !any ? -INFINITY : m == -INFINITY ? 0.f : m + static_cast<float>(e);
            p.ws_l[at] = any ? sum * gain : 0.f;
          }
        }
        f0[tid] = any ? w0 * units[0] * gain : 0.f;
        f1[tid] = any ? w1 * units[1] * gain : 0.f;
        row_at[tid] = tid < nrow ? to : -1;  // -1: not written
      }
      ptx::bar_sync(2 + g, 128);
      if (ok && had0)
        ok = __all_sync(0xffffffffu,
                        chunk_wait<false>(cta.bar(Lay::kODone), outs0 & 1, abort_flag));
      if (ok && had1)
        ok = __all_sync(0xffffffffu,
                        chunk_wait<false>(cta.bar(Lay::kODone + 1), outs1 & 1, abort_flag));
      ptx::tc_fence_after();
      outs0 += had0;
      outs1 += had1;
      // Half of the rows a group, a dim a thread.
#pragma unroll 1
      for (int c = g * (N / 2); c < min((g + 1) * (N / 2), nrow); c += 8) {
        float o[8] = {};
        if (ok && had0) {
          float v[8];
          tmem_ld8(tmem + kColOut + lane_off + c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = f0[c + e] != 0.f ? v[e] * f0[c + e] : 0.f;
        }
        if (ok && had1) {
          float v[8];
          tmem_ld8(tmem + kColOut + 128 + lane_off + c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += f1[c + e] != 0.f ? v[e] * f1[c + e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t to = row_at[c + e] + tid;
          if (to < tid) continue;
          if (p.S == 1)
            p.out[to] = f32_to_bf16_rn(o[e]);
          else
            p.ws_o[to] = o[e];
        }
      }
      ptx::tc_fence_before();
      ptx::bar_sync(1, 256);  // the accumulators and the rows' state were read
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) raise_status(p.st, DFLASH_DEV_WAIT_TIMEOUT);
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int N, bool kMany>
cudaError_t launch_form(const CUtensorMap &tm, const ChunkParams &p, const Cache8 &cache, dim3 grid,
                        cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit<chunk_attn8_few_kernel<N, kMany>>(kSmemMax);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = LayoutFew<N>::kBytes;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_attn8_few_kernel<N, kMany>, tm, p, cache);
}

template <int N>
cudaError_t launch_rows(const CUtensorMap &tm, const ChunkParams &p, const Cache8 &cache, dim3 grid,
                        cudaStream_t s) {
  return static_cast<int64_t>(grid.x) * grid.z > device_sm_count()
             ? launch_form<N, true>(tm, p, cache, grid, s)
             : launch_form<N, false>(tm, p, cache, grid, s);
}

}  // namespace

cudaError_t launch_attn8_few(int shift, const CUtensorMap &tm, const ChunkParams &p,
                             const Cache8 &cache, dim3 grid, cudaStream_t s) {
  return shift == 4 ? launch_rows<16>(tm, p, cache, grid, s)
                    : launch_rows<32>(tm, p, cache, grid, s);
}

}  // namespace dflash
