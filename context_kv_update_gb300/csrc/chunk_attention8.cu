// chunk_attention8.cu -- attention of a ragged chunk's rows over a cache held in 8 bits, on the
// 5th-generation tensor cores.
//
// The 16-bit kernel's scheme (work tiles of flat rows, two softmax groups, claims of blocks:
// chunk_attention.cu, chunk_work.cuh) over half the bytes.  What is its own:
//
// Scores.  K's codes go to the tensor cores as they are.  A row of Q is scaled by a power of two
// to at most 448 and split into two e4m3 numbers, q = hi + lo: four significant bits each hold a
// bf16 number's eight (what lies below 2^-18 of the row's largest value is lost).  Both multiply
// the same K tile, as one product of twice the depth, at twice the 16-bit rate.  The scales
// come in afterwards, in the softmax: one factor for 16 keys, since blocks have 16 tokens or more.
//
// Values.  P stays in 16 bits (e4m3 could not hold a small weight beside a large one), so V's
// codes are widened to fp16, exactly, by four warps, with the block's scale relative to the
// largest that the work met (2^E, the unit of the accumulator: it grows with E as it does with
// the running maximum).  fp16 holds code * 2^-14 exactly; a tile with a block further below E
// than that, and all tiles after it, are widened to bf16 with the scale itself instead, and E
// is 0: a power of two times four bits is a bf16 number.
//
// Four warpgroups, 128 registers a thread: warps 0-3 and 4-7 split Q, then softmax; 8 loads V; 9
// finds the CTA's next work tile and looks up its scales (four key tiles at a time, a ring of their
// own); 10 loads K; 11 issues every product; 12-15 widen V.  A row's 128 scores are read from
// tensor memory twice, 64 at a time: once for the maximum, once for the weights.
//
// What bounds it: for each group a chain of products (16 of 64 cycles, as many as in 16 bits: half
// the time an operand's, twice the operands), their latency (450), the softmax (1700) and its
// way back (450); two groups fill the tensor cores to about a half.  1024 rows behind 32768 keys,
// 32 heads of 128 over 8: 548 us, 1.02 PFLOP/s of the 558 GFLOP that attention is.  The
// softmax stays in short loops for the instruction cache: unrolled over a row's 128 scores, with no
// other change, 8 drafts of 16 tokens over up to 16384 keys took 90 us, so 74.
#include "chunk8_roles.cuh"

namespace dflash {
namespace {

// Shared memory: Q tiles; rings of K's tiles, of V's, and of V's in 16 bits; factors of Q's rows;
// scales; barriers; the work in hand.
template <int HD, bool kPairs>
struct Layout8 : Bars<HD == 64 ? 6 : kPairs ? 3 : 4, HD == 64 ? 4 : kPairs ? 2 : 3, 2, 2> {
  using B = Bars<HD == 64 ? 6 : kPairs ? 3 : 4, HD == 64 ? 4 : kPairs ? 2 : 3, 2, 2>;
  static constexpr int kHD = HD, kShift = kPairs ? 8 : 7, kWideners = 4;
  static constexpr bool kPair = kPairs, kFew = false;
  static constexpr uint32_t kTile = kKT * HD, kTile16 = 2 * kTile;
  static constexpr uint32_t kK = (kPair ? 2 : 1) * kTile16;
  static constexpr uint32_t kV = kK + B::kKs * kTile;
  static constexpr uint32_t kWide = kV + B::kVs * kTile;
  static constexpr uint32_t kQScale = kWide + B::kWides * kTile16;  // of two works: [2][256]
  static constexpr uint32_t kMeta = kQScale + 2048;
  static constexpr uint32_t kJoin = kMeta + kMetaBatch * kMetaBatches * sizeof(TileMeta);
  static constexpr uint32_t kPlaces = kJoin + 1024;  // m, then l, E, of a split tile [256]
  static constexpr uint32_t kWork = kPlaces + kSorted;
  static constexpr uint32_t kAnswer = kWork + 2 * sizeof(Work);
  static constexpr uint32_t kBars = kAnswer + 16;
  static constexpr uint32_t kWords = kBars + 8 * B::kBarCount;
  static constexpr uint32_t kBytes = 1024 + kWords + 16;
  static_assert(kBytes <= kSmemMax, "");
};

template <int HD, bool kPair, bool kMany>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn8_kernel(const __grid_constant__ CUtensorMap tm,
                       const __grid_constant__ ChunkParams p,
                       const __grid_constant__ Cache8 cache) {
  using Lay = Layout8<HD, kPair>;
  constexpr int kKs = Lay::kKs, kWides = Lay::kWides;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~static_cast<uintptr_t>(1023));
  const uint32_t sm0 = ptx::smem_u32(sm);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Lay::kWords);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  float *q_scale = reinterpret_cast<float *>(sm + Lay::kQScale);
  int *sort_tiles = reinterpret_cast<int *>(sm + Lay::kJoin);  // used before the works' joins
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
  if (sorted) sort_requests<kPair>(p, Lay::kShift, sort_tiles, sort_places);

  if (warp >= 12) {
    regs_less<kWidenRegs>();
    // ------------------------------------------------ V's widening
    const Widener<Lay> widener(warp, lane);
    int at = 0, batches = 0;  // V tiles and batches of scales so far
    bool ok = true;
    for (uint32_t w = 0; w == 0 || kMany; ++w) {
      const Work d = cta.next_work(w);
      cta.have_read();
      if (d.nrow == 0) break;
      if (d.n > 0 && ok) ok = widen_tiles(cta, widener, d, at, batches, [](int) {});
    }
  } else if (warp >= 8) {
    regs_less<kIssueRegs>();
    if (warp == 8) {
      load_tiles<kMany, true>(cta, p, tm);
    } else if (warp == 9) {
      schedule<kMany>(cta, p, cache, sorted, sort_tiles, sort_places);
    } else if (warp == 10) {
      load_tiles<kMany, false>(cta, p, tm);
    } else {
    // ------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_qk = idesc_of(128, kKT, 0, false);
    constexpr uint32_t idesc_f16 = idesc_of(128, HD, 0, true),
                       idesc_bf16 = idesc_of(128, HD, 1, true);
    // warp-uniform copies
    const uint32_t tm0 = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t base = __shfl_sync(0xffffffffu, sm0, 0);
    const uint64_t dq = ptx::desc_kmajor_sw128(base, 0);
    const uint64_t dk = ptx::smem_desc(base + Lay::kK, 16, 8 * HD,
                                       HD == 64 ? kSwizzle64B : ptx::kSwizzle128B);
    const uint64_t dv = ptx::smem_desc(base + Lay::kWide, kChunkBytes, 1024, ptx::kSwizzle128B);
    using At = typename Cta<Lay>::At;
    int at_k = 0, at_v = 0, batches = 0;  // of K tiles, V tiles, batches of scales
    uint32_t handed0 = 0u, handed1 = 0u, loads = 0u;  // phases of p_full and q_ready
    bool ok = true, pairs = false;
    auto slot = [&](int first, int at, int n) { return cta.full(first, at, n); };
    auto wait = [&](At a, At b, At e) {
      const bool got = cta.template wait<true>(a, b, e);
      ptx::tc_fence_after();
      return got;
    };
    auto qk = [&](int g, int at) {  // S_g = (hi + lo) K^T
      const uint64_t a = dq + (((pairs ? g : 0) * Lay::kTile16) >> 4);
      const uint64_t b = dk + (((at % kKs) * Lay::kTile) >> 4);
#pragma unroll
      for (int ks = 0; ks < 2 * HD / 32; ++ks) {
        const uint32_t oa = HD == 128 ? (ks >> 2) * kChunkBytes + (ks & 3) * 32 : ks * 32;
        const uint32_t ob = ks % (HD / 32) * 32;
        mma_e4m3(tm0 + 128 * g, a + (oa >> 4), b + (ob >> 4), idesc_qk, ks > 0 ? 1u : 0u);
      }
      ptx::mma_commit(cta.bar(Lay::kSFull + g));
    };
    auto pv = [&](int g, int at, bool first, uint32_t idesc) {  // O_g (+)= P V
      const uint64_t b = dv + (((at % kWides) * Lay::kTile16) >> 4);
#pragma unroll
      for (int ks = 0; ks < kKT / 16; ++ks)
        ptx::mma_bf16_ts(tm0 + kColO + HD * g, tm0 + 128 * g + ks * 8, b + ((ks * 2048) >> 4),
                         idesc, (!first || ks > 0) ? 1u : 0u);
    };
    for (uint32_t w = 0; w == 0 || kMany; ++w) {
      const Work d = cta.next_work(w);
      cta.have_read();
      if (d.nrow == 0) break;
      const int tiles = __shfl_sync(0xffffffffu, d.n, 0);
      if (!ok || tiles == 0) continue;
      pairs = kPair && __shfl_sync(0xffffffffu, d.nrow, 0) > 128;
      const int step = pairs ? 1 : 2;
      ok = wait(At{cta.bar(Lay::kQReady), loads & 1}, slot(Lay::kKFull, at_k, kKs),
                slot(Lay::kKFull, !pairs && tiles > 1 ? at_k + 1 : at_k, kKs));
      ++loads;
      if (ok && elect_one()) {
        qk(0, at_k);
        if (pairs) {
          qk(1, at_k);
          ptx::mma_commit(cta.bar(Lay::kKEmpty + at_k % kKs));
        } else {
          ptx::mma_commit(cta.bar(Lay::kKEmpty + at_k % kKs));
          if (tiles > 1) {
            qk(1, at_k + 1);
            ptx::mma_commit(cta.bar(Lay::kKEmpty + (at_k + 1) % kKs));
          }
        }
        if (tiles <= step) ptx::mma_commit(cta.bar(Lay::kQEmpty));
      }
      __syncwarp();
      int left = 0;
      for (int t = 0; ok && t < tiles; ++t) {
        const bool more = t + step < tiles;
        const int b = batches + t / kMetaBatch;
        uint32_t idesc = 0;
        for (int i = 0; ok && i < (pairs ? 2 : 1); ++i) {
          const int g = pairs ? i : t & 1;
          const At v = slot(Lay::kWFull, at_v + t, kWides);
          ok = wait(At{cta.bar(Lay::kPFull + g), (g ? handed1 : handed0) & 1}, v,
                    more ? slot(Lay::kKFull, at_k + t + step, kKs) : v);
          if (!ok) break;
          if (g) ++handed1; else ++handed0;
          // (the widening warps and the group that handed P over have seen the tile's scales)
          if (i == 0)
            idesc = __shfl_sync(
                0xffffffffu,
                cta.scales(b, t).far ? idesc_bf16 : idesc_f16,
                0);
          if (elect_one()) {
            pv(g, at_v + t, t < step, idesc);
            if (!pairs || i == 1) ptx::mma_commit(cta.bar(Lay::kWEmpty + (at_v + t) % kWides));
            if (more) qk(g, at_k + t + step);
            if (more && (!pairs || i == 1)) {
              ptx::mma_commit(cta.bar(Lay::kKEmpty + (at_k + t + step) % kKs));
              if (t + step == tiles - 1) ptx::mma_commit(cta.bar(Lay::kQEmpty));
            }
            if (!more) ptx::mma_commit(cta.bar(Lay::kODone + g));
          }
          __syncwarp();
        }
        if (t % kMetaBatch == kMetaBatch - 1 || t == tiles - 1) {
          if (lane == 0 && ok) ptx::mbar_arrive(cta.bar(Lay::kMEmpty + b % kMetaBatches));
          ++left;
        }
      }
      at_k += tiles;
      at_v += tiles;
      batches += left;
    }
    if (!ok) {
      if (elect_one()) ptx::mma_commit(cta.bar(Lay::kDrain));
      __syncwarp();
      volatile int dummy = 0;
      chunk_wait<false>(cta.bar(Lay::kDrain), 0u, &dummy);
    }
    }
  } else {
    regs_more<kSoftmaxRegs>();
    // ------------------------------------------------ softmax groups, which split Q first
    const int g = warp >> 2;
    const int tid = threadIdx.x & 127;  // TMEM lane = row of the group's tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + 128 * g + lane_off, tm_o = tmem + kColO + HD * g + lane_off;
    float *join = reinterpret_cast<float *>(sm + Lay::kJoin);
    int batches = 0;
    uint32_t loads = 0u, scores = 0u, outs0 = 0u, outs1 = 0u;  // of q_ready, s_full, o_done
    bool ok = true;
    for (uint32_t wk = 0; wk == 0 || kMany; ++wk) {
      // its fields are read again where they are needed: this slot is not written before
      // the next work is read
      const volatile Work &d = cta.shared_work[wk & 1];
      volatile int dummy = 0;
      int nrow = 0, n = 0;
      if (__all_sync(0xffffffffu, chunk_wait<false, 16>(cta.bar(Lay::kWorkFull), wk & 1, &dummy))) {
        nrow = d.nrow;
        n = d.n;
      } else {
        *abort_flag = 1;
      }
      cta.have_read();
      if (nrow == 0) break;
      const int lo_min = d.lo_min, hi_max = d.hi_max, t0 = d.t0;
      const bool split = !kPair || nrow <= 128;

      // this thread's row and the keys it sees
      const int rt = (split ? 0 : 128 * g) + tid;
      const bool real = rt < nrow;
      int lo = 0, hi = INT_MAX;  // no row: nothing to mask, its P may hold anything
      if (real) key_range(p, d.c + (d.row0 + rt) / p.G, d.kv, &lo, &hi);
      const bool active = (split ? 0 : 128 * g) + (warp & 3) * 32 < nrow;  // the warp holds rows
      float row_scale = 0.f;  // of the row's scores
      if (n > 0 && ok) {
        ok = split_rows(cta, p, cta.shared_work[wk & 1], loads,
                        [&](int row, int u, const uint32_t *hi, const uint32_t *lo, int e) {
          // HD 128: hi and lo in the two halves of 64 columns; 64: side by side in one
          uint8_t *dst = sm + (row >> 7) * Lay::kTile16 + (row & 127) * 128;
          if constexpr (HD == 128) {
            const int at16 = (u ^ (row & 7)) << 4;
            *reinterpret_cast<uint4 *>(dst + at16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(dst + kChunkBytes + at16) =
                make_uint4(lo[0], lo[1], lo[2], lo[3]);
          } else {
            const int half = (u & 1) * 8;
            *reinterpret_cast<uint2 *>(dst + (((u >> 1) ^ (row & 7)) << 4) + half) =
                make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(dst + (((4 + (u >> 1)) ^ (row & 7)) << 4) + half) =
                make_uint2(lo[0], lo[1]);
          }
          if (u == 0) q_scale[(wk & 1) * 256 + row] = exp2_int(e);
        });
        if (ok)
          ok = __all_sync(0xffffffffu,
                          chunk_wait<false>(cta.bar(Lay::kQReady), loads & 1, abort_flag));
        ++loads;
        if (ok && real) row_scale = q_scale[(wk & 1) * 256 + rt] * p.scale_log2;
      }

      float m_ref = -INFINITY, l = 0.f;
      int E = 0, left = 0;
      auto hand_back = [&](int to_batch) {
        __syncwarp();
        for (; left < to_batch; ++left)
          if (lane == 0) ptx::mbar_arrive(cta.bar(Lay::kMEmpty + (batches + left) % kMetaBatches));
      };
      const int step = split ? 2 : 1;
      for (int t = split ? g : 0; ok && t < n; t += step) {
        const int b = batches + t / kMetaBatch;
        hand_back(t / kMetaBatch);
        const typename Cta<Lay>::At s_full = {cta.bar(Lay::kSFull + g), scores & 1};
        ok = (t % kMetaBatch >= step || cta.arrived(Lay::kMFull, b, kMetaBatches)) &&
                   chunk_wait<false>(s_full.bar, s_full.phase, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++scores;
        ptx::tc_fence_after();
        if (!active) {  // its rows of P may hold anything: they reach no other row
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(cta.bar(Lay::kPFull + g));
          continue;
        }
        const TileMeta &tile = cta.scales(b, t);
        const int kb = (t0 + t) * kKT;
        const uint32_t bad = tile.bad;
        const bool cut = !(lo <= kb && hi >= kb + kKT - 1);  // (asked of each 64 keys: 2% slower)
        // Two passes of 64 scores a step, read from tensor memory each.  (Short loops: the tile's
        // 600 instructions, unrolled over the row, come at three cycles each, from a cache that
        // they share with the other warps' code.  32 a step: 1024 rows behind 32768 keys 591 us
        // instead of 548, for the loads' latency.)
        // the factor of 16 keys' scores; never 0 or NaN, which would make a masked one NaN
        auto factor = [&](int i) { return fmaxf(row_scale * tile.k[i], 0x1p-126f); };
        float tmax = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          float s[64];
          ptx::tmem_ld64f_sync(tm_s + 64 * c, s);
          // what the row does not see: -inf, for both passes
          if (__any_sync(0xffffffffu, cut) || bad) {
            if (bad >> 8) {  // K's scale is NaN
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (bad >> (8 + 4 * c + e / 16) & 1u) s[e] = NAN;
            }
#pragma unroll
            for (int h = 0; h < 64; h += 32) {
              const int k0 = kb + 64 * c + h, from = max(lo - k0, 0), to = min(hi - k0, 31);
              uint32_t vis = from <= to ? (0xffffffffu >> (31 - to + from)) << from : 0u;
              const uint32_t groups = bad >> (4 * c + h / 16);  // bits 0 and 1: the 32 keys'
              if (groups & 1u) vis &= 0xffff0000u;
              if (groups & 2u) vis &= 0x0000ffffu;
              uint32_t w[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if (!(vis >> e & 1u)) s[h + e] = -INFINITY;
                w[e] = __float_as_uint(s[h + e]);
              }
              tmem_st32(tm_s + 64 * c + h, w);
            }
            ptx::tmem_wait_st();
          }
#pragma unroll
          for (int i = 0; i < 64; i += 16) {
            float a = fmaxf(s[i], s[i + 1]), a2 = fmaxf(s[i + 2], s[i + 3]);
#pragma unroll
            for (int e = 4; e < 16; e += 4) {
              a = fmaxf(fmaxf(a, s[i + e]), s[i + e + 1]);
              a2 = fmaxf(fmaxf(a2, s[i + e + 2]), s[i + e + 3]);
            }
            tmax = fmaxf(tmax, fmaxf(a, a2) * factor(4 * c + i / 16));
          }
        }
        float corr = 1.f;
        if (m_ref == -INFINITY) {
          m_ref = tmax;
        } else if (tmax > m_ref + 8.f) {
          corr = ptx::ex2(m_ref - tmax);
          m_ref = tmax;
        }
        // the group's previous product completed before this S did
        if (__any_sync(0xffffffffu, corr != 1.f || tile.E != E)) {
          const float corr_o = corr * ptx::ex2(static_cast<float>(E - tile.E));
          E = tile.E;
          l *= corr;
#pragma unroll 1
          for (int c = 0; c < HD && t >= step; c += 16) {
            uint32_t ov[16];
            ptx::tmem_ld16_sync(tm_o + c, ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr_o);
            ptx::tmem_st16(tm_o + c, ov);
          }
        }
        // nothing seen yet: weights 2^-inf
        const float nm = m_ref == -INFINITY ? 0.f : kLift - m_ref;
        const bool far = tile.far != 0;
        const float2 nm2 = make_float2(nm, nm);
        float2 sum[2] = {};
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          float s[64];
          ptx::tmem_ld64f_sync(tm_s + 64 * c, s);
          uint32_t pk[32];
#pragma unroll
          for (int x = 0; x < 64; x += 2) {
            const float f = factor(4 * c + x / 16);
            float2 w = fma2(make_float2(s[x], s[x + 1]), make_float2(f, f), nm2);
            w.x = ptx::ex2(w.x);
            w.y = ptx::ex2(w.y);
            sum[x / 2 & 1] = add2(sum[x / 2 & 1], w);
            s[x] = w.x;
            s[x + 1] = w.y;
          }
          if (far) {
#pragma unroll
            for (int e = 0; e < 32; ++e) pk[e] = ptx::pack_bf16x2(s[2 * e], s[2 * e + 1]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) pk[e] = pack_f16x2(s[2 * e], s[2 * e + 1]);
          }
          tmem_st32(tm_s + 32 * c, pk);
        }
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(cta.bar(Lay::kPFull + g));
      }
      const int all = (n + kMetaBatch - 1) / kMetaBatch;
      hand_back(all);
      batches += all;
      // ---------------------------------------------- epilogue
      const bool had0 = n > 0, had1 = split ? n > 1 : n > 0;  // groups with products
      if (ok && (g ? had1 : had0)) {
        ok = __all_sync(0xffffffffu, chunk_wait<false>(cta.bar(Lay::kODone + g),
                                                       (g ? outs1 : outs0) & 1, abort_flag));
        ptx::tc_fence_after();
      }
      if (split && ok && (g ? had0 : had1)) {  // the other group's products
        ok = __all_sync(0xffffffffu, chunk_wait<false>(cta.bar(Lay::kODone + (g ^ 1)),
                                                       (g ? outs0 : outs1) & 1, abort_flag));
        ptx::tc_fence_after();
      }
      outs0 += had0;
      outs1 += had1;
      // the row's state over both groups, and this thread's share of its dims
      const int dims = split ? HD / 2 : HD, d0 = split ? g * (HD / 2) : 0;
      if (m_ref != -INFINITY) m_ref -= kLift;  // weights are relative to this
      float m = ok ? m_ref : -INFINITY, own = 1.f, other = 0.f;
      const float unit = exp2_int(min(max(E, -149), 127));  // of the accumulator
      if (split && n > 0) {
        // Both groups hold the row in the same TMEM lane: the states go through shared
        // memory, the other accumulator is read where it is.
        join[g * 128 + tid] = m;
        const bool broken = ptx::bar_or(1, 256, !ok);
        const float m2 = join[(g ^ 1) * 128 + tid];
        ptx::bar_sync(1, 256);
        join[g * 128 + tid] = l;
        ptx::bar_sync(1, 256);
        const float l2 = join[(g ^ 1) * 128 + tid];
        ptx::bar_sync(1, 256);
        join[g * 128 + tid] = unit;
        ptx::bar_sync(1, 256);
        const float unit2 = join[(g ^ 1) * 128 + tid];
        ok = ok && !broken;
        m = broken ? -INFINITY : fmaxf(m_ref, m2);
        own = broken || m_ref == -INFINITY ? 0.f : ptx::ex2(m_ref - m);
        other = broken || m2 == -INFINITY ? 0.f : ptx::ex2(m2 - m);
        l = l * own + l2 * other;
        other *= unit2;
      }
      own *= unit;
      // the row saw a key (where all its scores are NaN it has no reference, and a sum of NaN)
      const bool any = real && ok && (m != -INFINITY || l != 0.f);
      const int flat = d.row0 + (real ? rt : 0), tok = flat / p.G, seg = d.seg;
      const int h = d.kvh * p.G + flat - tok * p.G;
      const int64_t orow = static_cast<int64_t>(d.a) + tok;
      float gain = 1.f;
      if (p.S == 1) {
        float top = m, den = l;
        if (p.sinks && any) {
          const float sk = p.sinks[h] * kLog2e;
          top = fmaxf(m, sk);
          den = l * ptx::ex2(m - top) + ptx::ex2(sk - top);
        }
        gain = any ? ptx::ex2(m - top) / den : 0.f;
      } else if (any) {
        // A partial result is about the size of a value: a sum of weights times the largest that
        // the cache holds, 2^127, would not be an fp32 number.
        const int e = leading_exponent(l);
        m = m == -INFINITY ? 0.f : m + static_cast<float>(e);
        gain = exp2_int(-e);
        l *= gain;
      }
      if (p.S > 1 && real && (!split || g == 0)) {
        const int64_t w = (orow * p.hq + h) * p.S + seg;
        p.ws_m[w] = any ? m : -INFINITY;
        p.ws_l[w] = any ? l : 0.f;
      }
      own *= gain;
      other *= gain;
      const bool has = ok && (g ? had1 : had0);  // this group's accumulator was written
#pragma unroll
      for (int c = 0; c < HD; c += 32) {
        if (c >= dims || !active) break;
        float o[32];
        if (has) {  // warp-uniform: tensor memory loads take the whole warp
          ptx::tmem_ld32f_sync(tm_o + d0 + c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = own != 0.f ? o[e] * own : 0.f;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (split && ok && (g ? had0 : had1)) {
          float x[32];
          ptx::tmem_ld32f_sync(tmem + kColO + HD * (g ^ 1) + lane_off + d0 + c, x);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] += other != 0.f ? x[e] * other : 0.f;
        }
        if (!real) continue;
        if (p.S == 1) {
          uint16_t *dst = p.out + orow * p.os + static_cast<int64_t>(h) * HD + d0 + c;
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = ptx::pack_bf16x2(o[2 * e], o[2 * e + 1]);
          if (p.wide_out) {  // whole sectors: half the write requests
            store_32b(dst, w);
            store_32b(dst + 16, w + 8);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<uint4 *>(dst)[e] =
                  make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        } else if (any) {
          float *dst = p.ws_o + ((orow * p.hq + h) * p.S + seg) * HD + d0 + c;
          if ((reinterpret_cast<uintptr_t>(p.ws_o) & 31) == 0) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e]);
#pragma unroll
            for (int e = 0; e < 32; e += 8) store_32b(dst + e, w + e);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(dst + e) =
                  make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      }
      ptx::tc_fence_before();
      if (split && n > 0) ptx::bar_sync(1, 256);  // the other group's accumulator was read
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

template <int HD, bool kPair, bool kMany>
cudaError_t launch_form(const CUtensorMap &tm, const ChunkParams &p, const Cache8 &cache, dim3 grid,
                        cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit<chunk_attn8_kernel<HD, kPair, kMany>>(kSmemMax);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout8<HD, kPair>::kBytes;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_attn8_kernel<HD, kPair, kMany>, tm, p, cache);
}

template <int HD>
cudaError_t launch_main(bool pair, const CUtensorMap &tm, const ChunkParams &p,
                        const Cache8 &cache, dim3 grid, cudaStream_t s) {
  const bool many = static_cast<int64_t>(grid.x) * grid.z > device_sm_count();
  if (pair)
    return many ? launch_form<HD, true, true>(tm, p, cache, grid, s)
                : launch_form<HD, true, false>(tm, p, cache, grid, s);
  return many ? launch_form<HD, false, true>(tm, p, cache, grid, s)
              : launch_form<HD, false, false>(tm, p, cache, grid, s);
}

// Rows of a work tile, as a power of two.  Heads of 128 whose mean request has at most 32 rows take
// the kernel of chunk_attention8_few.cu: 64 single tokens of 4 rows a head over up to 8192 keys
// take 130 us there, 191 here with a row a softmax thread; 32 drafts of 32 rows over as many 93 and
// 103; 8 drafts of 64 rows 120 there (two works of 32 rows read the same keys), 73 here.
// The mean is all that the host knows: a long request among short ones goes there as well, in as many
// works of 32 rows, each over all its keys (63 single tokens and a piece of 400 tokens behind
// 32768 keys: 774 us there, 376 here; the piece at the start of its prompt 185 and 190).
// Heads of 64 have no such kernel: 64 single tokens take 176 us, in 16 bits 171.
int tile_shift(const dflash_geom &g, int B, int n_rows) {
  const int64_t rows = static_cast<int64_t>(n_rows) * (g.hq / g.nkv);
  if (g.head_dim == 128 && rows <= 32LL * B)
    return rows <= (1LL << kLeastFewShift) * B ? kLeastFewShift : kMostFewShift;
  return pair_form(g, B, n_rows) ? 8 : 7;
}

}  // namespace

int chunk_attention8_num_segments(const dflash_geom &g, int B, int n_rows, int window) {
  // Work tiles as if the requests had a mean's rows each (the most there can be is one more a
  // request: 16 requests of 16 tokens over up to 8192 keys took 102 us uncut for it, 83 in two).
  // Where a work begins and ends the key stream stops: ten to twelve tiles' time.  (Costs of heads
  // of 128; those of 64 take them as they are.)
  const int shift = tile_shift(g, B, n_rows);
  const int64_t flat = static_cast<int64_t>(n_rows) * (g.hq / g.nkv);
  const int64_t per = static_cast<int64_t>(B) << shift;
  const int64_t tiles = (flat + per - 1) / per * B;
  return shift <= kMostFewShift ? segments_of(g, B, n_rows, window, shift, tiles, 10.0, 2.0, 0.7)
                                : segments_of(g, B, n_rows, window, shift, tiles, 12.0, 2.0, 1.0);
}

size_t chunk_attention8_workspace_bytes(const dflash_geom &g, int B, int n_rows, int S) {
  if (B < 1 || n_rows < 1) return 0;
  return workspace_of(g, n_rows, S > 0 ? S : chunk_attention8_num_segments(g, B, n_rows, 0));
}

cudaError_t launch_chunk_attention8(const dflash_geom &g, int B, int layer, int n_rows,
                                    const void *q, int64_t q_stride, const dflash_cache8 &cache,
                                    const int32_t *tbl, const int32_t *cu, const int32_t *ctx,
                                    const int32_t *kv, int32_t window, const float *sinks,
                                    float scale, int mask_mode, int S, void *ws, void *out,
                                    int64_t out_stride, int32_t *st, cudaStream_t s) {
  const int shift = tile_shift(g, B, n_rows);
  const ChunkParams p = chunk_params(g, shift, B, layer, n_rows, q, q_stride, tbl, cu, ctx, kv,
                                     window, sinks, scale, mask_mode, S, ws, out, out_stride, st);
  CUtensorMap tm;
  const uint64_t rows = static_cast<uint64_t>(g.num_layers) * g.num_pool_pages * 2 * g.nkv *
                        static_cast<uint64_t>(g.page_size);
  cudaError_t e = code_tensor_map(&tm, cache.codes, rows, g.head_dim, p.box_rows);
  if (e != cudaSuccess) return e;
  const Cache8 c = cache8_of(g, cache, layer);
  const dim3 grid(static_cast<unsigned>(chunk_tiles(g, B, n_rows, shift) * g.nkv), 1, S);
  e = shift <= kMostFewShift ? launch_attn8_few(shift, tm, p, c, grid, s)
      : g.head_dim == 64     ? launch_main<64>(shift == 8, tm, p, c, grid, s)
                             : launch_main<128>(shift == 8, tm, p, c, grid, s);
  return e != cudaSuccess || S == 1 ? e : launch_merge(g, p, s);
}

}  // namespace dflash
