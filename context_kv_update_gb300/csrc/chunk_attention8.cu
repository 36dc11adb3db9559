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
// Four warpgroups, 128 registers a thread: warps 0-3 and 4-7 softmax, 8 finds the CTA's next work
// tile, 9 looks up scales (four key tiles at a time, a ring of its own), 10 issues the loads of K
// and V, 11 every product, 12-15 split Q and widen V.  A row's 128 scores are read from tensor
// memory twice, 64 at a time: once for the maximum, once for the weights.
#include "cache8.cuh"
#include "chunk_work.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 512;
// Registers: 512 threads launch with 128 each; the softmax groups take more (a row's 128 scores),
// the others give them up: 2 x 128 x 184 + 128 x 64 + 128 x 80 = 65536.
constexpr int kSoftmaxRegs = 184, kIssueRegs = 64, kWidenRegs = 80;
static_assert(256 * kSoftmaxRegs + 128 * (kIssueRegs + kWidenRegs) <= kThreads * 128, "");
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
  int bad;        // bits of the 16 keys each that are visible on a page outside the pool
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
constexpr uint32_t kSwizzle64B = 4;

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

// 128 columns in two loads (the compiler takes none of more registers than a thread launches
// with), one wait.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&r)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, %80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, %96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%129];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31]), "=f"(r[32]), "=f"(r[33]), "=f"(r[34]), "=f"(r[35]), "=f"(r[36]), "=f"(r[37]), "=f"(r[38]), "=f"(r[39]), "=f"(r[40]), "=f"(r[41]), "=f"(r[42]), "=f"(r[43]), "=f"(r[44]), "=f"(r[45]), "=f"(r[46]), "=f"(r[47]), "=f"(r[48]), "=f"(r[49]), "=f"(r[50]), "=f"(r[51]), "=f"(r[52]), "=f"(r[53]), "=f"(r[54]), "=f"(r[55]), "=f"(r[56]), "=f"(r[57]), "=f"(r[58]), "=f"(r[59]), "=f"(r[60]), "=f"(r[61]), "=f"(r[62]), "=f"(r[63]), "=f"(r[64]), "=f"(r[65]), "=f"(r[66]), "=f"(r[67]), "=f"(r[68]), "=f"(r[69]), "=f"(r[70]), "=f"(r[71]), "=f"(r[72]), "=f"(r[73]), "=f"(r[74]), "=f"(r[75]), "=f"(r[76]), "=f"(r[77]), "=f"(r[78]), "=f"(r[79]), "=f"(r[80]), "=f"(r[81]), "=f"(r[82]), "=f"(r[83]), "=f"(r[84]), "=f"(r[85]), "=f"(r[86]), "=f"(r[87]), "=f"(r[88]), "=f"(r[89]), "=f"(r[90]), "=f"(r[91]), "=f"(r[92]), "=f"(r[93]), "=f"(r[94]), "=f"(r[95]), "=f"(r[96]), "=f"(r[97]), "=f"(r[98]), "=f"(r[99]), "=f"(r[100]), "=f"(r[101]), "=f"(r[102]), "=f"(r[103]), "=f"(r[104]), "=f"(r[105]), "=f"(r[106]), "=f"(r[107]), "=f"(r[108]), "=f"(r[109]), "=f"(r[110]), "=f"(r[111]), "=f"(r[112]), "=f"(r[113]), "=f"(r[114]), "=f"(r[115]), "=f"(r[116]), "=f"(r[117]), "=f"(r[118]), "=f"(r[119]), "=f"(r[120]), "=f"(r[121]), "=f"(r[122]), "=f"(r[123]), "=f"(r[124]), "=f"(r[125]), "=f"(r[126]), "=f"(r[127])
      : "r"(taddr), "r"(taddr + 64)
      : "memory");
}
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Shared memory: Q tiles; rings of K's tiles, of V's, and of V's in 16 bits; factors of Q's rows;
// scales; barriers; the work in hand.
template <int HD, bool kPair>
struct Layout8 {
  static constexpr uint32_t kTile = kKT * HD, kTile16 = 2 * kTile;
  static constexpr int kKs = HD == 64 ? 6 : kPair ? 3 : 4, kVs = HD == 64 ? 4 : kPair ? 2 : 3;
  static constexpr int kWides = 2;
  static constexpr uint32_t kK = (kPair ? 2 : 1) * kTile16;
  static constexpr uint32_t kV = kK + kKs * kTile;
  static constexpr uint32_t kWide = kV + kVs * kTile;
  static constexpr uint32_t kQScale = kWide + kWides * kTile16;  // of two works: [2][256]
  static constexpr uint32_t kMeta = kQScale + 2048;
  static constexpr uint32_t kJoin = kMeta + kMetaBatch * kMetaBatches * sizeof(TileMeta);
  static constexpr uint32_t kPlaces = kJoin + 1024;  // m, then l, E, of a split tile [256]
  static constexpr uint32_t kWork = kPlaces + kSorted;
  static constexpr uint32_t kAnswer = kWork + 2 * sizeof(Work);
  static constexpr uint32_t kBars = kAnswer + 16;
  static constexpr int kBarCount = 2 * (kKs + kVs + kWides + kMetaBatches) + 12;
  static constexpr uint32_t kWords = kBars + 8 * kBarCount;
  static constexpr uint32_t kBytes = 1024 + kWords + 16;
  static_assert(kBytes <= kSmemMax, "");
};

template <int HD, bool kPair, bool kMany>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn8_kernel(const __grid_constant__ CUtensorMap tm,
                       const __grid_constant__ ChunkParams p, const __grid_constant__ Cache8 cache) {
  constexpr int kShift = kPair ? 8 : 7;
  using Lay = Layout8<HD, kPair>;
  constexpr int kKs = Lay::kKs, kVs = Lay::kVs, kWides = Lay::kWides;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~static_cast<uintptr_t>(1023));
  const uint32_t sm0 = ptx::smem_u32(sm);
  // barriers, by their place
  constexpr int kKFull = 0, kKEmpty = kKFull + kKs, kVFull = kKEmpty + kKs,
                kVEmpty = kVFull + kVs, kWFull = kVEmpty + kVs, kWEmpty = kWFull + kWides,
                kMFull = kWEmpty + kWides, kMEmpty = kMFull + kMetaBatches,
                kSFull = kMEmpty + kMetaBatches, kPFull = kSFull + 2, kODone = kPFull + 2,
                kQReady = kODone + 2, kQEmpty = kQReady + 1, kDrain = kQEmpty + 1,
                kWorkFull = kDrain + 1, kWorkRead = kWorkFull + 1, kClaim = kWorkRead + 1;
  static_assert(kClaim + 1 == Lay::kBarCount, "");
  auto bar = [&](int i) { return sm0 + Lay::kBars + 8u * static_cast<uint32_t>(i); };
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Lay::kWords);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  Work *shared_work = reinterpret_cast<Work *>(sm + Lay::kWork);
  float *q_scale = reinterpret_cast<float *>(sm + Lay::kQScale);
  TileMeta *meta = reinterpret_cast<TileMeta *>(sm + Lay::kMeta);
  int *sort_tiles = reinterpret_cast<int *>(sm + Lay::kJoin);  // used before the works' joins
  uint8_t *sort_places = sm + Lay::kPlaces;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    auto init = [&](int first, int n, uint32_t arrivals) {
      for (int i = 0; i < n; ++i) ptx::mbar_init(bar(first + i), arrivals);
    };
    init(kKFull, kKs, 1);
    init(kKEmpty, kKs, 1);
    init(kVFull, kVs, 1);
    init(kVEmpty, kVs, 4);  // the widening warps
    init(kWFull, kWides, 4);
    init(kWEmpty, kWides, 1);
    init(kMFull, kMetaBatches, 1);
    init(kMEmpty, kMetaBatches, 13);  // softmax, widening and issuing warps
    init(kSFull, 2, 1);
    init(kPFull, 2, 4);  // one arrival per warp of the group
    init(kODone, 2, 1);
    init(kQReady, 1, 4);
    init(kQEmpty, 1, 1);
    init(kDrain, 1, 1);
    init(kWorkFull, 1, 1);
    init(kWorkRead, 1, 15);  // every other warp
    init(kClaim, 1, 1);
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
  if (sorted) sort_requests<kPair>(p, kShift, sort_tiles, sort_places);

  // The CTA's works, one after the other, as in the 16-bit kernel.
  auto next_work = [&](uint32_t w) {
    volatile int dummy = 0;
    Work d = {};
    if (__all_sync(0xffffffffu, chunk_wait<false, 16>(bar(kWorkFull), w & 1, &dummy)))
      d = shared_work[w & 1];
    else
      *abort_flag = 1;
    return d;
  };
  auto have_read = [&] {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(kWorkRead));
  };
  // Whether the nth use of a ring of n slots may begin: its barrier and phase.
  auto reuse = [&](int first, int at, int n) {
    return at < n || chunk_wait<false>(bar(first + at % n),
                                       static_cast<uint32_t>((at / n - 1) & 1), abort_flag);
  };
  auto arrived = [&](int first, int at, int n) {
    return chunk_wait<false>(bar(first + at % n), static_cast<uint32_t>((at / n) & 1), abort_flag);
  };

  if (warp >= 12) {
    regs_less<kWidenRegs>();
    // ------------------------------------------------ Q's split, V's widening
    const int wr = 32 * (warp & 3);  // the warp's rows of a V tile
    // A lane's 16 codes of every eight rows (HD 64: once; 128: twice).  Eight lanes read and write
    // 16 bytes each of different banks: HD 64: of rows r and r + 1; 128: of r and r ^ 5, since a
    // row's chunks arrive at their number xor r, and leave at twice it xor r.
    constexpr int kSub = HD / 64;
    uint32_t from[kSub], to[kSub][2];
    int row8[kSub];  // the row of eight
#pragma unroll
    for (int e = 0; e < kSub; ++e) {
      const int pair = 2 * e + (lane >> 4), c = (lane & 3) + (HD == 64 ? 0 : lane >> 1 & 4);
      row8[e] = HD == 64 ? lane >> 2 : lane & 4 ? pair ^ 5 : pair;
      const int row = wr + row8[e];
      from[e] = row * HD + (HD == 64 ? c ^ (row8[e] >> 1) : c ^ row8[e]) * 16;
      for (int i = 0; i < 2; ++i)
        to[e][i] = (c >> 2) * kChunkBytes + row * 128 + (((2 * (c & 3) + i) ^ row8[e]) << 4);
    }
    int at = 0, batches = 0;  // V tiles and batches of scales so far
    uint32_t loads = 0u;
    bool ok = true;
    for (uint32_t w = 0; w == 0 || kMany; ++w) {
      const Work d = next_work(w);
      have_read();
      if (d.nrow == 0) break;
      if (d.n == 0 || !ok) continue;
      // Q: eight lanes a row, the next rows' loads under these.
      {
        constexpr int kLoads = HD / 64;  // of 8 values
        const int tok0 = d.row0 / p.G, rem0 = d.row0 - tok0 * p.G, u = lane & 7;
        auto fetch = [&](int row, uint4(&x)[kLoads]) {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) x[i] = make_uint4(0, 0, 0, 0);
          if (row >= d.nrow) return;
          const int f = rem0 + row, tok = p.G == 1 ? f : static_cast<int>(__umulhi(f, p.g_inv));
          const uint16_t *src = p.q + (d.a + tok0 + tok) * p.qs +
                                static_cast<int64_t>(d.kvh * p.G + f - tok * p.G) * HD +
                                u * 8 * kLoads;
#pragma unroll
          for (int i = 0; i < kLoads; ++i) x[i] = reinterpret_cast<const uint4 *>(src)[i];
        };
        uint4 x[kLoads];
        int row = 4 * (warp & 3) + (lane >> 3);
        fetch(row, x);
        if (loads > 0)
          ok = __all_sync(0xffffffffu,
                          chunk_wait<false>(bar(kQEmpty), (loads - 1) & 1, abort_flag));
#pragma unroll 1
        for (; ok && row - (lane >> 3) < d.nrow; row += 16) {
          uint4 ahead[kLoads];
          fetch(row + 16, ahead);
          float y[8 * kLoads], most = 0.f;
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[8 * i + 2 * e] = __uint_as_float(v[e] << 16);
              y[8 * i + 2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
            }
          }
#pragma unroll
          for (int e = 0; e < 8 * kLoads; ++e) {
            const float a = fabsf(y[e]);
            if (a < INFINITY) most = fmaxf(most, a);
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          const int e = scale8_exponent(most);
          const float down = exp2_int(-e);
          uint32_t hi[2 * kLoads], lo[2 * kLoads];
#pragma unroll
          for (int i = 0; i < 2 * kLoads; ++i) {
            uint32_t h[2], l[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float a = y[4 * i + 2 * j] * down, b = y[4 * i + 2 * j + 1] * down;
              if (!(fabsf(a) <= 448.f)) a = NAN;
              if (!(fabsf(b) <= 448.f)) b = NAN;
              h[j] = e4m3_pair(a, b);
              const float2 v = e4m3_values(h[j]);
              l[j] = e4m3_pair(a - v.x, b - v.y);
            }
            hi[i] = h[0] | h[1] << 16;
            lo[i] = l[0] | l[1] << 16;
          }
          if (row < d.nrow) {
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
            if (u == 0) q_scale[(w & 1) * 256 + row] = exp2_int(e);
          }
#pragma unroll
          for (int i = 0; i < kLoads; ++i) x[i] = ahead[i];
        }
        ++loads;
        if (!ok) continue;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kQReady));
      }
      int left = 0;  // batches of scales handed back
      auto hand_back = [&](int to_batch) {
        __syncwarp();
        for (; left < to_batch; ++left)
          if (lane == 0) ptx::mbar_arrive(bar(kMEmpty + (batches + left) % kMetaBatches));
      };
      const int n = d.n;
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        const int b = batches + t / kMetaBatch, raw = at % kVs, slot = at % kWides;
        hand_back(t / kMetaBatch);
        ok = (t % kMetaBatch != 0 || arrived(kMFull, b, kMetaBatches)) &&
             arrived(kVFull, at, kVs) && reuse(kWEmpty, at, kWides);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const TileMeta &tile = meta[b % kMetaBatches * kMetaBatch + t % kMetaBatch];
        const uint32_t v0 = tile.v[2 * (warp & 3)], v1 = tile.v[2 * (warp & 3) + 1];
        const int kb = (d.t0 + t) * kKT + wr;
        const uint8_t *src = sm + Lay::kV + raw * Lay::kTile;
        uint8_t *dst = sm + Lay::kWide + slot * Lay::kTile16;
        // Rows that no row of the work sees, and those of pages outside the pool, become zeros:
        // a weight of 0 does not silence a NaN.
        const bool whole = kb >= d.lo_min && kb + 31 <= d.hi_max && (v0 & v1) >> 24;
        const bool far = tile.far != 0;
        // Short loops: in a long run of instructions that other warps' code has driven out of the
        // cache each takes three cycles or four.
        if (whole && !far) {
          uint32_t f = (v0 & 0xffffu) * 0x10001u;
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            if (i == 2) f = (v1 & 0xffffu) * 0x10001u;
            uint4 x[kSub];
#pragma unroll
            for (int e = 0; e < kSub; ++e)
              x[e] = *reinterpret_cast<const uint4 *>(src + from[e] + i * 8 * HD);
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
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = i < 2 ? v0 : v1, f = (v & 0xffffu) * 0x10001u;
            const float scale = scale8_value(v >> 16 & 255u);
#pragma unroll
            for (int e = 0; e < kSub; ++e) {
              const int key = kb + row8[e] + i * 8;
              const bool keep = v >> 24 && key >= d.lo_min && key <= d.hi_max;
              const uint4 x = *reinterpret_cast<const uint4 *>(src + from[e] + i * 8 * HD);
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
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(kWFull + slot));
          ptx::mbar_arrive(bar(kVEmpty + raw));
        }
        ++at;
      }
      const int all = (n + kMetaBatch - 1) / kMetaBatch;
      hand_back(all);
      batches += all;
    }
  } else if (warp >= 8) {
    regs_less<kIssueRegs>();
    if (warp == 8) {
    // ------------------------------------------------ scheduler
    int block = blockIdx.x, seg = blockIdx.z;
    bool have = true, last = !kMany;
    uint32_t claims = 0;
    Order order = {};
    if (sorted) order = read_order(p, lane, sort_tiles, sort_places);
    for (uint32_t w = 0;; ++w) {
      Work d = {};
      while (true) {
        if (have) {
          d = sorted ? describe_sorted(p, order, block, seg, kShift)
                     : describe(p, block, seg, kShift, lane);
          have = false;
          if (d.nrow > 0) break;
        }
        if (last) break;
        const uint32_t answer = sm0 + Lay::kAnswer;
        if (lane == 0) {
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive_expect_tx(bar(kClaim), 16);
          claim_block(answer, bar(kClaim));
        }
        __syncwarp();
        volatile int dummy = 0;
        const bool told =
            __all_sync(0xffffffffu, chunk_wait<false, 4>(bar(kClaim), claims & 1, &dummy));
        if (!told) *abort_flag = 1;  // a block may be lost: reported
        have = told && claimed_block(answer, &block, &seg);
        __syncwarp();
        ++claims;
        last = !have;  // none left: not to be asked again
      }
      if (lane == 0) {
        shared_work[w & 1] = d;
        ptx::mbar_arrive(bar(kWorkFull));
      }
      __syncwarp();
      if (d.nrow == 0 || !kMany) break;
      volatile int dummy = 0;
      if (!__all_sync(0xffffffffu, chunk_wait<false, 4>(bar(kWorkRead), w & 1, &dummy)) ||
          *abort_flag)
        last = true;
    }
  } else if (warp == 9) {
    // ------------------------------------------------ scales
    // Lane 8 i + g: 16 keys g of tile i of four.  Pages are looked up two batches ahead, scales
    // one.
    const int mine = lane >> 3, g16 = 16 * (lane & 7);
    const int shift = 31 - __clz(cache.block), blocks = cache.P >> shift;
    int batches = 0;
    bool ok = true;
    for (uint32_t w = 0; w == 0 || kMany; ++w) {
      const Work d = next_work(w);
      have_read();
      if (d.nrow == 0) break;
      if (d.n == 0 || !ok) continue;
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
        ok = __all_sync(0xffffffffu, reuse(kMEmpty, batches, kMetaBatches));
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
                    mn = __shfl_sync(0xffffffffu, low, 8 * i), grown = max(E, mx);
          far = far || (mn != kNone && mn < grown - 14);
          if (!far) E = grown;
          if (i == mine) {
            my_E = far || E == -kNone ? 0 : E;
            my_far = far;
          }
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, page == -1);
        any_bad |= bad != 0;
        TileMeta &m = meta[batches % kMetaBatches * kMetaBatch + mine];
        m.k[lane & 7] = page >= 0 ? scale8_value(kb) : 1.f;
        const uint32_t factor =
            vb == 255u ? 0x7fffu : static_cast<uint32_t>(15 + static_cast<int>(vb) - 127 - my_E) << 10;
        m.v[lane & 7] = page >= 0 ? (factor & 0xffffu) | vb << 16 | 1u << 24 : 0u;
        if ((lane & 7) == 0) {
          m.E = my_E;
          m.far = my_far;
          m.bad = static_cast<int>(bad >> (8 * mine) & 255u);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kMFull + batches % kMetaBatches));
        ++batches;
        page = page1;
        page1 = page2;
        bytes = bytes1;
      }
      if (any_bad && lane == 0) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
    }
  } else if (warp == 10) {
    // ------------------------------------------------ TMA producer
    // A lane per box (page rows).  Boxes without a visible key and pages outside the pool are
    // not loaded.  The next work is claimed once the loads come to the last kAhead tiles.
    constexpr int kAhead = 3;
    const int boxes = kKT / p.box_rows;
    int at_k = 0, at_v = 0;
    bool ok = true;
    for (uint32_t w = 0; w == 0 || kMany; ++w) {
      const Work d = next_work(w);
      if (d.nrow == 0 || d.n == 0 || !ok) {
        have_read();
        if (d.nrow == 0) break;
        continue;
      }
      const int n = d.n;
      const uint64_t pol =
          d.total <= (1 << kShift) ? ptx::policy_evict_first() : ptx::policy_evict_normal();
      auto fetch = [&](int t) {  // page of box `lane` of tile t, -1 where it is not loaded
        int page = -1;
        if (lane < boxes && t < n) {
          const int key0 = (d.t0 + t) * kKT + lane * p.box_rows;
          if (key0 <= d.hi_max && key0 + p.box_rows > d.lo_min) {
            page = p.tbl[static_cast<int64_t>(d.r) * p.M + key0 / p.P];
            if (page >= p.NP) page = -1;
          }
        }
        return page;
      };
      auto load = [&](int t, int kv, int page) {
        if (!ok) return;
        int &at = kv ? at_v : at_k;
        const int slots = kv ? kVs : kKs, slot = at % slots;
        bool got = true;
        if (lane == 0) got = reuse(kv ? kVEmpty : kKEmpty, at, slots);
        ok = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
        if (!ok) return;
        const bool skip = t == p.skip_tile && kv == 0;
        const uint32_t full = bar((kv ? kVFull : kKFull) + slot);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * p.box_rows * HD;
        if (lane == 0 && !skip) ptx::mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (lane < boxes && page >= 0 && !skip) {
          const int key0 = (d.t0 + t) * kKT + lane * p.box_rows;
          const int64_t row =
              (((static_cast<int64_t>(p.layer) * p.NP + page) * 2 + kv) * p.nkv + d.kvh) * p.P +
              key0 % p.P;
          ptx::tma_load_2d_hint(sm0 + (kv ? Lay::kV : Lay::kK) + slot * Lay::kTile +
                                    lane * p.box_rows * HD,
                                &tm, 0, static_cast<int32_t>(row), full, pol);
        }
        ++at;
      };
      // a tile's pages are looked up at least one load ahead of their use
      if (kPair && d.nrow > 128) {
        int cur = fetch(0);
        for (int t = 0; t < n; ++t) {
          const int nxt = fetch(t + 1);
          if (t == max(n - kAhead, 0)) have_read();
          load(t, 0, cur);
          load(t, 1, cur);
          cur = nxt;
        }
      } else {
        int pa = fetch(0), pb = fetch(1);
        load(0, 0, pa);
        if (n > 1) load(1, 0, pb);
        for (int t = 0; t < n; ++t) {
          const int pc = fetch(t + 2);
          if (t == max(n - kAhead, 0)) have_read();
          load(t, 1, pa);
          if (t + 2 < n) load(t + 2, 0, pc);
          pa = pb;
          pb = pc;
        }
      }
    }
    if (*abort_flag && lane == 0) {  // wind down: the last copies land before the CTA ends
      volatile int dummy = 0;
      for (int i = max(at_k - kKs, 0); i < at_k; ++i)
        chunk_wait<false>(bar(kKFull + i % kKs), static_cast<uint32_t>((i / kKs) & 1), &dummy);
      for (int i = max(at_v - kVs, 0); i < at_v; ++i)
        chunk_wait<false>(bar(kVFull + i % kVs), static_cast<uint32_t>((i / kVs) & 1), &dummy);
    }
  } else if (warp == 11) {
    // ------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_qk = idesc_of(128, kKT, 0, false);
    constexpr uint32_t idesc_f16 = idesc_of(128, HD, 0, true), idesc_bf16 = idesc_of(128, HD, 1, true);
    // warp-uniform copies
    const uint32_t tm0 = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t base = __shfl_sync(0xffffffffu, sm0, 0);
    const uint64_t dq = ptx::desc_kmajor_sw128(base, 0);
    const uint64_t dk = ptx::smem_desc(base + Lay::kK, 16, 8 * HD,
                                       HD == 64 ? kSwizzle64B : ptx::kSwizzle128B);
    const uint64_t dv = ptx::smem_desc(base + Lay::kWide, kChunkBytes, 1024, ptx::kSwizzle128B);
    struct At {
      uint32_t bar, phase;
    };
    int at_k = 0, at_v = 0, batches = 0;  // of K tiles, V tiles, batches of scales
    uint32_t handed0 = 0u, handed1 = 0u, loads = 0u;  // phases of p_full and q_ready
    bool ok = true, pairs = false;
    auto slot = [&](int first, int at, int n) {
      return At{bar(first + at % n), static_cast<uint32_t>((at / n) & 1)};
    };
    // up to three barriers at the cost of one: each is polled by lanes of its own
    auto wait = [&](At a, At b, At c) {
      const At x = lane == 1 ? b : lane == 2 ? c : a;
      const bool got = __all_sync(0xffffffffu, chunk_wait<true>(x.bar, x.phase, abort_flag));
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
      ptx::mma_commit(bar(kSFull + g));
    };
    auto pv = [&](int g, int at, bool first, uint32_t idesc) {  // O_g (+)= P V
      const uint64_t b = dv + (((at % kWides) * Lay::kTile16) >> 4);
#pragma unroll
      for (int ks = 0; ks < kKT / 16; ++ks)
        ptx::mma_bf16_ts(tm0 + kColO + HD * g, tm0 + 128 * g + ks * 8, b + ((ks * 2048) >> 4),
                         idesc, (!first || ks > 0) ? 1u : 0u);
    };
    for (uint32_t w = 0; w == 0 || kMany; ++w) {
      const Work d = next_work(w);
      have_read();
      if (d.nrow == 0) break;
      const int tiles = __shfl_sync(0xffffffffu, d.n, 0);
      if (!ok || tiles == 0) continue;
      pairs = kPair && __shfl_sync(0xffffffffu, d.nrow, 0) > 128;
      const int step = pairs ? 1 : 2;
      ok = wait(At{bar(kQReady), loads & 1}, slot(kKFull, at_k, kKs),
                slot(kKFull, !pairs && tiles > 1 ? at_k + 1 : at_k, kKs));
      ++loads;
      if (ok && elect_one()) {
        qk(0, at_k);
        if (pairs) {
          qk(1, at_k);
          ptx::mma_commit(bar(kKEmpty + at_k % kKs));
        } else {
          ptx::mma_commit(bar(kKEmpty + at_k % kKs));
          if (tiles > 1) {
            qk(1, at_k + 1);
            ptx::mma_commit(bar(kKEmpty + (at_k + 1) % kKs));
          }
        }
        if (tiles <= step) ptx::mma_commit(bar(kQEmpty));
      }
      __syncwarp();
      int left = 0;
      for (int t = 0; ok && t < tiles; ++t) {
        const bool more = t + step < tiles;
        const int b = batches + t / kMetaBatch;
        uint32_t idesc = 0;
        for (int i = 0; ok && i < (pairs ? 2 : 1); ++i) {
          const int g = pairs ? i : t & 1;
          const At v = slot(kWFull, at_v + t, kWides);
          ok = wait(At{bar(kPFull + g), (g ? handed1 : handed0) & 1}, v,
                    more ? slot(kKFull, at_k + t + step, kKs) : v);
          if (!ok) break;
          if (g) ++handed1; else ++handed0;
          // (the widening warps and the group that handed P over have seen the tile's scales)
          if (i == 0)
            idesc = __shfl_sync(
                0xffffffffu,
                meta[b % kMetaBatches * kMetaBatch + t % kMetaBatch].far ? idesc_bf16 : idesc_f16,
                0);
          if (elect_one()) {
            pv(g, at_v + t, t < step, idesc);
            if (!pairs || i == 1) ptx::mma_commit(bar(kWEmpty + (at_v + t) % kWides));
            if (more) qk(g, at_k + t + step);
            if (more && (!pairs || i == 1)) {
              ptx::mma_commit(bar(kKEmpty + (at_k + t + step) % kKs));
              if (t + step == tiles - 1) ptx::mma_commit(bar(kQEmpty));
            }
            if (!more) ptx::mma_commit(bar(kODone + g));
          }
          __syncwarp();
        }
        if (t % kMetaBatch == kMetaBatch - 1 || t == tiles - 1) {
          if (lane == 0 && ok) ptx::mbar_arrive(bar(kMEmpty + b % kMetaBatches));
          ++left;
        }
      }
      at_k += tiles;
      at_v += tiles;
      batches += left;
    }
    if (!ok) {
      if (elect_one()) ptx::mma_commit(bar(kDrain));
      __syncwarp();
      volatile int dummy = 0;
      chunk_wait<false>(bar(kDrain), 0u, &dummy);
    }
    }
  } else {
    regs_more<kSoftmaxRegs>();
    // ------------------------------------------------ softmax groups
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
      const volatile Work &d = shared_work[wk & 1];
      volatile int dummy = 0;
      int nrow = 0, n = 0;
      if (__all_sync(0xffffffffu, chunk_wait<false, 16>(bar(kWorkFull), wk & 1, &dummy))) {
        nrow = d.nrow;
        n = d.n;
      } else {
        *abort_flag = 1;
      }
      have_read();
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
      if (n > 0) {
        if (ok)
          ok = __all_sync(0xffffffffu, chunk_wait<false>(bar(kQReady), loads & 1, abort_flag));
        ++loads;
        if (ok && real) row_scale = q_scale[(wk & 1) * 256 + rt] * p.scale_log2;
      }

      float m_ref = -INFINITY, l = 0.f;
      int E = 0, left = 0;
      auto hand_back = [&](int to_batch) {
        __syncwarp();
        for (; left < to_batch; ++left)
          if (lane == 0) ptx::mbar_arrive(bar(kMEmpty + (batches + left) % kMetaBatches));
      };
      const int step = split ? 2 : 1;
      for (int t = split ? g : 0; ok && t < n; t += step) {
        const int b = batches + t / kMetaBatch;
        hand_back(t / kMetaBatch);
        ok = arrived(kMFull, b, kMetaBatches) &&
             chunk_wait<false>(bar(kSFull + g), scores & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++scores;
        ptx::tc_fence_after();
        if (!active) {  // its rows of P may hold anything: they reach no other row
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(kPFull + g));
          continue;
        }
        const TileMeta &tile = meta[b % kMetaBatches * kMetaBatch + t % kMetaBatch];
        const int kb = (t0 + t) * kKT;
        const uint32_t bad = tile.bad;
        const bool cut = !(lo <= kb && hi >= kb + kKT - 1);
        float sv[128];
        tmem_ld128(tm_s, sv);
        if (bad) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if ((bad >> (c >> 4)) & 1u) sv[c] = -INFINITY;
        }
        if (cut) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (kb + c < lo || kb + c > hi) sv[c] = -INFINITY;
        }
        // the factor of 16 keys' scores; never 0, which would make a masked one NaN
        auto factor = [&](int i) { return fmaxf(row_scale * tile.k[i], 0x1p-126f); };
        float f[8], tmax = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = factor(i);
          float a = fmaxf(sv[16 * i], sv[16 * i + 1]);
#pragma unroll
          for (int c = 2; c < 16; c += 2) a = fmaxf(fmaxf(a, sv[16 * i + c]), sv[16 * i + c + 1]);
          tmax = fmaxf(tmax, a * f[i]);
        }
        const int grown = tile.E - E;
        float corr = 1.f, corr_o = 1.f;
        if (m_ref == -INFINITY) {
          m_ref = tmax;
        } else if (tmax > m_ref + 8.f) {
          corr = ptx::ex2(m_ref - tmax);
          m_ref = tmax;
        }
        corr_o = corr * ptx::ex2(static_cast<float>(-grown));
        E = tile.E;
        // the group's previous product completed before this S did
        if (t >= step && __any_sync(0xffffffffu, corr_o != 1.f)) {
          for (int c = 0; c < HD; c += 16) {
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
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int x = 64 * c; x < 64 * c + 64; x += 2) {
            const float2 f2 = make_float2(f[x / 16], f[x / 16]);
            float2 w = fma2(make_float2(sv[x], sv[x + 1]), f2, nm2);
            w.x = ptx::ex2(w.x);
            w.y = ptx::ex2(w.y);
            sum[x / 2 & 1] = add2(sum[x / 2 & 1], w);
            sv[x] = w.x;
            sv[x + 1] = w.y;
          }
          uint32_t pk[32];
          if (far) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              pk[e] = ptx::pack_bf16x2(sv[64 * c + 2 * e], sv[64 * c + 2 * e + 1]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              pk[e] = pack_f16x2(sv[64 * c + 2 * e], sv[64 * c + 2 * e + 1]);
          }
          tmem_st32(tm_s + 32 * c, pk);
        }
        sum[0] = add2(sum[0], sum[1]);
        l = l * corr + (sum[0].x + sum[0].y);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kPFull + g));
      }
      const int all = (n + kMetaBatch - 1) / kMetaBatch;
      hand_back(all);
      batches += all;
      // ---------------------------------------------- epilogue
      const bool had0 = n > 0, had1 = split ? n > 1 : n > 0;  // groups with products
      if (ok && (g ? had1 : had0)) {
        ok = __all_sync(0xffffffffu, chunk_wait<false>(bar(kODone + g), (g ? outs1 : outs0) & 1,
                                                       abort_flag));
        ptx::tc_fence_after();
      }
      if (split && ok && (g ? had0 : had1)) {  // the other group's products
        ok = __all_sync(0xffffffffu, chunk_wait<false>(bar(kODone + (g ^ 1)),
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
      const bool any = real && m != -INFINITY;  // the row saw a key
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
      } else if (real && (!split || g == 0)) {
        const int64_t w = (orow * p.hq + h) * p.S + seg;
        p.ws_m[w] = m;
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
          float4 *dst = reinterpret_cast<float4 *>(
              p.ws_o + ((orow * p.hq + h) * p.S + seg) * HD + d0 + c);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
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

// Rows of codes, one key of a head each.
cudaError_t code_tensor_map(CUtensorMap *m, const void *codes, uint64_t rows, uint32_t hd,
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

}  // namespace

int chunk_attention8_num_segments(const dflash_geom &g, int B, int n_rows, int window) {
  return segments_of(g, B, n_rows, window, 7.0, 3.0, 1.5);
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
  const ChunkParams p = chunk_params(g, B, layer, n_rows, q, q_stride, tbl, cu, ctx, kv, window,
                                     sinks, scale, mask_mode, S, ws, out, out_stride, st);
  CUtensorMap tm;
  const uint64_t rows = static_cast<uint64_t>(g.num_layers) * g.num_pool_pages * 2 * g.nkv *
                        static_cast<uint64_t>(g.page_size);
  cudaError_t e = code_tensor_map(&tm, cache.codes, rows, g.head_dim, p.box_rows);
  if (e != cudaSuccess) return e;
  const Cache8 c = cache8_of(g, cache, layer);
  const dim3 grid(static_cast<unsigned>(chunk_tiles(g, B, n_rows) * g.nkv), 1, S);
  const bool pair = pair_form(g, B, n_rows);
  e = g.head_dim == 64 ? launch_main<64>(pair, tm, p, c, grid, s)
                       : launch_main<128>(pair, tm, p, c, grid, s);
  return e != cudaSuccess || S == 1 ? e : launch_merge(g, p, s);
}

}  // namespace dflash
