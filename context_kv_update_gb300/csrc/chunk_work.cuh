// chunk_work.cuh -- what the attentions of a ragged chunk share (a 16-bit cache:
// chunk_attention.cu, one in 8 bits: chunk_attention8.cu): how requests are cut into work tiles,
// which CTA takes which, bounded waits.
#pragma once

#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "dflash_internal.cuh"
#include "f32x2.cuh"
#include "sm100_ptx.cuh"

namespace dflash {

cudaError_t make_tmap_bf16_2d(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols,
                              uint64_t row_stride_elems, uint32_t box_rows, uint32_t box_cols);
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled_fn();

struct ChunkParams {
  int B, n_rows, hq, nkv, G, wide_out, layer, NP, P, M, window, mask_mode, S;
  int box_rows, skip_tile, q_boxes;
  int tails;  // > 1: two segments of a main part and a tail (main_tiles)
  uint32_t g_inv;  // ceil(2^32 / G), for G > 1
  float scale_log2;
  const uint16_t *q;
  int64_t qs, os;
  const int32_t *tbl, *cu, *ctx, *kv;
  const float *sinks;
  float *ws_m, *ws_l, *ws_o;
  uint16_t *out;
  int32_t *st;
};
// Joins the segments' partial results (chunk_merge.cu).
cudaError_t launch_merge(const dflash_geom &g, const ChunkParams &p, cudaStream_t s);

namespace {

constexpr int kKT = kAttnTileKeys;  // 128 keys per tile
constexpr int kSmemMax = 227 * 1024;
constexpr uint32_t kChunkBytes = kKT * 128;  // 64 dims of 128 rows, 128-byte swizzled
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;  // S of group g at 128 g, O at 256 + HD g
constexpr float kLog2e = 1.4426950408889634f;


__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
// 32 bytes in one store, 32-byte aligned.
__device__ __forceinline__ void store_32b(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// Wait on phase `parity` of `bar`, bounded by the SM clock (a read of the
// global timer costs more than most of these waits): false, with *abort set,
// after about two seconds, or once another thread has set *abort.  kSpin: with
// the probe that does not suspend the thread (waking up takes longer than the
// wait does), for the waits between the products and the softmax.
template <bool kSpin, int kTimes = 1>
__device__ __forceinline__ bool chunk_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
  constexpr long long kLimit = kTimes * 4000000000ll;  // cycles
  auto probe = [&] { return kSpin ? ptx::mbar_test(bar, parity) : ptx::mbar_try_wait(bar, parity); };
  if (probe()) return true;
  const long long t0 = clock64();
  for (uint32_t n = 1;; ++n) {
    if (probe()) return true;
    if ((n & 255u) == 0) {
      if (*abort) return false;
      if (clock64() - t0 > kLimit) {
        *abort = 1;
        return false;
      }
    }
  }
}

// One lane of a converged warp, the same one at every call.  Issuing under it
// with warp-uniform operands lets the compiler keep descriptors in uniform
// registers: a lane-0 branch needs several times the instructions for each MMA,
// and they wait for the softmax warps that share the scheduler (measured with
// fma-bound neighbours: 262 cycles an MMA against 134; 64 without any).
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// The request whose tiles hold work tile x (tiles of 2^shift flat rows), found
// by the whole warp in a 32-ary search.
__device__ __forceinline__ int64_t first_tile(const ChunkParams &p, int r, int shift) {
  return ((static_cast<int64_t>(p.cu[r]) * p.G) >> shift) + r;
}
__device__ __forceinline__ int find_request(const ChunkParams &p, int64_t x, int shift, int lane) {
  int lo = 0, n = p.B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool at = lane * step < n && first_tile(p, lo + lane * step, shift) <= x;
    const int c = max(__popc(__ballot_sync(0xffffffffu, at)), 1) - 1;
    lo += c * step;
    n = min(step, n - c * step);
  }
  return lo;
}

// Chunk rows [a, b) of request r at positions from c over kv keys, or false
// (flagged) where its offsets or length make no sense.
struct Request {
  int a, b, c, kv;
};
__device__ __forceinline__ void load_request(const ChunkParams &p, int r, Request *q) {
  q->a = p.cu[r];
  q->b = p.cu[r + 1];
  q->c = p.ctx[r];
  q->kv = p.kv[r];
}
__device__ __forceinline__ bool check_request(const ChunkParams &p, bool report, Request *q) {
  if (q->a < 0 || q->b < q->a || q->b > p.n_rows || q->c < 0 || q->c > INT32_MAX - p.n_rows) {
    if (report) raise_status(p.st, DFLASH_DEV_BAD_ROWS);
    return false;
  }
  const int cap = p.M * p.P;
  if (q->kv < 0 || q->kv > cap) {
    if (report) raise_status(p.st, DFLASH_DEV_KV_LEN_RANGE);
    q->kv = q->kv < 0 ? 0 : cap;
  }
  return true;
}

// Keys [lo, hi] a row at position pos sees of kv.
__device__ __forceinline__ void key_range(const ChunkParams &p, int pos, int kv, int *lo, int *hi) {
  *hi = p.mask_mode == DFLASH_MASK_CAUSAL_TAIL ? min(pos, kv - 1) : kv - 1;
  *lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
}

// A work tile's rows [row0, row0 + nrow) of request r's flat rows, the keys
// [lo_min, hi_max] some of them sees, and its key tiles [t0, t0 + n).
struct __align__(16) Work {
  int r, kvh, seg, a, c, kv, total;  // chunk rows from a, positions from c, flat rows in all
  int row0, nrow, lo_min, hi_max, t0, n;
  int pad[3];
};

// Of n key tiles, those of the main segment where an SM that has no main one takes
// `tails` others, and each costs about two and a half key tiles on its own.
__host__ __device__ inline int main_tiles(int n, int tails) {
  const int64_t m =
      (2ll * tails * n + 5 * (tails - 1) + 2 * tails + 1) / (2 * tails + 2);  // rounded up
  return m < n ? static_cast<int>(m) : n;
}

// The work of rows from `first` on of request r, of S segments the seg-th; nrow 0 where
// there are none.
__device__ __forceinline__ Work work_of(const ChunkParams &p, int r, const Request &q,
                                        int64_t first, int kvh, int seg, int shift) {
  Work w = {};
  w.r = r;
  w.kvh = kvh;
  w.seg = seg;
  w.a = q.a;
  w.c = q.c;
  w.kv = q.kv;
  w.total = (q.b - q.a) * p.G;
  if (first < 0 || first >= w.total) return w;
  w.row0 = static_cast<int>(first);
  w.nrow = min(w.total - w.row0, 1 << shift);
  int lo, hi;
  key_range(p, w.c + w.row0 / p.G, w.kv, &w.lo_min, &hi);
  key_range(p, w.c + (w.row0 + w.nrow - 1) / p.G, w.kv, &lo, &w.hi_max);
  if (w.lo_min <= w.hi_max) {
    const int ta = w.lo_min / kKT, tb = w.hi_max / kKT + 1;
    if (p.tails > 1) {  // two segments of different lengths
      const int main = main_tiles(tb - ta, p.tails);
      w.t0 = ta + seg * main;
      w.n = seg ? tb - ta - main : main;
    } else {
      const int per = (tb - ta + p.S - 1) / p.S;
      w.t0 = ta + seg * per;
      w.n = max(min(tb - w.t0, per), 0);
    }
  }
  return w;
}

// Work tile (x, seg) of the grid, in the requests' order.  The whole warp.  Later rows
// see more keys, so the last tiles of all heads go first (heads one after the other
// leave a head's longest tiles for the end).
__device__ __forceinline__ Work describe(const ChunkParams &p, int block, int seg, int shift,
                                         int lane) {
  const int kvh = block % p.nkv;
  const int64_t x = gridDim.x / p.nkv - 1 - block / p.nkv;
  Request q;
  int r;
  if (p.B <= 32) {  // in one memory round trip: a request a lane
    const int i = min(lane, p.B - 1);
    load_request(p, i, &q);
    const int64_t tile = ((static_cast<int64_t>(q.a) * p.G) >> shift) + i;
    r = max(__popc(__ballot_sync(0xffffffffu, lane < p.B && tile <= x)), 1) - 1;
    q.a = __shfl_sync(0xffffffffu, q.a, r);
    q.b = __shfl_sync(0xffffffffu, q.b, r);
    q.c = __shfl_sync(0xffffffffu, q.c, r);
    q.kv = __shfl_sync(0xffffffffu, q.kv, r);
  } else {
    r = find_request(p, x, shift, lane);
    load_request(p, r, &q);
  }
  if (!check_request(p, lane == 0 && kvh == 0 && seg == 0, &q)) return Work{};
  const int64_t first = (x - (((static_cast<int64_t>(q.a) * p.G) >> shift) + r)) << shift;
  return work_of(p, r, q, first, kvh, seg, shift);
}

// The requests of a call with 2 to 256 of them in the order of their work tiles' cost,
// the dearest first: claimed in the requests' own order, a long one that comes late keeps one
// SM at work when the others have nothing left (64 single tokens over up to 8192 keys
// 226 us, so 210; 32 of them 139 and 107, 256 over up to 2048 keys 274 and 248).  Every
// block sorts for itself, all its threads together (one warp alone took 10 us for 256),
// and reports what makes no sense: which of them run is not known (a claimed one does
// not come here), and their order is not either.
constexpr int kSortLanes = 8, kSorted = 32 * kSortLanes;
struct Order {  // lane l holds places l, l + 32, ...
  int r[kSortLanes], end[kSortLanes];  // the request at a place, where its work tiles end
};
// By the whole block: into places[k] the request at place k, into tiles[k] its work tiles.
template <bool kPair>
__device__ __forceinline__ void sort_requests(const ChunkParams &p, int shift, int *tiles,
                                              uint8_t *places) {
  const int i = threadIdx.x, all = gridDim.x / p.nkv;
  int cost = -1, count = 0, rank = 0;
  if (i < p.B) {
    Request q;
    load_request(p, i, &q);
    const int from = static_cast<int>((static_cast<int64_t>(q.a) * p.G) >> shift) + i;
    const int to = i + 1 < p.B
                       ? static_cast<int>((static_cast<int64_t>(q.b) * p.G) >> shift) + i + 1
                       : all;
    count = min(max(to - from, 0), all);
    if (check_request(p, true, &q) && q.b > q.a) {
      int lo, hi;
      key_range(p, q.c + q.b - q.a - 1, q.kv, &lo, &hi);
      if (lo <= hi)  // one row tile is done in half the steps of two
        cost = (hi / kKT - lo / kKT + 1) * (kPair && (q.b - q.a) * p.G > 128 ? 2 : 1);
    }
  }
  if (i < kSorted) tiles[i] = i < p.B ? cost : -2;  // behind them all
  __syncthreads();
  if (i < p.B) {
    const int4 *costs = reinterpret_cast<const int4 *>(tiles);
#pragma unroll 4
    for (int j = 0; j < (p.B + 3) / 4; ++j) {
      const int4 c = costs[j];
      rank += (c.x > cost || (c.x == cost && 4 * j < i)) +
              (c.y > cost || (c.y == cost && 4 * j + 1 < i)) +
              (c.z > cost || (c.z == cost && 4 * j + 2 < i)) +
              (c.w > cost || (c.w == cost && 4 * j + 3 < i));
    }
    places[rank] = static_cast<uint8_t>(i);
  }
  __syncthreads();
  if (i < p.B) tiles[rank] = count;
  __syncthreads();
}
__device__ __forceinline__ Order read_order(const ChunkParams &p, int lane, const int *tiles,
                                            const uint8_t *places) {
  Order o;
  int before = 0;
#pragma unroll
  for (int k = 0; k < kSortLanes; ++k) {
    o.r[k] = 0;
    o.end[k] = INT32_MAX;
    if (32 * k < p.B) {
      const int at = lane + 32 * k;
      o.r[k] = at < p.B ? places[at] : 0;
      int end = at < p.B ? tiles[at] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, end, d);
        if (lane >= d) end += up;
      }
      o.end[k] = end + before;
      before = __shfl_sync(0xffffffffu, o.end[k], 31);
    }
  }
  return o;
}
__device__ __forceinline__ Work describe_sorted(const ChunkParams &p, const Order &o, int block,
                                                int seg, int shift) {
  const int x = block / p.nkv;
  int at = 0, r = 0, end = 0;
#pragma unroll
  for (int k = 0; k < kSortLanes; ++k)
    if (32 * k < p.B) at += __popc(__ballot_sync(0xffffffffu, o.end[k] <= x));
  if (at >= p.B) return Work{};
#pragma unroll
  for (int k = 0; k < kSortLanes; ++k)
    if (at >> 5 == k) {
      r = __shfl_sync(0xffffffffu, o.r[k], at & 31);
      end = __shfl_sync(0xffffffffu, o.end[k], at & 31);
    }
  Request q;
  load_request(p, r, &q);
  if (!check_request(p, false, &q)) return Work{};
  // its last tile first; the places past its rows are empty
  const int64_t first = static_cast<int64_t>(end - 1 - x) << shift;
  return work_of(p, r, q, first, block - x * p.nkv, seg, shift);
}

// Ask for a block of the grid that has not started, to do its work here; the
// answer (16 bytes) arrives on `bar`.
__device__ __forceinline__ void claim_block(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(answer),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool claimed_block(uint32_t answer, int *x, int *z) {
  uint32_t got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
      "ld.shared.b128 a, [%3];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::z.b32.b128 %2, a;\n\t}"
      : "=&r"(got), "=&r"(*x), "=&r"(*z)
      : "r"(answer)
      : "memory");
  return got != 0;
}
// Pair form where the mean request fills more than one 128-row tile.
inline bool pair_form(const dflash_geom &g, int B, int n_rows) {
  return static_cast<int64_t>(n_rows) * (g.hq / g.nkv) > 128LL * B;
}

// Work tiles of a chunk, at most (of 2^shift rows).
inline int64_t chunk_tiles(const dflash_geom &g, int B, int n_rows, int shift) {
  return ((static_cast<int64_t>(n_rows) * (g.hq / g.nkv)) >> shift) + B;
}

// Work tiles of a call with one request.
inline int64_t works_of_one(const dflash_geom &g, int n_rows, int shift) {
  const int tr = 1 << shift;
  return (static_cast<int64_t>(n_rows) * (g.hq / g.nkv) + tr - 1) / tr * g.nkv;
}

// Two segments of one request: its work tiles fill the SMs a whole number of times
// but for some; each SM left over takes the tails of this many tiles, cut so that all end
// together (1: halves).
inline int tail_tiles(const dflash_geom &g, int B, int n_rows, int shift) {
  if (B != 1) return 1;
  const int64_t works = works_of_one(g, n_rows, shift), sms = device_sm_count();
  const int64_t idle = (works + sms - 1) / sms * sms - works;
  return idle == 0 ? 1 : static_cast<int>(std::min<int64_t>((works + idle - 1) / idle, 64));
}

// `tiles`: work tiles expected; `fixed`: what a CTA costs beside its key tiles, `merge`: what the
// second launch does, both in key tiles, of `tile_us` each where few rows stream them.
inline int segments_of(const dflash_geom &g, int B, int n_rows, int window, int shift,
                       int64_t tiles, double fixed, double merge, double tile_us) {
  const double ctas = static_cast<double>(tiles) * g.nkv;
  const double sms = device_sm_count();
  double longest = static_cast<double>(g.max_pages) * g.page_size / kKT;
  if (window > 0) longest = std::min(longest, (static_cast<double>(window) + n_rows) / kKT + 1.0);
  const double mean = B >= 4 ? 0.6 * longest : longest;
  const bool alike = B == 1 && longest * kKT >= 2.0 * n_rows;
  const int64_t works = works_of_one(g, n_rows, shift), left = works % device_sm_count();
  // a segment's partial results, written and read: key tiles at 6 TB/s
  const double part = 8.0 * n_rows * g.hq * g.head_dim / (tile_us * 6e6);
  int best = 1;
  double least = 0.0;
  for (int S = 1; S == 1 || (S <= 64 && 4 * S <= longest && ctas * (S - 1) <= 4 * sms); ++S) {
    double one = fixed + longest / S;
    if (S == 2 && alike)
      one = fixed + main_tiles(static_cast<int>(longest), tail_tiles(g, B, n_rows, shift));
    double t = one;
    if (alike)
      t *= std::ceil(static_cast<double>(works) * (S == 2 && left ? 1 : S) / sms);
    else if (ctas * S > sms)  // in the order of cost the last ones are short
      t = std::max(one, ctas * (mean + fixed * S) / sms + (B > kSorted ? 0.5 : 0.25) * one);
    if (S > 1) t += merge + part * S;
    if (S == 1 || t < least) {
      least = t;
      best = S;
    }
  }
  return best;
}

inline size_t workspace_of(const dflash_geom &g, int n_rows, int S) {
  if (S == 1) return 0;
  const size_t rows = static_cast<size_t>(n_rows) * g.hq * S;
  return 2 * align_up(rows * sizeof(float), 256) + rows * g.head_dim * sizeof(float);
}

// What both kernels and the merge are given.
inline ChunkParams chunk_params(const dflash_geom &g, int shift, int B, int layer, int n_rows,
                                const void *q,
                                int64_t q_stride, const int32_t *tbl, const int32_t *cu,
                                const int32_t *ctx, const int32_t *kv, int32_t window,
                                const float *sinks, float scale, int mask_mode, int S, void *ws,
                                void *out, int64_t out_stride, int32_t *st) {
  ChunkParams p = {};
  p.B = B;
  p.n_rows = n_rows;
  p.hq = g.hq;
  p.nkv = g.nkv;
  p.G = g.hq / g.nkv;
  p.g_inv = p.G > 1 ? 0xffffffffu / p.G + 1u : 0u;
  p.wide_out = ((reinterpret_cast<uintptr_t>(out) | (2 * out_stride)) & 31u) == 0;
  p.layer = layer;
  p.NP = g.num_pool_pages;
  p.P = g.page_size;
  p.M = g.max_pages;
  p.window = window;
  p.mask_mode = mask_mode;
  p.S = S;
  p.box_rows = std::min(p.P, kKT);
  p.tails = S == 2 ? tail_tiles(g, B, n_rows, shift) : 1;
  p.skip_tile = attention_test_skip_tile_value();
  p.scale_log2 = scale * kLog2e;  // scale > 0 (validated by the caller)
  p.q = static_cast<const uint16_t *>(q);
  p.qs = q_stride;
  p.os = out_stride;
  p.tbl = tbl;
  p.cu = cu;
  p.ctx = ctx;
  p.kv = kv;
  p.sinks = sinks;
  const size_t rows = static_cast<size_t>(n_rows) * g.hq * S;
  char *w = static_cast<char *>(ws);
  p.ws_m = reinterpret_cast<float *>(w);
  p.ws_l = reinterpret_cast<float *>(w + align_up(rows * sizeof(float), 256));
  p.ws_o = reinterpret_cast<float *>(w + 2 * align_up(rows * sizeof(float), 256));
  p.out = static_cast<uint16_t *>(out);
  p.st = st;
  return p;
}

}  // namespace
}  // namespace dflash
