// chunk_attention.cuh -- attention of a ragged chunk's rows over the paged
// cache on the 5th-generation tensor cores: any number of rows per request,
// causal or bidirectional, sliding window, sinks.
//
// Mathematics: one pass over the keys in tiles of 128 with a running maximum
// and sum per row (fp32); the reference maximum only moves when a tile exceeds
// it by 2^8, so the accumulator in tensor memory is rarely rescaled; weights
// are rounded to bf16 for the second product, as its operands must be.
//
// A work tile is up to 128 (or 256) flat rows (token, head of the KV head's
// group) of one request, so the heads that share keys share their loads.
// Ragged requests are mapped to tiles without a prefix sum: request r's tiles
// start at floor(cu_r G / TR) + r, which leaves it room for ceil(rows G / TR).
//
// Three warpgroups a CTA, one CTA an SM: warps 0-3 and 4-7 are two softmax
// groups (one thread a row, 128 rows), warp 8 finds the CTA's next work tile and brings
// its Q with warp 9, warp 10 issues the loads of K and V, warp 11 every MMA.  Each group
// has its own scores S (128 columns of tensor memory; its weights P overwrite them) and
// accumulator O, so one group's softmax runs under the other's two products:
//   more than 128 rows: the groups hold two row tiles over the same key tiles;
//   otherwise the groups take the even and the odd key tiles of the one row tile
//   and their halves are joined at the end (few rows: the key stream is the work).
// kPair: work tiles of 256 rows; otherwise of 128, with more room for keys.
// K and V tiles come through one ring of 128-key slots in the order they are
// used; products of one issuing thread execute in order, so the next scores may
// be issued over the weights that the product before them reads.
//
// Where the grid has more work tiles than there are SMs, a CTA claims blocks that have
// not started (cluster launch control) and goes through its work tiles without a break
// between them: loads, Q and first scores of the next run under the end of the last (4096
// rows of a prompt 131 us with a CTA for each tile, 119 so; 2311 rows of 16 requests,
// window 1024: 75 and 65).
//
// Few row tiles: the keys are cut into S segments (grid z), each writes (m, l,
// O) to the workspace and chunk_merge_kernel joins them.
//
// Rows of K that no row of the tile sees are masked in the scores; such rows of
// V are zeroed in shared memory before the product reads them, since a weight
// of 0 does not silence a NaN.
//
// Bound: single tokens by HBM (64 of them over 1 to 8192 keys each, 32 heads over 8 of
// 128: 209 us, 5.9 TB/s), long chunks by the tensor cores (1024 rows behind 32768
// keys: 409 us, 1.36 PFLOP/s; 16384 rows of one prompt: 1.53).  In the 256-row form a
// key tile takes ~3250 cycles for 2048 of products: their operands and the loads keep
// shared memory busy for another ~2000 of 128 bytes each, and every hand-over between a
// softmax group and the issuing thread waits behind them.  A work tile ends with ~7000
// cycles in which a group has no scores to work on (its last product, its output, the next
// tile's row ranges), which bounds short key spans (the 2311 rows: 9 key tiles each).
#pragma once

#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "cache8.cuh"
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

namespace {

constexpr int kKT = kAttnTileKeys;  // 128 keys per tile
// Registers: 384 threads launch with 168 each, 64512 in all; the softmax groups
// take 200 (a row's 128 scores and 64 packed weights), the third group gives up the
// difference: 2 x 128 x 200 + 128 x 104 = 64512.  (224 and 56: 4% slower; 216 and 72: 1%.)
// The compiler reports 168 a thread for every form, and spills: those with claims reload 20
// to 148 bytes a thread, those without (kMany false) 388 to 428.
constexpr int kSoftmaxRegs = 200, kIssueRegs = 104;
static_assert(256 * kSoftmaxRegs + 128 * kIssueRegs <= 384 * 168, "register split");
// A cache in 8 bits takes a fourth warpgroup: 512 threads of 128 registers, which the compiler
// takes as its limit whatever the split, so the softmax goes over a row's scores twice, 64 at a
// time (tensor memory gives them again at little cost).
template <bool k8>
constexpr int kThreads = k8 ? 512 : 384;
constexpr int kSmemMax = 227 * 1024;
// Barriers of the events that free ring slots, more than can be between a slot's use
// and its next: each event frees a slot or two, of at most 12.
constexpr int kDone = 16;
constexpr uint32_t kChunkBytes = kKT * 128;  // 64 dims of 128 rows, 128-byte swizzled
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;  // S of group g at 128 g, O at 256 + HD g
constexpr float kLog2e = 1.4426950408889634f;

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
  const uint8_t *scales;   // a cache in 8 bits: its scales,
  int block_shift, blocks; // tokens that share one (a power of two), those of a page
};

__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&r)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, %64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, %80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, %96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]),
        "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]),
        "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31]), "=f"(r[32]), "=f"(r[33]), "=f"(r[34]),
        "=f"(r[35]), "=f"(r[36]), "=f"(r[37]), "=f"(r[38]), "=f"(r[39]), "=f"(r[40]), "=f"(r[41]),
        "=f"(r[42]), "=f"(r[43]), "=f"(r[44]), "=f"(r[45]), "=f"(r[46]), "=f"(r[47]), "=f"(r[48]),
        "=f"(r[49]), "=f"(r[50]), "=f"(r[51]), "=f"(r[52]), "=f"(r[53]), "=f"(r[54]), "=f"(r[55]),
        "=f"(r[56]), "=f"(r[57]), "=f"(r[58]), "=f"(r[59]), "=f"(r[60]), "=f"(r[61]), "=f"(r[62]),
        "=f"(r[63]), "=f"(r[64]), "=f"(r[65]), "=f"(r[66]), "=f"(r[67]), "=f"(r[68]), "=f"(r[69]),
        "=f"(r[70]), "=f"(r[71]), "=f"(r[72]), "=f"(r[73]), "=f"(r[74]), "=f"(r[75]), "=f"(r[76]),
        "=f"(r[77]), "=f"(r[78]), "=f"(r[79]), "=f"(r[80]), "=f"(r[81]), "=f"(r[82]), "=f"(r[83]),
        "=f"(r[84]), "=f"(r[85]), "=f"(r[86]), "=f"(r[87]), "=f"(r[88]), "=f"(r[89]), "=f"(r[90]),
        "=f"(r[91]), "=f"(r[92]), "=f"(r[93]), "=f"(r[94]), "=f"(r[95]), "=f"(r[96]), "=f"(r[97]),
        "=f"(r[98]), "=f"(r[99]), "=f"(r[100]), "=f"(r[101]), "=f"(r[102]), "=f"(r[103]),
        "=f"(r[104]), "=f"(r[105]), "=f"(r[106]), "=f"(r[107]), "=f"(r[108]), "=f"(r[109]),
        "=f"(r[110]), "=f"(r[111]), "=f"(r[112]), "=f"(r[113]), "=f"(r[114]), "=f"(r[115]),
        "=f"(r[116]), "=f"(r[117]), "=f"(r[118]), "=f"(r[119]), "=f"(r[120]), "=f"(r[121]),
        "=f"(r[122]), "=f"(r[123]), "=f"(r[124]), "=f"(r[125]), "=f"(r[126]), "=f"(r[127])
      : "r"(taddr)
      : "memory");
}
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
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
// Box of a [tokens][heads][dims] tensor.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, int32_t c0,
                                            int32_t c1, int32_t c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four e4m3 codes as bf16 numbers times 2^120 f, f a bf16 pair: a code's bits, moved to a bf16
// number's place, stand for its value times 2^-120.  Exact.  (A code for NaN comes out as 480.)
__device__ __forceinline__ uint2 widen4(uint32_t w, uint32_t f) {
  const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
  return make_uint2(mul_bf16x2((a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), f),
                    mul_bf16x2((b & 0x80008000u) | ((b >> 4) & 0x07f007f0u), f));
}
// A scale byte's f; the scales past 134 have a factor of their own beside it.
__device__ __forceinline__ uint32_t widen_factor(uint32_t scale) {
  return (min(scale + 120u, 254u) << 7) * 0x10001u;
}
// Bits 7, 15, 23, 31: whether a code is NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }
// 16 codes, whatever they and the scale are.
__device__ __forceinline__ void widen16(const uint4 &codes, uint32_t scale, uint4 *lo, uint4 *hi) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  const uint32_t g = (min(max(scale, 134u) - 7u, 254u) << 7) * 0x10001u;  // 2^(scale - 134)
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint2 v = widen4(w[i], widen_factor(scale));
    const uint32_t bad = scale == 255 ? ~0u : nan_codes(w[i]);
    r[2 * i] = mul_bf16x2(v.x, g) | (bad & 0x80u ? 0x7fffu : 0u) | (bad & 0x8000u ? 0x7fff0000u : 0u);
    r[2 * i + 1] = mul_bf16x2(v.y, g) | (bad & 0x800000u ? 0x7fffu : 0u) |
                   (bad & 0x80000000u ? 0x7fff0000u : 0u);
  }
  *lo = make_uint4(r[0], r[1], r[2], r[3]);
  *hi = make_uint4(r[4], r[5], r[6], r[7]);
}

// Shared memory: Q tiles, the slot ring, a ring of tiles in 8 bits as they arrive, barriers,
// the work in hand.
template <int HD, bool kPair, bool k8>
struct Layout {
  static constexpr uint32_t kSlotBytes = HD / 64 * kChunkBytes;
  static constexpr uint32_t kRing = (kPair ? 2 : 1) * kSlotBytes;
  static constexpr uint32_t kRawBytes = k8 ? kKT * HD : 0;
  static constexpr int kRaws = !k8 ? 1 : HD == 64 ? 8 : kPair ? 4 : 6;
  static constexpr uint32_t kWords = (12 + kDone + 13 + 2 * kRaws) * 8;  // barriers, then 3 words
  static constexpr uint32_t kWork = (kWords + 12 + 15) / 16 * 16;
  static constexpr uint32_t kAnswer = kWork + 2 * sizeof(Work);
  static constexpr uint32_t kJoin = kAnswer + 16;  // m, then l, of a split tile [256]
  static constexpr uint32_t kPlaces = kJoin + 1024;
  static constexpr uint32_t kBarBytes = kPlaces + kSorted;
  static constexpr int kFit =
      (kSmemMax - 1024 - kBarBytes - kRing - kRaws * kRawBytes) / kSlotBytes;
  static constexpr int kSlots = kFit < 12 ? kFit : 12;
  static constexpr uint32_t kRaw = kRing + kSlots * kSlotBytes;
  static constexpr uint32_t kBars = kRaw + kRaws * kRawBytes;
  static constexpr uint32_t kBytes = 1024 + kBars + kBarBytes;
  static_assert(kSlots >= (k8 ? 3 : 5) && kBytes <= kSmemMax, "");
};

// kMany: more blocks than SMs.  A grid that fits them has one work a block, and the form
// without the rest is shorter: cold instructions cost the shortest calls 0.5 us.
//
// k8: a cache in 8 bits.  Its tiles arrive in a ring of their own, and a fourth warpgroup widens
// them to bf16 in the slots that the products read, with their scales: a power of two times four
// significant bits is a bf16 number exactly, so everything behind is as for a 16-bit cache.
template <int HD, bool kPair, bool kMany, bool k8>
__global__ void __launch_bounds__(kThreads<k8>, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm,
                      const __grid_constant__ CUtensorMap tq,
                      const __grid_constant__ ChunkParams p) {
  constexpr int kChunks = HD / 64;
  constexpr int kShift = kPair ? 8 : 7;
  using Lay = Layout<HD, kPair, k8>;
  constexpr uint32_t kSlotBytes = Lay::kSlotBytes;
  constexpr int kSlots = Lay::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~static_cast<uintptr_t>(1023));
  uint8_t *ring = sm + Lay::kRing;  // Q tiles come first
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + Lay::kBars), *done = full + 12;
  uint64_t *s_full = done + kDone, *p_full = s_full + 2, *o_done = p_full + 2;
  uint64_t *q_full = o_done + 2, *q_empty = q_full + 1, *drain = q_empty + 1;
  uint64_t *work_full = drain + 1, *work_read = work_full + 1, *claim = work_read + 1;
  uint64_t *pages_seen = claim + 1;
  [[maybe_unused]] uint64_t *raw_full = pages_seen + 1, *raw_empty = raw_full + Lay::kRaws;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Lay::kBars + Lay::kWords);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  volatile int *bad_flag = abort_flag + 1;  // the work's segment has pages outside the pool
  Work *shared_work = reinterpret_cast<Work *>(sm + Lay::kBars + Lay::kWork);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) ptx::mbar_init(ptx::smem_u32(&full[i]), k8 ? 4 : 1);
    for (int i = 0; i < Lay::kRaws; ++i) {
      ptx::mbar_init(ptx::smem_u32(&raw_full[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&raw_empty[i]), 4);  // the widening warps
    }
    for (int i = 0; i < kDone; ++i) ptx::mbar_init(ptx::smem_u32(&done[i]), 1);
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(ptx::smem_u32(&s_full[g]), 1);
      ptx::mbar_init(ptx::smem_u32(&p_full[g]), 4);  // one arrival per warp of the group
      ptx::mbar_init(ptx::smem_u32(&o_done[g]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(q_full), 2);  // the loading warps
    ptx::mbar_init(ptx::smem_u32(q_empty), 1);
    ptx::mbar_init(ptx::smem_u32(work_full), 1);
    ptx::mbar_init(ptx::smem_u32(work_read), k8 ? 15 : 11);  // every other warp
    ptx::mbar_init(ptx::smem_u32(claim), 1);
    ptx::mbar_init(ptx::smem_u32(pages_seen), 1);
    ptx::mbar_init(ptx::smem_u32(drain), 1);
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
  if (sorted)  // in memory that the works' joins use later
    sort_requests<kPair>(p, kShift, reinterpret_cast<int *>(sm + Lay::kBars + Lay::kJoin),
                         sm + Lay::kBars + Lay::kPlaces);

  // The CTA's works, one after the other: its own block of the grid, then blocks that
  // have not started (there are none where the grid fits the SMs).  The next one is
  // claimed when the loads come to this one's last key tiles, so its own loads and first
  // scores run under the last values and the output of this one; claimed as this
  // one begins, long works pile up on some SMs (64 single tokens over up to 8192 keys 258 us
  // instead of 226).  Every warp sees every work; wound down, it passes over them.
  // (Its wait for one is longer than all that the scheduler can spend before it
  // announces one, so no warp of the softmax groups gives up alone and leaves the others in
  // a barrier.)
  auto next_work = [&](uint32_t w) {
    volatile int dummy = 0;
    Work d = {};
    if (__all_sync(0xffffffffu,
                   chunk_wait<false, 16>(ptx::smem_u32(work_full), w & 1, &dummy)))
      d = shared_work[w & 1];
    else
      *abort_flag = 1;
    return d;
  };
  auto have_read = [&] {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(work_read));
  };
  // A work's Q rows into shared memory, K-major, 128-byte swizzle, once the scores of
  // the work before are done.  Many rows whose tiles begin with a token (the
  // group's heads divide 128) come as tensor boxes: 64 KB took two warps of 16-byte
  // copies 8000 to 12000 cycles, in the way of the next work.  Otherwise each of two warps
  // copies half of them.  Rows past the end are left as they are: they reach no other
  // row.
  auto q_in_boxes = [&](const Work &d) { return p.q_boxes && d.nrow > 64; };
  auto load_q = [&](const Work &d, int half, uint32_t count) {
    bool ok = true;
    if (count > 0)
      ok = __all_sync(0xffffffffu,
                      chunk_wait<false>(ptx::smem_u32(q_empty), (count - 1) & 1, abort_flag));
    if (!ok) return false;
    if (q_in_boxes(d)) {
      if (half == 0 && lane == 0) {
        const int tiles = kPair && d.nrow > 128 ? 2 : 1, tok0 = d.row0 / p.G;
        ptx::mbar_arrive_expect_tx(ptx::smem_u32(q_full), tiles * kSlotBytes);
        for (int t = 0; t < tiles; ++t)
          for (int c = 0; c < kChunks; ++c)
            tma_load_3d(ptx::smem_u32(sm) + t * kSlotBytes + c * kChunkBytes, &tq, 64 * c,
                        d.kvh * p.G, d.a + tok0 + t * (128 / p.G), ptx::smem_u32(q_full));
      }
      __syncwarp();
      return true;
    }
    constexpr int kUnits = HD / 8, kAtOnce = 64 / kUnits;  // 16-byte units of a row
    const int u = lane % kUnits, tok0 = d.row0 / p.G, rem0 = d.row0 - tok0 * p.G;
    const uint32_t base = ptx::smem_u32(sm) + (u >> 3) * kChunkBytes;
    for (int row = half * (kAtOnce / 2) + lane / kUnits; row < d.nrow; row += kAtOnce) {
      const int x = rem0 + row;
      // x / G by the reciprocal, exact for x G < 2^32
      const int tok = p.G == 1 ? x : static_cast<int>(__umulhi(x, p.g_inv));
      const uint16_t *from = p.q + (d.a + tok0 + tok) * p.qs +
                             static_cast<int64_t>(d.kvh * p.G + x - tok * p.G) * HD;
      copy_async16(base + (row >> 7) * kSlotBytes + (row & 127) * 128 +
                       (((u & 7) ^ (row & 7)) << 4),
                   from + 8 * u);
    }
    return true;
  };
  auto q_copied = [&] {
    asm volatile("cp.async.wait_all;" ::: "memory");
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(q_full));
  };

  if (k8 && warp >= 12) {
    // ------------------------------------------------ widening: 32 rows of a tile a warp
    // Of K's and V's tiles in the order they arrive.  Rows of V that no row of the work sees,
    // and those of pages outside the pool, become zeros; what such rows of K hold is masked
    // in the scores.
    const int wr = 32 * (warp & 3);  // the warp's first row
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
      from[e] = row * HD + (HD == 64 ? c : c ^ row8[e]) * 16;
      for (int i = 0; i < 2; ++i)
        to[e][i] = (c >> 2) * kChunkBytes + row * 128 + (((2 * (c & 3) + i) ^ row8[e]) << 4);
    }
    int at = 0, events = 0, freed_by = 0;  // as the loads of a 16-bit cache count them
    bool ok = true;
    for (uint32_t w = 0; w == 0 || kMany; ++w) {
      const Work d = next_work(w);
      have_read();
      if (d.nrow == 0) break;
      if (d.n == 0 || !ok) continue;
      const int n = d.n, t0 = d.t0;
      const bool pairs = kPair && d.nrow > 128;
      const int first = pairs ? 1 : min(n, 2);  // events before V 0's
      // Scales: the rows of a warp have two a tile at most for each of K and V; lanes 2 i and
      // 2 i + 1 look up those of tile i of 16, 16 tiles ahead of their use.
      auto look = [&](int t) {
        const int key = (t0 + t + (lane >> 1)) * kKT + wr + 16 * (lane & 1);
        int page = -1;
        if (t + (lane >> 1) < n && key <= d.hi_max && key + 15 >= d.lo_min) {
          page = p.tbl[static_cast<int64_t>(d.r) * p.M + key / p.P];
          if (page >= p.NP) page = -1;
        }
        return page;
      };
      auto scales_of = [&](int t, int page) {  // K's, V's, and whether the rows are there
        uint32_t s = 0;
        if (page >= 0) {
          const int key = (t0 + t + (lane >> 1)) * kKT + wr + 16 * (lane & 1);
          const uint8_t *at_k =
              p.scales +
              ((static_cast<int64_t>(p.layer) * p.NP + page) * 2 * p.nkv + d.kvh) * p.blocks +
              ((key % p.P) >> p.block_shift);
          s = 0x10000u | at_k[0] | static_cast<uint32_t>(at_k[p.nkv * p.blocks]) << 8;
        }
        return s;
      };
      uint32_t sc = scales_of(0, look(0)), sc_next = 0, sc_last = 0;
      int page = look(16), base = 0;  // first tile of `sc`
      // One place for both kinds and both orders: unrolled at several, the warps wait for
      // instructions.
      for (int i = 0; i < 2 * n; ++i) {
        // two row tiles: K0 V0 K1 V1 ...; one: K0 K1 V0 K2 V1 K3 ... and the last two tiles' V
        int t = i >> 1, kv = i & 1;
        if (!pairs && n > 1) {
          const int j = i - 2;
          kv = j >= 0 && (j >= 2 * (n - 2) || (j & 1) == 0);
          t = j < 0 ? i : kv == 0 ? 2 + (j >> 1) : j >= 2 * (n - 2) ? j - (n - 2) : j >> 1;
        }
        if (kv == 0) {  // K comes first: the scales of 16 tiles more when it gets there
          if (t >= base + 16) {
            sc_last = sc;
            sc = sc_next;
            base += 16;
            page = look(base + 16);
          }
          if (t == base + 8) sc_next = scales_of(base + 16, page);
        }
        const uint32_t scales = t < base ? sc_last : sc;
        const int raw = at % Lay::kRaws, slot = at % kSlots;
        const int last = __shfl_sync(0xffffffffu, freed_by, slot);
        ok = chunk_wait<false>(ptx::smem_u32(&raw_full[raw]),
                               static_cast<uint32_t>((at / Lay::kRaws) & 1), abort_flag);
        if (ok && at >= kSlots)
          ok = chunk_wait<false>(ptx::smem_u32(&done[last % kDone]),
                                 static_cast<uint32_t>((last / kDone) & 1), abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == slot) freed_by = events + t + (kv ? first : 0);
        const uint8_t *src = sm + Lay::kRaw + raw * Lay::kRawBytes;
        uint8_t *dst = ring + slot * kSlotBytes;
        const uint32_t a0 = __shfl_sync(0xffffffffu, scales, 2 * (t & 15)),
                       a1 = __shfl_sync(0xffffffffu, scales, 2 * (t & 15) + 1);
        const uint32_t s0 = kv ? a0 >> 8 & 255 : a0 & 255, s1 = kv ? a1 >> 8 & 255 : a1 & 255;
        const int kb = (t0 + t) * kKT + wr;
        // rows that stay, scales and codes that need nothing more: as a rule
        uint32_t bad = (kv == 0 || (kb >= d.lo_min && kb + 31 <= d.hi_max && (a0 & a1) >> 16)) &&
                               max(s0, s1) <= 134
                           ? 0u
                           : 0x80u;
        uint32_t f = widen_factor(s0);
        uint4 v[kSub], next[kSub];
#pragma unroll
        for (int e = 0; e < kSub; ++e) next[e] = *reinterpret_cast<const uint4 *>(src + from[e]);
        // A short loop: in a long run of instructions that other warps' code drives out of the
        // cache each costs four cycles.
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int e = 0; e < kSub; ++e) v[e] = next[e];
          if (i < 3) {
#pragma unroll
            for (int e = 0; e < kSub; ++e)
              next[e] = *reinterpret_cast<const uint4 *>(src + from[e] + (i + 1) * 8 * HD);
          }
          if (i == 2) f = widen_factor(s1);
#pragma unroll
          for (int e = 0; e < kSub; ++e) {
            const uint2 x = widen4(v[e].x, f), y = widen4(v[e].y, f), z = widen4(v[e].z, f),
                        w = widen4(v[e].w, f);
            bad |= nan_codes(v[e].x) | nan_codes(v[e].y);
            bad |= nan_codes(v[e].z) | nan_codes(v[e].w);
            uint8_t *o = dst + i * 1024;
            *reinterpret_cast<uint4 *>(o + to[e][0]) = make_uint4(x.x, x.y, y.x, y.y);
            *reinterpret_cast<uint4 *>(o + to[e][1]) = make_uint4(z.x, z.y, w.x, w.y);
          }
        }
        if (__any_sync(0xffffffffu, (bad & 0x80808080u) != 0)) {
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const uint32_t mine = i < 2 ? a0 : a1;
#pragma unroll
            for (int e = 0; e < kSub; ++e) {
              const int key = kb + row8[e] + i * 8;
              uint4 lo, hi;
              widen16(*reinterpret_cast<const uint4 *>(src + from[e] + i * 8 * HD), i < 2 ? s0 : s1,
                      &lo, &hi);
              if (kv && (!(mine >> 16) || key < d.lo_min || key > d.hi_max))
                lo = hi = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4 *>(dst + i * 1024 + to[e][0]) = lo;
              *reinterpret_cast<uint4 *>(dst + i * 1024 + to[e][1]) = hi;
            }
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(ptx::smem_u32(&full[slot]));
          ptx::mbar_arrive(ptx::smem_u32(&raw_empty[raw]));
        }
        ++at;
      }
      events += first + n;
    }
  } else if (warp >= 8) {
    if constexpr (!k8) regs_less<kIssueRegs>();
    if (warp == 8) {
      // ---------------------------------------------- scheduler, half of Q
      int block = blockIdx.x, seg = blockIdx.z;
      bool have = true, last = !kMany;
      uint32_t claims = 0, loads = 0;
      Order order = {};
      if (sorted)
        order = read_order(p, lane, reinterpret_cast<const int *>(sm + Lay::kBars + Lay::kJoin),
                           sm + Lay::kBars + Lay::kPlaces);
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
          const uint32_t answer = ptx::smem_u32(sm) + Lay::kBars + Lay::kAnswer;
          if (lane == 0) {
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive_expect_tx(ptx::smem_u32(claim), 16);
            claim_block(answer, ptx::smem_u32(claim));
          }
          __syncwarp();
          volatile int dummy = 0;
          const bool told = __all_sync(
              0xffffffffu, chunk_wait<false, 4>(ptx::smem_u32(claim), claims & 1, &dummy));
          if (!told) *abort_flag = 1;  // a block may be lost: reported
          have = told && claimed_block(answer, &block, &seg);
          __syncwarp();
          ++claims;
          last = !have;  // none left: not to be asked again
        }
        if (lane == 0) {
          shared_work[w & 1] = d;
          ptx::mbar_arrive(ptx::smem_u32(work_full));
        }
        __syncwarp();
        if (d.nrow == 0) break;
        if (d.n > 0 && load_q(d, 0, loads++) && !q_in_boxes(d)) q_copied();
        if (!kMany) break;
        volatile int dummy = 0;
        if (!__all_sync(0xffffffffu,
                        chunk_wait<false, 4>(ptx::smem_u32(work_read), w & 1, &dummy)) ||
            *abort_flag)
          last = true;
      }
      if (*abort_flag && loads > 0) {  // wind down: Q's last boxes land before the CTA ends
        volatile int dummy = 0;
        chunk_wait<false>(ptx::smem_u32(q_full), (loads - 1) & 1, &dummy);
      }
    } else if (warp == 9) {
      // ---------------------------------------------- half of Q, the pages' check
      uint32_t loads = 0;
      for (uint32_t w = 0; w == 0 || kMany; ++w) {
        const Work d = next_work(w);
        have_read();
        if (d.nrow == 0) break;
        if (d.n == 0) continue;
        // pages of the segment outside the pool: none, as a rule
        const int32_t *pages = p.tbl + static_cast<int64_t>(d.r) * p.M;
        const int last_page = min(d.hi_max, (d.t0 + d.n) * kKT - 1) / p.P;
        int lp = max(d.lo_min, d.t0 * kKT) / p.P + lane;
        const int first = lp <= last_page ? pages[lp] : 0;
        if (load_q(d, 1, loads++)) q_copied();
        bool bad = first < 0 || first >= p.NP;
        while ((lp += 32) <= last_page) bad |= pages[lp] < 0 || pages[lp] >= p.NP;
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
          *bad_flag = bad;
          if (bad) raise_status(p.st, DFLASH_DEV_BAD_PAGE);
          ptx::mbar_arrive(ptx::smem_u32(pages_seen));
        }
        __syncwarp();
      }
    } else if (warp == 10) {
      // ---------------------------------------------- TMA producer
      // A lane per box (page rows x 64 dims).  Boxes without a visible key and
      // pages outside the pool are not loaded; their keys are masked below.
      // The next work is claimed once the loads come to the last kAhead tiles.
      constexpr int kAhead = 3;
      const int boxes = kKT / p.box_rows;
      int at = 0;  // place of the next load in the ring's order
      // The events that free slots, counted over all works.  Two row tiles: the
      // work's event 0 is the first scores, 1 + t tile t's values and tile t + 1's
      // scores; one: events 0 and 1 (with one key tile 0) the first scores, then one for tile
      // t's values and tile t + 2's scores.  Lane s keeps the one that frees slot s.
      int events = 0, freed_by = 0;
      bool ok = true;
      for (uint32_t w = 0; w == 0 || kMany; ++w) {
        const Work d = next_work(w);
        if (d.nrow == 0 || d.n == 0 || !ok) {
          have_read();
          if (d.nrow == 0) break;
          continue;
        }
        const int n = d.n, t0 = d.t0, lo_min = d.lo_min, hi_max = d.hi_max;
        const int first = kPair && d.nrow > 128 ? 1 : min(n, 2);  // events before V 0's
        const uint64_t pol =
            d.total <= (1 << kShift) ? ptx::policy_evict_first() : ptx::policy_evict_normal();
        auto fetch = [&](int t) {  // page of box `lane` of tile t, -1 where it is not loaded
          int page = -1;
          if (lane < boxes && t < n) {
            const int key0 = (t0 + t) * kKT + lane * p.box_rows;
            if (key0 <= hi_max && key0 + p.box_rows > lo_min) {
              page = p.tbl[static_cast<int64_t>(d.r) * p.M + key0 / p.P];
              if (page >= p.NP) page = -1;
            }
          }
          return page;
        };
        auto load = [&](int t, int kv, int page) {
          if (!ok) return;
          bool got = true;
          if constexpr (k8) {  // into the ring of tiles in 8 bits
            const int raw = at % Lay::kRaws;
            if (lane == 0 && at >= Lay::kRaws)
              got = chunk_wait<false>(ptx::smem_u32(&raw_empty[raw]),
                                      static_cast<uint32_t>((at / Lay::kRaws - 1) & 1), abort_flag);
            ok = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
            if (!ok) return;
            const bool skip = t == p.skip_tile && kv == 0;
            const uint32_t bar = ptx::smem_u32(&raw_full[raw]);
            const uint32_t bytes =
                __popc(__ballot_sync(0xffffffffu, page >= 0)) * p.box_rows * HD;
            if (lane == 0 && !skip) ptx::mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            // other lanes for each load: one thread's copies complete one after another
            const int b = (lane - at * boxes) & 31;
            const int pg = __shfl_sync(0xffffffffu, page, b);
            if (b < boxes && pg >= 0 && !skip) {
              const int key0 = (t0 + t) * kKT + b * p.box_rows;
              const int64_t row =
                  (((static_cast<int64_t>(p.layer) * p.NP + pg) * 2 + kv) * p.nkv + d.kvh) * p.P +
                  key0 % p.P;
              ptx::tma_load_2d_hint(
                  ptx::smem_u32(sm + Lay::kRaw + raw * Lay::kRawBytes + b * p.box_rows * HD), &tm,
                  0, static_cast<int32_t>(row), bar, pol);
            }
            ++at;
            return;
          }
          const int last = __shfl_sync(0xffffffffu, freed_by, at % kSlots);
          if (lane == 0 && at >= kSlots)
            got = chunk_wait<false>(ptx::smem_u32(&done[last % kDone]),
                                    static_cast<uint32_t>((last / kDone) & 1), abort_flag);
          ok = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
          if (!ok) return;
          const bool skip = t == p.skip_tile && kv == 0;
          const int slot = at % kSlots;
          if (lane == slot) freed_by = events + t + (kv ? first : 0);
          const uint32_t bar = ptx::smem_u32(&full[slot]);
          const uint32_t bytes =
              __popc(__ballot_sync(0xffffffffu, page >= 0)) * kChunks * p.box_rows * 128u;
          if (lane == 0 && !skip) ptx::mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          // other lanes for each load: one thread's copies complete one after another
          const int j = (lane - at * boxes * kChunks) & 31, b = j / kChunks, c = j % kChunks;
          const int pg = __shfl_sync(0xffffffffu, page, b & 31);
          if (b < boxes && pg >= 0 && !skip) {
            const int key0 = (t0 + t) * kKT + b * p.box_rows;
            const int64_t row =
                (((static_cast<int64_t>(p.layer) * p.NP + pg) * 2 + kv) * p.nkv + d.kvh) * p.P +
                key0 % p.P;
            ptx::tma_load_2d_hint(ptx::smem_u32(ring + slot * kSlotBytes + c * kChunkBytes +
                                                b * p.box_rows * 128),
                                  &tm, c * 64, static_cast<int32_t>(row), bar, pol);
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
        events += first + n;
      }
      if (*abort_flag && lane == 0) {  // wind down: the last copies land before the CTA ends
        constexpr int kIn = k8 ? Lay::kRaws : kSlots;
        uint64_t *arrived = k8 ? raw_full : full;
        for (int i = max(at - kIn, 0); i < at; ++i) {
          volatile int dummy = 0;
          chunk_wait<false>(ptx::smem_u32(&arrived[i % kIn]), static_cast<uint32_t>((i / kIn) & 1),
                            &dummy);
        }
      }
    } else {
      // ---------------------------------------------- MMA issuer
      // One thread for both groups: their blocks of products go into the pipe in
      // turn (mixed by two issuers, both groups wait for the pipe and then leave
      // it idle together: 570 us where one issuer took 430, 1024 rows behind 32768 keys).
      constexpr uint32_t idesc_qk = ptx::idesc_bf16_f32(128, kKT, false);
      constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(128, HD, true);
      // warp-uniform copies
      const uint32_t tm0 = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t qbase = __shfl_sync(0xffffffffu, ptx::smem_u32(sm), 0);
      const uint32_t rbase = __shfl_sync(0xffffffffu, ptx::smem_u32(ring), 0);
      const uint64_t dq = ptx::desc_kmajor_sw128(qbase, 0);
      const uint64_t dk = ptx::desc_kmajor_sw128(rbase, 0);
      const uint64_t dv = ptx::smem_desc(rbase, kChunkBytes, 1024, ptx::kSwizzle128B);
      const uint32_t full0 = ptx::smem_u32(full);
      // Waits on up to three barriers at the cost of one: each is polled by lanes
      // of its own.  A slot in the ring's order, or a barrier and its phase.
      struct At {
        uint32_t bar, phase;
      };
      int base = 0, events = 0;  // the work's first place in the ring's order, its first event
      uint32_t handed0 = 0u, handed1 = 0u, loads = 0u;  // phases of p_full and q_full
      bool ok = true, pairs = false;
      auto slot = [&](int at) {
        return At{full0 + 8u * (at % kSlots), static_cast<uint32_t>((at / kSlots) & 1)};
      };
      auto wait = [&](At a, At b, At c) {
        const At x = lane == 1 ? b : lane == 2 ? c : a;
        const bool got = __all_sync(0xffffffffu, chunk_wait<true>(x.bar, x.phase, abort_flag));
        ptx::tc_fence_after();
        return got;
      };
      auto qk = [&](int g, int at) {  // S_g = Q K^T
        const uint64_t a = dq + (((pairs ? g : 0) * kSlotBytes) >> 4);
        const uint64_t b = dk + (((at % kSlots) * kSlotBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * kChunkBytes + (ks & 3) * 32) >> 4;
          ptx::mma_bf16(tm0 + 128 * g, a + off, b + off, idesc_qk, ks > 0 ? 1u : 0u);
        }
        ptx::mma_commit(ptx::smem_u32(&s_full[g]));
      };
      auto pv = [&](int g, int at, bool first) {  // O_g (+)= P V
        const uint64_t b = dv + (((at % kSlots) * kSlotBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < kKT / 16; ++ks)
          ptx::mma_bf16_ts(tm0 + kColO + HD * g, tm0 + 128 * g + ks * 8, b + ((ks * 2048) >> 4),
                           idesc_pv, (!first || ks > 0) ? 1u : 0u);
      };
      auto event = [&](int e) { ptx::mma_commit(ptx::smem_u32(&done[(events + e) % kDone])); };
      for (uint32_t w = 0; w == 0 || kMany; ++w) {
        const Work d = next_work(w);
        have_read();
        if (d.nrow == 0) break;
        const int tiles = __shfl_sync(0xffffffffu, d.n, 0);
        if (!ok || tiles == 0) continue;
        pairs = kPair && __shfl_sync(0xffffffffu, d.nrow, 0) > 128;
        const int step = pairs ? 1 : 2, first = min(step, tiles);
        ok = wait(At{ptx::smem_u32(q_full), loads & 1}, slot(base),
                  slot(!pairs && tiles > 1 ? base + 1 : base));
        ++loads;
        if (ok && elect_one()) {
          qk(0, base);
          if (pairs) {
            qk(1, base);
            event(0);
          } else {
            event(0);
            if (tiles > 1) {
              qk(1, base + 1);
              event(1);
            }
          }
          if (tiles <= step) ptx::mma_commit(ptx::smem_u32(q_empty));
        }
        __syncwarp();
        for (int t = 0; ok && t < tiles; ++t) {
          // V's place in the ring's order: two row tiles K0 V0 K1 V1 ..., one
          // K0 K1 V0 K2 V1 K3 ...
          const int av = base + (pairs ? 2 * t + 1 : min(t + 2, tiles) + t);
          const bool more = t + step < tiles;
          for (int i = 0; ok && i < (pairs ? 2 : 1); ++i) {
            const int g = pairs ? i : t & 1;
            const At k = slot(more ? av + 1 : av);
            ok = wait(At{ptx::smem_u32(&p_full[g]), (g ? handed1 : handed0) & 1}, slot(av), k);
            if (!ok) break;
            if (g) ++handed1; else ++handed0;
            if (elect_one()) {
              pv(g, av, t < step);
              if (more) qk(g, av + 1);
              if (!more) ptx::mma_commit(ptx::smem_u32(&o_done[g]));
              if (!pairs || i == 1) {
                event(first + t);
                if (t + step == tiles - 1) ptx::mma_commit(ptx::smem_u32(q_empty));
              }
            }
            __syncwarp();
          }
        }
        base += 2 * tiles;
        events += first + tiles;
      }
      if (!ok) {
        if (elect_one()) ptx::mma_commit(ptx::smem_u32(drain));
        __syncwarp();
        volatile int dummy = 0;
        chunk_wait<false>(ptx::smem_u32(drain), 0u, &dummy);
      }
    }
  } else {
    if constexpr (!k8) regs_more<kSoftmaxRegs>();
    // ------------------------------------------------ softmax groups
    const int g = warp >> 2;
    const int tid = threadIdx.x & 127;  // TMEM lane = row of the group's tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + 128 * g + lane_off, tm_o = tmem + kColO + HD * g + lane_off;
    float *join = reinterpret_cast<float *>(sm + Lay::kBars + Lay::kJoin);
    int base = 0;  // the work's first place in the ring's order
    uint32_t loads = 0u, scores = 0u, outs0 = 0u, outs1 = 0u;  // of pages_seen, s_full, o_done
    bool ok = true;
    for (uint32_t wk = 0; wk == 0 || kMany; ++wk) {
      // its fields are read again where they are needed: this slot is not written before
      // the next work is read
      const volatile Work &d = shared_work[wk & 1];
      volatile int dummy = 0;
      int nrow = 0, n = 0;
      if (__all_sync(0xffffffffu,
                     chunk_wait<false, 16>(ptx::smem_u32(work_full), wk & 1, &dummy))) {
        nrow = d.nrow;
        n = d.n;
      } else {
        *abort_flag = 1;
      }
      bool bad_pages = false;
      if (n > 0) {
        if (ok)
          ok = __all_sync(0xffffffffu,
                          chunk_wait<false>(ptx::smem_u32(pages_seen), loads & 1, abort_flag));
        ++loads;
        bad_pages = ok && *bad_flag != 0;
      }
      have_read();
      if (nrow == 0) break;
      const int lo_min = d.lo_min, hi_max = d.hi_max, t0 = d.t0;
      const bool split = !kPair || nrow <= 128;

      // this thread's row and the keys it sees
      const int rt = (split ? 0 : 128 * g) + tid;
      const bool real = rt < nrow;
      int lo = 0, hi = -1;
      if (real) key_range(p, d.c + (d.row0 + rt) / p.G, d.kv, &lo, &hi);

      const bool active = (split ? 0 : 128 * g) + (warp & 3) * 32 < nrow;  // the warp holds rows
      float m_ref = -INFINITY, l = 0.f;
      int u = 0;
      for (int t = split ? g : 0; ok && t < n; t += split ? 2 : 1, ++u) {
        ok = __all_sync(0xffffffffu, chunk_wait<false>(ptx::smem_u32(&s_full[g]), scores & 1,
                                                       abort_flag));
        if (!ok) break;
        ++scores;
        ptx::tc_fence_after();
        const int kb = (t0 + t) * kKT;
        // the tile holds keys that some row of the CTA does not see, or bad pages
        const bool edge = bad_pages || kb < lo_min || kb + kKT - 1 > hi_max;
        constexpr int kCols = k8 ? 64 : 128;  // scores of a row held at once
        float sv[kCols];
        if constexpr (!k8) tmem_ld128(tm_s, sv);
        uint32_t okm[4] = {~0u, ~0u, ~0u, ~0u};  // keys on pages of the pool
        if (edge) {
          if (bad_pages) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int lp = (kb + 32 * w + lane) / p.P;
              const int page = lp < p.M ? p.tbl[static_cast<int64_t>(d.r) * p.M + lp] : -1;
              okm[w] = __ballot_sync(0xffffffffu, page >= 0 && page < p.NP);
            }
          }
          if constexpr (!k8) {  // (the widening warps did it)
            // V rows no row of this tile sees: zero, before P is handed over
            const int at = base + (split ? min(t + 2, n) + t : 2 * t + 1);  // V's place in the ring
            const int slot = at % kSlots;
            ok = __all_sync(0xffffffffu,
                            chunk_wait<false>(ptx::smem_u32(&full[slot]),
                                              static_cast<uint32_t>((at / kSlots) & 1), abort_flag));
            if (!ok) break;
            const int key = kb + tid, w4 = warp & 3;
            const uint32_t mine = w4 == 0 ? okm[0] : w4 == 1 ? okm[1] : w4 == 2 ? okm[2] : okm[3];
            if (key < lo_min || key > hi_max || !((mine >> lane) & 1u)) {
#pragma unroll
              for (int c = 0; c < kChunks; ++c) {
                uint4 *v = reinterpret_cast<uint4 *>(ring + slot * kSlotBytes + c * kChunkBytes +
                                                     tid * 128);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[(e + tid) & 7] = make_uint4(0, 0, 0, 0);
              }
            }
            ptx::fence_proxy_async_smem();
          }
        }
        if (!active) {  // its rows of P may hold anything: they reach no other row
          ptx::tc_fence_before();
          __syncwarp();  // all lanes' zeros are written
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&p_full[g]));
          continue;
        }
        const bool cut = !(lo <= kb && hi >= kb + kKT - 1);
        auto mask = [&](int c0) {  // columns c0 on, in sv
          if (bad_pages) {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (!((okm[(c0 + c) >> 5] >> (c & 31)) & 1u)) sv[c] = -INFINITY;
          }
          if (cut) {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (kb + c0 + c < lo || kb + c0 + c > hi) sv[c] = -INFINITY;
          }
        };
        float mx[4];
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += kCols) {
          if constexpr (k8) ptx::tmem_ld64f_sync(tm_s + c0, sv);
          mask(c0);
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = c0 ? fmaxf(mx[c], sv[c]) : sv[c];
#pragma unroll
          for (int c = 4; c < kCols; c += 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (c + e + 4 < kCols) mx[e] = fmaxf(fmaxf(mx[e], sv[c + e]), sv[c + e + 4]);
              else mx[e] = fmaxf(mx[e], sv[c + e]);
          }
        }
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        float corr = 1.f;
        bool need = false;
        if (m_ref == -INFINITY) {
          m_ref = tmax;
        } else if (tmax > m_ref + 8.f) {
          corr = ptx::ex2(m_ref - tmax);
          m_ref = tmax;
          need = true;
        }
        // the group's previous product completed before this S did
        if (__any_sync(0xffffffffu, need)) {
          for (int c = 0; c < HD; c += 16) {
            uint32_t ov[16];
            ptx::tmem_ld16_sync(tm_o + c, ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr);
            ptx::tmem_st16(tm_o + c, ov);
          }
        }
        const float nm = m_ref == -INFINITY ? 0.f : -m_ref;  // nothing seen yet: weights 2^-inf
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(nm, nm);
        float2 sum[2] = {};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if constexpr (k8) {  // P of the first half lies over scores that were used
            ptx::tmem_ld64f_sync(tm_s + 64 * c, sv);
            mask(64 * c);
          }
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int x = (k8 ? 0 : 64 * c) + 2 * e;
            float2 w = fma2(make_float2(sv[x], sv[x + 1]), sc2, nm2);
            w.x = ptx::ex2(w.x);
            w.y = ptx::ex2(w.y);
            sum[e & 1] = add2(sum[e & 1], w);
            pk[e] = ptx::pack_bf16x2(w.x, w.y);
          }
          tmem_st32(tm_s + 32 * c, pk);
        }
        sum[0] = add2(sum[0], sum[1]);
        l = l * corr + (sum[0].x + sum[0].y);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&p_full[g]));
      }
      // ---------------------------------------------- epilogue
      const bool had0 = n > 0, had1 = split ? n > 1 : n > 0;  // groups with products
      if (ok && (g ? had1 : had0)) {
        ok = __all_sync(0xffffffffu, chunk_wait<false>(ptx::smem_u32(&o_done[g]),
                                                       (g ? outs1 : outs0) & 1, abort_flag));
        ptx::tc_fence_after();
      }
      if (split && ok && (g ? had0 : had1)) {  // the other group's products
        ok = __all_sync(0xffffffffu, chunk_wait<false>(ptx::smem_u32(&o_done[g ^ 1]),
                                                       (g ? outs0 : outs1) & 1, abort_flag));
        ptx::tc_fence_after();
      }
      outs0 += had0;
      outs1 += had1;
      base += 2 * n;
      // the row's state over both groups, and this thread's share of its dims
      const int dims = split ? HD / 2 : HD, d0 = split ? g * (HD / 2) : 0;
      float m = ok ? m_ref : -INFINITY, own = 1.f, other = 0.f;
      if (split && n > 0) {
        // Both groups hold the row in the same TMEM lane: the states go through shared
        // memory, the other accumulator is read where it is.
        join[g * 128 + tid] = m;
        const bool bad = ptx::bar_or(1, 256, !ok);
        const float m2 = join[(g ^ 1) * 128 + tid];
        ptx::bar_sync(1, 256);
        join[g * 128 + tid] = l;
        ptx::bar_sync(1, 256);
        const float l2 = join[(g ^ 1) * 128 + tid];
        ok = ok && !bad;
        m = bad ? -INFINITY : fmaxf(m_ref, m2);
        own = bad || m_ref == -INFINITY ? 0.f : ptx::ex2(m_ref - m);
        other = bad || m2 == -INFINITY ? 0.f : ptx::ex2(m2 - m);
        l = l * own + l2 * other;
      }
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

// Joins the S partial states of a row: one warp per (row, head), HD / 32 dims a
// lane.  All of a batch's loads are issued before any is used (one memory round
// trip for up to 20 segments; four and two where there are no more, since the places past S
// are read too).  Rows of no request are passed over, as the main
// kernel passes them; O of a segment without keys is not written, so what is read
// there is selected away.
template <int HD, int kBatch>
__global__ void __launch_bounds__(128) chunk_merge_kernel(const ChunkParams p) {
  constexpr int E = HD / 32;
  ptx::griddep_launch();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / p.hq), h = static_cast<int>(w % p.hq);
  if (t >= p.n_rows) return;
  const float *o = p.ws_o + w * p.S * HD + lane * E;
  float m = p.sinks ? p.sinks[h] * kLog2e : -INFINITY, l = p.sinks ? 1.f : 0.f;
  float acc[E] = {};
  for (int s0 = 0; s0 < p.S; s0 += kBatch) {
    const bool in = lane < kBatch && s0 + lane < p.S;
    const float mj = in ? __ldcg(p.ws_m + w * p.S + s0 + lane) : -INFINITY;
    const float lj = in ? __ldcg(p.ws_l + w * p.S + s0 + lane) : 0.f;
    float ov[kBatch][E];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float *from = o + static_cast<int64_t>(min(s0 + j, p.S - 1)) * HD;
      if constexpr (E == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(from));
        ov[j][0] = v.x;
        ov[j][1] = v.y;
        ov[j][2] = v.z;
        ov[j][3] = v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(from));
        ov[j][0] = v.x;
        ov[j][1] = v.y;
      }
    }
    const float mn = fmaxf(m, warp_max(mj));
    if (mn == -INFINITY) continue;
    const float sc = m == -INFINITY ? 0.f : ptx::ex2(m - mn);
    const float wj = mj == -INFINITY ? 0.f : ptx::ex2(mj - mn);
    l = l * sc + warp_sum(wj * lj);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= sc;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float ws = __shfl_sync(0xffffffffu, wj, j);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += ws != 0.f ? ws * ov[j][e] : 0.f;
    }
    m = mn;
  }
  // the row's request
  int lo = 0, n = p.B;  // the last request whose first row is <= t
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool at = lane * step < n && p.cu[lo + lane * step] <= t;
    const int c = max(__popc(__ballot_sync(0xffffffffu, at)), 1) - 1;
    lo += c * step;
    n = min(step, n - c * step);
  }
  Request rq;
  load_request(p, lo, &rq);
  if (!check_request(p, false, &rq) || t < rq.a || t >= rq.b) return;
  float f[E];
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = l > 0.f ? acc[e] / l : 0.f;
  uint16_t *dst = p.out + t * p.os + static_cast<int64_t>(h) * HD + lane * E;
  const uint32_t a = ptx::pack_bf16x2(f[0], f[1]);
  if constexpr (E == 4)
    *reinterpret_cast<uint2 *>(dst) = make_uint2(a, ptx::pack_bf16x2(f[2], f[3]));
  else
    *reinterpret_cast<uint32_t *>(dst) = a;
}

// Pair form where the mean request fills more than one 128-row tile.
bool pair_form(const dflash_geom &g, int B, int n_rows) {
  return static_cast<int64_t>(n_rows) * (g.hq / g.nkv) > 128LL * B;
}

// Work tiles of a chunk, at most.
int64_t chunk_tiles(const dflash_geom &g, int B, int n_rows) {
  return ((static_cast<int64_t>(n_rows) * (g.hq / g.nkv)) >> (pair_form(g, B, n_rows) ? 8 : 7)) + B;
}

// Work tiles of a call with one request.
int64_t works_of_one(const dflash_geom &g, int n_rows) {
  const int tr = pair_form(g, 1, n_rows) ? 256 : 128;
  return (static_cast<int64_t>(n_rows) * (g.hq / g.nkv) + tr - 1) / tr * g.nkv;
}

// Two segments of one request: its work tiles fill the SMs a whole number of times
// but for some; each SM left over takes the tails of this many tiles, cut so that all end
// together (1: halves).
int tail_tiles(const dflash_geom &g, int B, int n_rows) {
  if (B != 1) return 1;
  const int64_t works = works_of_one(g, n_rows), sms = device_sm_count();
  const int64_t idle = (works + sms - 1) / sms * sms - works;
  return idle == 0 ? 1 : static_cast<int>(std::min<int64_t>((works + idle - 1) / idle, 64));
}

// Segments the keys are cut into, by a model of the call's time in key tiles: a CTA
// costs its tiles and kFixed more, and a merge costs kMerge and its bytes.  Lengths are on
// the device: the table's width, or the window, stands for the longest span, so the
// figures below hold for tables about as wide as the longest request.  Behind 32768 keys of
// table a prompt of 4096 rows takes two segments and 181 us instead of 117, 64 single tokens
// over up to 8192 keys 227 instead of 211, 16 over up to 2048 keys 34.9 (three) instead of
// 29.8, 3 short requests 10.8 (25) instead of 7.2; one token over 1000 keys gains (13.9, 11.8).
//
// One request whose rows are few beside its keys: all work tiles are about as long,
// and the SMs take them in rounds; two segments are cut so that the last round leaves no
// SM without work (1024 rows behind 32768 keys, 32 heads over 8, us: 410 with one
// segment, 388 so; 2048 rows 812 and 767, and 893 with three).  Otherwise the SMs share the
// CTAs, and the last ones run alone for a part of their time; 0.6 of the longest
// span stands for the mean of four requests or more (16 single tokens over up to
// 16384 keys 162 with one segment, 105 with two, 124 with three; over up to 2048 keys 31
// and 32 with two; one token over 32768 keys 33 with 19).
int segments_of(const dflash_geom &g, int B, int n_rows, int window) {
  constexpr double kFixed = 7.0, kMerge = 3.0;
  const double ctas = static_cast<double>(chunk_tiles(g, B, n_rows)) * g.nkv;
  const double sms = device_sm_count();
  double longest = static_cast<double>(g.max_pages) * g.page_size / kKT;
  if (window > 0) longest = std::min(longest, (static_cast<double>(window) + n_rows) / kKT + 1.0);
  const double mean = B >= 4 ? 0.6 * longest : longest;
  const bool alike = B == 1 && longest * kKT >= 2.0 * n_rows;
  const int64_t works = works_of_one(g, n_rows), left = works % device_sm_count();
  // a segment's partial results, written and read: key tiles (of 1.5 us) at 6 TB/s
  const double part = 8.0 * n_rows * g.hq * g.head_dim / 9e6;
  int best = 1;
  double least = 0.0;
  for (int S = 1; S == 1 || (S <= 64 && 4 * S <= longest && ctas * (S - 1) <= 4 * sms); ++S) {
    double one = kFixed + longest / S;
    if (S == 2 && alike)
      one = kFixed + main_tiles(static_cast<int>(longest), tail_tiles(g, B, n_rows));
    double t = one;
    if (alike)
      t *= std::ceil(static_cast<double>(works) * (S == 2 && left ? 1 : S) / sms);
    else if (ctas * S > sms)  // in the order of cost the last ones are short
      t = std::max(one, ctas * (mean + kFixed * S) / sms + (B > kSorted ? 0.5 : 0.25) * one);
    if (S > 1) t += kMerge + part * S;
    if (S == 1 || t < least) {
      least = t;
      best = S;
    }
  }
  return best;
}

size_t workspace_of(const dflash_geom &g, int B, int n_rows, int S) {
  if (B < 1 || n_rows < 1) return 0;
  if (S <= 0) S = segments_of(g, B, n_rows, 0);
  if (S == 1) return 0;
  const size_t rows = static_cast<size_t>(n_rows) * g.hq * S;
  return 2 * align_up(rows * sizeof(float), 256) + rows * g.head_dim * sizeof(float);
}

// [n_rows][hq][head_dim] in boxes of 128 rows (token, head of a group) by 64 dims.
cudaError_t q_tensor_map(CUtensorMap *m, const dflash_geom &g, int n_rows, const void *q,
                         int64_t q_stride) {
  const EncodeTiled encode = encode_tiled_fn();
  if (!encode) return cudaErrorNotSupported;
  const cuuint32_t G = g.hq / g.nkv;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(g.head_dim), static_cast<cuuint64_t>(g.hq),
                              static_cast<cuuint64_t>(n_rows)};
  const cuuint64_t strides[2] = {2ull * g.head_dim, 2ull * static_cast<cuuint64_t>(q_stride)};
  const cuuint32_t box[3] = {64, G, 128 / G}, each[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box,
                each, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
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
                hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int HD, bool kPair, bool kMany, bool k8>
cudaError_t launch_form(const CUtensorMap &tm, const CUtensorMap &tq, const ChunkParams &p,
                        dim3 grid, cudaStream_t s) {
  const cudaError_t e = ensure_smem_limit<chunk_attn_kernel<HD, kPair, kMany, k8>>(kSmemMax);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads<k8>);
  cfg.dynamicSmemBytes = Layout<HD, kPair, k8>::kBytes;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_attn_kernel<HD, kPair, kMany, k8>, tm, tq, p);
}

template <int HD, bool k8>
cudaError_t launch_main(bool pair, const CUtensorMap &tm, const CUtensorMap &tq,
                        const ChunkParams &p, dim3 grid, cudaStream_t s) {
  const bool many = static_cast<int64_t>(grid.x) * grid.z > device_sm_count();
  if (pair)
    return many ? launch_form<HD, true, true, k8>(tm, tq, p, grid, s)
                : launch_form<HD, true, false, k8>(tm, tq, p, grid, s);
  return many ? launch_form<HD, false, true, k8>(tm, tq, p, grid, s)
              : launch_form<HD, false, false, k8>(tm, tq, p, grid, s);
}

// pool: the 16-bit cache, or the codes of c8.
template <bool k8>
cudaError_t launch_attention(const dflash_geom &g, int B, int layer, int n_rows, const void *q,
                             int64_t q_stride, const void *pool, const dflash_cache8 *c8,
                             const int32_t *tbl, const int32_t *cu, const int32_t *ctx,
                             const int32_t *kv, int32_t window, const float *sinks, float scale,
                             int mask_mode, int S, void *ws, void *out, int64_t out_stride,
                             int32_t *st, cudaStream_t s) {
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
  p.tails = S == 2 ? tail_tiles(g, B, n_rows) : 1;
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
  CUtensorMap tm;
  const uint64_t pool_rows = static_cast<uint64_t>(g.num_layers) * g.num_pool_pages * 2 * g.nkv *
                             static_cast<uint64_t>(g.page_size);
  cudaError_t e;
  if constexpr (k8) {
    p.scales = static_cast<const uint8_t *>(c8->scales);
    p.block_shift = c8->block == 16 ? 4 : c8->block == 32 ? 5 : 6;
    p.blocks = p.P / c8->block;
    e = code_tensor_map(&tm, pool, pool_rows, g.head_dim, p.box_rows);
  } else {
    e = make_tmap_bf16_2d(&tm, pool, pool_rows, g.head_dim, g.head_dim, p.box_rows, 64);
  }
  if (e != cudaSuccess) return e;
  // Q in boxes: not worth its tensor map where the mean request has few rows
  CUtensorMap tq = {};
  p.q_boxes = 128 % p.G == 0 && static_cast<int64_t>(n_rows) * p.G > 64LL * B &&
              q_stride < (1LL << 38);
  if (p.q_boxes && (e = q_tensor_map(&tq, g, n_rows, q, q_stride)) != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(chunk_tiles(g, B, n_rows) * g.nkv), 1, S);
  const bool pair = pair_form(g, B, n_rows);
  e = g.head_dim == 64 ? launch_main<64, k8>(pair, tm, tq, p, grid, s)
                       : launch_main<128, k8>(pair, tm, tq, p, grid, s);
  if (e != cudaSuccess || S == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(n_rows) * g.hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (g.head_dim == 64)
    return cudaLaunchKernelEx(&cfg, S > 4   ? chunk_merge_kernel<64, 20>
                                    : S > 2 ? chunk_merge_kernel<64, 4>
                                            : chunk_merge_kernel<64, 2>, p);
  return cudaLaunchKernelEx(&cfg, S > 4   ? chunk_merge_kernel<128, 20>
                                  : S > 2 ? chunk_merge_kernel<128, 4>
                                          : chunk_merge_kernel<128, 2>, p);
}

}  // namespace
}  // namespace dflash
