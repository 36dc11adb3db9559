// chunk_merge.cu -- joins what the segments of a chunk's attention leave, over a 16-bit cache
// (chunk_attention.cu) or one in 8 bits (chunk_attention8.cu, chunk_attention8_few.cu).
#include "chunk_work.cuh"

namespace dflash {
namespace {

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
  bool any = false;  // the row saw a key
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
    const float top = warp_max(mj);
    if (top == -INFINITY) continue;
    any = true;
    const float mn = fmaxf(m, top);
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
  float f[E];  // (a sum of NaN, from any segment or the sink, makes the row NaN)
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = any ? acc[e] / l : 0.f;
  uint16_t *dst = p.out + t * p.os + static_cast<int64_t>(h) * HD + lane * E;
  const uint32_t a = ptx::pack_bf16x2(f[0], f[1]);
  if constexpr (E == 4)
    *reinterpret_cast<uint2 *>(dst) = make_uint2(a, ptx::pack_bf16x2(f[2], f[3]));
  else
    *reinterpret_cast<uint32_t *>(dst) = a;
}

}  // namespace

cudaError_t launch_merge(const dflash_geom &g, const ChunkParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.n_rows) * g.hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (g.head_dim == 64)
    return cudaLaunchKernelEx(&cfg, p.S > 4   ? chunk_merge_kernel<64, 20>
                                    : p.S > 2 ? chunk_merge_kernel<64, 4>
                                            : chunk_merge_kernel<64, 2>, p);
  return cudaLaunchKernelEx(&cfg, p.S > 4   ? chunk_merge_kernel<128, 20>
                                  : p.S > 2 ? chunk_merge_kernel<128, 4>
                                          : chunk_merge_kernel<128, 2>, p);
}

}  // namespace dflash
