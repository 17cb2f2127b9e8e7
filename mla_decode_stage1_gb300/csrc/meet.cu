// meet.cu -- the partial results of a shared-prefix decode become its output:
// for every query token and head the decode kernel's partials over the request's
// own end and the prefix kernel's over the prefix, weighted by their log-sum-exp.
//
//     M = max_s lse_s, w_s = 2^(lse_s - M), out = sum_s w_s o_s / sum_s w_s,
//     lse = (M + log2 sum w) ln 2.
//
// A part without keys, or without weight, has lse = -inf and adds nothing; one
// whose lse is NaN makes the row NaN.
//
// Bound: latency, and memory for many rows.  The prefix kernel's partials stand as
// [dim / 8][row][dim % 8], so that both kernels move whole lines: a CTA takes a
// token's 16 rows and 128 of the 512 dims, a thread 8 dims of a row (16 rows of 32
// bytes stand together), with up to 8 partials in flight.

#include "shared.h"

namespace mla {
namespace {

constexpr int kThreads = 256;                 // 16 rows x 16 groups of 8 dims

template <int kAhead>
__global__ void __launch_bounds__(kThreads) meet_kernel(const MeetParams p) {
  const int64_t token = blockIdx.x / 4;
  const int row = threadIdx.x & 15, group = blockIdx.x % 4 * 16 + (threadIdx.x >> 4);
  const MeetJob j = p.jobs[token];
  const bool sound = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp &&
                     check_of(j, p.stamp) == j.check;
  if (!sound) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrStale);
    return;
  }
  const int n = j.own_count + j.prefix_count;
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the partials are there
  float M = -INFINITY, wsum = 0.0f, acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int s0 = 0; s0 < n; s0 += kAhead) {
    float lse[kAhead];
    float4 v[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = s0 + u;
      lse[u] = -INFINITY;
      v[u][0] = v[u][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (s >= n) continue;
      const float* src;
      if (s < j.own_count) {
        const int64_t at = static_cast<int64_t>(j.own_first + s) * p.own_rows + j.own_row + row;
        lse[u] = p.own_lse[at];
        src = p.own_o + at * kVDim + 8 * group;
      } else {
        const int64_t block = j.prefix_first + static_cast<int64_t>(s - j.own_count) * p.blocks;
        lse[u] = p.prefix_lse[block * kSpRows + j.prefix_row + row];
        src = p.prefix_o + block * kSpRows * kVDim + (group * kSpRows + j.prefix_row + row) * 8;
      }
      v[u][0] = reinterpret_cast<const float4*>(src)[0];
      v[u][1] = reinterpret_cast<const float4*>(src)[1];
    }
    // the maximum so far (NaN stays: what it scales is NaN)
    float top = M;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) top = lse[u] != lse[u] ? lse[u] : fmaxf(top, lse[u]);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) top = lse[u] != lse[u] ? lse[u] : top;
    if (top == -INFINITY) continue;
    const float f = M == -INFINITY ? 0.0f : ex2(M - top);
    M = top;
    wsum *= f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float w = ex2(lse[u] - M);
      wsum += w;
      if (w == 0.0f) continue;        // (a partial without weight may hold 0 / 0)
      acc[0] += w * v[u][0].x; acc[1] += w * v[u][0].y;
      acc[2] += w * v[u][0].z; acc[3] += w * v[u][0].w;
      acc[4] += w * v[u][1].x; acc[5] += w * v[u][1].y;
      acc[6] += w * v[u][1].z; acc[7] += w * v[u][1].w;
    }
  }
  const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    o[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
  const int64_t at = token * kHeads + row;
  reinterpret_cast<uint4*>(p.out + at * kVDim)[group] = make_uint4(o[0], o[1], o[2], o[3]);
  if (group == 0 && p.lse != nullptr)
    p.lse[at] = wsum == 0.0f ? -INFINITY : (M + __log2f(wsum)) * kLn2;
}

}  // namespace

cudaError_t launch_meet(const MeetParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tokens * 4));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.most <= 4 ? cudaLaunchKernelEx(&cfg, meet_kernel<4>, p)
                     : cudaLaunchKernelEx(&cfg, meet_kernel<8>, p);
}

}  // namespace mla
