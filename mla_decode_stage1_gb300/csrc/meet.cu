// meet.cu -- the partial results of a shared-prefix decode become its output:
// for every query token and head the decode kernel's partials over the request's
// own end and the prefix kernel's over the prefix, weighted by their log-sum-exp.
//
//     M = max_s lse_s, w_s = 2^(lse_s - M), out = sum_s w_s o_s / sum_s w_s,
//     lse = (M + log2 sum w) ln 2.
//
// A part without keys, or without weight, has lse = -inf and adds nothing; one
// whose lse is NaN makes the row NaN.  A warp per row, a lane 16 of the 512 dims.

#include "shared.h"

namespace mla {
namespace {

__global__ void __launch_bounds__(256) meet_kernel(const MeetParams p) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t token = row / kHeads;
  const int h = static_cast<int>(row % kHeads);
  if (token >= p.tokens) return;
  const MeetJob j = p.jobs[token];
  const bool sound = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp &&
                     check_of(j, p.stamp) == j.check;
  if (!sound) {
    if (lane == 0) atomicOr(p.err, kErrStale);
    return;
  }
  const int n = j.own_count + j.prefix_count;
  // row of partial s in its array of rows
  auto at = [&](int s) {
    return s < j.own_count
               ? static_cast<int64_t>(j.own_first + s) * p.own_rows + j.own_row + h
               : static_cast<int64_t>(j.prefix_first + s - j.own_count) * kSpRows + j.prefix_row + h;
  };
  auto lse_of = [&](int s) { return (s < j.own_count ? p.own_lse : p.prefix_lse)[at(s)]; };
  float M = -INFINITY;
  bool bad = false;
  for (int s = lane; s < n; s += 32) {
    const float l = lse_of(s);
    bad |= l != l;
    M = fmaxf(M, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (__any_sync(0xffffffffu, bad)) M = __uint_as_float(0x7fc00000u);
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  float wsum = 0.0f;
  if (M != -INFINITY) {
    for (int s0 = 0; s0 < n; s0 += 4) {
      float w[4];
      float4 v[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int s = min(s0 + u, n - 1);
        w[u] = lse_of(s);
        const float4* src =
            reinterpret_cast<const float4*>((s < j.own_count ? p.own_o : p.prefix_o) + at(s) * kVDim);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = src[lane + 32 * i];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = s0 + u < n ? ex2(w[u] - M) : 0.0f;
        wsum += f;
        // (a partial without weight is left out: it may hold 0 / 0)
        const bool none = f == 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[4 * i + 0] += none ? 0.0f : f * v[u][i].x;
          acc[4 * i + 1] += none ? 0.0f : f * v[u][i].y;
          acc[4 * i + 2] += none ? 0.0f : f * v[u][i].z;
          acc[4 * i + 3] += none ? 0.0f : f * v[u][i].w;
        }
      }
    }
  }
  const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
  uint16_t* out = p.out + row * kVDim;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc[4 * i + 0] * inv, acc[4 * i + 1] * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv);
    reinterpret_cast<uint2*>(out)[lane + 32 * i] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = wsum == 0.0f ? -INFINITY : (M + __log2f(wsum)) * kLn2;
}

}  // namespace

cudaError_t launch_meet(const MeetParams& p, cudaStream_t stream) {
  const int64_t ctas = (p.tokens * kHeads + 7) / 8;
  meet_kernel<<<static_cast<unsigned>(ctas), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
