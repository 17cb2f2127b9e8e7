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
// Bound: latency, and memory for many rows.  A CTA per row, a warp per 128 of the
// 512 dims, the loads of up to 16 partials in flight (4 where no row has more:
// registers for twice as many CTAs an SM).

#include "shared.h"

namespace mla {
namespace {

template <int kAhead>
__global__ void __launch_bounds__(128) meet_kernel(const MeetParams p) {
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int col = threadIdx.x;                  // this lane's float4 of the row
  const int64_t token = row / kHeads;
  const int h = static_cast<int>(row % kHeads);
  const MeetJob j = p.jobs[token];
  const bool sound = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp &&
                     check_of(j, p.stamp) == j.check;
  if (!sound) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrStale);
    return;
  }
  const int n = j.own_count + j.prefix_count;
  // row of partial s in its array of rows
  auto at = [&](int s) {
    return s < j.own_count
               ? static_cast<int64_t>(j.own_first + s) * p.own_rows + j.own_row + h
               : (j.prefix_first + static_cast<int64_t>(s - j.own_count) * p.blocks) * kSpRows + j.prefix_row + h;
  };
  auto lse_of = [&](int s) { return (s < j.own_count ? p.own_lse : p.prefix_lse)[at(s)]; };
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the partials are there
  float M = -INFINITY, wsum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s0 = 0; s0 < n; s0 += kAhead) {
    float4 v[kAhead];
    const float mine = lane < kAhead && s0 + lane < n ? lse_of(s0 + lane) : -INFINITY;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = s0 + u;
      v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (s < n)
        v[u] = reinterpret_cast<const float4*>((s < j.own_count ? p.own_o : p.prefix_o) +
                                               at(s) * kVDim)[col];
    }
    // the maximum so far (NaN stays: what it scales is NaN)
    float top = mine;
#pragma unroll
    for (int o = kAhead / 2; o > 0; o >>= 1)
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(M, __shfl_sync(0xffffffffu, top, 0));
    if (__any_sync(0xffffffffu, mine != mine)) top = __uint_as_float(0x7fc00000u);
    if (top == -INFINITY) continue;
    const float f = M == -INFINITY ? 0.0f : ex2(M - top);
    M = top;
    wsum *= f;
    acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
    const float weight = ex2(mine - M);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float w = __shfl_sync(0xffffffffu, weight, u);
      if (w == 0.0f) continue;        // (a partial without weight may hold 0 / 0)
      wsum += w;
      acc.x += w * v[u].x;
      acc.y += w * v[u].y;
      acc.z += w * v[u].z;
      acc.w += w * v[u].w;
    }
  }
  const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(p.out + row * kVDim)[col] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (threadIdx.x == 0 && p.lse != nullptr)
    p.lse[row] = wsum == 0.0f ? -INFINITY : (M + __log2f(wsum)) * kLn2;
}

}  // namespace

cudaError_t launch_meet(const MeetParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tokens * kHeads));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.most <= 4   ? cudaLaunchKernelEx(&cfg, meet_kernel<4>, p)
         : p.most <= 8 ? cudaLaunchKernelEx(&cfg, meet_kernel<8>, p)
                       : cudaLaunchKernelEx(&cfg, meet_kernel<16>, p);
}

}  // namespace mla
