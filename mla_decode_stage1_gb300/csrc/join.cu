// join.cu -- joins the partial results of key ranges of the expanded form by
// their log-sum-exp.  Latency: 16 heads x 77 rows in 18 parts (11 MB), cold:
// 12 us with the parts one after the other, 9.4 us with eight in flight.

#include <cuda_bf16.h>

#include "prefill.h"

namespace mla {
namespace {

// out = sum_s w_s o_s / sum_s w_s with w_s = 2^(lse_s - max lse): one warp per
// row of a job, four dims a lane.
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");      // a programmatic dependent
  if (reinterpret_cast<const WsHeader*>(p.err)->stamp != p.stamp) return;   // reported by attn_kernel
  const int lane = threadIdx.x & 31;
  const JoinJob j = p.jobs[blockIdx.x];
  if (check_of(j, p.stamp) != j.check) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrStale);
    return;
  }
  const int i = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (i >= j.rows) return;
  // Weights first, a part per lane and 32 at a time, then the parts' rows,
  // eight in flight.
  float M = -INFINITY;
  bool nan = false;
  for (int s = lane; s < j.count; s += 32) {
    const float v = p.part_lse[static_cast<int64_t>(j.first + s * j.span) * kPfRows + i];
    nan |= v != v;
    M = fmaxf(M, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (__any_sync(0xffffffffu, nan)) M = __uint_as_float(0x7fc00000u);
  float wsum = 0.0f;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s0 = 0; s0 < j.count; s0 += 8) {
    float v[8];
    float4 o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int s = min(s0 + u, j.count - 1);
      const int64_t at = static_cast<int64_t>(j.first + s * j.span) * kPfRows + i;
      v[u] = s0 + u < j.count ? p.part_lse[at] : -INFINITY;
      o[u] = reinterpret_cast<const float4*>(p.part_o + at * kVHead)[lane];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (v[u] == -INFINITY) continue;       // no key of this range is seen
      const float w = exp2f(v[u] - M);
      wsum += w;
      a.x += w * o[u].x;
      a.y += w * o[u].y;
      a.z += w * o[u].z;
      a.w += w * o[u].w;
    }
  }
  // a row that sees no key at all is zero; one whose keys all score -inf is 0 / 0
  const float inv = j.vis0 + i <= 0 ? 0.0f : 1.0f / wsum;
  const int64_t at = (static_cast<int64_t>(j.q_row) + i) * p.heads + j.head;
  const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv);
  const __nv_bfloat162 y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
  uint2 v;
  v.x = *reinterpret_cast<const uint32_t*>(&x);
  v.y = *reinterpret_cast<const uint32_t*>(&y);
  reinterpret_cast<uint2*>(p.out + at * kVHead)[lane] = v;
  if (lane == 0 && p.lse != nullptr)
    p.lse[at] = wsum == 0.0f ? -INFINITY : (M + log2f(wsum)) * kLn2;
}

}  // namespace

cudaError_t launch_join(const JoinParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.num_jobs, 2 * kPfRows / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel, p);
}

}  // namespace mla
