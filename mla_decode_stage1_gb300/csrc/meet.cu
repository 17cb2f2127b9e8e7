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
// bytes stand together), with up to 4 partials in flight.  Of tokens with many
// partials (kSlices 4) a CTA takes 32 dims, and a thread every fourth partial.  64
// tokens of 9 or 10 partials, 22 MB, take 9.4 us with all of it in DRAM; in a call it
// comes from L2.

#include "shared.h"

namespace mla {
namespace {

constexpr int kThreads = 256;                 // 16 rows x 16 groups of 8 dims (or slices)

// The larger of two maxima; NaN stays.
__device__ __forceinline__ float top_of(float a, float b) {
  return a != a ? a : b != b ? b : fmaxf(a, b);
}

template <int kAhead, int kSlices>
__global__ void __launch_bounds__(kThreads) meet_kernel(const MeetParams p) {
  constexpr int kGroups = 16 / kSlices;                  // of a CTA
  const int64_t token = blockIdx.x / (4 * kSlices);
  const int row = threadIdx.x & 15, slice = threadIdx.x / (16 * kGroups);
  const int group = blockIdx.x % (4 * kSlices) * kGroups + (threadIdx.x >> 4) % kGroups;
  // (behind another kernel of the call, the table is there already)
  if (p.alone) asm volatile("griddepcontrol.wait;" ::: "memory");
  const MeetJob j = p.jobs[token];
  const bool sound = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp &&
                     check_of(j, p.stamp) == j.check;
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the partials are there
  if (!sound) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrStale);
    return;
  }
  const int n = j.own_count + j.prefix_count;
  float M = -INFINITY, wsum = 0.0f, acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int s0 = slice; s0 < n; s0 += kAhead * kSlices) {
    float lse[kAhead];
    float4 v[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = s0 + u * kSlices;
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
    for (int u = 0; u < kAhead; ++u) top = top_of(top, lse[u]);
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
  if constexpr (kSlices > 1) {
    // the slices' sums, by the first one's threads
    constexpr int kPer = 16 * kGroups;
    __shared__ float parts[kSlices - 1][10][kPer];
    const int at = threadIdx.x % kPer;
    if (slice > 0) {
      parts[slice - 1][0][at] = M;
      parts[slice - 1][1][at] = wsum;
#pragma unroll
      for (int i = 0; i < 8; ++i) parts[slice - 1][2 + i][at] = acc[i];
    }
    __syncthreads();
    if (slice > 0) return;
    float top = M;
#pragma unroll
    for (int k = 0; k < kSlices - 1; ++k) top = top_of(top, parts[k][0][at]);
    if (top != -INFINITY) {
      const float f = M == -INFINITY ? 0.0f : ex2(M - top);
      wsum *= f;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] *= f;
#pragma unroll
      for (int k = 0; k < kSlices - 1; ++k) {
        const float w = parts[k][0][at] == -INFINITY ? 0.0f : ex2(parts[k][0][at] - top);
        wsum += w * parts[k][1][at];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += w * parts[k][2 + i][at];
      }
    }
    M = top;
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
  // In slices: 2 tokens of 65 partials 21 us a call, 28 not; 4 tokens of 9 12.5 and 14.5,
  // but 32 tokens of 9 22.6 and 20.6.  (4 in flight where 8 took 73.5 instead of 71.8:
  // 256 tokens of 4 or 5.)
  const bool wide = p.most > 16 || (p.most > 6 && p.tokens * 4 < 152);
  const dim3 grid(static_cast<unsigned>(p.tokens * (wide ? 16 : 4)));
  auto* kernel = wide ? meet_kernel<8, 4> : meet_kernel<4, 1>;
  return launch_dependent(kernel, grid, kThreads, 0, stream, p);
}

}  // namespace mla
