// rotate.cu -- the rotation of the queries' last 64 dims for the expanded
// form, into the workspace: qr[t][h] = rotate(q[t][h][128:192]).  The rotated
// values are rounded to bf16 as operands of the attention's products.
//
// Bound: memory (128 bytes in and out a row).  A kernel of its own: in the
// attention kernel the rotation held up every item's first product (about 7k
// cycles an item), and as part of the expansion it took that kernel's
// registers and end (8192 tokens of 16 heads: expansion 37 -> 49 us; alone 8.6 us,
// 3.9 TB/s).
// Four lanes to a row, eight pairs a lane.

#include <cuda_bf16.h>

#include "prefill.h"

namespace mla {
namespace {

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(256) rotate_kernel(const RotateParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (reinterpret_cast<const WsHeader*>(p.err)->stamp != p.stamp) return;   // reported by the others
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x >> 2);
  if (r >= p.q_tokens * p.heads) return;
  const int64_t t = r / p.heads;
  const int h = static_cast<int>(r - t * p.heads);
  const int lane4 = threadIdx.x & 3, half = p.rot.half;
  // the two granules of eight dims that this lane turns
  const int g0 = half ? lane4 : 2 * lane4, g1 = half ? lane4 + 4 : 2 * lane4 + 1;
  const uint4* q = reinterpret_cast<const uint4*>(p.q + t * p.q_token_stride +
                                                  h * p.q_head_stride + kNope);
  const uint4 x = q[g0], y = q[g1];
  const float4* f = reinterpret_cast<const float4*>(
      rotation_row(p.rot, t, lane4 == 0 && h == 0 ? p.err : nullptr) + 8 * lane4);
  const float4 c0 = f[0], c1 = f[1], s0 = f[kRope / 8], s1 = f[kRope / 8 + 1];
  uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
  auto lo = [](uint32_t v) { return __uint_as_float(v << 16); };
  auto hi = [](uint32_t v) { return __uint_as_float(v & 0xffff0000u); };
  if (half) {
    // element k of the first granule turns with element k of the second
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a0 = lo(u[k]), b0 = lo(u[4 + k]), a1 = hi(u[k]), b1 = hi(u[4 + k]);
      rotate(a0, b0, cs[2 * k], sn[2 * k]);
      rotate(a1, b1, cs[2 * k + 1], sn[2 * k + 1]);
      u[k] = bf16x2(a0, a1);
      u[4 + k] = bf16x2(b0, b1);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a = lo(u[k]), b = hi(u[k]);
      rotate(a, b, cs[k], sn[k]);
      u[k] = bf16x2(a, b);
    }
  }
  uint4* out = reinterpret_cast<uint4*>(p.qr + r * kRope);
  out[g0] = make_uint4(u[0], u[1], u[2], u[3]);
  out[g1] = make_uint4(u[4], u[5], u[6], u[7]);
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, cudaStream_t stream) {
  const int64_t ctas = (p.q_tokens * p.heads + 63) / 64;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  rotate_kernel<<<static_cast<unsigned>(ctas), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
