// prefill.cu -- kernels of the expanded form, in their simplest form: one
// thread per expanded dim, one warp per (query token, head).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "prefill.h"

namespace mla {
namespace {

__device__ __forceinline__ float bf16f(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ uint16_t bf16r(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

__device__ __forceinline__ bool stamp_ok(int32_t* err, uint64_t stamp) {
  if (reinterpret_cast<const WsHeader*>(err)->stamp == stamp) return true;
  if (threadIdx.x == 0) atomicOr(err, kErrStale);
  return false;
}

// Pool row of token `tok` of a request (bounds: see kv_indices).
__device__ __forceinline__ int64_t pool_row(const ExpandParams& p, const ExpandTile& t, int tok) {
  const int e = tok / p.page_size;
  int64_t page = static_cast<int64_t>(t.page_base) + e;
  if (p.kv_indices != nullptr) {
    page = p.kv_indices[page];
    if (page < 0 || page >= p.pool_rows / p.page_size) {
      atomicOr(p.err, kErrBadPage);
      page = 0;
    }
  }
  return page * p.page_size + (tok - e * p.page_size);
}

__device__ __forceinline__ float stored(const ExpandParams& p, int64_t row, int d) {
  if (p.kv_dtype == MLA_DTYPE_BF16)
    return bf16f(reinterpret_cast<const uint16_t*>(p.kv)[row * kQkDim + d]);
  if (p.kv_dtype == MLA_DTYPE_FP8_E4M3) {
    const uint32_t h = e4m3x2_to_f16x2(p.kv[row * kQkDim + d]);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu))) * *p.kv_scale;
  }
  const uint32_t c = (p.kv[row * (kQkDim / 2) + (d >> 1)] >> (4 * (d & 1))) & 15u;
  const int e = p.e8m0[row * p.e8m0_stride + d / 32];
  const float s = e == 255 ? __uint_as_float(0x7fc00000u)
                           : __uint_as_float(e > 0 ? static_cast<uint32_t>(e) << 23 : 0x00400000u);
  return __half2float(__ushort_as_half(
             static_cast<unsigned short>(e2m1x2_to_f16x2(c) & 0xffffu))) * s;
}

__global__ void __launch_bounds__(256) expand_kernel(const ExpandParams p) {
  __shared__ float x[kQkDim];
  if (!stamp_ok(p.err, p.stamp)) return;
  const ExpandTile t = p.tiles[blockIdx.x];
  const int h = blockIdx.y, n = threadIdx.x;
  const uint16_t* w = p.w + (static_cast<int64_t>(h) * kWRows + n) * kVDim;
  for (int r = 0; r < kPfTile; ++r) {
    const int tok = t.tok0 + r;
    const bool live = tok < t.len;
    __syncthreads();
    if (live) {
      const int64_t row = pool_row(p, t, tok);
      for (int d = n; d < kQkDim; d += 256) x[d] = stored(p, row, d);
    }
    __syncthreads();
    float s = 0.0f;
    if (live)
      for (int c = 0; c < kVDim; ++c) s += x[c] * bf16f(w[c]);
    const int64_t orow = static_cast<int64_t>(t.out_row) + r;
    p.kx[(static_cast<int64_t>(h) * p.kx_rows + orow) * kWRows + n] = bf16r(s);
    if (h == 0 && n < kRope) p.kr[orow * kRope + n] = live ? bf16r(x[kVDim + n]) : 0;
  }
}

__global__ void __launch_bounds__(256) attn_kernel(const AttnParams p) {
  if (!stamp_ok(p.err, p.stamp)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int it = p.cta_indptr[blockIdx.x]; it < p.cta_indptr[blockIdx.x + 1]; ++it) {
    const AttnItem w = p.items[it];
    const uint16_t* kx = p.kx + (static_cast<int64_t>(w.head) * p.kx_rows + w.kv_row) * kWRows;
    const uint16_t* kr = p.kr + static_cast<int64_t>(w.kv_row) * kRope;
    for (int i = warp; i < w.rows; i += 8) {
      const int64_t t = static_cast<int64_t>(w.q_row) + i;
      const uint16_t* q = p.q + t * p.q_token_stride + w.head * p.q_head_stride;
      float qv[4], ra, rb;
      for (int d = 0; d < 4; ++d) qv[d] = bf16f(q[lane + 32 * d]);
      const int d0 = rope_dim0(lane, p.rot.half), d1 = rope_dim1(lane, p.rot.half);
      ra = bf16f(q[kNope + d0]);
      rb = bf16f(q[kNope + d1]);
      if (p.rot.cos_sin != nullptr) {
        const float* cs = rotation_row(p.rot, t, lane == 0 ? p.err : nullptr);
        rotate(ra, rb, cs[lane], cs[kRope / 2 + lane]);
        ra = bf16f(bf16r(ra));
        rb = bf16f(bf16r(rb));
      }
      float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int end = min(w.kv_end, w.vis0 + i);
      for (int k = w.kv_begin; k < end; ++k) {
        const uint16_t* kk = kx + static_cast<int64_t>(k) * kWRows;
        float s = ra * bf16f(kr[static_cast<int64_t>(k) * kRope + d0]) +
                  rb * bf16f(kr[static_cast<int64_t>(k) * kRope + d1]);
        for (int d = 0; d < 4; ++d) s += qv[d] * bf16f(kk[lane + 32 * d]);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s);
        const float a = m == -INFINITY ? 0.0f : exp2f(m - mn);
        // a score of -inf adds nothing, whatever the maximum so far; NaN stays NaN
        const float e = s == -INFINITY ? 0.0f : exp2f(s - mn);
        m = mn;
        l = l * a + e;
        for (int d = 0; d < 4; ++d) o[d] = o[d] * a + e * bf16f(kk[kNope + lane + 32 * d]);
      }
      // no key in reach: zeros (a row whose keys all score -inf is 0 / 0)
      const float inv = end <= w.kv_begin ? 0.0f : 1.0f / l;
      if (w.slot >= 0) {
        const int64_t at = static_cast<int64_t>(w.slot) * kPfRows + i;
        for (int d = 0; d < 4; ++d) p.part_o[at * kVHead + lane + 32 * d] = o[d] * inv;
        if (lane == 0) p.part_lse[at] = l == 0.0f ? -INFINITY : m + log2f(l);
      } else {
        const int64_t at = t * p.heads + w.head;
        for (int d = 0; d < 4; ++d) p.out[at * kVHead + lane + 32 * d] = bf16r(o[d] * inv);
        if (lane == 0 && p.lse != nullptr)
          p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
  }
}

// out = sum_s w_s o_s / sum_s w_s with w_s = 2^(lse_s - max lse): one warp per
// row of a job, four dims a lane.
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p) {
  if (!stamp_ok(p.err, p.stamp)) return;
  const int lane = threadIdx.x & 31;
  const JoinJob j = p.jobs[blockIdx.x];
  const int i = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (i >= j.rows) return;
  float M = -INFINITY;
  bool nan = false;
  for (int s = 0; s < j.count; ++s) {
    const float v = p.part_lse[static_cast<int64_t>(j.first + s) * kPfRows + i];
    nan |= v != v;
    M = fmaxf(M, v);
  }
  if (nan) M = __uint_as_float(0x7fc00000u);
  float wsum = 0.0f;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < j.count; ++s) {
    const int64_t at = static_cast<int64_t>(j.first + s) * kPfRows + i;
    const float v = p.part_lse[at];
    if (v == -INFINITY) continue;          // no key of this range is seen
    const float w = exp2f(v - M);
    const float4 o = reinterpret_cast<const float4*>(p.part_o + at * kVHead)[lane];
    wsum += w;
    a.x += w * o.x;
    a.y += w * o.y;
    a.z += w * o.z;
    a.w += w * o.w;
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

cudaError_t launch_expand(const ExpandParams& p, int, cudaStream_t stream) {
  expand_kernel<<<dim3(p.num_tiles, p.heads), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_attn(const AttnParams& p, int num_ctas, cudaStream_t stream) {
  attn_kernel<<<num_ctas, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_join(const JoinParams& p, cudaStream_t stream) {
  join_kernel<<<dim3(p.num_jobs, kPfRows / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
