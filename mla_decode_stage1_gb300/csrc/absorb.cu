// absorb.cu -- the absorbed form's two products, in their simplest form: one
// thread per output dim of one (token, head).

#include <cuda_bf16.h>

#include "layer.h"

namespace mla {
namespace {

struct AbsorbQParams {
  const uint16_t* q;
  int64_t token_stride, head_stride;
  const uint16_t* w;
  int64_t tokens;
  int32_t heads;
  float factor;                // 24 sm_scale
  Rotation rot;
  const float* q_scale;        // null: bf16 out
  void* out;
  int32_t* err;
};

__device__ __forceinline__ float bf16f(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ uint16_t bf16r(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

__device__ __forceinline__ void store_q(const AbsorbQParams& p, int64_t at, float v) {
  if (p.q_scale == nullptr)
    static_cast<uint16_t*>(p.out)[at] = bf16r(v);
  else
    static_cast<uint8_t*>(p.out)[at] =
        static_cast<uint8_t>(to_e4m3x2(__fdiv_rn(v, *p.q_scale), 0.0f) & 0xff);
}

__global__ void __launch_bounds__(kVDim) absorb_q_kernel(const AbsorbQParams p) {
  __shared__ float x[kQHead];
  const int c = threadIdx.x, h = blockIdx.y;
  const int64_t t = blockIdx.x;
  const uint16_t* q = p.q + t * p.token_stride + h * p.head_stride;
  if (c < kQHead) x[c] = bf16f(q[c]);
  __syncthreads();
  const uint16_t* w = p.w + static_cast<int64_t>(h) * kWRows * kVDim + c;
  float s = 0.0f;
  for (int d = 0; d < kNope; ++d) s += x[d] * bf16f(w[d * kVDim]);
  const int64_t at = (t * p.heads + h) * kQkDim;
  store_q(p, at + c, s * p.factor);
  if (c < kRope / 2) {
    const int d0 = rope_dim0(c, p.rot.half), d1 = rope_dim1(c, p.rot.half);
    float a = x[kNope + d0], b = x[kNope + d1];
    if (p.rot.cos_sin != nullptr) {
      const float* cs = rotation_row(p.rot, t, c == 0 ? p.err : nullptr);
      rotate(a, b, cs[c], cs[kRope / 2 + c]);
    }
    store_q(p, at + kVDim + d0, a * p.factor);
    store_q(p, at + kVDim + d1, b * p.factor);
  }
}

__global__ void __launch_bounds__(kVHead) absorb_out_kernel(const uint16_t* o, const uint16_t* w,
                                                            uint16_t* out, int32_t heads) {
  __shared__ float x[kVDim];
  const int v = threadIdx.x, h = blockIdx.y;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * heads + h;
  for (int c = v; c < kVDim; c += kVHead) x[c] = bf16f(o[at * kVDim + c]);
  __syncthreads();
  const uint16_t* wr = w + (static_cast<int64_t>(h) * kWRows + kNope + v) * kVDim;
  float s = 0.0f;
  for (int c = 0; c < kVDim; ++c) s += x[c] * bf16f(wr[c]);
  out[at * kVHead + v] = bf16r(s);
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_absorb_q(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                   const void* w, int64_t num_tokens, int32_t heads,
                                   float sm_scale, const float* cos_sin, int64_t max_positions,
                                   const int32_t* positions, mla_rope rope, mla_dtype q_dtype,
                                   const float* q_scale, void* q_out, int32_t* err,
                                   mla_stream_t stream) {
  using mla::ptr_aligned;
  if (num_tokens < 0 || num_tokens > INT32_MAX || heads < 1 || heads > 1024 ||
      !(sm_scale > 0.0f) || !(sm_scale < 1e30f))
    return MLA_ERR_INVALID_ARG;
  if (q_dtype != MLA_DTYPE_BF16 && q_dtype != MLA_DTYPE_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  if (q_dtype == MLA_DTYPE_FP8_E4M3 && q_scale == nullptr) return MLA_ERR_INVALID_ARG;
  const mla::Rotation rot{cos_sin, positions, max_positions, rope == MLA_ROPE_HALF ? 1 : 0};
  if (!mla::rotation_ok(rot, rope) || !ptr_aligned(positions, 4) || !ptr_aligned(q_scale, 4) ||
      !ptr_aligned(err, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (q == nullptr || w == nullptr || q_out == nullptr) return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(w, 16) || !ptr_aligned(q_out, 16) ||
      q_token_stride < mla::kQHead || q_head_stride < mla::kQHead || q_token_stride % 8 != 0 ||
      q_head_stride % 8 != 0)
    return MLA_ERR_INVALID_ARG;
  const mla::AbsorbQParams p{static_cast<const uint16_t*>(q), q_token_stride, q_head_stride,
                             static_cast<const uint16_t*>(w), num_tokens, heads,
                             24.0f * sm_scale, rot,
                             q_dtype == MLA_DTYPE_FP8_E4M3 ? q_scale : nullptr, q_out, err};
  mla::absorb_q_kernel<<<dim3(static_cast<unsigned>(num_tokens), heads), mla::kVDim, 0,
                         reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_absorb_out(const void* o, const void* w, int64_t num_tokens,
                                     int32_t heads, void* out, mla_stream_t stream) {
  using mla::ptr_aligned;
  if (num_tokens < 0 || num_tokens > INT32_MAX || heads < 1 || heads > 1024)
    return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (o == nullptr || w == nullptr || out == nullptr || !ptr_aligned(o, 16) ||
      !ptr_aligned(w, 16) || !ptr_aligned(out, 16))
    return MLA_ERR_INVALID_ARG;
  mla::absorb_out_kernel<<<dim3(static_cast<unsigned>(num_tokens), heads), mla::kVHead, 0,
                           reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(o), static_cast<const uint16_t*>(w),
      static_cast<uint16_t*>(out), heads);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
