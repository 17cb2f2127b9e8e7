// gather.cu -- the rows of shared prefixes, from the pool's pages and encoding
// to bf16 rows that stand one behind the other in the workspace (the last tile
// of a group is filled up with zeros).
//
// e4m3 values have four significant bits and MXFP4 values two, bf16 has eight and a
// wider range of exponents, so the values are exact (MXFP4 values of 2^128 and more
// are infinite); an e4m3 pool's scale is applied to scores and outputs, not here.
//
// Bound: memory.  One 16-byte load a thread and step, all of a thread's loads
// in flight together.  8,192 rows of e4m3 (4.7 MB in, 9.4 out) take 6.8 us; the prefix
// kernel starts beside it.

#include <cuda_fp16.h>

#include "shared.h"

namespace mla {
namespace {

constexpr int kThreads = 288;                // 72 pieces of 16 bytes (bf16 row) x 4
constexpr int kRowsPerCta = 32;
constexpr int kParts = kSpTile / kRowsPerCta;

__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t h) {
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  const float2 f = __half22float2(v);
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int KV>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherParams p) {
  // pieces of a stored row, and of rows that a step of the CTA covers
  constexpr int kPieces = KV == MLA_DTYPE_BF16 ? 72 : KV == MLA_DTYPE_FP8_E4M3 ? 36 : 18;
  constexpr int kStep = kThreads / kPieces, kSteps = kRowsPerCta / kStep;
  constexpr int kRowBytes = kPieces * 16;
  // (launched while the kernel before it ends; what follows may count on that end too)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const ExpandTile t = p.tiles[blockIdx.x / kParts];
  if (reinterpret_cast<const WsHeader*>(p.err)->stamp != p.stamp || check_of(t, p.stamp) != t.check) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrStale);
    return;
  }
  const int piece = threadIdx.x % kPieces;
  const int row0 = blockIdx.x % kParts * kRowsPerCta + threadIdx.x / kPieces;
  uint4 v[kSteps];
  uint32_t e[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int tok = t.tok0 + row0 + i * kStep;
    v[i] = make_uint4(0, 0, 0, 0);
    e[i] = 127;
    if (tok >= t.len) continue;
    int64_t page = t.page_base + tok / p.page_size;
    const int64_t in = tok % p.page_size;
    if (p.indices != nullptr) page = p.indices[page];
    int64_t row = page * p.page_size + in;
    if (page < 0 || row >= p.pool_rows) {
      atomicOr(p.err, kErrBadPage);
      row = in < p.pool_rows ? in : 0;
    }
    v[i] = ld_na_v4(p.kv + row * kRowBytes + piece * 16);
    if constexpr (KV == MLA_DTYPE_MXFP4) e[i] = ld_u8(p.e8m0 + row * p.e8m0_stride + piece);
  }
  uint16_t* dst = p.rows + (static_cast<int64_t>(t.out_row) + row0) * kQkDim;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    uint16_t* at = dst + static_cast<int64_t>(i) * kStep * kQkDim;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    if constexpr (KV == MLA_DTYPE_BF16) {
      reinterpret_cast<uint4*>(at)[piece] = v[i];
    } else if constexpr (KV == MLA_DTYPE_FP8_E4M3) {
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[2 * k] = bf16x2_of_f16x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[k])));
        o[2 * k + 1] = bf16x2_of_f16x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[k] >> 16)));
      }
      st_global_32(at + 16 * piece, o);
    } else {
      const uint32_t scale = e8m0_to_bf16x2(e[i]);
      uint32_t o[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e2m1x4_to_bf16(w[k], scale, o[4 * k], o[4 * k + 1]);
        e2m1x4_to_bf16(w[k] >> 16, scale, o[4 * k + 2], o[4 * k + 3]);
      }
      st_global_32(at + 32 * piece, o);
      st_global_32(at + 32 * piece + 16, o + 8);
    }
  }
}

}  // namespace

cudaError_t launch_gather(const GatherParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.num_tiles) * kParts);
  auto* kernel = p.kv_dtype == MLA_DTYPE_BF16       ? gather_kernel<MLA_DTYPE_BF16>
                 : p.kv_dtype == MLA_DTYPE_FP8_E4M3 ? gather_kernel<MLA_DTYPE_FP8_E4M3>
                                                    : gather_kernel<MLA_DTYPE_MXFP4>;
  return launch_dependent(kernel, grid, kThreads, 0, stream, p);
}

}  // namespace mla
