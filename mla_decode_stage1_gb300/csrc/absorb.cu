// absorb.cu -- the absorbed form's two products.
//
//     mla_absorb_q    q_out[t,h,c] = f sum_d q[t,h,d] w[h][d][c]        (K = 128, N = 512)
//                     q_out[t,h,512:] = f rotate(q[t,h,128:192])
//     mla_absorb_out  out[t,h,v] = sum_c o[t,h,c] w[h][128+v][c]        (K = 512, N = 128)
//
// Bound: one pass over the weights (128 KB a head, each) for few tokens,
// where the call is latency; memory for many.  Heads do not share weights, so
// a CTA is (head, 128 tokens, slice of the output dims): slices are narrow
// while there are few token tiles, so that the weights stream through all
// SMs.  Operands come by TMA, the product runs on the tensor cores (rows past
// the last token are computed from whatever the shared memory holds and never
// written), the epilogue scales, rounds once and writes whole sectors.
//
// A wait that gives up is noted in the caller's error word, if there is one, and
// in any case the tile's products are written as NaN: what the output held
// before must not pass for a result.
//
// Measured (16 heads, kernel alone, warm L2): absorb_q 3.5 us for 4 tokens to
// bf16 and 6.1 us for 256 to fp8; absorb_out 3.8 us for 61 tokens and 5.8 us
// for 1024 (2.1 GFLOP, 23 MB: 4.0 TB/s).  Their bytes take 0.3, 0.9, 0.5 and
// 3.4 us at 6.8 TB/s: launch, descriptor fetch, one trip to memory and one to
// the tensor cores make up the rest.

#include <cuda.h>
#include <cuda_bf16.h>

#include "layer.h"
#include "plan.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kTokens = 128;                       // tokens of a CTA
constexpr uint32_t kPanel = kTokens * 128;         // a row panel: 128 tokens x 64 bf16
constexpr int kAbsorbThreads = 128;

// The wait for operands: on their barrier, or (the self-test) on one that
// nothing arrives on, with a limit of its own.
struct OperandWait {
  uint64_t limit_ns = kWaitLimitNs;
  bool stalled = false;
};

struct AbsorbQParams {
  CUtensorMap map_q;           // {192, heads, tokens}, boxes {64, 1, box_rows}
  CUtensorMap map_w;           // {512, 256, heads}, boxes {64, 128, 1}
  const uint16_t* q;
  int64_t token_stride, head_stride;
  int64_t tokens;
  int32_t heads;
  int32_t box_rows;            // tokens a box brings (128, or fewer when there are fewer)
  float factor;                // 24 sm_scale
  Rotation rot;
  const float* q_scale;        // null: bf16 out
  void* out;
  int32_t* err;
  OperandWait wait;
};

struct AbsorbOutParams {
  CUtensorMap map_o;           // {512, heads, tokens}, boxes {64, 1, box_rows}
  CUtensorMap map_w;           // {512, 256, heads}, boxes {64, N, 1}
  int64_t tokens;
  int32_t heads;
  int32_t box_rows;
  uint16_t* out;
  int32_t* err;
  OperandWait wait;
};

__device__ __forceinline__ float bf16f(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One rotated pair of a row, scaled and stored at dims d0 and d1 behind the
// 512 latent ones.
__device__ __forceinline__ void store_pair(const AbsorbQParams& p, const Fp8Scale& fs, int64_t row,
                                           int d0, int d1, float a, float b) {
  const int64_t at = row * kQkDim + kVDim;
  if (p.q_scale == nullptr) {
    uint16_t* out = static_cast<uint16_t*>(p.out) + at;
    const uint32_t v = bf16x2(a, b);
    out[d0] = static_cast<uint16_t>(v & 0xffffu);
    out[d1] = static_cast<uint16_t>(v >> 16);
  } else {
    uint8_t* out = static_cast<uint8_t*>(p.out) + at;
    const float pair[2] = {a, b};
    uint32_t v;
    to_e4m3<2>(pair, fs, &v);
    out[d0] = static_cast<uint8_t>(v & 0xff);
    out[d1] = static_cast<uint8_t>(v >> 8);
  }
}

// N output dims a CTA; kSlices = 512 / N CTAs share a (head, token tile) and
// the rotation of its rows.
template <int N>
__global__ void __launch_bounds__(kAbsorbThreads)
    absorb_q_kernel(const __grid_constant__ AbsorbQParams p) {
  constexpr int kSlices = kVDim / N;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full, done, never;
  __shared__ uint32_t tmem_base, gave_up;
  __shared__ int32_t unreported;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t a_smem = smem_u32(smem), b_smem = a_smem + 2 * kPanel;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int slice = blockIdx.x % kSlices, h = blockIdx.y;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / kSlices) * kTokens;
  int32_t* err = p.err != nullptr ? p.err : &unreported;
  if (warp == 0) {
    if (elect_one()) {
      mbar_init(smem_u32(&full), 1);
      mbar_init(smem_u32(&never), 1);
      mbar_init(smem_u32(&done), 2);            // the products' commit, and `gave_up` is set
      fence_mbar_init();
      mbar_arrive_expect_tx(smem_u32(&full), 2 * p.box_rows * 128 + N / 64 * kPanel);
      const uint64_t keep = l2_policy_evict_normal();
      for (int ch = 0; ch < N / 64; ++ch)
        tma_load_3d(b_smem + ch * kPanel, &p.map_w, smem_u32(&full), slice * N + 64 * ch, 0, h,
                    keep);
      for (int ch = 0; ch < 2; ++ch)
        tma_load_3d(a_smem + ch * kPanel, &p.map_q, smem_u32(&full), 64 * ch, h,
                    static_cast<int32_t>(t0), keep);
    }
    __syncwarp();
    tmem_alloc(smem_u32(&tmem_base), N);
    tmem_relinquish();
  }
  // rows slice, slice + kSlices, ... of the tile are rotated here, a warp per
  // row and a pair per lane, while the operands are on their way
  // (all of a warp's rows are loaded before the first is turned)
  constexpr int kRows = kTokens / (4 * kSlices);
  const Fp8Scale fs = p.q_scale != nullptr ? load_fp8_scale(p.q_scale) : Fp8Scale{1.0f, 1.0f, true};
  const int d0 = rope_dim0(lane, p.rot.half), d1 = rope_dim1(lane, p.rot.half);
  float a[kRows], b[kRows], c[kRows], s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t t = t0 + slice + kSlices * (warp + 4 * i);
    if (t >= p.tokens) continue;
    const uint16_t* q = p.q + t * p.token_stride + h * p.head_stride + kNope;
    a[i] = bf16f(q[d0]);
    b[i] = bf16f(q[d1]);
    if (p.rot.cos_sin != nullptr) {
      const float* cs = rotation_row(p.rot, t, lane == 0 && h == 0 ? p.err : nullptr);
      c[i] = cs[lane];
      s[i] = cs[kRope / 2 + lane];
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t t = t0 + slice + kSlices * (warp + 4 * i);
    if (t >= p.tokens) continue;
    if (p.rot.cos_sin != nullptr) rotate(a[i], b[i], c[i], s[i]);
    store_pair(p, fs, t * p.heads + h, d0, d1, a[i] * p.factor, b[i] * p.factor);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(tmem_base);
  if (warp == 0) {
    const bool ok = __all_sync(
        0xffffffffu, mbar_wait_for(smem_u32(p.wait.stalled ? &never : &full), 0, err, kErrProducer,
                                   p.wait.limit_ns));
    tc_fence_after();
    if (elect_one()) {
      if (ok) {
        constexpr uint32_t idesc = make_idesc(1, 1, false, true, 128, N);
        const uint64_t a = smem_desc(a_smem, 16, 1024, kSwizzle128B);
        const uint64_t b = smem_desc(b_smem, kPanel, 1024, kSwizzle128B);
#pragma unroll
        for (int kk = 0; kk < kNope / 16; ++kk)      // 16 dims: 32 bytes of A, 2 row groups of B
          umma_f16(tmem, a + (((kk >> 2) * kPanel + (kk & 3) * 32) >> 4), b + ((kk * 2048) >> 4),
                   idesc, kk != 0);
      }
      gave_up = ok ? 0 : 1;
      mbar_arrive(smem_u32(&done));
      tc_commit(smem_u32(&done));
    }
    __syncwarp();
    // no copy may land after the CTA has gone
    if (!ok) mbar_wait(smem_u32(&full), 0, err, kErrProducer);
  }
  bool ok = mbar_wait(smem_u32(&done), 0, err, kErrDrain);
  ok = __all_sync(0xffffffffu, ok) && gave_up == 0;
  tc_fence_after();
  const int64_t t = t0 + warp * 32 + lane;
  const int64_t at = (t * p.heads + h) * kQkDim + slice * N;
  if (!ok) {
    const uint32_t nan = p.q_scale == nullptr ? 0x7fff7fffu : 0x7f7f7f7fu;
    const uint32_t u[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
    const int size = p.q_scale == nullptr ? 2 : 1;
    if (t < p.tokens)
      for (int i = 0; i < N * size; i += 32)
        st_global_32(static_cast<uint8_t*>(p.out) + at * size + i, u);
  } else {
    const uint32_t acc = tmem + (static_cast<uint32_t>(warp) << 21);
#pragma unroll
    for (int c = 0; c < N / 32; ++c) {
      uint32_t x[32], u[16];
      __syncwarp();
      tmem_ld32(acc + 32 * c, x);
      tmem_wait_ld();
      if (t >= p.tokens) {
        // past the last token
      } else if (p.q_scale == nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          u[i] = bf16x2(__uint_as_float(x[2 * i]) * p.factor,
                        __uint_as_float(x[2 * i + 1]) * p.factor);
        uint16_t* out = static_cast<uint16_t*>(p.out) + at + 32 * c;
        st_global_32(out, u);
        st_global_32(out + 16, u + 8);
      } else {
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(x[i]) * p.factor;
        to_e4m3<32>(f, fs, u);
        st_global_32(static_cast<uint8_t*>(p.out) + at + 32 * c, u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, N);
}

// N output dims a CTA, S stages of 64 latent dims.
template <int N, int S>
__global__ void __launch_bounds__(kAbsorbThreads)
    absorb_out_kernel(const __grid_constant__ AbsorbOutParams p) {
  constexpr int kSlices = kVHead / N, kSteps = kVDim / 64;
  constexpr uint32_t kStage = kPanel + N * 128;
  constexpr uint32_t kCols = N < 32 ? 32 : N;        // tensor memory comes in 32 columns
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[S], empty[S], done, never;
  __shared__ uint32_t tmem_base, gave_up;
  __shared__ int32_t unreported;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int slice = blockIdx.x % kSlices, h = blockIdx.y;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / kSlices) * kTokens;
  int32_t* err = p.err != nullptr ? p.err : &unreported;
  const uint64_t keep = l2_policy_evict_normal();
  auto load = [&](int step) {
    const int s = step % S;
    const uint32_t bar = smem_u32(&full[s]);
    mbar_arrive_expect_tx(bar, p.box_rows * 128 + N * 128);
    tma_load_3d(base + s * kStage + kPanel, &p.map_w, bar, 64 * step, kNope + slice * N, h, keep);
    tma_load_3d(base + s * kStage, &p.map_o, bar, 64 * step, h, static_cast<int32_t>(t0), keep);
  };
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < S; ++s) {
        mbar_init(smem_u32(&full[s]), 1);
        mbar_init(smem_u32(&empty[s]), 1);
      }
      mbar_init(smem_u32(&never), 1);
      mbar_init(smem_u32(&done), 2);            // the products' commit, and `gave_up` is set
      fence_mbar_init();
      for (int s = 0; s < S; ++s) load(s);
    }
    __syncwarp();
    tmem_alloc(smem_u32(&tmem_base), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(tmem_base);
  if (warp == 0) {
    bool ok = true;
    int seen = 0, issued = S;           // copies waited for, and under way
    constexpr uint32_t idesc = make_idesc(1, 1, false, false, 128, N);
    const uint64_t a0 = smem_desc(base, 16, 1024, kSwizzle128B);
#pragma unroll
    for (int step = 0; step < kSteps; ++step) {
      if (!ok) break;
      const int s = step % S;
      ok = __all_sync(0xffffffffu, mbar_wait_for(smem_u32(p.wait.stalled ? &never : &full[s]),
                                                 p.wait.stalled ? 0 : (step / S) & 1, err,
                                                 kErrProducer, p.wait.limit_ns));
      if (!ok) break;
      ++seen;
      tc_fence_after();
      const uint64_t a = a0 + ((s * kStage) >> 4), b = a + (kPanel >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16(tmem, a + 2 * kk, b + 2 * kk, idesc, (step | kk) != 0);
        tc_commit(smem_u32(&empty[s]));
      }
      // refill the stage of the step before: its products are behind this one's
      if (step >= 1 && step - 1 + S < kSteps) {
        const int back = step - 1;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[back % S]), (back / S) & 1, err,
                                               kErrMma));
        if (ok) {
          ++issued;
          if (elect_one()) load(back + S);
        }
      }
    }
    // a wait gave up: no copy may land after the CTA has gone
    for (int k = seen; !ok && k < issued; ++k)
      mbar_wait(smem_u32(&full[k % S]), (k / S) & 1, err, kErrProducer);
    if (elect_one()) {
      gave_up = ok ? 0 : 1;
      mbar_arrive(smem_u32(&done));
      tc_commit(smem_u32(&done));
    }
    __syncwarp();
  }
  bool ok = mbar_wait(smem_u32(&done), 0, err, kErrDrain);
  ok = __all_sync(0xffffffffu, ok) && gave_up == 0;
  tc_fence_after();
  const int64_t t = t0 + warp * 32 + lane;
  uint16_t* out = p.out + (t * p.heads + h) * kVHead + slice * N;
  if (!ok) {
    const uint32_t nan = 0x7fff7fffu, u[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
    if (t < p.tokens)
      for (int c = 0; c < N / 16; ++c) st_global_32(out + 16 * c, u);
  } else {
    const uint32_t acc = tmem + (static_cast<uint32_t>(warp) << 21);
#pragma unroll
    for (int c = 0; c < N / 16; ++c) {
      float x[16];
      uint32_t u[8];
      __syncwarp();
      tmem_ld16(acc + 16 * c, x);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = bf16x2(x[2 * i], x[2 * i + 1]);
      if (t < p.tokens) st_global_32(out + 16 * c, u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kCols);
}

// A 3-D tensor of bf16 in 64-element boxes with the 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* ptr, cuuint64_t d0, cuuint64_t d1, cuuint64_t d2,
              cuuint64_t s1, cuuint64_t s2, cuuint32_t b1, cuuint32_t b2) {
  const TiledEncoder enc = tiled_encoder();
  const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1 * 2, s2 * 2};
  const cuuint32_t box[3] = {64, b1, b2}, one[3] = {1, 1, 1};
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens that a box brings: all 128 of a tile, or, when there are fewer in
// all, a multiple of 8 that holds them.
int32_t box_rows_for(int64_t tokens) {
  return tokens >= kTokens ? kTokens : static_cast<int32_t>((tokens + 7) / 8 * 8);
}

template <int N>
cudaError_t launch_q(const AbsorbQParams& p, int64_t tiles, cudaStream_t stream) {
  constexpr int bytes = (2 + N / 64) * kPanel + 1024;
  const cudaError_t e = cudaFuncSetAttribute(absorb_q_kernel<N>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  absorb_q_kernel<N><<<dim3(static_cast<unsigned>(tiles * (kVDim / N)), p.heads), kAbsorbThreads,
                       bytes, stream>>>(p);
  return cudaGetLastError();
}

template <int N, int S>
cudaError_t launch_out(AbsorbOutParams& p, const void* w, int64_t tiles, cudaStream_t stream) {
  constexpr int bytes = S * (kPanel + N * 128) + 1024;
  if (!make_map(&p.map_w, w, kVDim, kWRows, p.heads, kVDim, kVDim * kWRows, N, 1))
    return cudaErrorUnknown;
  const cudaError_t e = cudaFuncSetAttribute(absorb_out_kernel<N, S>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  absorb_out_kernel<N, S><<<dim3(static_cast<unsigned>(tiles * (kVHead / N)), p.heads),
                            kAbsorbThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

// Arguments as for mla_absorb_q and mla_absorb_out_ex.
mla_status absorb_q(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* w,
                    int64_t num_tokens, int32_t heads, float sm_scale, const Rotation& rot,
                    int rope, mla_dtype q_dtype, const float* q_scale, void* q_out, int32_t* err,
                    const OperandWait& wait, cudaStream_t stream) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || heads < 1 || heads > 1024 ||
      !(sm_scale > 0.0f) || !(sm_scale < 1e30f))
    return MLA_ERR_INVALID_ARG;
  if (q_dtype != MLA_DTYPE_BF16 && q_dtype != MLA_DTYPE_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  if (q_dtype == MLA_DTYPE_FP8_E4M3 && q_scale == nullptr) return MLA_ERR_INVALID_ARG;
  if (!rotation_ok(rot, rope, num_tokens) || !ptr_aligned(rot.positions, 4) ||
      !ptr_aligned(q_scale, 4) || !ptr_aligned(err, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (q == nullptr || w == nullptr || q_out == nullptr) return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(w, 16) || !ptr_aligned(q_out, 32) ||
      q_token_stride >= (1LL << 39) || q_head_stride >= (1LL << 39) ||
      q_token_stride < kQHead || q_head_stride < kQHead || q_token_stride % 8 != 0 ||
      q_head_stride % 8 != 0)
    return MLA_ERR_INVALID_ARG;
  AbsorbQParams p{};
  p.box_rows = box_rows_for(num_tokens);
  if (!make_map(&p.map_q, q, kQHead, heads, num_tokens, q_head_stride, q_token_stride, 1,
                p.box_rows) ||
      !make_map(&p.map_w, w, kVDim, kWRows, heads, kVDim, kVDim * kWRows, kNope, 1))
    return MLA_ERR_CUDA;
  p.q = static_cast<const uint16_t*>(q);
  p.token_stride = q_token_stride;
  p.head_stride = q_head_stride;
  p.tokens = num_tokens;
  p.heads = heads;
  p.factor = 24.0f * sm_scale;
  p.rot = rot;
  p.q_scale = q_dtype == MLA_DTYPE_FP8_E4M3 ? q_scale : nullptr;
  p.out = q_out;
  p.err = err;
  p.wait = wait;
  const int64_t tiles = (num_tokens + kTokens - 1) / kTokens;
  // eight slices of 64 dims until the (head, token tile)s alone fill the SMs
  const cudaError_t e =
      tiles * heads < 76 ? launch_q<64>(p, tiles, stream) : launch_q<128>(p, tiles, stream);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status absorb_out(const void* o, const void* w, int64_t num_tokens, int32_t heads, void* out,
                      int32_t* err, const OperandWait& wait, cudaStream_t stream) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || heads < 1 || heads > 1024 ||
      !ptr_aligned(err, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (o == nullptr || w == nullptr || out == nullptr || !ptr_aligned(o, 16) ||
      !ptr_aligned(w, 16) || !ptr_aligned(out, 32))
    return MLA_ERR_INVALID_ARG;
  AbsorbOutParams p{};
  p.box_rows = box_rows_for(num_tokens);
  if (!make_map(&p.map_o, o, kVDim, heads, num_tokens, kVDim,
                static_cast<int64_t>(heads) * kVDim, 1, p.box_rows))
    return MLA_ERR_CUDA;
  p.tokens = num_tokens;
  p.heads = heads;
  p.out = static_cast<uint16_t*>(out);
  p.err = err;
  p.wait = wait;
  const int64_t tiles = (num_tokens + kTokens - 1) / kTokens, units = tiles * heads;
  // narrower slices of the 128 output dims while there are few (head, token tile)s
  const cudaError_t e = units < 24    ? launch_out<16, 8>(p, w, tiles, stream)
                        : units < 48  ? launch_out<32, 8>(p, w, tiles, stream)
                        : units < 96  ? launch_out<64, 4>(p, w, tiles, stream)
                                      : launch_out<128, 3>(p, w, tiles, stream);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

extern "C" {

mla_status mla_absorb_q(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                        const void* w, int64_t num_tokens, int32_t heads, float sm_scale,
                        const float* cos_sin, int64_t max_positions, const int32_t* positions,
                        mla_rope rope, mla_dtype q_dtype, const float* q_scale, void* q_out,
                        int32_t* err, mla_stream_t stream) {
  const mla::Rotation rot{cos_sin, positions, max_positions, rope == MLA_ROPE_HALF ? 1 : 0};
  return mla::absorb_q(q, q_token_stride, q_head_stride, w, num_tokens, heads, sm_scale, rot, rope,
                       q_dtype, q_scale, q_out, err, {}, reinterpret_cast<cudaStream_t>(stream));
}

mla_status mla_absorb_out(const void* o, const void* w, int64_t num_tokens, int32_t heads,
                          void* out, mla_stream_t stream) {
  return mla_absorb_out_ex(o, w, num_tokens, heads, out, nullptr, stream);
}

mla_status mla_absorb_out_ex(const void* o, const void* w, int64_t num_tokens, int32_t heads,
                             void* out, int32_t* err, mla_stream_t stream) {
  return mla::absorb_out(o, w, num_tokens, heads, out, err, {},
                         reinterpret_cast<cudaStream_t>(stream));
}

mla_status mla_selftest_absorb_wait(const void* x, const void* w, int64_t num_tokens,
                                    int32_t heads, const float* q_scale, void* y, int32_t to_out,
                                    uint32_t limit_us, int32_t* err, mla_stream_t stream) {
  if (limit_us == 0 || limit_us > 20000) return MLA_ERR_INVALID_ARG;
  mla::OperandWait wait;
  wait.limit_ns = static_cast<uint64_t>(limit_us) * 1000u;
  wait.stalled = true;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (to_out != 0) return mla::absorb_out(x, w, num_tokens, heads, y, err, wait, st);
  return mla::absorb_q(x, static_cast<int64_t>(heads) * mla::kQHead, mla::kQHead, w, num_tokens,
                       heads, 1.0f, mla::Rotation{}, MLA_ROPE_HALF,
                       q_scale != nullptr ? MLA_DTYPE_FP8_E4M3 : MLA_DTYPE_BF16, q_scale, y, err,
                       wait, st);
}

}  // extern "C"
