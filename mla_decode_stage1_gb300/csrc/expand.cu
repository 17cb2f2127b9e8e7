// expand.cu -- expansion of cached rows into keys and values: for every
// cached token t and head h
//     kx[h][t][0:128] = W_UK[h] c_t,   kx[h][t][128:256] = W_UV[h] c_t
// (one matrix product, K = 512, N = 256 a head), and kr[t] = the 64 rotated
// dims.  The rows are gathered through the page table and decoded on the way
// into shared memory; nothing is written back in between.
//
// Bound: 2 x 512 x 256 flops per (token, head) against 512 bytes written; the
// weights (256 KB a head) come from L2.  A CTA keeps 128 rows (128 KB of bf16)
// in shared memory and runs heads over them, so rows are read and decoded
// once per CTA that meets them; units (tile, head) are split evenly over the
// CTAs.  Two 256-column accumulators let the epilogue of one head run under
// the products of the next.
//
// Roundings: e4m3 and e2m1 values with their block exponents are exact in
// bf16; the per-tensor scale goes into the fp32 epilogue; keys and values are
// rounded to bf16 once, as operands of the attention's products.
//
// A value row that is not finite would reach every query through 0 x NaN in
// the attention's product, also those that must not see the token.  Such a
// row's values are written as zeros and its key as NaN: the queries that see
// the token get NaN through their scores, the others nothing.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "prefill.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kExpandThreads = 448;        // 4 epilogue, 8 row, 1 weight, 1 product warps
constexpr uint32_t kAChunk = 128 * 128;    // 128 rows x 64 bf16
constexpr uint32_t kWChunk = 256 * 128;    // 256 weight rows x 64 bf16
constexpr int kChunks = kVDim / 64;
constexpr int kWSlots = 3;
constexpr int kAhead = 4;                  // row chunks loaded ahead of their use
constexpr uint32_t kExpandSmem = kChunks * kAChunk + kWSlots * kWChunk;

struct ExpandMisc {
  uint64_t a_full[kChunks], a_empty[kChunks];
  uint64_t w_full[kWSlots], w_empty[kWSlots];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem, ours;
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Pool row of token `tok` of a tile's request; a page outside the pool is
// reported and read as page 0.
__device__ __forceinline__ int64_t pool_row(const ExpandParams& p, int page_base, int tok) {
  const int e = tok / p.page_size;
  int64_t page = static_cast<int64_t>(page_base) + e;
  if (p.kv_indices != nullptr) {
    page = p.kv_indices[page];
    if (page < 0 || page >= p.pool_rows / p.page_size) {
      atomicOr(p.err, kErrBadPage);
      page = 0;
    }
  }
  return page * p.page_size + (tok - e * p.page_size);
}

// Eight consecutive stored values as they lie in memory.
template <int KV>
struct Raw;
template <>
struct Raw<MLA_DTYPE_BF16> { uint4 v; };
template <>
struct Raw<MLA_DTYPE_FP8_E4M3> { uint2 v; };
template <>
struct Raw<MLA_DTYPE_MXFP4> { uint32_t v; uint32_t e; };

// Values 8 g .. 8 g + 7 of a row (g = 0..71).
template <int KV>
__device__ __forceinline__ Raw<KV> load_raw(const ExpandParams& p, int64_t row, int g) {
  Raw<KV> r;
  if constexpr (KV == MLA_DTYPE_BF16) {
    r.v = *reinterpret_cast<const uint4*>(p.kv + row * (kQkDim * 2) + g * 16);
  } else if constexpr (KV == MLA_DTYPE_FP8_E4M3) {
    r.v = *reinterpret_cast<const uint2*>(p.kv + row * kQkDim + g * 8);
  } else {
    r.v = *reinterpret_cast<const uint32_t*>(p.kv + row * (kQkDim / 2) + g * 4);
    r.e = p.e8m0[row * p.e8m0_stride + (g >> 2)];
  }
  return r;
}

// The same values as bf16 (exactly; e4m3 without the per-tensor scale `sc`
// unless it is given).
template <int KV>
__device__ __forceinline__ uint4 decode(const Raw<KV>& r, float sc) {
  if constexpr (KV == MLA_DTYPE_BF16) {
    return r.v;
  } else {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h;
      if constexpr (KV == MLA_DTYPE_FP8_E4M3)
        h = e4m3x2_to_f16x2(static_cast<uint16_t>((i < 2 ? r.v.x : r.v.y) >> (16 * (i & 1))));
      else
        h = e2m1x2_to_f16x2((r.v >> (8 * i)) & 0xffu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      float m = sc;
      if constexpr (KV == MLA_DTYPE_MXFP4)
        m = r.e == 255u ? __uint_as_float(0x7fc00000u)
                        : __uint_as_float(r.e > 0 ? r.e << 23 : 0x00400000u);
      o[i] = bf16x2(f.x * m, f.y * m);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int KV>
__device__ void run_rows(const ExpandParams& p, ExpandMisc* ms, uint8_t* a_smem, int u0, int u1,
                         int tid) {
  const int g = tid & 7, r0 = tid >> 3;      // granule of a chunk; rows r0 + 32 i
  const float sc = KV == MLA_DTYPE_FP8_E4M3 ? *p.kv_scale : 1.0f;
  uint32_t lap = 0;
  for (int u = u0; u < u1; ++lap) {
    const int tile = u / p.heads;
    const ExpandTile t = p.tiles[tile];
    int64_t row[4];
    bool live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = t.tok0 + r0 + 32 * i;
      live[i] = tok < t.len;
      row[i] = live[i] ? pool_row(p, t.page_base, tok) : 0;
    }
    Raw<KV> raw[kAhead][4];                  // chunks in flight from memory
    auto fetch = [&](int c) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (live[i]) raw[c % kAhead][i] = load_raw<KV>(p, row[i], 8 * c + g);
    };
#pragma unroll
    for (int c = 0; c < kAhead; ++c) fetch(c);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = live[i] ? decode<KV>(raw[c % kAhead][i], 1.0f) : make_uint4(0, 0, 0, 0);
      if (c + kAhead <= kChunks) fetch(c + kAhead);     // chunk 8: the rotated dims
      if (lap > 0 && !mbar_wait(smem_u32(&ms->a_empty[c]), (lap - 1) & 1, p.err, kErrProducer))
        return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i;
        *reinterpret_cast<uint4*>(a_smem + c * kAChunk + r * 128 + ((g ^ (r & 7)) << 4)) = v[i];
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&ms->a_full[c]));
    }
    if (u % p.heads == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(p.kr + (static_cast<int64_t>(t.out_row) + r0 + 32 * i) * kRope +
                                  8 * g) =
            live[i] ? decode<KV>(raw[kChunks % kAhead][i], sc) : make_uint4(0, 0, 0, 0);
    }
    u = min(u1, (tile + 1) * p.heads);
  }
}

__device__ void run_weights(const ExpandParams& p, ExpandMisc* ms, uint32_t w_smem, int u0,
                            int u1) {
  const uint64_t keep = l2_policy_evict_normal();
  uint32_t n = 0;
  bool ok = true;
  for (int u = u0; u < u1 && ok; ++u) {
    const int h = u % p.heads;
    for (int c = 0; c < kChunks; ++c, ++n) {
      const uint32_t s = n % kWSlots, lap = n / kWSlots;
      if (lap > 0 &&
          !mbar_wait(smem_u32(&ms->w_empty[s]), (lap - 1) & 1, p.err, kErrProducer)) {
        ok = false;
        break;
      }
      mbar_arrive_expect_tx(smem_u32(&ms->w_full[s]), kWChunk);
      tma_load_3d(w_smem + s * kWChunk, &p.map_w, smem_u32(&ms->w_full[s]), 64 * c, 0, h, keep);
    }
  }
  if (!ok)      // a wait gave up: no copy may land after the CTA has gone
    for (uint32_t k = n > kWSlots ? n - kWSlots : 0; k < n; ++k)
      mbar_wait(smem_u32(&ms->w_full[k % kWSlots]), (k / kWSlots) & 1, p.err, kErrProducer);
}

// The whole warp walks the units; one lane issues.
__device__ void run_products(const ExpandParams& p, ExpandMisc* ms, uint32_t a_smem,
                             uint32_t w_smem, uint32_t tmem, int u0, int u1) {
  constexpr uint32_t idesc = make_idesc(1, 1, false, false, 128, kWRows);
  const uint64_t ad = smem_desc(a_smem, 16, 1024, kSwizzle128B);
  const uint64_t wd = smem_desc(w_smem, 16, 1024, kSwizzle128B);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.err, kErrMma));
  };
  uint32_t slot = 0, phase = 0, lap = 0, k = 0;
  for (int u = u0; u < u1; ++u, ++k) {
    const bool first = u == u0 || u % p.heads == 0;          // first unit of its tile here
    const bool last = u + 1 == u1 || (u + 1) % p.heads == 0;
    const uint32_t buf = k & 1;
    if (k >= 2 && !wait(&ms->acc_empty[buf], ((k >> 1) - 1) & 1)) return;
    tc_fence_after();
    const uint32_t d = tmem + buf * kWRows;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (first && !wait(&ms->a_full[c], lap & 1)) return;
      if (!wait(&ms->w_full[slot], phase)) return;
      tc_fence_after();
      const uint64_t a = ad + ((c * kAChunk) >> 4), w = wd + ((slot * kWChunk) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_f16(d, a + 2 * kk, w + 2 * kk, idesc, (c | kk) != 0);
        tc_commit(smem_u32(&ms->w_empty[slot]));
        if (last) tc_commit(smem_u32(&ms->a_empty[c]));
      }
      if (++slot == kWSlots) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (elect_one()) tc_commit(smem_u32(&ms->acc_full[buf]));
    if (last) ++lap;
  }
}

__device__ void run_epilogue(const ExpandParams& p, ExpandMisc* ms, uint32_t tmem, int u0, int u1,
                             int warp, int lane) {
  const float sc = p.kv_dtype == MLA_DTYPE_FP8_E4M3 ? *p.kv_scale : 1.0f;
  uint32_t k = 0;
  for (int u = u0; u < u1; ++u, ++k) {
    const uint32_t buf = k & 1;
    const int tile = u / p.heads, h = u - tile * p.heads;
    const int64_t row = static_cast<int64_t>(p.tiles[tile].out_row) + warp * 32 + lane;
    uint16_t* dst = p.kx + (static_cast<int64_t>(h) * p.kx_rows + row) * kWRows;
    const bool ok = mbar_wait(smem_u32(&ms->acc_full[buf]), (k >> 1) & 1, p.err, kErrDrain);
    if (!__all_sync(0xffffffffu, ok)) return;
    tc_fence_after();
    const uint32_t acc = tmem + buf * kWRows + (static_cast<uint32_t>(warp) << 21);
    // values first: whether they are finite decides what the key becomes
    uint32_t v[64];
    __nv_bfloat162 top = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t x[64];
      tmem_ld32(acc + kNope + 64 * half, x);
      tmem_ld32(acc + kNope + 64 * half + 32, x + 32);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        v[32 * half + i] =
            bf16x2(__uint_as_float(x[2 * i]) * sc, __uint_as_float(x[2 * i + 1]) * sc);
        top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[32 * half + i])));
      }
    }
    const bool finite = fmaxf(__low2float(top), __high2float(top)) < INFINITY &&
                        !__isnanf(__low2float(top)) && !__isnanf(__high2float(top));
    // (a sector per store: with 16-byte stores the write path was the limit)
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = finite ? v[i] : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) st_global_32(dst + kNope + 16 * i, v + 8 * i);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t x[64];
      tmem_ld32(acc + 64 * half, x);
      tmem_ld32(acc + 64 * half + 32, x + 32);
      tmem_wait_ld();
      if (half == 1) {
        tc_fence_before();
        mbar_arrive(smem_u32(&ms->acc_empty[buf]));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          o[q] = finite ? bf16x2(__uint_as_float(x[16 * i + 2 * q]) * sc,
                                 __uint_as_float(x[16 * i + 2 * q + 1]) * sc)
                        : 0x7fc07fc0u;
        st_global_32(dst + 64 * half + 16 * i, o);
      }
    }
  }
}

template <int KV>
__global__ void __launch_bounds__(kExpandThreads, 1)
    expand_kernel(const __grid_constant__ ExpandParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ExpandMisc misc;
  ExpandMisc* ms = &misc;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t a_smem = smem_u32(smem), w_smem = a_smem + kChunks * kAChunk;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kChunks; ++i) {
      mbar_init(smem_u32(&ms->a_full[i]), 256);
      mbar_init(smem_u32(&ms->a_empty[i]), 1);
    }
    for (int i = 0; i < kWSlots; ++i) {
      mbar_init(smem_u32(&ms->w_full[i]), 1);
      mbar_init(smem_u32(&ms->w_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ms->acc_full[i]), 1);
      mbar_init(smem_u32(&ms->acc_empty[i]), 128);
    }
    mbar_init(smem_u32(&ms->drain), 1);
    fence_mbar_init();
    ms->ours = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp ? 1 : 0;
    if (!ms->ours) atomicOr(p.err, kErrStale);
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(&ms->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(ms->tmem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (ms->ours) {
    const int64_t units = static_cast<int64_t>(p.num_tiles) * p.heads;
    const int u0 = static_cast<int>(units * blockIdx.x / gridDim.x);
    const int u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    if (warp < 4) {
      run_epilogue(p, ms, tmem, u0, u1, warp, lane);
    } else if (warp < 12) {
      run_rows<KV>(p, ms, smem, u0, u1, threadIdx.x - 128);
    } else if (warp == 12) {
      if (lane == 0) run_weights(p, ms, w_smem, u0, u1);
    } else {
      run_products(p, ms, a_smem, w_smem, tmem, uniform(u0), uniform(u1));
      // no product may run on after the CTA has gone
      if (elect_one()) {
        tc_commit(smem_u32(&ms->drain));
        mbar_wait(smem_u32(&ms->drain), 0, p.err, kErrDrain);
      }
    }
    __syncwarp();
  }
  // Nothing here needs the rotation of the queries; what follows needs both.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

template <int KV>
cudaError_t launch(const ExpandParams& p, int ctas, bool dependent, cudaStream_t stream) {
  constexpr int bytes = kExpandSmem + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(expand_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kExpandThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, expand_kernel<KV>, p);
}

}  // namespace

cudaError_t launch_expand(const ExpandParams& p, int num_ctas, bool dependent,
                          cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(p.num_tiles) * p.heads;
  const int ctas = static_cast<int>(units < num_ctas ? units : num_ctas);
  if (p.kv_dtype == MLA_DTYPE_BF16) return launch<MLA_DTYPE_BF16>(p, ctas, dependent, stream);
  if (p.kv_dtype == MLA_DTYPE_FP8_E4M3)
    return launch<MLA_DTYPE_FP8_E4M3>(p, ctas, dependent, stream);
  return launch<MLA_DTYPE_MXFP4>(p, ctas, dependent, stream);
}

}  // namespace mla
