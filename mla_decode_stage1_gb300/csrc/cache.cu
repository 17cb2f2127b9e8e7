// cache.cu -- the latent cache's bookkeeping and its writes: the cache step
// (pages handed out, page table, slots and positions from request lengths),
// the cache write (norm, rotation, storage encoding, scatter) and the read of
// their device error word.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "layer.h"
#include "ptx.cuh"

namespace mla {
namespace {

// ---------------------------------------------------------------- cache step
//
// With pages(n) = ceil(n / page_size), request b has pages(old_b) pages and
// needs pages(old_b + new_b); it takes the missing ones from the free list at
// the sum of the earlier requests' needs.  All offsets are exclusive sums over
// the requests, so a CTA adds up the requests before its own (8 bytes each,
// from L2) instead of waiting for another CTA: one launch, no order between
// CTAs, and the result does not depend on it.  Latency-bound: 4.6 us for a step
// of 256 requests near 8192 tokens (1.6 MB), for 32 prompts as well.

struct StepParams {
  const int32_t* old_lens;
  const int32_t* new_lens;      // null: one new token per request
  int32_t bs, page_size;
  int32_t* table;
  int64_t table_stride;
  int32_t table_pages;
  const int32_t* free_pages;
  int32_t num_free;
  int32_t* kv_indptr;
  int32_t* last_page;
  int32_t* kv_indices;
  int64_t max_indices;
  int32_t* qo_indptr;
  int64_t* slots;
  int32_t* positions;
  int64_t max_tokens;
  int32_t* pages_used;
  int32_t* err;
  int32_t per_cta;              // requests per CTA (grid.x chunks)
};

constexpr int kStepThreads = 256;

struct Request {
  int64_t len;                  // tokens after the step, within the table's reach
  int32_t old_len, new_len, have, pages;
  int32_t bad;
};

__device__ __forceinline__ Request load_request(const StepParams& p, int32_t b) {
  Request r;
  int32_t o = p.old_lens[b], n = p.new_lens != nullptr ? p.new_lens[b] : 1;
  r.bad = 0;
  if (o < 0 || n < 0) r.bad |= kErrBadLength;
  o = max(o, 0);
  n = max(n, 0);
  const int64_t reach = static_cast<int64_t>(p.table_pages) * p.page_size;
  r.len = static_cast<int64_t>(o) + n;
  if (r.len > reach) r.bad |= kErrCapacity;
  r.len = min(r.len, min(reach, static_cast<int64_t>(INT32_MAX)));
  r.old_len = o;
  r.new_len = n;
  const int64_t kept = min(static_cast<int64_t>(o), r.len);
  r.have = static_cast<int32_t>((kept + p.page_size - 1) / p.page_size);
  r.pages = static_cast<int32_t>((r.len + p.page_size - 1) / p.page_size);
  return r;
}

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kStepThreads / 32; ++w) v += red[w];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kStepThreads) cache_step_kernel(const StepParams p) {
  __shared__ int64_t red[kStepThreads / 32];
  const int tid = threadIdx.x;
  const int32_t b0 = blockIdx.x * p.per_cta, b1 = min(p.bs, b0 + p.per_cta);
  const int64_t lane0 = static_cast<int64_t>(blockIdx.y) * kStepThreads + tid;
  const int64_t step = static_cast<int64_t>(gridDim.y) * kStepThreads;
  int64_t need0 = 0, page0 = 0, tok0 = 0;
  for (int32_t b = tid; b < b0; b += kStepThreads) {
    const Request r = load_request(p, b);
    need0 += r.pages - r.have;
    page0 += r.pages;
    tok0 += r.new_len;
  }
  need0 = block_sum(need0, red);
  page0 = block_sum(page0, red);
  tok0 = block_sum(tok0, red);
  int32_t bad = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const Request r = load_request(p, b);
    bad |= r.bad;
    int32_t* row = p.table + b * p.table_stride;
    // the page that table column j of this request holds
    auto page_of = [&](int32_t j) -> int32_t {
      if (j < r.have) return row[j];
      const int64_t f = need0 + (j - r.have);
      return f < p.num_free ? p.free_pages[f] : -1;
    };
    for (int64_t j = lane0; j < r.pages; j += step) {
      const int32_t page = page_of(static_cast<int32_t>(j));
      if (j >= r.have) row[j] = page;
      if (page < 0) bad |= j < r.have ? kErrBadPage : kErrCapacity;
      if (page0 + j < p.max_indices) p.kv_indices[page0 + j] = page;
      else bad |= kErrCapacity;
    }
    for (int64_t i = lane0; i < r.new_len; i += step) {
      const int64_t pos = static_cast<int64_t>(r.old_len) + i;
      int64_t slot = -1;
      if (pos < r.len) {
        const int32_t j = static_cast<int32_t>(pos) / p.page_size;
        const int32_t page = page_of(j);
        if (page >= 0)
          slot = static_cast<int64_t>(page) * p.page_size +
                 (static_cast<int32_t>(pos) - j * p.page_size);
      }
      if (tok0 + i < p.max_tokens) {
        p.slots[tok0 + i] = slot;
        p.positions[tok0 + i] =
            static_cast<int32_t>(min(pos, static_cast<int64_t>(INT32_MAX)));
      } else {
        bad |= kErrCapacity;
      }
    }
    if (lane0 == 0) {
      p.kv_indptr[b] = static_cast<int32_t>(min(page0, static_cast<int64_t>(INT32_MAX)));
      p.qo_indptr[b] = static_cast<int32_t>(min(tok0, static_cast<int64_t>(INT32_MAX)));
      p.last_page[b] =
          r.pages > 0 ? static_cast<int32_t>(r.len - (r.pages - 1LL) * p.page_size) : 0;
    }
    need0 += r.pages - r.have;
    page0 += r.pages;
    tok0 += r.new_len;
  }
  if (b1 == p.bs) {
    // past the last request: the totals, and tokens that do not exist
    if (lane0 == 0) {
      if (page0 > INT32_MAX || tok0 > INT32_MAX) bad |= kErrCapacity;
      p.kv_indptr[p.bs] = static_cast<int32_t>(min(page0, static_cast<int64_t>(INT32_MAX)));
      p.qo_indptr[p.bs] = static_cast<int32_t>(min(tok0, static_cast<int64_t>(INT32_MAX)));
      if (p.pages_used != nullptr)
        *p.pages_used = static_cast<int32_t>(min(need0, static_cast<int64_t>(p.num_free)));
    }
    for (int64_t i = tok0 + lane0; i < p.max_tokens; i += step) {
      p.slots[i] = -1;
      p.positions[i] = 0;
    }
  }
  if (bad != 0 && p.err != nullptr) atomicOr(p.err, bad);
}

// --------------------------------------------------------------- cache write
//
// One warp per token: y = x r g with r = 1 / sqrt(mean(x^2) + eps) over the
// 512 latent dims, the 64 rotated dims behind them, encoded as the pool
// stores them and written to the token's slot.  One pass: the row stays in
// registers (16 latent dims and one rotation pair a lane).  16,384 tokens to fp8
// take 9.9 us: neither memory (3.3 TB/s) nor issue (about 480 instructions a
// token, 47 % busy) is full, but each of 2.7 waves loads, then computes, then
// stores.  5003 to MXFP4 5.2 us, 32 to bf16 2.2 us.
// Several tokens a warp with the next one's loads ahead took 13.9 us (90
// registers, a quarter of the warps).
//
// The squares of bf16 values are exact in 32 bits and are added with their
// rounding errors kept (an error-free sum of two terms), so the mean is the
// exact one rounded to 32 bits whatever the order of the sum; the rest is
// rounded operation by operation.  A value next to a rounding border of the
// storage type then gets the code that plain 32-bit arithmetic gives it.

struct WriteParams {
  const uint16_t* latent;
  const uint16_t* k_rope;
  int64_t latent_stride, rope_stride;
  const uint16_t* weight;       // null: no norm
  float eps;
  Rotation rot;
  const int64_t* slots;
  int64_t tokens;
  uint8_t* kv;
  const float* kv_scale;
  uint8_t* e8m0;
  int64_t e8m0_stride;
  int64_t pool_rows;
  uint16_t* rows;               // null: not wanted
  int32_t* err;
};

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint16_t one_bf16(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}
__device__ __forceinline__ float f16_lo(uint32_t v) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(v & 0xffffu)));
}
__device__ __forceinline__ float f16_hi(uint32_t v) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(v >> 16)));
}

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {      // (a - b, rounded once)
  return fma_f32x2(b, pack_f32x2(-1.0f, -1.0f), a);
}
// (hi, lo) += v with the rounding error of the sum added to lo (Knuth's
// error-free sum), two sums side by side or one.
__device__ __forceinline__ void sum_exactly2(uint64_t& hi, uint64_t& lo, uint64_t v) {
  const uint64_t s = add_f32x2(hi, v), t = sub2(s, hi);
  lo = add_f32x2(lo, add_f32x2(sub2(hi, sub2(s, t)), sub2(v, t)));
  hi = s;
}
__device__ __forceinline__ void sum_exactly(float& hi, float& lo, float v) {
  const float s = __fadd_rn(hi, v);
  const float t = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(v, t)));
  hi = s;
}

// The biased exponent that a block of 32 values with this largest magnitude
// shares: floor(log2 amax) - 2, at least 2^-127; 255 (NaN) if not finite.
__device__ __forceinline__ int mx_exponent(float amax) {
  const int ex = static_cast<int>(__float_as_uint(amax) >> 23);
  return ex == 255 ? 255 : max(ex - 2, 0);
}
// 2^(e - 127) and its reciprocal, for e in [0, 254].
__device__ __forceinline__ float exp2_biased(int e) {
  return __uint_as_float(e > 0 ? static_cast<uint32_t>(e) << 23 : 0x00400000u);
}
// max of magnitudes that lets NaN through (as all-ones bits)
__device__ __forceinline__ float mag_max(float a, float b) {
  const uint32_t x = __float_as_uint(a) & 0x7fffffffu, y = __float_as_uint(b) & 0x7fffffffu;
  return __uint_as_float(max(x, y));
}

// What one warp loads of a token before it computes.
struct TokenIn {
  int64_t slot;
  uint4 raw[2];                 // dims 8 lane .. and 256 + 8 lane ..
  float ra, rb, c, s;           // rotation pair `lane` and its angle
};

__device__ __forceinline__ TokenIn load_token(const WriteParams& p, int64_t t, int lane, int d0,
                                              int d1) {
  TokenIn in;
  in.slot = p.slots[t];
  const uint16_t* src = p.latent + t * p.latent_stride;
  in.raw[0] = *reinterpret_cast<const uint4*>(src + 8 * lane);
  in.raw[1] = *reinterpret_cast<const uint4*>(src + 256 + 8 * lane);
  const uint16_t* rsrc = p.k_rope + t * p.rope_stride;
  in.ra = __uint_as_float(static_cast<uint32_t>(rsrc[d0]) << 16);
  in.rb = __uint_as_float(static_cast<uint32_t>(rsrc[d1]) << 16);
  if (p.rot.cos_sin != nullptr) {
    const float* cs = rotation_row(p.rot, t, lane == 0 ? p.err : nullptr);
    in.c = cs[lane];
    in.s = cs[kRope / 2 + lane];
  }
  return in;
}

// Norm, rotation, encoding and store of one token.
template <int KV>
__device__ __forceinline__ void write_token(const WriteParams& p, int64_t t, const TokenIn& in,
                                            int lane, int d0, int d1, const uint4& w0,
                                            const uint4& w1) {
  int64_t slot = in.slot;
  if (slot < -1 || slot >= p.pool_rows) {
    if (lane == 0 && p.err != nullptr) atomicOr(p.err, kErrBadSlot);
    slot = -1;
  }
  float ra = in.ra, rb = in.rb;
  if (p.rot.cos_sin != nullptr) rotate(ra, rb, in.c, in.s);
  float y[16];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t u[4] = {in.raw[g].x, in.raw[g].y, in.raw[g].z, in.raw[g].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[8 * g + 2 * i] = bf16_lo(u[i]);
      y[8 * g + 2 * i + 1] = bf16_hi(u[i]);
    }
  }
  if (p.weight != nullptr) {
    uint64_t hi2 = 0, lo2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t v = pack_f32x2(y[2 * i], y[2 * i + 1]);
      sum_exactly2(hi2, lo2, mul_f32x2(v, v));
    }
    float hi, lo, h1, l1;
    unpack_f32x2(hi2, hi, h1);
    unpack_f32x2(lo2, lo, l1);
    lo = __fadd_rn(lo, l1);
    sum_exactly(hi, lo, h1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float oh = __shfl_xor_sync(0xffffffffu, hi, o);
      const float ol = __shfl_xor_sync(0xffffffffu, lo, o);
      // the same operands in the same order in both lanes of a pair
      float a = (lane & o) ? oh : hi, b = (lane & o) ? hi : oh;
      float c = __fadd_rn(lo, ol);
      sum_exactly(a, c, b);
      hi = a;
      lo = c;
    }
    float sum = __fadd_rn(hi, lo);
    // a sum that is not finite has no error term
    if (!(fabsf(hi) < INFINITY)) sum = hi;
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(sum * (1.0f / kVDim), p.eps)));
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    const uint64_t r2 = pack_f32x2(r, r);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      unpack_f32x2(mul_f32x2(mul_f32x2(pack_f32x2(y[2 * i], y[2 * i + 1]), r2),
                        pack_f32x2(bf16_lo(w[i]), bf16_hi(w[i]))),
                   y[2 * i], y[2 * i + 1]);
  }
  uint16_t* out = p.rows != nullptr ? p.rows + t * kQkDim : nullptr;
  if constexpr (KV == MLA_DTYPE_BF16) {
    uint16_t* dst = slot >= 0 ? reinterpret_cast<uint16_t*>(p.kv) + slot * kQkDim : nullptr;
    const uint16_t a = one_bf16(ra), b = one_bf16(rb);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint4 v;
      v.x = pack_bf16(y[8 * g + 0], y[8 * g + 1]);
      v.y = pack_bf16(y[8 * g + 2], y[8 * g + 3]);
      v.z = pack_bf16(y[8 * g + 4], y[8 * g + 5]);
      v.w = pack_bf16(y[8 * g + 6], y[8 * g + 7]);
      if (dst) *reinterpret_cast<uint4*>(dst + 256 * g + 8 * lane) = v;
      if (out) *reinterpret_cast<uint4*>(out + 256 * g + 8 * lane) = v;
    }
    if (dst) { dst[kVDim + d0] = a; dst[kVDim + d1] = b; }
    if (out) { out[kVDim + d0] = a; out[kVDim + d1] = b; }
  } else if constexpr (KV == MLA_DTYPE_FP8_E4M3) {
    const Fp8Scale fs = load_fp8_scale(p.kv_scale);
    const float sc = fs.sc;
    uint8_t* dst = slot >= 0 ? p.kv + slot * kQkDim : nullptr;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t v8[2];
      to_e4m3<8>(y + 8 * g, fs, v8);
      const uint32_t c[4] = {v8[0] & 0xffffu, v8[0] >> 16, v8[1] & 0xffffu, v8[1] >> 16};
      if (dst)
        *reinterpret_cast<uint2*>(dst + 256 * g + 8 * lane) = make_uint2(v8[0], v8[1]);
      if (out) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(c[i]));
          v[i] = pack_bf16(f16_lo(h) * sc, f16_hi(h) * sc);
        }
        *reinterpret_cast<uint4*>(out + 256 * g + 8 * lane) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    const float pair[2] = {ra, rb};
    uint32_t c2;
    to_e4m3<2>(pair, fs, &c2);
    const uint16_t c = static_cast<uint16_t>(c2);
    if (dst && !p.rot.half) {
      *reinterpret_cast<uint16_t*>(dst + kVDim + d0) = c;
    } else if (dst) {
      dst[kVDim + d0] = static_cast<uint8_t>(c & 0xff);
      dst[kVDim + d1] = static_cast<uint8_t>(c >> 8);
    }
    if (out) {
      const uint32_t h = e4m3x2_to_f16x2(c);
      out[kVDim + d0] = one_bf16(f16_lo(h) * sc);
      out[kVDim + d1] = one_bf16(f16_hi(h) * sc);
    }
  } else {
    uint8_t* dst = slot >= 0 ? p.kv + slot * (kQkDim / 2) : nullptr;
    uint8_t* sdst = slot >= 0 ? p.e8m0 + slot * p.e8m0_stride : nullptr;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      // 4 lanes hold a block of 32
      float am = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) am = mag_max(am, y[8 * g + i]);
      am = mag_max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = mag_max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int e = mx_exponent(am);
      const float up = exp2_biased(254 - e);       // 2^(127 - e); e = 255 stores zeros below
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = e == 255 ? 0u : to_e2m1x2(y[8 * g + 2 * i] * up, y[8 * g + 2 * i + 1] * up);
      if (dst) {
        *reinterpret_cast<uint32_t*>(dst + 128 * g + 4 * lane) =
            c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
        if ((lane & 3) == 0) sdst[8 * g + (lane >> 2)] = static_cast<uint8_t>(e);
      }
      if (out) {
        const float down = e == 255 ? __uint_as_float(0x7fc00000u) : exp2_biased(e);
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t h = e2m1x2_to_f16x2(c[i]);
          v[i] = pack_bf16(f16_lo(h) * down, f16_hi(h) * down);
        }
        *reinterpret_cast<uint4*>(out + 256 * g + 8 * lane) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    // The rotated dims are two blocks.  In pairs (2i, 2i+1), lanes 0..15 hold
    // the first; in halves, every lane holds one dim of each.  Lane i then
    // stores byte i, the dims (2i, 2i+1), and lanes 0 and 16 the exponents.
    float va = ra, vb = rb;
    if (p.rot.half) {
      // dims (2i, 2i+1) are the a (i < 16) or b (i >= 16) of lanes 2i, 2i+1 (mod 32)
      const int s0 = (2 * lane) & 31, s1 = (2 * lane + 1) & 31;
      const float a0 = __shfl_sync(0xffffffffu, ra, s0), a1 = __shfl_sync(0xffffffffu, ra, s1);
      const float b0 = __shfl_sync(0xffffffffu, rb, s0), b1 = __shfl_sync(0xffffffffu, rb, s1);
      va = lane < 16 ? a0 : b0;
      vb = lane < 16 ? a1 : b1;
    }
    float am = mag_max(va, vb);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) am = mag_max(am, __shfl_xor_sync(0xffffffffu, am, o));
    const int e = mx_exponent(am);
    const float up = exp2_biased(254 - e);
    const uint32_t c = e == 255 ? 0u : to_e2m1x2(va * up, vb * up);
    if (dst) {
      dst[kVDim / 2 + lane] = static_cast<uint8_t>(c);
      if ((lane & 15) == 0) sdst[kVDim / 32 + (lane >> 4)] = static_cast<uint8_t>(e);
    }
    if (out) {
      const float down = e == 255 ? __uint_as_float(0x7fc00000u) : exp2_biased(e);
      const uint32_t h = e2m1x2_to_f16x2(c);
      *reinterpret_cast<uint32_t*>(out + kVDim + 2 * lane) =
          pack_bf16(f16_lo(h) * down, f16_hi(h) * down);
    }
  }
}

template <int KV>
__global__ void __launch_bounds__(256, 5) cache_write_kernel(const WriteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const int d0 = rope_dim0(lane, p.rot.half), d1 = rope_dim1(lane, p.rot.half);
  const TokenIn in = load_token(p, t, lane, d0, d1);
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (p.weight != nullptr) {
    w0 = *reinterpret_cast<const uint4*>(p.weight + 8 * lane);
    w1 = *reinterpret_cast<const uint4*>(p.weight + 256 + 8 * lane);
  }
  write_token<KV>(p, t, in, lane, d0, d1, w0, w1);
}

}  // namespace
}  // namespace mla

extern "C" mla_status mla_cache_step(const int32_t* old_lens, const int32_t* new_lens,
                                     int32_t batch_size, int32_t page_size, int32_t* block_table,
                                     int64_t table_stride, int32_t table_pages,
                                     const int32_t* free_pages, int32_t num_free,
                                     int32_t* kv_indptr, int32_t* kv_last_page_len,
                                     int32_t* kv_indices, int64_t max_indices, int32_t* qo_indptr,
                                     int64_t* slots, int32_t* positions, int64_t max_tokens,
                                     int32_t* pages_used, int32_t* err, mla_stream_t stream) {
  if (batch_size < 1 || page_size < 1 || table_pages < 0 || num_free < 0 || max_indices < 0 ||
      max_tokens < 0 || table_stride < table_pages)
    return MLA_ERR_INVALID_ARG;
  if (old_lens == nullptr || (block_table == nullptr && table_pages > 0) ||
      (free_pages == nullptr && num_free > 0) || kv_indptr == nullptr ||
      kv_last_page_len == nullptr || (kv_indices == nullptr && max_indices > 0) ||
      qo_indptr == nullptr || ((slots == nullptr || positions == nullptr) && max_tokens > 0))
    return MLA_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(old_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                        static_cast<const void*>(kv_indptr),
                        static_cast<const void*>(kv_last_page_len),
                        static_cast<const void*>(kv_indices), static_cast<const void*>(qo_indptr),
                        static_cast<const void*>(positions), static_cast<const void*>(pages_used),
                        static_cast<const void*>(err)})
    if (!mla::ptr_aligned(q, 4)) return MLA_ERR_INVALID_ARG;
  if (!mla::ptr_aligned(slots, 8)) return MLA_ERR_INVALID_ARG;
  mla::StepParams p{old_lens, new_lens, batch_size, page_size, block_table, table_stride,
                    table_pages, free_pages, num_free, kv_indptr, kv_last_page_len, kv_indices,
                    max_indices, qo_indptr, slots, positions, max_tokens, pages_used, err, 1};
  // At most 1024 chunks of requests; where the output arrays are long for the
  // number of chunks, several CTAs share one, about 1024 entries each.
  p.per_cta = (batch_size + 1023) / 1024;
  const int32_t chunks = (batch_size + p.per_cta - 1) / p.per_cta;
  const int64_t per = (max_indices + max_tokens) / chunks / 1024 + 1;
  const int32_t slices = static_cast<int32_t>(std::min<int64_t>(per, std::max(1, 1216 / chunks)));
  mla::cache_step_kernel<<<dim3(chunks, slices), mla::kStepThreads, 0,
                           reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_cache_write(const void* latent, int64_t latent_stride,
                                      const void* k_rope, int64_t k_rope_stride,
                                      const void* norm_weight, float eps, const float* cos_sin,
                                      int64_t max_positions, const int32_t* positions,
                                      mla_rope rope, const int64_t* slots, int64_t num_tokens,
                                      mla_dtype kv_dtype, void* kv, const float* kv_scale,
                                      uint8_t* kv_e8m0, int64_t kv_e8m0_row_stride,
                                      int64_t kv_pool_rows, void* rows, int32_t* err,
                                      mla_stream_t stream_) {
  if (num_tokens < 0 || kv_pool_rows < 1 || kv_pool_rows > INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (kv_dtype < MLA_DTYPE_BF16 || kv_dtype > MLA_DTYPE_MXFP4) return MLA_ERR_INVALID_ARG;
  if (kv == nullptr || (kv_dtype == MLA_DTYPE_FP8_E4M3 && kv_scale == nullptr) ||
      (kv_dtype == MLA_DTYPE_MXFP4 && (kv_e8m0 == nullptr || kv_e8m0_row_stride < 18)))
    return MLA_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !mla::ptr_aligned(kv, 16) || !mla::ptr_aligned(kv_scale, 4) ||
      !mla::ptr_aligned(err, 4))
    return MLA_ERR_INVALID_ARG;
  mla::Rotation rot{cos_sin, positions, max_positions, rope == MLA_ROPE_HALF ? 1 : 0};
  if (!mla::rotation_ok(rot, rope, num_tokens) || !mla::ptr_aligned(positions, 4)) return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (latent == nullptr || k_rope == nullptr || slots == nullptr) return MLA_ERR_INVALID_ARG;
  if (latent_stride < mla::kVDim || k_rope_stride < mla::kRope) return MLA_ERR_INVALID_ARG;
  if (!mla::ptr_aligned(latent, 16) || latent_stride % 8 != 0 || !mla::ptr_aligned(k_rope, 2) ||
      !mla::ptr_aligned(norm_weight, 16) || !mla::ptr_aligned(slots, 8) ||
      !mla::ptr_aligned(rows, 16))
    return MLA_ERR_INVALID_ARG;
  const int64_t ctas = (num_tokens + 7) / 8;
  if (ctas > INT32_MAX) return MLA_ERR_INVALID_ARG;
  mla::WriteParams p{static_cast<const uint16_t*>(latent), static_cast<const uint16_t*>(k_rope),
                     latent_stride, k_rope_stride, static_cast<const uint16_t*>(norm_weight), eps,
                     rot, slots, num_tokens, static_cast<uint8_t*>(kv), kv_scale, kv_e8m0,
                     kv_e8m0_row_stride, kv_pool_rows, static_cast<uint16_t*>(rows), err};
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const dim3 grid(static_cast<unsigned>(ctas));
  if (kv_dtype == MLA_DTYPE_BF16)
    mla::cache_write_kernel<MLA_DTYPE_BF16><<<grid, 256, 0, stream>>>(p);
  else if (kv_dtype == MLA_DTYPE_FP8_E4M3)
    mla::cache_write_kernel<MLA_DTYPE_FP8_E4M3><<<grid, 256, 0, stream>>>(p);
  else
    mla::cache_write_kernel<MLA_DTYPE_MXFP4><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_error_check(int32_t* err, mla_stream_t stream_) {
  if (err == nullptr || !mla::ptr_aligned(err, 4)) return MLA_ERR_INVALID_ARG;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  int32_t word = 0;
  if (cudaMemcpyAsync(&word, err, sizeof(word), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (word == 0) return MLA_OK;
  if (cudaMemsetAsync(err, 0, sizeof(word), stream) != cudaSuccess) return MLA_ERR_CUDA;
  if (word & mla::kErrTimeout) return MLA_ERR_DEVICE_TIMEOUT;
  return word == mla::kErrCapacity ? MLA_ERR_CAPACITY : MLA_ERR_INVALID_ARG;
}
