// layer.h -- internal declarations shared by the operators around the
// decode call (cache.cu, absorb.cu, prefill_api.cu and its kernels): their
// geometry, the bits of their device error word and the rotation of the 64
// position dims.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "mla_decode.h"
#ifdef __CUDACC__
#include "ptx.cuh"
#endif

namespace mla {

constexpr int kRope = 64;                 // rotated dims of a query head and of the cached row
constexpr int kNope = MLA_NOPE_DIM;       // unrotated query / key dims per head (expanded form)
constexpr int kVHead = MLA_V_HEAD_DIM;    // value dims per head (expanded form)
constexpr int kQHead = kNope + kRope;     // query dims per head (expanded form)
constexpr int kWRows = kNope + kVHead;    // weight rows per head: keys, then values

// Bits of the operators' device error word beside kErrBadPage (kernels.h).
enum : int32_t {
  kErrBadLength = 1 << 8,      // a negative length
  kErrCapacity = 1 << 9,       // pages, table columns or output entries ran out
  kErrBadSlot = 1 << 10,       // a slot outside the pool (other than -1)
  kErrBadPosition = 1 << 11    // a position outside the rotation table
};

inline bool ptr_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// The rotation's arguments: a table row holds 32 cosines, then 32 sines.
struct Rotation {
  const float* cos_sin;        // [max_positions, 64], or null: no rotation
  const int32_t* positions;    // [tokens]
  int64_t max_positions;
  int32_t half;                // 0: pairs (2i, 2i+1); 1: pairs (i, i + 32)
};

// Checks shared by the calls that rotate: both pointers or neither (the
// positions of no token may be anywhere: an empty array often has no address).
inline bool rotation_ok(const Rotation& r, int rope, int64_t tokens) {
  if (rope != MLA_ROPE_INTERLEAVED && rope != MLA_ROPE_HALF) return false;
  if (tokens == 0) return true;
  if ((r.cos_sin == nullptr) != (r.positions == nullptr)) return false;
  return r.cos_sin == nullptr || (r.max_positions >= 1 && ptr_aligned(r.cos_sin, 16));
}

#ifdef __CUDACC__
// Token t's table row.  A position outside the table is reported and read as 0.
__device__ __forceinline__ const float* rotation_row(const Rotation& r, int64_t t, int32_t* err) {
  int64_t pos = r.positions[t];
  if (pos < 0 || pos >= r.max_positions) {
    if (err != nullptr) atomicOr(err, kErrBadPosition);
    pos = 0;
  }
  return r.cos_sin + pos * kRope;
}

// The two dims of rotation pair i.
__device__ __forceinline__ int rope_dim0(int i, int half) { return half ? i : 2 * i; }
__device__ __forceinline__ int rope_dim1(int i, int half) { return half ? i + kRope / 2 : 2 * i + 1; }

// (a, b) turned by the angle with cosine c and sine s.  Products and sum are
// rounded one by one (no fused multiply-add), so that the stored codes are
// those of the formula in plain 32-bit arithmetic.
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
  b = y;
}

// Two values to e4m3 (round to nearest even, saturating at 448; NaN stays
// NaN), `lo` in the low byte.
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// A per-tensor scale.  x / sc as plain division rounds it, in three operations
// where the division instruction's sequence takes about 80 cycles: q0 = x r
// with r = 1 / sc rounded, then q0 + (x - q0 sc) r, which is the rounded
// quotient while nothing over- or underflows (Markstein 1990).  The negative of
// it is computed and the codes' signs turned: x = -0 keeps its sign that way.
struct Fp8Scale {
  float sc, r;
  bool normal;                // 2^-60 < sc < 2^60
};
__device__ __forceinline__ Fp8Scale load_fp8_scale(const float* p) {
  const float sc = *p;
  return Fp8Scale{sc, __fdiv_rn(1.0f, sc), sc > 0x1p-60f && sc < 0x1p60f};
}
// N values divided by the scale to e4m3, four a word.  Values that are not
// finite, or whose quotient is not, go through the division instruction.
template <int N>
__device__ __forceinline__ void to_e4m3(const float* y, const Fp8Scale& s, uint32_t* out) {
  uint32_t top = 0;           // largest magnitude, as bits: NaN above all
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
  uint16_t c[N / 2];
  const bool fast =
      s.normal && __uint_as_float(top) < 1e30f && __uint_as_float(top) * s.r < 1e30f;
  if (fast) {
    const uint64_t n2 = pack_f32x2(-s.r, -s.r), s2 = pack_f32x2(s.sc, s.sc);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t x = pack_f32x2(y[i], y[i + 1]), q0 = mul_f32x2(x, n2);
      float a, b;
      unpack_f32x2(fma_f32x2(fma_f32x2(q0, s2, x), n2, q0), a, b);
      c[i / 2] = to_e4m3x2(a, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2)
      c[i / 2] = to_e4m3x2(__fdiv_rn(y[i], s.sc), __fdiv_rn(y[i + 1], s.sc));
  }
#pragma unroll
  for (int i = 0; i < (N + 3) / 4; ++i)
    out[i] = (c[2 * i] | (N > 2 ? static_cast<uint32_t>(c[2 * i + 1]) << 16 : 0u)) ^
             (fast ? 0x80808080u : 0u);
}
// Two e4m3 codes as half precision (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// Two values to e2m1 (round to nearest even, saturating at 6), `lo` in the low nibble.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
      "cvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}
// Two e2m1 codes (one byte) as half precision (exact).
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.u8.u32 t, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four e2m1 codes (the low 16 bits of x) times a power of two given as a bf16
// pair, exactly: the magnitudes' bf16 bytes are looked up by byte permutes, the
// code's three low bits being the selector.
__device__ __forceinline__ void e2m1x4_to_bf16(uint32_t x, uint32_t scale, uint32_t& lo,
                                               uint32_t& hi) {
  const uint32_t sel = x & 0x7777u;
  // 0, 0.5, 1, 1.5, 2, 3, 4, 6: high bytes, low bytes; selector bit 3 copies a
  // byte's top bit, which makes 0xff of a negative code and 0x80 of another
  uint32_t h = prmt(0x3f3f3f00u, 0x40404040u, sel);
  const uint32_t l = prmt(0xc0800000u, 0xc0804000u, sel);
  h |= (prmt(0x80808080u, 0x80808080u, x) << 7) & 0x80808080u;
  lo = mul_bf16x2(prmt(l, h, 0x5140), scale);
  hi = mul_bf16x2(prmt(l, h, 0x7362), scale);
}
// The power of two of an e8m0 byte as a bf16 pair (255: NaN).
__device__ __forceinline__ uint32_t e8m0_to_bf16x2(uint32_t e) {
  const uint32_t s = e == 255u ? 0x7fc0u : e > 0 ? e << 7 : 0x0040u;
  return s | (s << 16);
}
#endif

}  // namespace mla
