// attn.cu -- the attention kernel of the expanded form: causal attention of
// 256-row query blocks over the expanded keys and values of one head, one
// pass over the keys with the running maximum and sum of a softmax.
//
// For query rows i and keys k of 192 dims (128 expanded, 64 rotated):
//     s[i,k] = sm_scale q_i . k,   m_i = max_k s[i,k],   p = 2^(s log2 e - m),
//     out_i = sum_k p v_k / sum_k p,   lse_i = (m + log2 sum p) ln 2.
//
// Bound: matrix products, 2 (192 + 128) flops per (query, key); the exponents
// (one per pair) come next.  An item holds two 128-row query tiles so that
// one tile's softmax runs under the other's products: per 128-key step the
// tensor pipe has QK^T (12 K steps) and PV (8) of both tiles, and S, P and O
// of both fill the 512 columns of tensor memory exactly (S 2 x 128, P over
// S's first 64 columns, O 2 x 128).
//
// Roles (512 threads): warps 0-3 and 4-7 hold the softmax of tile 0 and 1, a
// thread per row; warps 8-11 rotate the query's last 64 dims in shared
// memory; warp 12 loads (TMA), warp 13 issues the products.

#include <cuda_bf16.h>

#include "prefill.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 512;
constexpr uint32_t kChunkBytes = 128 * 128;        // 128 rows x 64 bf16
constexpr uint32_t kQTileBytes = 3 * kChunkBytes;
constexpr uint32_t kQBytes = 2 * kQTileBytes;
constexpr int kSlots = 8;                          // ring of 16 KB: K tiles take 3, V tiles 2
constexpr uint32_t kSmemBytes = kQBytes + kSlots * kChunkBytes;
constexpr uint32_t kColS = 0, kColO = 256;         // tile t: + 128 t
// A row's maximum is kept until a score exceeds it by 2^8: the probabilities
// (bf16 has the exponent range of fp32) and their fp32 sums stay finite, and
// rescaling O is rare.
constexpr float kLag = 8.0f;

struct Misc {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full[2], q_ready[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem;
  uint32_t ours;
};

// Key steps of tile t of an item: those with a key that the tile's last row sees.
__device__ __forceinline__ int tile_steps(const AttnItem& w, int t) {
  if (w.rows <= t * kPfTile) return 0;
  const int last = min(w.rows, (t + 1) * kPfTile) - 1;
  const int end = min(w.kv_end, w.vis0 + last);
  return end > w.kv_begin ? (end - w.kv_begin + kPfTile - 1) / kPfTile : 0;
}

__device__ __forceinline__ AttnItem load_item(const AttnItem* p) {
  const int4 a = reinterpret_cast<const int4*>(p)[0], b = reinterpret_cast<const int4*>(p)[1];
  return AttnItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// A wait of the whole warp, which goes on (or gives up) together.
__device__ __forceinline__ bool all_waited(bool ok) { return __all_sync(0xffffffffu, ok); }

struct RingCursor {
  uint32_t n = 0;
  __device__ uint32_t slot() const { return n % kSlots; }
  __device__ uint32_t lap() const { return n / kSlots; }
};

// ---------------------------------------------------------------- loads
__device__ void run_loads(const AttnParams& p, Misc* ms, uint32_t q_smem, uint32_t ring, int it0,
                          int it1) {
  RingCursor c;
  uint32_t nq0 = 0, nq1 = 0;        // query tiles loaded of either kind
  bool ok = true;
  auto open = [&](uint32_t bytes) -> uint32_t {
    const uint32_t s = c.slot();
    if (c.lap() > 0 &&
        !mbar_wait(smem_u32(&ms->empty[s]), (c.lap() - 1) & 1, p.err, kErrProducer)) {
      ok = false;
      return 0;
    }
    mbar_arrive_expect_tx(smem_u32(&ms->full[s]), bytes);
    ++c.n;
    return s;
  };
  const uint64_t keep = l2_policy_evict_normal();
  auto load_k = [&](const AttnItem& w, int j) {
    const int row = w.kv_row + w.kv_begin + j * kPfTile;
#pragma unroll 1
    for (int ch = 0; ch < 3 && ok; ++ch) {
      const uint32_t s = open(kChunkBytes);
      if (!ok) return;
      const uint32_t dst = ring + s * kChunkBytes, bar = smem_u32(&ms->full[s]);
      for (int half = 0; half < 2; ++half) {
        if (ch < 2)
          tma_load_3d(dst + half * 8192, &p.map_kx, bar, ch * 64, row + half * 64, w.head, keep);
        else
          tma_load_3d(dst + half * 8192, &p.map_kr, bar, 0, row + half * 64, 0, keep);
      }
    }
  };
  auto load_v = [&](const AttnItem& w, int j) {
    const int row = w.kv_row + w.kv_begin + j * kPfTile;
#pragma unroll 1
    for (int half = 0; half < 2 && ok; ++half) {
      const uint32_t s = open(kChunkBytes);
      if (!ok) return;
      const uint32_t dst = ring + s * kChunkBytes, bar = smem_u32(&ms->full[s]);
      for (int ch = 0; ch < 2; ++ch)
        tma_load_3d(dst + ch * 8192, &p.map_kx, bar, kNope + ch * 64, row + half * 64, w.head,
                    keep);
    }
  };
  for (int it = it0; it < it1 && ok; ++it) {
    const AttnItem w = load_item(p.items + it);
    const int n0 = tile_steps(w, 0), n1 = tile_steps(w, 1), n = max(n0, n1);
    if (n == 0) continue;
    load_k(w, 0);
    if (!ok) break;
    for (int t = 0; t < 2 && ok; ++t) {
      if ((t ? n1 : n0) == 0) continue;
      const uint32_t k = t ? nq1++ : nq0++;
      if (k > 0 && !mbar_wait(smem_u32(&ms->q_empty[t]), (k - 1) & 1, p.err, kErrProducer)) {
        --(t ? nq1 : nq0);
        ok = false;
        break;
      }
      const uint32_t bar = smem_u32(&ms->q_full[t]);
      mbar_arrive_expect_tx(bar, kQTileBytes);
      for (int ch = 0; ch < 3; ++ch)
        tma_load_3d(q_smem + t * kQTileBytes + ch * kChunkBytes, &p.map_q, bar, ch * 64, w.head,
                    w.q_row + t * kPfTile, keep);
    }
    if (!ok) break;
    load_v(w, 0);
    for (int j = 1; j < n && ok; ++j) {
      load_k(w, j);
      load_v(w, j);
    }
  }
  if (!ok) {
    // a wait gave up: no copy may land after the CTA has gone
    for (uint32_t k = c.n > kSlots ? c.n - kSlots : 0; k < c.n; ++k)
      mbar_wait(smem_u32(&ms->full[k % kSlots]), (k / kSlots) & 1, p.err, kErrProducer);
    if (nq0 > 0) mbar_wait(smem_u32(&ms->q_full[0]), (nq0 - 1) & 1, p.err, kErrProducer);
    if (nq1 > 0) mbar_wait(smem_u32(&ms->q_full[1]), (nq1 - 1) & 1, p.err, kErrProducer);
  }
}

// ------------------------------------------------------------- products
// The whole warp walks the steps; one lane issues.
__device__ void run_products(const AttnParams& p, Misc* ms, uint32_t q_smem, uint32_t ring,
                             uint32_t tmem, int it0, int it1) {
  constexpr uint32_t idesc_qk = make_idesc(1, 1, false, false, 128, 128);
  constexpr uint32_t idesc_pv = make_idesc(1, 1, false, true, 128, 128);
  uint32_t n = 0;                   // ring chunks consumed
  uint32_t nq0 = 0, nq1 = 0;        // query tiles used of either kind
  uint32_t np0 = 0, np1 = 0;        // P tiles consumed of query tile 0, 1
  const uint64_t qd = smem_desc(q_smem, 16, 1024, kSwizzle128B);
  const uint64_t kd = smem_desc(ring, 16, 1024, kSwizzle128B);
  const uint64_t vd = smem_desc(ring, 8192, 1024, kSwizzle128B);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return all_waited(mbar_wait(smem_u32(bar), parity, p.err, kErrMma));
  };
  // S_t = Q_t K^T, K in ring chunks k, k + 1, k + 2 (waited for by the first tile that meets them)
  // ; `last`: this query tile's last step of the item
  auto qk = [&](int t, uint32_t k, bool fresh, bool last) {
#pragma unroll
    for (int ch = 0; ch < 3; ++ch) {
      const uint32_t s = (k + ch) % kSlots;
      if (fresh && !wait(&ms->full[s], ((k + ch) / kSlots) & 1)) return false;
      if (fresh) tc_fence_after();
      const uint64_t a = qd + ((t * kQTileBytes + ch * kChunkBytes) >> 4);
      const uint64_t b = kd + ((s * kChunkBytes) >> 4);
      const uint32_t d = tmem + kColS + 128 * t;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16(d, a + 2 * kk, b + 2 * kk, idesc_qk, (ch | kk) != 0);
      }
    }
    if (elect_one()) {
      tc_commit(smem_u32(&ms->s_full[t]));
      if (last) tc_commit(smem_u32(&ms->q_empty[t]));
    }
    return true;
  };
  // O_t (+)= P_t V, V in ring chunks k, k + 1 (64 keys each)
  auto pv = [&](int t, uint32_t k, bool fresh, bool first) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t s = (k + half) % kSlots;
      if (fresh && !wait(&ms->full[s], ((k + half) / kSlots) & 1)) return false;
      if (fresh) tc_fence_after();
      const uint64_t b = vd + ((s * kChunkBytes) >> 4);
      const uint32_t d = tmem + kColO + 128 * t, a = tmem + kColS + 128 * t + 32 * half;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ta(d, a + 8 * kk, b + 128 * kk, idesc_pv, !(first && half == 0 && kk == 0));
      }
    }
    return true;
  };
  auto release = [&](uint32_t k, int count) {
    if (elect_one()) {
      for (int i = 0; i < count; ++i) tc_commit(smem_u32(&ms->empty[(k + i) % kSlots]));
    }
  };
  for (int it = it0; it < it1; ++it) {
    const AttnItem w = load_item(p.items + it);
    const int n0 = uniform(tile_steps(w, 0)), n1 = uniform(tile_steps(w, 1));
    const int steps = max(n0, n1);
    if (steps == 0) continue;
    if (n0 > 0) {
      if (!wait(&ms->q_ready[0], nq0++ & 1)) return;
      tc_fence_after();
      if (!qk(0, n, true, n0 == 1)) return;
    }
    if (n1 > 0) {
      if (!wait(&ms->q_ready[1], nq1++ & 1)) return;
      tc_fence_after();
      if (!qk(1, n, n0 == 0, n1 == 1)) return;
    }
    release(n, 3);
    n += 3;
    for (int j = 0; j < steps; ++j) {
      const uint32_t v = n, k = n + 2;
      bool fresh_v = true, fresh_k = true;
      if (j < n0) {
        if (!wait(&ms->p_full[0], np0++ & 1)) return;
        tc_fence_after();
        if (!pv(0, v, true, j == 0)) return;
        fresh_v = false;
        if (j + 1 == n0 && elect_one()) tc_commit(smem_u32(&ms->o_full[0]));
        if (j + 1 < n0) {
          if (!qk(0, k, true, j + 2 == n0)) return;
          fresh_k = false;
        }
      }
      if (j < n1) {
        if (!wait(&ms->p_full[1], np1++ & 1)) return;
        tc_fence_after();
        if (!pv(1, v, fresh_v, j == 0)) return;
        if (j + 1 == n1 && elect_one()) tc_commit(smem_u32(&ms->o_full[1]));
      }
      // the values' chunks are free before the next scores are through
      release(v, 2);
      n += 2;
      if (j + 1 < steps) {
        if (j + 1 < n1 && !qk(1, k, fresh_k, j + 2 == n1)) return;
        release(k, 3);
        n += 3;
      }
    }
  }
}

// ------------------------------------------------------------- rotation
// Rotates dims 128..191 of the item's query rows in place (chunk 2 of each
// tile; 16-byte granule g of row r sits at g ^ (r & 7)).  Four lanes a row,
// eight pairs a lane, four rows a thread and tile.  The rotated values are
// rounded to bf16 once more: they are operands of a bf16 product.
__device__ __forceinline__ void rotate_row(const Rotation& rot, uint8_t* row, int r, int lane4,
                                           const float4 (&c)[2], const float4 (&s)[2]) {
  const int g0 = rot.half ? lane4 : 2 * lane4, g1 = rot.half ? lane4 + 4 : 2 * lane4 + 1;
  uint4* p0 = reinterpret_cast<uint4*>(row + ((g0 ^ (r & 7)) << 4));
  uint4* p1 = reinterpret_cast<uint4*>(row + ((g1 ^ (r & 7)) << 4));
  const uint4 x = *p0, y = *p1;
  uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  const float cs[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
  const float sn[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
  auto lo = [](uint32_t v) { return __uint_as_float(v << 16); };
  auto hi = [](uint32_t v) { return __uint_as_float(v & 0xffff0000u); };
  auto pack = [](float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  };
  if (rot.half) {
    // element i of the first granule turns with element i of the second
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a0 = lo(u[i]), b0 = lo(u[4 + i]), a1 = hi(u[i]), b1 = hi(u[4 + i]);
      rotate(a0, b0, cs[2 * i], sn[2 * i]);
      rotate(a1, b1, cs[2 * i + 1], sn[2 * i + 1]);
      u[i] = pack(a0, a1);
      u[4 + i] = pack(b0, b1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a = lo(u[i]), b = hi(u[i]);
      rotate(a, b, cs[i], sn[i]);
      u[i] = pack(a, b);
    }
  }
  *p0 = make_uint4(u[0], u[1], u[2], u[3]);
  *p1 = make_uint4(u[4], u[5], u[6], u[7]);
}

__device__ void run_rotation(const AttnParams& p, Misc* ms, uint8_t* q_smem, int it0, int it1,
                             int tid) {
  const int lane4 = tid & 3;
  uint32_t nq0 = 0, nq1 = 0;
  for (int it = it0; it < it1; ++it) {
    const AttnItem w = load_item(p.items + it);
    for (int t = 0; t < 2; ++t) {
      if (tile_steps(w, t) == 0) continue;
      const uint32_t k = t ? nq1++ : nq0++;
      const int rows = min(kPfTile, w.rows - t * kPfTile), r0 = tid >> 2;
      const float* at[4];           // this lane's cosines of its four rows
      if (p.rot.cos_sin != nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + 32 * i;
          at[i] = r < rows ? rotation_row(p.rot, static_cast<int64_t>(w.q_row) + t * kPfTile + r,
                                          lane4 == 0 ? p.err : nullptr) + 8 * lane4
                           : p.rot.cos_sin;
        }
      }
      float4 c[2][2], s[2][2];
      auto fetch = [&](int i, int b) {
        const float4* f = reinterpret_cast<const float4*>(at[i]);
        c[b][0] = f[0];
        c[b][1] = f[1];
        s[b][0] = f[kRope / 8];
        s[b][1] = f[kRope / 8 + 1];
      };
      if (p.rot.cos_sin != nullptr) {
        fetch(0, 0);
        fetch(1, 1);
      }
      if (!mbar_wait(smem_u32(&ms->q_full[t]), k & 1, p.err, kErrQPrep)) return;
      if (p.rot.cos_sin != nullptr) {
        uint8_t* base = q_smem + t * kQTileBytes + 2 * kChunkBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + 32 * i;
          if (r < rows) rotate_row(p.rot, base + r * 128, r, lane4, c[i & 1], s[i & 1]);
          if (i < 2) fetch(i + 2, i);
        }
        fence_proxy_async_smem();
      }
      mbar_arrive(smem_u32(&ms->q_ready[t]));
    }
  }
}

// -------------------------------------------------------------- softmax
__device__ void run_softmax(const AttnParams& p, Misc* ms, uint32_t tmem, int it0, int it1, int t,
                            int warp, int lane) {
  const int row = t * kPfTile + warp * 32 + lane;     // of the item
  const uint32_t lanes = static_cast<uint32_t>(warp) << 21;      // TMEM lane 32 warp
  const uint32_t ts = tmem + lanes + kColS + 128 * t, to = tmem + lanes + kColO + 128 * t;
  const uint32_t s_full = smem_u32(&ms->s_full[t]), p_full = smem_u32(&ms->p_full[t]);
  uint32_t ns = 0, no = 0;
  const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
  for (int it = it0; it < it1; ++it) {
    const AttnItem w = load_item(p.items + it);
    const int n = tile_steps(w, t);
    const int limit = min(w.kv_end, w.vis0 + row) - w.kv_begin;  // keys of this range it sees
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < n; ++j) {
      if (!all_waited(mbar_wait(s_full, ns & 1, p.err, kErrSoftmax))) return;
      ++ns;
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, s + 32 * q);
      tmem_wait_ld();
      const int left = limit - j * kPfTile;            // keys of this step that the row sees
      if (__any_sync(0xffffffffu, left < kPfTile)) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          s[i] = i < left ? s[i] : 0xff800000u;
      }
      float a = -INFINITY, b = -INFINITY;
#pragma unroll
      for (int i = 0; i < 128; i += 4) {
        a = max3(a, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        b = max3(b, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
      }
      const float top = fmaxf(a, b) * p.scale_log2;
      // the maximum moves for the whole warp when one of its rows needs it
      if (__any_sync(0xffffffffu, top > m + kLag)) {
        const float nm = fmaxf(m, top);
        const float f = nm == -INFINITY ? 1.0f : ex2(m - nm);
        m = nm;
        l *= f;
        if (j > 0) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float o[16];
            tmem_ld16(to + 16 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            tmem_st16(to + 16 * q, o);
          }
        }
      }
      // a row that has seen no key keeps p = 2^(-inf) = 0
      const float off = m == -INFINITY ? 0.0f : -m;
      const uint64_t off2 = pack_f32x2(off, off);
      uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const uint32_t* v = s + 64 * h + i;
          float x0, x1, x2, x3;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[0]), __uint_as_float(v[1])), scale2,
                                 off2), x0, x1);
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[2]), __uint_as_float(v[3])), scale2,
                                 off2), x2, x3);
          x0 = ex2(x0); x1 = ex2(x1); x2 = ex2(x2); x3 = ex2(x3);
          sum0 = add_f32x2(sum0, pack_f32x2(x0, x1));
          sum1 = add_f32x2(sum1, pack_f32x2(x2, x3));
          const __nv_bfloat162 c = __floats2bfloat162_rn(x0, x1), d = __floats2bfloat162_rn(x2, x3);
          pk[i / 2] = *reinterpret_cast<const uint32_t*>(&c);
          pk[i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&d);
        }
        tmem_st32(ts + 32 * h, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full);
      float u0, u1;
      unpack_f32x2(add_f32x2(sum0, sum1), u0, u1);
      l += u0 + u1;
    }
    if (n > 0) {
      if (!all_waited(mbar_wait(smem_u32(&ms->o_full[t]), no & 1, p.err, kErrDrain))) return;
      ++no;
      tc_fence_after();
    }
    const bool live = row < w.rows, seen = limit > 0;
    // a row that sees no key: zeros (one whose keys all score -inf: 0 / 0)
    const float inv = 1.0f / l;
    const int64_t token = static_cast<int64_t>(w.q_row) + row;
    const int64_t part = static_cast<int64_t>(w.slot) * kPfRows + row;
    const int64_t at = token * p.heads + w.head;
#pragma unroll 2
    for (int q = 0; q < 8; ++q) {
      float o[16];
      __syncwarp();
      if (n > 0) {
        tmem_ld16(to + 16 * q, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = seen ? o[i] * inv : 0.0f;
      if (!live) {
        // past the item's rows: nothing to write
      } else if (w.slot >= 0) {
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i]);
        float* dst = p.part_o + part * kVHead + 16 * q;
        st_global_32(dst, u);
        st_global_32(dst + 8, u + 8);
      } else {
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
          u[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        st_global_32(p.out + at * kVHead + 16 * q, u);
      }
    }
    if (live) {
      const float lse2 = seen ? m + __log2f(l) : -INFINITY;
      if (w.slot >= 0)
        p.part_lse[part] = lse2;
      else if (p.lse != nullptr)
        p.lse[at] = lse2 * kLn2;
    }
    __syncwarp();
    tc_fence_before();
  }
}

__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Misc misc;
  Misc* ms = &misc;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t q_smem = smem_u32(smem), ring = q_smem + kQBytes;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&ms->full[i]), 1);
      mbar_init(smem_u32(&ms->empty[i]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&ms->q_full[t]), 1);
      mbar_init(smem_u32(&ms->q_ready[t]), 128);
      mbar_init(smem_u32(&ms->q_empty[t]), 1);
      mbar_init(smem_u32(&ms->s_full[t]), 1);
      mbar_init(smem_u32(&ms->p_full[t]), 128);
      mbar_init(smem_u32(&ms->o_full[t]), 1);
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
  if (ms->ours) {
    const int it0 = p.cta_indptr[blockIdx.x], it1 = p.cta_indptr[blockIdx.x + 1];
    if (warp < 8) {
      regs_raise<192>();
      run_softmax(p, ms, tmem, it0, it1, warp >> 2, warp & 3, lane);
    } else {
      regs_lower<64>();
      if (warp < 12) {
        run_rotation(p, ms, smem, it0, it1, threadIdx.x - 256);
      } else if (warp == 12) {
        if (lane == 0) run_loads(p, ms, q_smem, ring, it0, it1);
      } else if (warp == 13) {
        run_products(p, ms, q_smem, ring, tmem, uniform(it0), uniform(it1));
        // no product may run on after the CTA has gone
        if (elect_one()) {
          tc_commit(smem_u32(&ms->drain));
          mbar_wait(smem_u32(&ms->drain), 0, p.err, kErrDrain);
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_attn(const AttnParams& p, int num_ctas, cudaStream_t stream) {
  constexpr int bytes = kSmemBytes + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  attn_kernel<<<num_ctas, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
