// prefix.cu -- the attention of a group's queries to their shared prefix: up to
// 128 query rows (8 tokens x 16 heads) against a range of the prefix's rows, one
// pass over the keys with the running maximum and sum of a softmax.
//
// For query rows i and gathered rows k (576 dims, the first 512 the value):
//     s[i,k] = scale q_i . k,  m_i = max_k s[i,k],  p = 2^(s log2 e - m),
//     o_i = sum_k p k[0:512] / sum_k p,  lse_i = m + log2 sum p.
//
// Bound: matrix products, 2 (576 + 512) flops per (row, key).
//
// Two CTAs of a cluster work on one item.  The output of 128 rows alone fills
// the 512 columns of a CTA's tensor memory, so the scores stand in the other
// CTA's.  The even CTA holds the queries (512 dims in tensor memory, 64 in
// shared memory) and streams key tiles through QK^T; eight warps make
// probabilities of its scores and send them to the odd CTA's shared memory (bulk
// copies, 64 keys at a time), with the factors by which the output's rows are to
// be rescaled.  The odd CTA streams value tiles through PV; its eight warps
// rescale the output, rarely, and write it.  The two halves' work is nearly equal: a
// tile of 128 keys takes 36 K steps of N = 128 in the even CTA (2,304 cycles)
// and 16 of N = 256 in the odd one (2,048).
//
// Probabilities are rounded to bf16, the type of the values that they meet; the
// sums that divide the output are of the unrounded ones.  Scores, sums, maxima
// and outputs are fp32.
//
// Roles (352 threads): warps 0-3 and 4-7 of the even CTA hold the softmax, a
// thread per row and half of a tile's keys (both see the tile's maximum, so that
// they keep the same m); of the odd CTA the output's dims 0-255 and 256-511.
// Warp 8 (and in the even CTA warp 10) loads, warp 9 issues the products.
//
// What those single threads do for each piece counts: a wait that is over takes
// 100 cycles, announcing bytes 25, issuing a copy 64.  With a loop over 9 chunks a
// tile that waits for each, a tile took 4,900 cycles.  So key chunks are loaded by
// two warps and waited for by threes, and a wait is looked at before the products
// ahead of it are issued.  A chunk takes 1,800 to 2,500 cycles to come from L2:
// eleven stand in the ring.

#include <cuda_fp16.h>

#include "shared.h"

namespace mla {
namespace {

constexpr int kThreads = 352;
constexpr uint32_t kHalfBytes = 128 * 128;         // 128 rows x 64 bf16 (or 64 keys)
// even CTA: probabilities of either half of a tile on their way, rotated query
// dims, K ring; odd CTA: the probabilities of two tiles received, V ring
constexpr uint32_t kStageAt = 0, kQrAt = 2 * kHalfBytes, kKRingAt = 3 * kHalfBytes;
constexpr int kChunks = kQkDim / 64;               // of a tile: 128 keys x 64 dims
constexpr int kGroup = 3, kGroups = 4;             // chunks waited for together; groups under way
constexpr uint32_t kKSlots = 11;
constexpr uint32_t kPAt = 0, kVRingAt = 4 * kHalfBytes;
constexpr int kVSlots = 5;                         // 64 keys x 256 dims each
constexpr uint32_t kVBytes = 64 * 256 * 2;
constexpr uint32_t kSmemBytes = kVRingAt + kVSlots * kVBytes;
static_assert(kKRingAt + kKSlots * kHalfBytes <= kSmemBytes, "the even CTA's arrays fit");
// even CTA: queries' dims 0-511, then two buffers of scores; odd CTA: the output
constexpr uint32_t kColQ = 0, kColS = 256, kColO = 0;
// A row's maximum is kept until a score exceeds it by a factor of 2^8, and then
// moves by a power of two, so that a byte tells the factor.
constexpr float kLag = 8.0f;

struct Misc {
  uint64_t full[kVSlots], empty[kKSlots];          // rings: even: a group's bytes, a chunk's
                                                   // slot is free; odd: a slot's
  uint64_t q_ready;                                // even: the item's queries are in place
  uint64_t s_full[2], s_empty[2];                  // even: score buffers
  uint64_t p_empty[4];                             // even: P buffers (tile & 1, half) are free
  uint64_t landed[2];                              // even: a half's copy has arrived
  uint64_t sum_full;                               // even: the second half's sums
  uint64_t p_full[4];                              // odd: P buffers and factors
  uint64_t o_ready[2], pv_done;                    // odd: output rescaled (tiles in turn, as the
                                                   // warps may be a tile ahead); a tile's PV through
  uint64_t fin_full[2];                            // odd: 1 / sums of an item
  uint64_t drain;
  uint32_t tmem;
  // of tiles, and of items, in turn; odd CTA: received, even CTA: being sent
  alignas(16) uint8_t factor[4][kSpRows];          // rows are to be scaled by 2^-factor
  alignas(16) float fin[2][kSpRows];               // 1 / sums (even CTA: first the half sums)
};
static_assert(sizeof(Misc) + kSmemBytes + 1024 <= 232448, "fits a CTA's shared memory");

__device__ __forceinline__ PrefixItem load_item(const PrefixItem* p) {
  const int4 a = reinterpret_cast<const int4*>(p)[0], b = reinterpret_cast<const int4*>(p)[1];
  PrefixItem w{};
  w.q_row = a.x; w.rows = a.y; w.key0 = a.z; w.keys = a.w;
  w.slot = b.x; w.check = static_cast<uint32_t>(b.y);
  return w;
}
__device__ __forceinline__ int tiles_of(const PrefixItem& w) {
  return (w.keys + kSpTile - 1) / kSpTile;
}
// About a millisecond, in which every copy under way lands (a wait gave up).
__device__ __forceinline__ void linger() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 1000000) {}
}
__device__ __forceinline__ bool all_waited(bool ok) { return __all_sync(0xffffffffu, ok); }
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(bar));
}
// Copy of this CTA's shared memory to the other's, counted on a barrier there.
__device__ __forceinline__ void bulk_to_peer(uint32_t dst, uint32_t src, uint32_t bytes,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// One arrival on the even CTA's barrier of that name once every product that
// this thread has issued is through.
__device__ __forceinline__ void commit_to_even(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 even;\n\t"
      "mov.b16 even, 1;\n\t"
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], even;\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// ---------------------------------------------------------------- loads
//
// Even CTA: every other group of three chunks, from `first` (0 or 1) on.
__device__ void load_keys(const PrefixParams& p, Misc* ms, uint32_t ring, int it0, int it1, int first) {
  // group of the whole walk, its barrier; the next chunk's slot and, of the slots
  // from it on, the parity of the release to wait for
  uint32_t g = 0, s = 0, parity = 1;
  bool ok = true;
  const uint64_t keep = l2_policy_evict_normal();
  const CUtensorMap* map = &p.map_k;
  fence_proxy_async();               // (the rows were written by another kernel)
  for (int it = it0; it < it1 && ok; ++it) {
    const PrefixItem w = load_item(p.items + it);
    const int tiles = tiles_of(w);
    for (int j = 0; j < tiles && ok; ++j) {
      const int key = w.key0 + j * kSpTile;
      for (int ch = 0; ch < kChunks && ok; ch += kGroup, ++g) {
        if ((g & 1) != static_cast<uint32_t>(first)) {
          s += kGroup;
          if (s >= kKSlots) {
            s -= kKSlots;
            parity ^= 1;
          }
          continue;
        }
        const uint32_t bar = smem_u32(&ms->full[g % kGroups]);
        bool ready = mbar_test(smem_u32(&ms->empty[s]), parity);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          if (!ready && !mbar_wait_poll(smem_u32(&ms->empty[s]), parity, p.err, kErrProducer)) {
            ok = false;
            break;
          }
          if (i == 0) mbar_arrive_expect_tx(bar, kGroup * kHalfBytes);
          const uint32_t at = s;
          if (++s == kKSlots) {
            s = 0;
            parity ^= 1;
          }
          if (i + 1 < kGroup) ready = mbar_test(smem_u32(&ms->empty[s]), parity);
          tma_load_3d(ring + at * kHalfBytes, map, bar, 0, key, ch + i, keep);
        }
      }
    }
  }
  if (!ok) linger();                 // no copy may land after the CTA has gone
}

// Odd CTA: slots of 64 keys and 256 dims.
__device__ void load_values(const PrefixParams& p, Misc* ms, uint32_t ring, int it0, int it1) {
  uint32_t s = 0, parity = 1;        // (of the first lap: nothing to wait for)
  bool ok = true;
  const uint64_t keep = l2_policy_evict_normal();
  const CUtensorMap* map = &p.map_v;
  fence_proxy_async();
  for (int it = it0; it < it1 && ok; ++it) {
    const PrefixItem w = load_item(p.items + it);
    const int tiles = tiles_of(w);
    for (int j = 0; j < tiles && ok; ++j) {
      const int key = w.key0 + j * kSpTile;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!mbar_wait_poll(smem_u32(&ms->empty[s]), parity, p.err, kErrProducer)) {
          ok = false;
          break;
        }
        const uint32_t bar = smem_u32(&ms->full[s]);
        mbar_arrive_expect_tx(bar, kVBytes);
        tma_load_3d(ring + s * kVBytes, map, bar, 0, key + 64 * (u >> 1), 4 * (u & 1), keep);
        if (++s == kVSlots) {
          s = 0;
          parity ^= 1;
        }
      }
    }
  }
  if (!ok) linger();
}

// ------------------------------------------------------------- products
__device__ void run_scores(const PrefixParams& p, Misc* ms, uint32_t smem, uint32_t tmem, int it0,
                           int it1) {
  constexpr uint32_t idesc = make_idesc(1, 1, false, false, 128, 128);
  const uint64_t qd = smem_desc(smem + kQrAt, 16, 1024, kSwizzle128B);
  const uint64_t kd = smem_desc(smem + kKRingAt, 16, 1024, kSwizzle128B);
  uint32_t tile = 0, g = 0, s = 0;
  auto wait = [&](bool ready, uint64_t* bar, uint32_t parity) {
    return all_waited(ready) ||
           all_waited(mbar_wait_poll(smem_u32(bar), parity, p.err, kErrMma));
  };
  auto group_ready = [&](uint32_t g) {
    return mbar_test(smem_u32(&ms->full[g % kGroups]), (g / kGroups) & 1);
  };
  for (int it = it0; it < it1; ++it) {
    const int tiles = uniform(tiles_of(load_item(p.items + it)));
    if (!wait(false, &ms->q_ready, (it - it0) & 1)) return;
    for (int j = 0; j < tiles; ++j, ++tile) {
      const uint32_t b = tile & 1;
      bool ready = group_ready(g);
      if (tile >= 2 && !wait(false, &ms->s_empty[b], ((tile >> 1) - 1) & 1)) return;
      const uint32_t d = tmem + kColS + 128 * b;
#pragma unroll
      for (int u = 0; u < kChunks / kGroup; ++u, ++g) {
        if (!wait(ready, &ms->full[g % kGroups], (g / kGroups) & 1)) return;
        ready = group_ready(g + 1);
        tc_fence_after();
        uint32_t at[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          at[i] = s;
          s = s + 1 == kKSlots ? 0 : s + 1;
        }
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const int ch = kGroup * u + i;
            const uint64_t kb = kd + ((at[i] * kHalfBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (ch < 8)
                umma_f16_ta(d, tmem + kColQ + 32 * ch + 8 * kk, kb + 2 * kk, idesc, (ch | kk) != 0);
              else
                umma_f16(d, qd + 2 * kk, kb + 2 * kk, idesc, 1);
            }
            tc_commit(smem_u32(&ms->empty[at[i]]));
          }
          if (u == kChunks / kGroup - 1) tc_commit(smem_u32(&ms->s_full[b]));
        }
        __syncwarp();
      }
    }
  }
}

constexpr uint32_t kPHalfBytes = kHalfBytes;
constexpr uint32_t kFactorBytes = kSpRows, kFinBytes = kSpRows * 4;

__device__ void run_values(const PrefixParams& p, Misc* ms, uint32_t smem, uint32_t tmem, int it0,
                           int it1) {
  constexpr uint32_t idesc = make_idesc(1, 1, false, true, 128, 256);
  const uint64_t pd = smem_desc(smem + kPAt, 16, 1024, kSwizzle128B);
  const uint64_t vd = smem_desc(smem + kVRingAt, 64 * 128, 1024, kSwizzle128B);
  uint32_t s = 0, lap = 0, tile = 0;
  auto wait = [&](bool ready, uint64_t* bar, uint32_t parity) {
    return all_waited(ready) ||
           all_waited(mbar_wait_poll(smem_u32(bar), parity, p.err, kErrMma));
  };
  for (int it = it0; it < it1; ++it) {
    const int tiles = uniform(tiles_of(load_item(p.items + it)));
    for (int j = 0; j < tiles; ++j, ++tile) {
      const uint32_t turn = (tile >> 1) & 1;
      bool p_ready = mbar_test(smem_u32(&ms->p_full[2 * (tile & 1)]), turn);
      if (!wait(false, &ms->o_ready[tile & 1], turn)) return;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t buf = 2 * (tile & 1) + h;
        bool v_ready = mbar_test(smem_u32(&ms->full[s]), lap);
        if (!wait(p_ready, &ms->p_full[buf], turn)) return;
        // (the next one's bytes, which cannot come before this buffer is given back)
        if (elect_one())
          mbar_arrive_expect_tx(smem_u32(&ms->p_full[buf]), kPHalfBytes + kFactorBytes);
        const uint64_t a = pd + ((buf * kHalfBytes) >> 4);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait(v_ready, &ms->full[s], lap)) return;
          const uint32_t at = s;
          if (++s == kVSlots) {
            s = 0;
            lap ^= 1;
          }
          if (half == 0) v_ready = mbar_test(smem_u32(&ms->full[s]), lap);
          if (half == 1 && h == 0) p_ready = mbar_test(smem_u32(&ms->p_full[buf + 1]), turn);
          tc_fence_after();
          const uint64_t vb = vd + ((at * kVBytes) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16(tmem + kColO + 256 * half, a + 2 * kk, vb + 128 * kk, idesc,
                       (j | h | kk) != 0);
            tc_commit(smem_u32(&ms->empty[at]));
            if (half == 1) commit_to_even(&ms->p_empty[buf]);
            if (half == 1 && h == 1) tc_commit(smem_u32(&ms->pv_done));
          }
          __syncwarp();
        }
      }
    }
  }
}

// -------------------------------------------------------------- softmax
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void st_shared_16(uint32_t at, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// 2^-drop (0 where that is no normal number).
__device__ __forceinline__ float factor_of(uint32_t drop) {
  return drop < 127 ? __uint_as_float((127u - drop) << 23) : 0.0f;
}

// kChunks64 x 64 dims of a query row (zeros past the item's rows) as bf16 pairs,
// all loads in flight together.
template <int kChunks64>
__device__ __forceinline__ void load_query(const PrefixParams& p, int64_t row, bool live, int chunk,
                                           uint32_t* v) {
  if (p.q_fp8) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) +
                                                      row * kQkDim + chunk * 64);
    uint4 x[4 * kChunks64];
#pragma unroll
    for (int i = 0; i < 4 * kChunks64; ++i) x[i] = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4 * kChunks64; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[8 * i + k] = bf16x2_of(f.x, f.y);
      }
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                      row * kQkDim + chunk * 64);
#pragma unroll
    for (int i = 0; i < 8 * kChunks64; ++i) {
      const uint4 x = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
      v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    }
  }
}

__device__ void run_softmax(const PrefixParams& p, Misc* ms, uint32_t smem, uint32_t tmem, int it0,
                            int it1, int h, int warp, int lane) {
  const int row = warp * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>(warp) << 21;      // TMEM lane 32 warp
  const uint32_t tq = tmem + lanes + kColQ, ts = tmem + lanes + kColS;
  const uint32_t stage = smem + kStageAt + h * kHalfBytes, turn = row & 7;
  const uint32_t peer_p = dsmem_addr(smem + kPAt + h * kHalfBytes, 1);
  const uint32_t peer_full = dsmem_addr(smem_u32(&ms->p_full[h]), 1);
  const uint32_t peer_factor = dsmem_addr(smem_u32(ms->factor[h]), 1);
  const bool sender = warp == 0 && lane == 0;
  const float qs = p.q_scale != nullptr ? *p.q_scale : 1.0f;
  const float ks = p.kv_scale != nullptr ? *p.kv_scale : 1.0f;
  const float scale = qs * ks * (kLog2e / 24.0f);
  const uint64_t scale2 = pack_f32x2(scale, scale);
  uint32_t tile = 0;
  // A wait that gave up is kept until the warpgroup's next barrier, where its
  // four warps leave together: none is left alone at one.
  bool ok = true;
  for (int it = it0; it < it1; ++it) {
    const PrefixItem w = load_item(p.items + it);
    const int tiles = tiles_of(w);
    {
      const int64_t q_row = static_cast<int64_t>(w.q_row) + row;
      const bool live = row < w.rows;
      // (the lines of the second step, on their way beside the first one's)
      if (live) {
        const char* line = static_cast<const char*>(p.q) + q_row * kQkDim * (p.q_fp8 ? 1 : 2);
        const int bytes = 64 * (p.q_fp8 ? 1 : 2);
        for (int c = 2; c < 5; ++c)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(line + (c < 4 ? 4 * h + c : 8) * bytes));
      }
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        uint32_t v[64];
        load_query<2>(p, q_row, live, 4 * h + c, v);
        __syncwarp();
        tmem_st32(tq + 128 * h + 32 * c, v);
        tmem_st32(tq + 128 * h + 32 * c + 32, v + 32);
      }
      if (h == 0) {
        uint32_t r[32];
        load_query<1>(p, q_row, live, 8, r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_16(smem + kQrAt + row * 128 + ((i ^ turn) << 4), r[4 * i], r[4 * i + 1],
                       r[4 * i + 2], r[4 * i + 3]);
        fence_proxy_async_smem();
      }
      __syncwarp();
      tmem_wait_st();
      tc_fence_before();
      arrive_warp(&ms->q_ready, lane);
    }
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < tiles; ++j, ++tile) {
      const uint32_t b = tile & 1;
      ok = all_waited(ok && mbar_wait_poll(smem_u32(&ms->s_full[b]), (tile >> 1) & 1, p.err, kErrSoftmax));
      tc_fence_after();
      // the scores of this half, and the maxima of both
      uint32_t s[64], other[32];
      const uint32_t mine = ts + 128 * b + 64 * h, theirs = ts + 128 * b + 64 * (1 - h);
      float tops[4];
      const int left = w.keys - j * kSpTile;             // keys of this tile
      tops[2] = tmem_ld32_max(theirs, other);
      tmem_wait_ld();
      if (left < kSpTile) {
        tops[2] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          tops[2] = fmaxf(tops[2], 64 * (1 - h) + i < left ? __uint_as_float(other[i]) : -INFINITY);
      }
      tops[3] = tmem_ld32_max(theirs + 32, other);
      tops[0] = tmem_ld32_max(mine, s);
      tops[1] = tmem_ld32_max(mine + 32, s + 32);
      tmem_wait_ld();
      tc_fence_before();
      arrive_warp(&ms->s_empty[b], lane);
      if (left < kSpTile) {
        tops[0] = tops[1] = tops[3] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          tops[3] = fmaxf(tops[3],
                          64 * (1 - h) + 32 + i < left ? __uint_as_float(other[i]) : -INFINITY);
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          s[i] = 64 * h + i < left ? s[i] : 0xff800000u;
          tops[0] = fmaxf(tops[0], __uint_as_float(s[i]));
        }
      }
      // The staging buffer is free once its last copy has landed, the odd CTA's once
      // the tile before the last is through PV: looked at here, waited for below.
      const uint32_t buf = 2 * b + h;
      const bool landed =
          tile < 1 || mbar_test_cluster(smem_u32(&ms->landed[h]), (tile - 1) & 1);
      const bool taken =
          tile < 2 || mbar_test_cluster(smem_u32(&ms->p_empty[buf]), ((tile >> 1) - 1) & 1);
      const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * scale;
      uint32_t drop = 0;
      if (top > m + kLag) {
        const float d = ceilf(top - m);                  // (the first tile: infinite)
        drop = d < 200.0f ? static_cast<uint32_t>(d) : 200u;
        m = m == -INFINITY ? top : m + d;
        l *= factor_of(drop);
      }
      // a row that has seen no score above -inf keeps p = 2^(-inf) = 0
      const float off = m == -INFINITY ? 0.0f : -m;
      const uint64_t off2 = pack_f32x2(off, off);
      uint64_t sum0 = 0, sum1 = 0;
      uint32_t pk[32];
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        float x0, x1, x2, x3;
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), scale2,
                               off2), x0, x1);
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])),
                               scale2, off2), x2, x3);
        x0 = ex2(x0); x1 = ex2(x1); x2 = ex2(x2); x3 = ex2(x3);
        sum0 = add_f32x2(sum0, pack_f32x2(x0, x1));
        sum1 = add_f32x2(sum1, pack_f32x2(x2, x3));
        pk[i / 2] = bf16x2_of(x0, x1);
        pk[i / 2 + 1] = bf16x2_of(x2, x3);
      }
      float u0, u1;
      unpack_f32x2(add_f32x2(sum0, sum1), u0, u1);
      l += u0 + u1;
      if (!all_waited(landed))
        ok = ok && all_waited(mbar_wait_cluster(smem_u32(&ms->landed[h]), (tile - 1) & 1, p.err,
                                                kErrSoftmax));
      if (!all_waited(taken))
        ok = ok && all_waited(mbar_wait_cluster(smem_u32(&ms->p_empty[buf]), ((tile >> 1) - 1) & 1,
                                                p.err, kErrSoftmax));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        st_shared_16(stage + row * 128 + ((i ^ turn) << 4), pk[4 * i], pk[4 * i + 1], pk[4 * i + 2],
                     pk[4 * i + 3]);
      ms->factor[buf][row] = static_cast<uint8_t>(drop);
      fence_proxy_async_smem();
      if (named_bar_any(1 + h, 128, !ok)) return;
      if (sender) {
        bulk_to_peer(peer_p + b * 2 * kHalfBytes, stage, kPHalfBytes, peer_full + 16 * b);
        bulk_to_peer(peer_factor + b * 2 * kSpRows, smem_u32(ms->factor[buf]), kFactorBytes,
                     peer_full + 16 * b);
      }
      __syncwarp();
    }
    // Sums of both halves; 1 / sum (times the values' scale) to the odd CTA.  The
    // buffers on both sides are those of the item before the last: its output is
    // written before the last item's PV begins, and that is through here.
    const uint32_t turn_of = (it - it0) & 1;
    if (sender && ok && tile >= 2)
      ok = mbar_wait_cluster<true>(smem_u32(&ms->p_empty[2 * (tile & 1) + h]),
                                   ((tile - 2) >> 1) & 1, p.err, kErrSoftmax);
    if (named_bar_any(1 + h, 128, !ok)) return;
    if (h == 1) {
      ms->fin[turn_of][row] = l;
      arrive_warp(&ms->sum_full, lane);
    } else {
      ok = all_waited(ok && mbar_wait_poll(smem_u32(&ms->sum_full), turn_of, p.err, kErrSoftmax));
      l += ms->fin[turn_of][row];
      if (row < w.rows)
        p.part_lse[static_cast<int64_t>(w.slot) * kSpRows + row] = l == 0.0f ? -INFINITY : m + __log2f(l);
      ms->fin[turn_of][row] = l == 0.0f ? 0.0f : ks / l;
      fence_proxy_async_smem();
      if (named_bar_any(1, 128, !ok)) return;
      if (sender)
        bulk_to_peer(dsmem_addr(smem_u32(ms->fin[turn_of]), 1), smem_u32(ms->fin[turn_of]),
                     kFinBytes, dsmem_addr(smem_u32(&ms->fin_full[turn_of]), 1));
    }
  }
  // what was sent is there before either CTA goes
  if (sender && tile > 0)
    mbar_wait_cluster(smem_u32(&ms->landed[h]), (tile - 1) & 1, p.err, kErrSoftmax);
}

// --------------------------------------------------------------- output
// (false: a wait gave up)
__device__ bool run_output(const PrefixParams& p, Misc* ms, uint32_t tmem, int it0, int it1, int half,
                           int warp, int lane) {
  const int row = warp * 32 + lane;
  const uint32_t to = tmem + (static_cast<uint32_t>(warp) << 21) + kColO + 256 * half;
  uint32_t tile = 0;
  for (int it = it0; it < it1; ++it) {
    const PrefixItem w = load_item(p.items + it);
    const int tiles = tiles_of(w);
    for (int j = 0; j < tiles; ++j, ++tile) {
      const uint32_t buf = 2 * (tile & 1) + half;
      if (!all_waited(mbar_wait_poll(smem_u32(&ms->p_full[buf]), (tile >> 1) & 1, p.err, kErrDrain)))
        return false;
      if (warp == 0 && lane == 0) mbar_arrive_cluster_relaxed(dsmem_addr(smem_u32(&ms->landed[half]), 0));
      const uint32_t drop = ms->factor[buf][row];
      if (j > 0 && __any_sync(0xffffffffu, drop != 0)) {
        const float f = factor_of(drop);
        if (!all_waited(mbar_wait_poll(smem_u32(&ms->pv_done), (tile - 1) & 1, p.err, kErrDrain)))
          return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 16; ++c) {
          float o[16];
          tmem_ld16(to + 16 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] *= f;
          tmem_st16(to + 16 * c, o);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      arrive_warp(&ms->o_ready[tile & 1], lane);
    }
    const uint32_t turn_of = (it - it0) & 1;
    // (P of the last tile came when the tile two before it was through: two
    // phases may be left, of which a wait for the last alone would see neither)
    if (!all_waited((tile < 2 || mbar_wait_poll(smem_u32(&ms->pv_done), tile & 1, p.err, kErrDrain)) &&
                    mbar_wait_poll(smem_u32(&ms->pv_done), (tile - 1) & 1, p.err, kErrDrain)) ||
        !all_waited(mbar_wait_poll(smem_u32(&ms->fin_full[turn_of]), ((it - it0) >> 1) & 1, p.err,
                                   kErrDrain)))
      return false;
    tc_fence_after();
    const float inv = ms->fin[turn_of][row];
    float* dst = p.part_o + (static_cast<int64_t>(w.slot) * kSpRows + row) * kVDim + 256 * half;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t o[64];
      __syncwarp();
      tmem_ld32(to + 64 * c, o);
      tmem_ld32(to + 64 * c + 32, o + 32);
      tmem_wait_ld();
      if (row < w.rows) {
#pragma unroll
        for (int i = 0; i < 64; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
#pragma unroll
        for (int i = 0; i < 8; ++i) st_global_32(dst + 64 * c + 8 * i, o + 8 * i);
      }
    }
    tc_fence_before();
    // the odd CTA's thread re-arms the buffer for the item after the next
    if (half == 0 && row == 0) mbar_arrive_expect_tx(smem_u32(&ms->fin_full[turn_of]), kFinBytes);
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    prefix_kernel(const __grid_constant__ PrefixParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) Misc misc;
  Misc* ms = &misc;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kVSlots; ++i) mbar_init(smem_u32(&ms->full[i]), 1);
    for (uint32_t i = 0; i < kKSlots; ++i) mbar_init(smem_u32(&ms->empty[i]), 1);
    mbar_init(smem_u32(&ms->q_ready), 8);
    mbar_init(smem_u32(&ms->sum_full), 4);
    mbar_init(smem_u32(&ms->pv_done), 1);
    mbar_init(smem_u32(&ms->drain), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ms->s_full[i]), 1);
      mbar_init(smem_u32(&ms->s_empty[i]), 8);
      mbar_init(smem_u32(&ms->landed[i]), 1);
      mbar_init(smem_u32(&ms->o_ready[i]), 8);
      for (int b = i; b < 4; b += 2) {
        mbar_init(smem_u32(&ms->p_empty[b]), 1);
        mbar_init(smem_u32(&ms->p_full[b]), 1);
      }
      mbar_init(smem_u32(&ms->fin_full[i]), 1);
    }
    fence_mbar_init();
    if (rank == 1) {
      for (int b = 0; b < 4; ++b)
        mbar_arrive_expect_tx(smem_u32(&ms->p_full[b]), kPHalfBytes + kFactorBytes);
      mbar_arrive_expect_tx(smem_u32(&ms->fin_full[0]), kFinBytes);
      mbar_arrive_expect_tx(smem_u32(&ms->fin_full[1]), kFinBytes);
    }
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&ms->tmem), 512);
    tmem_relinquish();
  }
  // the pair's items, all checked before the first is taken up (both CTAs check
  // the same ones)
  const int4 mine = reinterpret_cast<const int4*>(p.pairs)[blockIdx.x / 2];
  bool sound = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp &&
               check_of(CtaItems{mine.x, mine.y, 0u, 0}, p.stamp) == static_cast<uint32_t>(mine.z);
  const int it0 = sound ? mine.x : 0;
  for (int it = it0 + static_cast<int>(threadIdx.x); sound && it < mine.y; it += kThreads) {
    const PrefixItem w = load_item(p.items + it);
    sound = check_of(w, p.stamp) == w.check;
  }
  sound = __syncthreads_and(sound);
  if (!sound && threadIdx.x == 0) atomicOr(p.err, kErrStale);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                    // the other CTA's barriers are set up too
  tc_fence_after();
  const uint32_t tmem = uniform(ms->tmem);
  const int first = uniform(it0), last = uniform(sound ? mine.y : it0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp < 8) {
    if (rank == 0) {
      run_softmax(p, ms, smem, tmem, first, last, warp >> 2, warp & 3, lane);
    } else if (!run_output(p, ms, tmem, first, last, warp >> 2, warp & 3, lane)) {
      linger();                      // copies on their way land before this CTA goes
    }
  } else if (warp == 8) {
    if (lane == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");      // the gathered rows are there
      if (rank == 0)
        load_keys(p, ms, smem + kKRingAt, first, last, 0);
      else
        load_values(p, ms, smem + kVRingAt, first, last);
    }
  } else if (warp == 10) {
    if (lane == 0 && rank == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      load_keys(p, ms, smem + kKRingAt, first, last, 1);
    }
  } else {
    if (rank == 0)
      run_scores(p, ms, smem, tmem, first, last);
    else
      run_values(p, ms, smem, tmem, first, last);
    // no product may run on after the CTAs have gone
    if (elect_one()) {
      tc_commit(smem_u32(&ms->drain));
      mbar_wait_poll(smem_u32(&ms->drain), 0, p.err, kErrDrain);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();                    // nothing of the pair is under way any more
  if (warp == 9) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, int num_pairs, cudaStream_t stream) {
  constexpr int bytes = kSmemBytes + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * num_pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_kernel, p);
}

}  // namespace mla
