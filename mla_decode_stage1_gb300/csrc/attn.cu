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
// On its own a CTA reads 8 KB of operands for each 64-cycle product of the
// scores, all that its shared memory gives, and takes in its keys beside that:
// a step takes about 3,700 cycles where the products need 2,560.  Two CTAs as a
// pair (one product of M = 256, half of each key and value tile in either)
// take 2,790: 8192 tokens, 16 heads, causal: 210 us on single CTAs, 196 us in
// pairs (1.75 PFLOP/s, tensor pipe 79 % busy; what is left is 3 items a CTA
// filling and draining, 5 % each).  Against many keys and few rows HBM bounds
// it: 77 rows, 32,845 keys: 57 us for 274 MB (4.8 TB/s).
//
// Probabilities are rounded to the type of the values that they meet, fp16 or
// bf16 by groups of 32 keys (expand.cu); each 16-key product is of that type.
// (bf16 alone: 1 % faster in pairs and 5 % on single CTAs, but an error of the
// output of 0.0026 to 0.0031 instead of 0.0021 to 0.0023, 0.0017 of it the
// rounding of the output.)
// Sums, maxima and O are fp32.
//
// Roles (384 threads): warps 0-3 and 4-7 hold the softmax of tile 0 and 1, a
// thread per row; warp 8 loads (TMA), warp 9 issues the products (warps 10 and
// 11 only hold up the third warpgroup, whose registers the softmax takes).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "prefill.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kChunkBytes = 128 * 128;        // 128 rows x 64 bf16
constexpr uint32_t kQTileBytes = 3 * kChunkBytes;
constexpr uint32_t kQBytes = 2 * kQTileBytes;
constexpr uint32_t kRingBytes = 8 * kChunkBytes;
constexpr uint32_t kSmemBytes = kQBytes + kRingBytes;

// A CTA on its own, or a pair that shares every key and value tile.  Query
// tile t of an item is kTileRows<P> rows, 128 in each CTA.
//
// The ring hands out units.  On its own, a CTA's unit is a chunk of 16 KB: a K
// tile takes three (64 dims each), a V tile two (64 keys each), so that 128 KB
// hold 1.6 tiles.  In a pair a CTA holds keys 64 rank .. of a K tile and dims
// 64 rank .. of a V tile; a unit is such a half tile, in one of three stages
// of 24 KB (K) or 16 KB (V): fewer barriers a step, and three tiles deep.
template <bool P>
constexpr int kTileRows = P ? 256 : 128;
constexpr int kSlots = 8;                          // units of a CTA on its own
constexpr int kStages = 3;
constexpr uint32_t kPieceBytes = 64 * 128;         // 64 rows x 64 bf16
constexpr uint32_t kVStages = kStages * 3 * kPieceBytes;      // V stages stand behind K's
constexpr uint32_t kColS = 0, kColO = 256;         // tile t: + 128 t
// A row's maximum is kept until a score exceeds it by a factor of 2^8, so that
// rescaling O is rare.  Probabilities are 2^7 times their value against that
// maximum: at most 2^15 in fp16's 2^16, and down to 2^-21 of the largest with
// all of fp16's bits, 2^-31 as its smallest (a first token with nearly all of
// the weight and a small value leaves the output to such keys).
constexpr float kLag = 8.0f, kLift = 7.0f;

struct Misc {
  uint64_t full[kSlots], empty[kSlots];            // units (a pair: K stages, then V stages)
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem;
  uint32_t ours;
  int32_t expanded;
};

// What query tile t of an item works on: rows from `first` of the item on,
// keys [begin, end).
struct Stream {
  int first, begin, end, slot;
};
template <bool P>
__device__ __forceinline__ Stream stream_of(const AttnItem& w, int t) {
  if (!P && halved(w)) {
    const int mid = middle_key(w);
    return Stream{0, t ? mid : w.kv_begin, t ? w.kv_end : mid, w.slot + t};
  }
  return Stream{t * kTileRows<P>, w.kv_begin, w.kv_end, w.slot};
}

// Key steps of query tile t: those with a key that the tile's last row sees.
template <bool P>
__device__ __forceinline__ int tile_steps(const AttnItem& w, int t) {
  const Stream s = stream_of<P>(w, t);
  if (w.rows <= s.first) return 0;
  const int last = min(w.rows, s.first + kTileRows<P>) - 1;
  const int end = min(s.end, w.vis0 + last);
  return end > s.begin ? (end - s.begin + kPfTile - 1) / kPfTile : 0;
}

__device__ __forceinline__ AttnItem load_item(const AttnItem* p) {
  const int4 a = reinterpret_cast<const int4*>(p)[0], b = reinterpret_cast<const int4*>(p)[1];
  return AttnItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Types of the values of key step j of a query tile: a byte per 32 keys, 1 = fp16.
__device__ __forceinline__ uint32_t value_types(const AttnParams& p, const AttnItem& w,
                                                const Stream& s, int j) {
  return __ldcg(reinterpret_cast<const uint32_t*>(
      p.v_half + (w.head * p.kx_rows + w.kv_row + s.begin + j * kPfTile) / kPfGroup));
}
constexpr uint32_t kAllHalf = 0x01010101u;

// A wait of the whole warp, which goes on (or gives up) together.
__device__ __forceinline__ bool all_waited(bool ok) { return __all_sync(0xffffffffu, ok); }

// Barriers that the issuing CTA waits on: its own, or the even CTA's of a pair.
template <bool P>
__device__ __forceinline__ uint32_t issuer_bar(uint64_t* bar) {
  return P ? dsmem_addr(smem_u32(bar), 0) : smem_u32(bar);
}
// One arrival of the (converged) warp on tensor memory that it wrote.
template <bool P>
__device__ __forceinline__ void arrive_at_issuer(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane != 0) return;
  if constexpr (P)
    mbar_arrive_cluster_relaxed(issuer_bar<P>(bar));
  else
    mbar_arrive(smem_u32(bar));
}
template <bool P>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (P)
    tc_commit_pair(smem_u32(bar));
  else
    tc_commit(smem_u32(bar));
}

// ---------------------------------------------------------------- loads
template <bool P>
__device__ void run_loads(const AttnParams& p, Misc* ms, uint32_t q_smem, uint32_t ring, int it0,
                          int it1, int rank) {
  uint32_t n = 0;                   // chunks opened (a pair: K tiles; its V tiles: nv)
  uint32_t nv = 0;
  uint32_t nq0 = 0, nq1 = 0;        // query tiles loaded of either kind
  bool ok = true;
  const uint64_t keep = l2_policy_evict_normal();
  fence_proxy_async();              // (behind the expansion, if word was left of it)
  // unit `s` is free in its lap; its bytes are announced (a pair's on the even
  // CTA, for both)
  auto open = [&](uint32_t s, uint32_t lap, uint32_t bytes) {
    if (lap > 0 && !mbar_wait_poll(smem_u32(&ms->empty[s]), (lap - 1) & 1, p.err, kErrProducer))
      ok = false;
    else if (rank == 0)
      mbar_arrive_expect_tx(smem_u32(&ms->full[s]), bytes);
    return ok;
  };
  auto load = [&](uint32_t dst, uint64_t* bar, const CUtensorMap* map, int x, int y, int z) {
    if constexpr (P)
      tma_load_3d_pair(dst, map, issuer_bar<P>(bar), x, y, z, keep);
    else
      tma_load_3d(dst, map, smem_u32(bar), x, y, z, keep);
  };
  // K and V tiles whose first key stands in workspace row `key`
  auto load_k = [&](const AttnItem& w, int key) {
    const int row = key + 64 * rank;
    if constexpr (P) {
      const uint32_t s = n % kStages;
      if (!open(s, n / kStages, 2 * 3 * kPieceBytes)) return;
      ++n;
      const uint32_t dst = ring + s * 3 * kPieceBytes;
      for (int ch = 0; ch < 3; ++ch)
        load(dst + ch * kPieceBytes, &ms->full[s], ch < 2 ? &p.map_kx : &p.map_kr,
             ch < 2 ? ch * 64 : 0, row, ch < 2 ? w.head : 0);
    } else {
#pragma unroll 1
      for (int ch = 0; ch < 3; ++ch) {
        const uint32_t s = n % kSlots;
        if (!open(s, n / kSlots, kChunkBytes)) return;
        ++n;
        for (int i = 0; i < 2; ++i)
          load(ring + s * kChunkBytes + i * kPieceBytes, &ms->full[s],
               ch < 2 ? &p.map_kx : &p.map_kr, ch < 2 ? ch * 64 : 0, row + 64 * i,
               ch < 2 ? w.head : 0);
      }
    }
  };
  auto load_v = [&](const AttnItem& w, int row) {
    if constexpr (P) {
      const uint32_t s = nv % kStages;
      if (!open(kStages + s, nv / kStages, 2 * 2 * kPieceBytes)) return;
      ++nv;
      const uint32_t dst = ring + kVStages + s * 2 * kPieceBytes;
      for (int half = 0; half < 2; ++half)
        load(dst + half * kPieceBytes, &ms->full[kStages + s], &p.map_kx, kNope + 64 * rank,
             row + half * 64, w.head);
    } else {
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const uint32_t s = n % kSlots;
        if (!open(s, n / kSlots, kChunkBytes)) return;
        ++n;
        for (int i = 0; i < 2; ++i)
          load(ring + s * kChunkBytes + i * kPieceBytes, &ms->full[s], &p.map_kx, kNope + 64 * i,
               row + half * 64, w.head);
      }
    }
  };
  // (the next item's description is loaded one item ahead, here and below)
  AttnItem next = load_item(p.items + it0);
  for (int it = it0; it < it1 && ok; ++it) {
    const AttnItem w = next;
    if (it + 1 < it1) next = load_item(p.items + it + 1);
    const int n0 = tile_steps<P>(w, 0), n1 = tile_steps<P>(w, 1), steps = max(n0, n1);
    if (steps == 0) continue;
    const bool two = !P && halved(w);      // each query tile has keys of its own
    const Stream s0 = stream_of<P>(w, 0), s1 = stream_of<P>(w, 1);
    const int key0 = w.kv_row + s0.begin, key1 = w.kv_row + s1.begin;
    if (!two || n0 > 0) load_k(w, key0);
    if (!ok) break;
    for (int t = 0; t < 2 && ok; ++t) {
      if ((t ? n1 : n0) == 0) continue;
      if (two && t == 1) load_k(w, key1);
      const uint32_t k = t ? nq1 : nq0;
      if (!ok || (k > 0 && !mbar_wait_poll(smem_u32(&ms->q_empty[t]), (k - 1) & 1, p.err,
                                           kErrProducer))) {
        ok = false;
        break;
      }
      ++(t ? nq1 : nq0);
      if (rank == 0)
        mbar_arrive_expect_tx(smem_u32(&ms->q_full[t]), (P ? 2 : 1) * kQTileBytes);
      for (int ch = 0; ch < 3; ++ch)
        load(q_smem + t * kQTileBytes + ch * kChunkBytes, &ms->q_full[t],
             ch < 2 ? &p.map_q : &p.map_qr, ch < 2 ? ch * 64 : p.qr_x, w.head,
             w.q_row + (t ? s1.first : s0.first) + rank * kPfTile);
    }
    for (int j = 0; j < steps && ok; ++j) {
      if (!two) {
        load_v(w, key0 + j * kPfTile);
        if (ok && j + 1 < steps) load_k(w, key0 + (j + 1) * kPfTile);
      } else {
        if (j < n0) load_v(w, key0 + j * kPfTile);
        if (ok && j + 1 < n0) load_k(w, key0 + (j + 1) * kPfTile);
        if (ok && j < n1) load_v(w, key1 + j * kPfTile);
        if (ok && j + 1 < n1) load_k(w, key1 + (j + 1) * kPfTile);
      }
    }
  }
  if (!ok && rank == 0) {
    // a wait gave up: no copy may land after the CTA has gone (a pair's copies
    // are counted on the even CTA, and both leave together)
    auto landed = [&](uint64_t* bars, uint32_t count, uint32_t units) {
      for (uint32_t k = count > units ? count - units : 0; k < count; ++k)
        mbar_wait_poll(smem_u32(&bars[k % units]), (k / units) & 1, p.err, kErrProducer);
    };
    landed(ms->full, n, P ? kStages : kSlots);
    landed(ms->full + kStages, nv, kStages);
    landed(&ms->q_full[0], nq0, 1);
    landed(&ms->q_full[1], nq1, 1);
  }
}

// ------------------------------------------------------------- products
// The whole warp walks the steps; one lane issues (of the even CTA, for a pair).
template <bool P>
__device__ void run_products(const AttnParams& p, Misc* ms, uint32_t q_smem, uint32_t ring,
                             uint32_t tmem, int it0, int it1) {
  constexpr uint32_t idesc_qk = make_idesc(1, 1, false, false, kTileRows<P>, 128);
  constexpr uint32_t idesc_pv = make_idesc(1, 1, false, true, kTileRows<P>, 128);
  constexpr uint32_t idesc_pv_half = make_idesc(0, 0, false, true, kTileRows<P>, 128);
  uint32_t n = 0;                   // chunks consumed (a pair: K tiles; its V tiles: nv)
  uint32_t nv = 0;
  uint32_t nq0 = 0, nq1 = 0;        // query tiles used of either kind
  uint32_t np0 = 0, np1 = 0;        // P tiles consumed of query tile 0, 1
  const uint64_t qd = smem_desc(q_smem, 16, 1024, kSwizzle128B);
  const uint64_t kd = smem_desc(ring, 16, 1024, kSwizzle128B);
  const uint64_t vd = smem_desc(ring, kPieceBytes, 1024, kSwizzle128B);
  // A wait that is ready costs its latency all the same (about 80 cycles, twice
  // that under load), so each is looked at (`peek`) before the products ahead
  // of it are issued, and waited for only if it was not ready by then.  Bytes
  // of copies, and arrivals of threads (of both CTAs).
  auto peek = [&](uint64_t* bar, uint32_t parity) { return mbar_test(smem_u32(bar), parity); };
  auto peek_threads = [&](uint64_t* bar, uint32_t parity) {
    return P ? mbar_test_cluster(smem_u32(bar), parity) : mbar_test(smem_u32(bar), parity);
  };
  auto wait = [&](bool ready, uint64_t* bar, uint32_t parity) {
    return all_waited(ready) ||
           all_waited(mbar_wait_poll(smem_u32(bar), parity, p.err, kErrMma));
  };
  auto wait_threads = [&](bool ready, uint64_t* bar, uint32_t parity) {
    return all_waited(ready) ||
           all_waited(P ? mbar_wait_cluster(smem_u32(bar), parity, p.err, kErrMma)
                        : mbar_wait_poll(smem_u32(bar), parity, p.err, kErrMma));
  };
  // barrier of chunk (or stage) k of K, and of V
  auto k_bar = [&](uint32_t k) { return &ms->full[P ? k % kStages : k % kSlots]; };
  auto v_bar = [&](uint32_t k) { return &ms->full[P ? kStages + k % kStages : k % kSlots]; };
  auto lap = [&](uint32_t k) { return (P ? k / kStages : k / kSlots) & 1; };
  // S_t = Q_t K^T with the K tile from unit k on; `fresh`: not waited for
  // yet (`ready`: its first unit was seen); `last`: this query tile's last
  // step of the item
  auto qk = [&](int t, uint32_t k, bool fresh, bool ready, bool last) {
#pragma unroll
    for (int ch = 0; ch < 3; ++ch) {
      if (fresh && (ch == 0 || !P)) {
        if (!wait(ch == 0 && ready, k_bar(k + ch), lap(k + ch))) return false;
        tc_fence_after();
      }
      const uint32_t at = P ? (k % kStages) * 3 * kPieceBytes + ch * kPieceBytes
                            : ((k + ch) % kSlots) * kChunkBytes;
      const uint64_t a = qd + ((t * kQTileBytes + ch * kChunkBytes) >> 4);
      const uint64_t b = kd + (at >> 4);
      const uint32_t d = tmem + kColS + 128 * t;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if constexpr (P)
            umma_f16_pair(d, a + 2 * kk, b + 2 * kk, idesc_qk, (ch | kk) != 0);
          else
            umma_f16(d, a + 2 * kk, b + 2 * kk, idesc_qk, (ch | kk) != 0);
        }
      }
    }
    if (elect_one()) {
      commit<P>(&ms->s_full[t]);
      if (last) commit<P>(&ms->q_empty[t]);
    }
    return true;
  };
  // O_t (+)= P_t V with the V tile from unit k on, a half of 64 keys as soon as
  // its probabilities are there; looks at K's barrier k_next on the way
  auto pv = [&](int t, uint32_t k, uint32_t types, uint32_t parity, bool fresh, bool ready,
                bool first, uint32_t k_next, bool* k_ready) {
    bool p_ready = false;
    // Descriptors as uniform data.  (A branch to constant ones where all keys'
    // values are fp16 cost 2.5 % of the long prompt's kernel with its test up
    // here, 5 % with a test at each half.)
    const uint32_t idesc0 = uniform(types & 0x1 ? idesc_pv_half : idesc_pv);
    const uint32_t idesc1 = uniform(types & 0x100 ? idesc_pv_half : idesc_pv);
    const uint32_t idesc2 = uniform(types & 0x10000 ? idesc_pv_half : idesc_pv);
    const uint32_t idesc3 = uniform(types & 0x1000000 ? idesc_pv_half : idesc_pv);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (fresh && (half == 0 || !P))
        if (!wait(half == 0 && ready, v_bar(k + half), lap(k + half))) return false;
      if (!wait_threads(p_ready, half == 0 ? &ms->p_half[t] : &ms->p_full[t], parity))
        return false;
      if (half == 0)
        p_ready = peek_threads(&ms->p_full[t], parity);
      else
        *k_ready = peek(k_bar(k_next), lap(k_next));
      tc_fence_after();
      const uint32_t at = P ? kVStages + (k % kStages) * 2 * kPieceBytes + half * kPieceBytes
                            : ((k + half) % kSlots) * kChunkBytes;
      const uint64_t b = vd + (at >> 4);
      const uint32_t d = tmem + kColO + 128 * t, a = tmem + kColS + 128 * t + 32 * half;
      const uint32_t first_pair = half ? idesc2 : idesc0, second_pair = half ? idesc3 : idesc1;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const bool add = !(first && half == 0 && kk == 0);
          const uint32_t idesc = kk < 2 ? first_pair : second_pair;
          if constexpr (P)
            umma_f16_ta_pair(d, a + 8 * kk, b + 128 * kk, idesc, add);
          else
            umma_f16_ta(d, a + 8 * kk, b + 128 * kk, idesc, add);
        }
      }
    }
    return true;
  };
  // the K (V) tile from unit k on is free once everything issued so far is through
  auto release_k = [&](uint32_t k) {
    if (elect_one()) {
      if constexpr (P)
        commit<P>(&ms->empty[k % kStages]);
      else
        for (int i = 0; i < 3; ++i) commit<P>(&ms->empty[(k + i) % kSlots]);
    }
  };
  auto release_v = [&](uint32_t k) {
    if (elect_one()) {
      if constexpr (P)
        commit<P>(&ms->empty[kStages + k % kStages]);
      else
        for (int i = 0; i < 2; ++i) commit<P>(&ms->empty[(k + i) % kSlots]);
    }
  };
  AttnItem next = load_item(p.items + it0);
  bool begun = false;               // the item's first scores of tile 0 are issued
  for (int it = it0; it < it1; ++it) {
    const AttnItem w = next;
    if (it + 1 < it1) next = load_item(p.items + it + 1);
    const int n0 = uniform(tile_steps<P>(w, 0)), n1 = uniform(tile_steps<P>(w, 1));
    const int steps = max(n0, n1);
    if (steps == 0) continue;
    // types of the values, a step ahead (of either tile's keys)
    const Stream s0 = stream_of<P>(w, 0), s1 = stream_of<P>(w, 1);
    uint32_t types0 = n0 > 0 ? value_types(p, w, s0, 0) : 0;
    uint32_t types1 = n1 > 0 ? value_types(p, w, s1, 0) : 0;
    auto next_types = [&](const Stream& s, int j, int steps_of) {
      return j + 1 < steps_of ? value_types(p, w, s, j + 1) : 0u;
    };
    if constexpr (!P) if (halved(w)) {
      // the query tiles have keys of their own, in turn
      for (int t = 0; t < 2; ++t) {
        const int nt = t ? n1 : n0;
        if (nt == 0) continue;
        if (!wait(false, &ms->q_full[t], (t ? nq1++ : nq0++) & 1)) return;
        tc_fence_after();
        if (!qk(t, n, true, false, nt == 1)) return;
        release_k(n);
        n += 3;
      }
      for (int j = 0; j < steps; ++j)
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          const int nt = t ? n1 : n0;
          if (j >= nt) continue;
          bool k_ready = false;
          const uint32_t types = uniform(t ? types1 : types0);
          if (t) types1 = next_types(s1, j, nt); else types0 = next_types(s0, j, nt);
          if (!pv(t, n, types, (t ? np1++ : np0++) & 1, true, false, j == 0, n + 2, &k_ready))
            return;
          if (j + 1 == nt && elect_one()) commit<P>(&ms->o_full[t]);
          release_v(n);
          n += 2;
          if (j + 1 < nt) {
            if (!qk(t, n, true, k_ready, j + 2 == nt)) return;
            release_k(n);
            n += 3;
          }
        }
      continue;
    }
    if (n0 > 0 && !begun) {
      if (!wait(false, &ms->q_full[0], nq0++ & 1)) return;
      tc_fence_after();
      if (!qk(0, n, true, false, n0 == 1)) return;
    }
    begun = false;
    if (n1 > 0) {
      if (!wait(false, &ms->q_full[1], nq1++ & 1)) return;
      tc_fence_after();
      if (!qk(1, n, n0 == 0, false, n1 == 1)) return;
    }
    release_k(n);
    n += P ? 1 : 3;
    for (int j = 0; j < steps; ++j) {
      const uint32_t v = P ? nv : n, k = P ? n : n + 2;
      bool fresh_v = true, fresh_k = true, k_ready = false;
      const bool v_ready = peek(v_bar(v), lap(v));
      // (the tiles share their keys)
      const uint32_t types = uniform(n1 > j ? types1 : types0);
      types0 = next_types(s0, j, n0);
      types1 = next_types(s1, j, n1);
      if (j < n0) {
        if (!pv(0, v, types, np0++ & 1, true, v_ready, j == 0, k, &k_ready)) return;
        fresh_v = false;
        if (j + 1 == n0 && elect_one()) commit<P>(&ms->o_full[0]);
        if (j + 1 < n0) {
          if (!qk(0, k, true, k_ready, j + 2 == n0)) return;
          fresh_k = false;
        }
      }
      // The next item's first scores of tile 0, if its query is there, ahead of
      // this item's last values: its softmax has them when it is through with
      // this item's output.  (8192 tokens: 198.6 -> 196.6 us; on single CTAs a
      // ragged batch lost by it, 102.3 -> 105.4 us.)
      if (P && j + 1 == steps && it + 1 < it1) {
        const int next0 = uniform(tile_steps<P>(next, 0));
        if (next0 > 0 && all_waited(peek(&ms->q_full[0], nq0 & 1))) {
          ++nq0;
          tc_fence_after();
          if (!qk(0, k, true, false, next0 == 1)) return;
          begun = true;
        }
      }
      if (j < n1) {
        if (!pv(1, v, types, np1++ & 1, fresh_v, v_ready, j == 0, k, &k_ready)) return;
        if (j + 1 == n1 && elect_one()) commit<P>(&ms->o_full[1]);
      }
      // the values are free before the next scores are through
      release_v(v);
      if constexpr (P) ++nv; else n += 2;
      if (j + 1 < steps) {
        if (j + 1 < n1 && !qk(1, k, fresh_k, k_ready, j + 2 == n1)) return;
        release_k(k);
        n += P ? 1 : 3;
      }
    }
  }
}

// -------------------------------------------------------------- softmax
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool P>
__device__ void run_softmax(const AttnParams& p, Misc* ms, uint32_t tmem, int it0, int it1,
                            int rank, int t, int warp, int lane) {
  const uint32_t lanes = static_cast<uint32_t>(warp) << 21;      // TMEM lane 32 warp
  const uint32_t ts = tmem + lanes + kColS + 128 * t, to = tmem + lanes + kColO + 128 * t;
  const uint32_t s_full = smem_u32(&ms->s_full[t]);
  uint32_t ns = 0, no = 0;
  const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
  AttnItem next = load_item(p.items + it0);
  for (int it = it0; it < it1; ++it) {
    const AttnItem w = next;
    if (it + 1 < it1) next = load_item(p.items + it + 1);
    const Stream st = stream_of<P>(w, t);
    const int n = tile_steps<P>(w, t);
    const int row = st.first + rank * kPfTile + warp * 32 + lane;     // of the item
    const int limit = min(st.end, w.vis0 + row) - st.begin;           // keys of this range it sees
    float m = -INFINITY, l = 0.0f;
    uint32_t next_types = n > 0 ? value_types(p, w, st, 0) : 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t types = next_types;
      if (j + 1 < n) next_types = value_types(p, w, st, j + 1);
      if (!all_waited(mbar_wait_poll(s_full, ns & 1, p.err, kErrSoftmax))) return;
      ++ns;
      tc_fence_after();
      // the scores, and with them (from the load itself) their maximum
      uint32_t s[128];
      float tops[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) tops[q] = tmem_ld32_max(ts + 32 * q, s + 32 * q);
      tmem_wait_ld();
      const int left = limit - j * kPfTile;            // keys of this step that the row sees
      if (__any_sync(0xffffffffu, left < kPfTile)) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          s[i] = i < left ? s[i] : 0xff800000u;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tops[q] = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            tops[q] = max3(tops[q], __uint_as_float(s[32 * q + i]),
                           __uint_as_float(s[32 * q + i + 1]));
        }
      }
      // Probabilities of 64 keys with the maximum so far, their sum, and pairs
      // in the values' types.
      uint64_t sum0 = 0, sum1 = 0;
      uint32_t pk[32];
      auto exponents = [&](const uint32_t* v, auto all_half, uint32_t bits) {
        // a row that has seen no key keeps p = 2^(-inf) = 0
        const float off = m == -INFINITY ? 0.0f : kLift - m;
        const uint64_t off2 = pack_f32x2(off, off);
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          float x0, x1, x2, x3;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])),
                                 scale2, off2), x0, x1);
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])),
                                 scale2, off2), x2, x3);
          x0 = ex2(x0); x1 = ex2(x1); x2 = ex2(x2); x3 = ex2(x3);
          sum0 = add_f32x2(sum0, pack_f32x2(x0, x1));
          sum1 = add_f32x2(sum1, pack_f32x2(x2, x3));
          if (decltype(all_half)::value || ((bits >> (8 * (i / 32))) & 1)) {
            pk[i / 2] = half2_of(x0, x1);
            pk[i / 2 + 1] = half2_of(x2, x3);
          } else {
            pk[i / 2] = bf16x2_of(x0, x1);
            pk[i / 2 + 1] = bf16x2_of(x2, x3);
          }
        }
      };
      auto hand_over = [&](int half) {
        tmem_st32(ts + 32 * half, pk);
        tmem_wait_st();
        tc_fence_before();
        arrive_at_issuer<P>(half == 0 ? &ms->p_half[t] : &ms->p_full[t], lane);
      };
      const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * p.scale_log2;
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
      auto probabilities = [&](auto all_half) {
        exponents(s, all_half, types);
        hand_over(0);
        exponents(s + 64, all_half, types >> 16);
        hand_over(1);
      };
      if (__all_sync(0xffffffffu, types == kAllHalf))
        probabilities(std::true_type());
      else
        probabilities(std::false_type());
      float u0, u1;
      unpack_f32x2(add_f32x2(sum0, sum1), u0, u1);
      l += u0 + u1;
    }
    if (n > 0) {
      if (!all_waited(mbar_wait_poll(smem_u32(&ms->o_full[t]), no & 1, p.err, kErrDrain))) return;
      ++no;
      tc_fence_after();
    }
    const bool live = row < w.rows, seen = limit > 0;
    // a row that sees no key: zeros (one whose keys all score -inf: 0 / 0)
    const float inv = 1.0f / l;
    const int64_t token = static_cast<int64_t>(w.q_row) + row;
    const int64_t part = static_cast<int64_t>(st.slot) * kPfRows + row;
    const int64_t at = token * p.heads + w.head;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      uint32_t o[64];
      __syncwarp();
      tmem_ld32(to + 64 * half, o);              // (of an item without steps: not used)
      tmem_ld32(to + 64 * half + 32, o + 32);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 64; ++i)
        o[i] = seen ? __float_as_uint(__uint_as_float(o[i]) * inv) : 0u;
      if (!live) {
        // past the item's rows: nothing to write
      } else if (w.slot >= 0) {
        float* dst = p.part_o + part * kVHead + 64 * half;
#pragma unroll
        for (int q = 0; q < 8; ++q) st_global_32(dst + 8 * q, o + 8 * q);
      } else {
        uint16_t* dst = p.out + at * kVHead + 64 * half;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[16 * q + 2 * i]),
                                                           __uint_as_float(o[16 * q + 2 * i + 1]));
            u[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          st_global_32(dst + 16 * q, u);
        }
      }
    }
    tc_fence_before();
    if (live) {
      const float lse2 = seen ? m - kLift + __log2f(l) : -INFINITY;
      if (w.slot >= 0)
        p.part_lse[part] = lse2;
      else if (p.lse != nullptr)
        p.lse[at] = lse2 * kLn2;
    }
    __syncwarp();
  }
}

template <bool P>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Misc misc;
  Misc* ms = &misc;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t q_smem = smem_u32(smem), ring = q_smem + kQBytes;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = P ? static_cast<int>(cluster_ctarank()) : 0;
  constexpr int kCtas = P ? 2 : 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&ms->full[i]), 1);
      mbar_init(smem_u32(&ms->empty[i]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&ms->q_full[t]), 1);
      mbar_init(smem_u32(&ms->q_empty[t]), 1);
      mbar_init(smem_u32(&ms->s_full[t]), 1);
      mbar_init(smem_u32(&ms->p_half[t]), 4 * kCtas);       // a warp's arrival each
      mbar_init(smem_u32(&ms->p_full[t]), 4 * kCtas);
      mbar_init(smem_u32(&ms->o_full[t]), 1);
    }
    mbar_init(smem_u32(&ms->drain), 1);
    fence_mbar_init();
    ms->ours = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp ? 1 : 0;
    if (!ms->ours) atomicOr(p.err, kErrStale);
    ms->expanded = p.after_attn ? ld_acquire_gpu(expanded_word(p.err)) : 0;
  }
  if (warp == 9) {
    if constexpr (P) {
      tmem_alloc_pair(smem_u32(&ms->tmem), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&ms->tmem), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (P) cluster_sync();      // the other CTA's barriers are set up too
  tc_fence_after();
  const uint32_t tmem = uniform(ms->tmem);
  if (ms->ours) {
    const int at = P ? blockIdx.x / 2 : blockIdx.x;
    // the CTA's items, all checked before the first is taken up (a pair's two
    // CTAs check the same ones)
    const int4 mine = reinterpret_cast<const int4*>(p.ctas)[at];
    bool sound = check_of(CtaItems{mine.x, mine.y, 0u, 0}, p.stamp) ==
                 static_cast<uint32_t>(mine.z);
    const int it0 = sound ? mine.x : 0;
    for (int it = it0 + static_cast<int>(threadIdx.x); sound && it < mine.y; it += kThreads)
      sound = check_of(load_item(p.items + it), p.stamp) == p.item_checks[it];
    sound = __syncthreads_and(sound);
    if (!sound && threadIdx.x == 0) atomicOr(p.err, kErrStale);
    const int it1 = uniform(sound ? mine.y : it0);
    // Launched as a programmatic dependent: the kernels before this one have to
    // be through before anything of theirs is read.  One that follows an
    // attention kernel (`after_attn`) reads nothing of that one, only of the
    // expansion, which the first kernel has waited for before it lets this one
    // go.  It leaves word of that, by a release here and an acquire there, so
    // that this kernel may start beside the first one's last items and wait for
    // it only before it ends (mixed batches: 2 to 7 % less than with the wait up
    // here).  Without the word it waits.
    if (!p.after_attn || !ms->expanded) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (P && threadIdx.x == 0) st_release_gpu(expanded_word(p.err), 1);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp < 8) {
      regs_raise<208>();
      run_softmax<P>(p, ms, tmem, it0, it1, rank, warp >> 2, warp & 3, lane);
    } else {
      regs_lower<88>();            // 2 x 208 + 88 = 3 x 168, the registers at launch
    }
    if (warp == 8) {
      if (lane == 0) run_loads<P>(p, ms, q_smem, ring, it0, it1, rank);
    } else if (warp == 9 && rank == 0) {
      run_products<P>(p, ms, q_smem, ring, tmem, uniform(it0), uniform(it1));
      // no product may run on after the CTAs have gone
      if (elect_one()) {
        commit<P>(&ms->drain);
        mbar_wait_poll(smem_u32(&ms->drain), 0, p.err, kErrDrain);
      }
    }
    __syncwarp();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if constexpr (P) {
    cluster_sync();                     // nothing of the pair is under way any more
    if (warp == 9) tmem_dealloc_pair(tmem, 512);
  } else {
    if (warp == 9) tmem_dealloc(tmem, 512);
  }
}

template <bool P>
cudaError_t launch(const AttnParams& p, int ctas, cudaStream_t stream) {
  constexpr int bytes = kSmemBytes + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * (P ? 2 : 1));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = P ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, attn_kernel<P>, p);
}

}  // namespace

cudaError_t launch_attn(const AttnParams& p, int num_ctas, cudaStream_t stream) {
  return launch<false>(p, num_ctas, stream);
}
cudaError_t launch_attn_pairs(const AttnParams& p, int num_pairs, cudaStream_t stream) {
  return launch<true>(p, num_pairs, stream);
}

}  // namespace mla
