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
// The output of 128 rows alone fills the 512 columns of a CTA's tensor memory, so
// the scores stand in another CTA's.  A score CTA holds 128 query rows (512 dims
// in tensor memory, 64 in shared memory) and streams key tiles through QK^T; eight
// warps make probabilities of its scores and send them to a value CTA's shared
// memory (bulk copies, 64 keys at a time), with the factors by which the output's
// rows are to be rescaled.  The value CTA streams the keys' first 512 dims through
// PV; its eight warps rescale the output, rarely, and write it.  The work of the two
// is nearly equal: a tile of 128 keys takes 36 K steps of N = 128 of the one (2,304
// cycles) and 16 of N = 256 of the other (2,048).
//
// A cluster is a score and a value CTA, or two of each (kPaired) for 256 rows,
// whose products are those of a pair of CTAs (M = 256): either holds half of a
// tile's keys (of the values: half of their dims).  On their own the two kinds read
// and write 350 KB of shared memory a tile, 2,800 cycles' worth, and a tile takes
// 3,300 cycles; paired, each moves half of the keys, and it takes 2,300 to 2,600.
//
// Measured: 1,024 rows (64 requests) against 32,768 keys, 73 GFLOP, 50 us on 36
// clusters, 1.46 PFLOP/s.  Of these 1.5 us pass until a cluster's CTAs have met, 4 with
// the queries on their way (147 KB, and as many of keys, come to a score CTA in that
// time, at 37 bytes a cycle; an SM takes up to 69, so what holds them up is not known),
// 2 with the first scores, 34 with the other tiles, 3.5 with the last products and 4 with
// the output, 256 KB a CTA at 32 bytes a cycle.  Copies of keys to both CTAs at once
// (multicast) changed nothing, nor did queries that were asked for earlier or taken up
// in thirds.
//
// Probabilities are rounded to bf16, the type of the values that they meet; the
// sums that divide the output are of the unrounded ones.  Scores, sums, maxima
// and outputs are fp32.
//
// Roles (384 threads): warps 0-3 and 4-7 of a score CTA hold the softmax, a
// thread per row and half of a tile's keys (both see the tile's maximum, so that
// they keep the same m); of a value CTA the output's dims 0-255 and 256-511.
// Warp 8 (and in a score CTA warp 10) loads, warp 9 issues the products, in the
// first CTA of a pair for both; warp 11 of a score CTA sends.
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

constexpr int kThreads = 384;
constexpr uint32_t kHalfBytes = 128 * 128;         // 128 rows x 64 keys of P (or 64 dims)
constexpr uint32_t kPanelBytes = 64 * 128;         // 64 keys x 64 dims
// score CTA: probabilities of either half of a tile or two on their way, rotated
// query dims, K ring; value CTA: the probabilities of some tiles received, V ring
constexpr uint32_t kStageAt = 0, kPAt = 0;
constexpr uint32_t kSmemBytes = 14 * kHalfBytes;
constexpr int kChunks = kQkDim / 64;               // of a tile: its keys' dims by 64
constexpr int kGroup = 3;                          // chunks that are waited for together

// What a CTA holds of a tile.  K: 64 or 128 keys and 64 dims a slot; V: 64 keys and
// 128 or 256 dims a slot.
template <bool kPaired>
struct Ring {
  static constexpr uint32_t kPanels = kPaired ? 1 : 2;          // of a K slot, 64 keys each
  static constexpr uint32_t kKBytes = kPanels * kPanelBytes;
  // tiles of P on their way: a copy lands 2,000 cycles after its tile was staged,
  // and chunks take as long to come from L2, which a CTA on its own has less room for
  static constexpr uint32_t kStages = kPaired ? 2 : 1;
  static constexpr uint32_t kQrAt = kStages * 2 * kHalfBytes, kKRingAt = kQrAt + kHalfBytes;
  static constexpr uint32_t kKSlots = kPaired ? 18 : 11;
  static constexpr uint32_t kGroups = kPaired ? 8 : 4;          // of chunks, under way
  static constexpr uint32_t kVPanels = kPaired ? 2 : 4;         // of a V slot, 64 dims each
  static constexpr uint32_t kVBytes = kVPanels * kPanelBytes;
  static constexpr uint32_t kVSlots = kPaired ? 8 : 5;
  // tiles of P in the value CTA: the word that one is there takes 1,500 cycles to
  // the other CTA of a pair
  static constexpr uint32_t kPTiles = kPaired ? 3 : 2;
  static_assert(kPTiles == 2 || kPTiles == 3, "buffers of P");
  static constexpr uint32_t kVRingAt = kPAt + kPTiles * 2 * kHalfBytes;
  static constexpr int kCtas = kPaired ? 2 : 1;                 // of either kind in a cluster
  static_assert(kKRingAt + kKSlots * kKBytes <= kSmemBytes, "the score CTA's arrays fit");
  static_assert(kVRingAt + kVSlots * kVBytes <= kSmemBytes, "the value CTA's arrays fit");
  // (a group's barrier is used again once its chunks have left the ring)
  static_assert(kGroups * kGroup > kKSlots, "groups under way");
};
// score CTA: queries' dims 0-511, then two buffers of scores; value CTA: the output
constexpr uint32_t kColQ = 0, kColS = 256, kColO = 0;
// A row's maximum is kept until a score exceeds it by a factor of 2^8, and then
// moves by a power of two, so that a byte tells the factor.
constexpr float kLag = 8.0f;
// From here on a maximum, which is rounded, may be far from the product that it was
// rounded from (half a step): scores are then rounded in the same way before it is
// taken off.
constexpr float kFar = 16777216.0f;
constexpr uint32_t kPHalfBytes = kHalfBytes;
constexpr uint32_t kFactorBytes = kSpRows, kFinBytes = kSpRows * 4;

struct Misc {
  uint64_t full[8], empty[22];                     // rings: score: a group's bytes, a chunk's
                                                   // slot is free; value: a slot's
  union {
    struct {                                       // score CTA
      uint64_t q_ready;                            // the item's queries are in place
      uint64_t s_full[2], s_empty[2];              // score buffers
      uint64_t staged[4];                          // a half's probabilities are to be sent
      uint64_t landed[4];                          // they have arrived (both: tiles in turn)
      uint64_t p_empty[6];                         // the value CTA's P buffers are free
      uint64_t sum_full, fin_staged;               // the second half's sums; 1 / sums
    };
    struct {                                       // value CTA
      uint64_t p_full[6];                          // P buffers and factors
      uint64_t o_ready[3];                         // a tile's P is there, the output rescaled
      uint64_t pv_done[3];                         // its PV is through
      uint64_t fin_full[2];                        // 1 / sums of an item
    };
  };
  uint64_t drain;
  uint32_t tmem;
  PrefixItem first;                                // the cluster's first item
  // of tiles, and of items, in turn; value CTA: received, score CTA: being sent
  alignas(16) uint8_t factor[6][kSpRows];          // rows are to be scaled by 2^-factor
  alignas(16) float fin[2][kSpRows];               // 1 / sums (score CTA: first the half sums)
};
static_assert(kSmemBytes + sizeof(Misc) <= 232448, "fits a CTA's shared memory");

// Buffer of a tile in a ring of N, and how often the ring has gone round (its
// lowest bit).
template <uint32_t N>
struct Turn {
  uint32_t at = 0, lap = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      lap ^= 1;
    }
  }
};

__device__ __forceinline__ PrefixItem load_item(const PrefixItem* p) {
  const int4 a = reinterpret_cast<const int4*>(p)[0], b = reinterpret_cast<const int4*>(p)[1];
  return PrefixItem{a.x, a.y, a.z, a.w, b.x, b.y, static_cast<uint32_t>(b.z), 0};
}
// Item `it` of a cluster's items from `it0` on.
__device__ __forceinline__ PrefixItem item_at(const PrefixParams& p, const Misc* ms, int it, int it0) {
  return it == it0 ? ms->first : load_item(p.items + it);
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

// This CTA's place: its kind, and which of its kind.  The first of a kind issues
// the products and holds the barriers that they wait for.
struct Place {
  int kind, half;                                  // kind 0: scores, 1: values
  uint32_t first;                                  // rank of the first CTA of this kind
  uint32_t peer;                                   // rank of the other kind's CTA of these rows
};

// One arrival of the (converged) warp at the first CTA's barrier.  kRelease: it
// hands over shared memory, or data that came there; else tensor memory alone,
// which the tcgen05 fences order.
template <bool kPaired, bool kRelease>
__device__ __forceinline__ void arrive_at_first(const Place& at, uint64_t* bar, int lane) {
  __syncwarp();
  if (lane != 0) return;
  if constexpr (!kPaired) {
    mbar_arrive(smem_u32(bar));
  } else {
    const uint32_t there = dsmem_addr(smem_u32(bar), at.first);
    if constexpr (kRelease)
      mbar_arrive_cluster_release(there);
    else
      mbar_arrive_cluster_relaxed(there);
  }
}
template <bool kPaired>
__device__ __forceinline__ void commit(const Place& at, uint64_t* bar) {
  if constexpr (kPaired)
    tc_commit_mask<true>(smem_u32(bar), static_cast<uint16_t>(3u << at.first));
  else
    tc_commit(smem_u32(bar));
}
// Copy of this CTA's shared memory to another's, counted on a barrier there.
__device__ __forceinline__ void bulk_to_peer(uint32_t dst, uint32_t src, uint32_t bytes,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// ---------------------------------------------------------------- loads
template <bool kPaired>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row,
                                         int panel, uint64_t policy) {
  if constexpr (kPaired)
    tma_load_3d_pair(dst, map, bar, 0, row, panel, policy);
  else
    tma_load_3d(dst, map, bar, 0, row, panel, policy);
}

// Row of the tensor map of 64 keys of the item's group, from key `key` on.  In the
// pool itself (`direct`), behind the group's last key it is that of the last 64 keys:
// such keys have no weight, but what stands in their place must not be NaN.
__device__ __forceinline__ int key_row(const PrefixParams& p, const PrefixItem& w, int key) {
  if (!p.direct) return key;
  key = min(key, w.key0 + (w.keys - 1) / 64 * 64);       // (with boxes of 128 keys: a whole tile)
  int64_t page = w.page_base + key / p.page_size;
  if (p.indices != nullptr) page = p.indices[page];
  const int64_t row = page * p.page_size + key % p.page_size;
  if (page < 0 || row + 64 > p.pool_rows) {
    atomicOr(p.err, kErrBadPage);
    return 0;
  }
  return static_cast<int>(row);
}

// Score CTA: every other group of three chunks, from `first` (0 or 1) on.
template <bool kPaired>
__device__ void load_keys(const PrefixParams& p, Misc* ms, const Place& at, uint32_t ring, int it0,
                          int it1, int first) {
  using R = Ring<kPaired>;
  // group of the whole walk, its barrier; the next chunk's slot and, of the slots
  // from it on, the parity of the release to wait for
  uint32_t g = 0, s = 0, parity = 1;
  bool ok = true;
  const uint64_t keep = l2_policy_evict_normal();
  const CUtensorMap* map = &p.map_k;
  const uint32_t full = kPaired ? dsmem_addr(smem_u32(ms->full), at.first) : smem_u32(ms->full);
  for (int it = it0; it < it1 && ok; ++it) {
    const PrefixItem w = item_at(p, ms, it, it0);
    const int tiles = tiles_of(w);
    const int mine = w.key0 + (kPaired ? 64 * at.half : 0);
    int next0 = key_row(p, w, mine), next1 = kPaired ? 0 : key_row(p, w, mine + 64);
    for (int j = 0; j < tiles && ok; ++j) {
      const int row0 = next0, row1 = next1;
      if (j + 1 < tiles) {
        next0 = key_row(p, w, mine + (j + 1) * kSpTile);
        if (!kPaired) next1 = key_row(p, w, mine + (j + 1) * kSpTile + 64);
      }
      for (int ch = 0; ch < kChunks && ok; ch += kGroup, ++g) {
        if ((g & 1) != static_cast<uint32_t>(first)) {
          s += kGroup;
          if (s >= R::kKSlots) {
            s -= R::kKSlots;
            parity ^= 1;
          }
          continue;
        }
        const uint32_t bar = full + 8 * (g % R::kGroups);
        bool ready = mbar_test(smem_u32(&ms->empty[s]), parity);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          if (!ready && !mbar_wait_poll(smem_u32(&ms->empty[s]), parity, p.err, kErrProducer)) {
            ok = false;
            break;
          }
          if (i == 0 && at.half == 0)
            mbar_arrive_expect_tx(smem_u32(&ms->full[g % R::kGroups]), R::kCtas * kGroup * R::kKBytes);
          const uint32_t dst = ring + s * R::kKBytes;
          if (++s == R::kKSlots) {
            s = 0;
            parity ^= 1;
          }
          if (i + 1 < kGroup) ready = mbar_test(smem_u32(&ms->empty[s]), parity);
          load_box<kPaired>(dst, map, bar, row0, ch + i, keep);
          if (!kPaired && !p.tall) load_box<kPaired>(dst + kPanelBytes, map, bar, row1, ch + i, keep);
        }
      }
    }
  }
  if (!ok) linger();                 // no copy may land after the CTA has gone
}

// Value CTA: for each 64 keys the output's dims 0-255 and 256-511 (of a pair:
// this CTA's half of either).
template <bool kPaired>
__device__ void load_values(const PrefixParams& p, Misc* ms, const Place& at, uint32_t ring, int it0,
                            int it1) {
  using R = Ring<kPaired>;
  uint32_t s = 0, parity = 1;        // (of the first lap: nothing to wait for)
  bool ok = true;
  const uint64_t keep = l2_policy_evict_normal();
  const CUtensorMap* map = &p.map_v;
  const uint32_t full = kPaired ? dsmem_addr(smem_u32(ms->full), at.first) : smem_u32(ms->full);
  for (int it = it0; it < it1 && ok; ++it) {
    const PrefixItem w = item_at(p, ms, it, it0);
    const int tiles = tiles_of(w);
    int next0 = key_row(p, w, w.key0), next1 = key_row(p, w, w.key0 + 64);
    for (int j = 0; j < tiles && ok; ++j) {
      const int row0 = next0, row1 = next1;
      if (j + 1 < tiles) {
        next0 = key_row(p, w, w.key0 + (j + 1) * kSpTile);
        next1 = key_row(p, w, w.key0 + (j + 1) * kSpTile + 64);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!mbar_wait_poll(smem_u32(&ms->empty[s]), parity, p.err, kErrProducer)) {
          ok = false;
          break;
        }
        if (at.half == 0) mbar_arrive_expect_tx(smem_u32(&ms->full[s]), R::kCtas * R::kVBytes);
        const int row = u < 2 ? row0 : row1, panel = 4 * (u & 1) + 2 * at.half;
        const uint32_t dst = ring + s * R::kVBytes, bar = full + 8 * s;
        load_box<kPaired>(dst, map, bar, row, panel, keep);
        if (++s == R::kVSlots) {
          s = 0;
          parity ^= 1;
        }
      }
    }
  }
  if (!ok) linger();
}

// ------------------------------------------------------------- products
template <bool kPaired>
__device__ void run_scores(const PrefixParams& p, Misc* ms, const Place& at, uint32_t smem,
                           uint32_t tmem, int it0, int it1) {
  using R = Ring<kPaired>;
  constexpr uint32_t idesc = make_idesc(1, 1, false, false, kPaired ? 256 : 128, 128);
  const uint64_t qd = smem_desc(smem + R::kQrAt, 16, 1024, kSwizzle128B);
  const uint64_t kd = smem_desc(smem + R::kKRingAt, 16, 1024, kSwizzle128B);
  uint32_t tile = 0, g = 0, s = 0;
  auto wait = [&](bool ready, uint64_t* bar, uint32_t parity) {
    return all_waited(ready) ||
           all_waited(mbar_wait_poll(smem_u32(bar), parity, p.err, kErrMma));
  };
  // (arrivals of both CTAs' threads)
  auto wait_queries = [&](uint32_t parity) {
    return all_waited(kPaired ? mbar_wait_cluster<true>(smem_u32(&ms->q_ready), parity, p.err, kErrMma)
                              : mbar_wait_poll(smem_u32(&ms->q_ready), parity, p.err, kErrMma));
  };
  auto wait_buffer = [&](uint32_t b, uint32_t parity) {
    return all_waited(kPaired ? mbar_wait_cluster(smem_u32(&ms->s_empty[b]), parity, p.err, kErrMma)
                              : mbar_wait_poll(smem_u32(&ms->s_empty[b]), parity, p.err, kErrMma));
  };
  auto group_ready = [&](uint32_t g) {
    return mbar_test(smem_u32(&ms->full[g % R::kGroups]), (g / R::kGroups) & 1);
  };
  for (int it = it0; it < it1; ++it) {
    const int tiles = uniform(tiles_of(item_at(p, ms, it, it0)));
    if (!wait_queries((it - it0) & 1)) return;
    if constexpr (kPaired) fence_proxy_async();      // (the other CTA's rotated query dims)
    for (int j = 0; j < tiles; ++j, ++tile) {
      const uint32_t b = tile & 1;
      bool ready = group_ready(g);
      if (tile >= 2 && !wait_buffer(b, ((tile >> 1) - 1) & 1)) return;
      const uint32_t d = tmem + kColS + 128 * b;
#pragma unroll
      for (int u = 0; u < kChunks / kGroup; ++u, ++g) {
        if (!wait(ready, &ms->full[g % R::kGroups], (g / R::kGroups) & 1)) return;
        ready = group_ready(g + 1);
        tc_fence_after();
        uint32_t slot[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          slot[i] = s;
          s = s + 1 == R::kKSlots ? 0 : s + 1;
        }
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const int ch = kGroup * u + i;
            const uint64_t kb = kd + ((slot[i] * R::kKBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t qa = tmem + kColQ + 32 * ch + 8 * kk;
              if constexpr (kPaired) {
                if (ch < 8)
                  umma_f16_ta_pair(d, qa, kb + 2 * kk, idesc, (ch | kk) != 0);
                else
                  umma_f16_pair(d, qd + 2 * kk, kb + 2 * kk, idesc, 1);
              } else {
                if (ch < 8)
                  umma_f16_ta(d, qa, kb + 2 * kk, idesc, (ch | kk) != 0);
                else
                  umma_f16(d, qd + 2 * kk, kb + 2 * kk, idesc, 1);
              }
            }
            commit<kPaired>(at, &ms->empty[slot[i]]);
          }
          if (u == kChunks / kGroup - 1) commit<kPaired>(at, &ms->s_full[b]);
        }
        __syncwarp();
      }
    }
  }
}

template <bool kPaired>
__device__ void run_values(const PrefixParams& p, Misc* ms, const Place& at, uint32_t smem,
                           uint32_t tmem, int it0, int it1) {
  using R = Ring<kPaired>;
  constexpr uint32_t idesc = make_idesc(1, 1, false, true, kPaired ? 256 : 128, 256);
  // (the score CTAs of these rows: those before the value CTAs)
  const uint16_t scores = kPaired ? 3 : 1;
  const uint64_t pd = smem_desc(smem + kPAt, 16, 1024, kSwizzle128B);
  const uint64_t vd = smem_desc(smem + R::kVRingAt, kPanelBytes, 1024, kSwizzle128B);
  uint32_t s = 0, lap = 0;
  Turn<R::kPTiles> turn;
  for (int it = it0; it < it1; ++it) {
    const int tiles = uniform(tiles_of(item_at(p, ms, it, it0)));
    for (int j = 0; j < tiles; ++j, turn.next()) {
      bool ready = mbar_test(smem_u32(&ms->full[s]), lap);
      uint64_t* o_ready = &ms->o_ready[turn.at];
      if (!all_waited(kPaired ? mbar_wait_cluster<true>(smem_u32(o_ready), turn.lap, p.err, kErrMma)
                              : mbar_wait_poll(smem_u32(o_ready), turn.lap, p.err, kErrMma)))
        return;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int h = u >> 1, dims = u & 1;
        const uint32_t buf = 2 * turn.at + h;
        const uint64_t a = pd + ((buf * kHalfBytes) >> 4);
        if (!all_waited(ready) &&
            !all_waited(mbar_wait_poll(smem_u32(&ms->full[s]), lap, p.err, kErrMma)))
          return;
        const uint32_t slot = s;
        if (++s == R::kVSlots) {
          s = 0;
          lap ^= 1;
        }
        if (u < 3) ready = mbar_test(smem_u32(&ms->full[s]), lap);
        tc_fence_after();
        const uint64_t vb = vd + ((slot * R::kVBytes) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t d = tmem + kColO + 256 * dims;
            if constexpr (kPaired)
              umma_f16_pair(d, a + 2 * kk, vb + 128 * kk, idesc, (j | h | kk) != 0);
            else
              umma_f16(d, a + 2 * kk, vb + 128 * kk, idesc, (j | h | kk) != 0);
          }
          commit<kPaired>(at, &ms->empty[slot]);
          if (dims == 1) tc_commit_mask<kPaired>(smem_u32(&ms->p_empty[buf]), scores);
          if (u == 3) commit<kPaired>(at, &ms->pv_done[turn.at]);
        }
        __syncwarp();
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

// 64 dims of a warp's 32 query rows (zeros past the item's `live` rows) on their
// way, whole lines at a time: a lane holds 16 bytes of bf16 in steps of 4 rows, or of
// e4m3 in steps of 8.  `src`: the lane's piece of its first row.
template <bool kFp8>
__device__ __forceinline__ void fetch_query(const uint8_t* src, int live, int lane,
                                            uint4 (&x)[kFp8 ? 4 : 8]) {
  constexpr int kLanes = kFp8 ? 4 : 8;                   // of a row
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    const int r = 32 / kLanes * i + lane / kLanes;
    x[i] = r < live ? ld_na_v4(src + 32 / kLanes * i * kQkDim * (kFp8 ? 1 : 2)) : make_uint4(0, 0, 0, 0);
  }
}
// The same as bf16 rows of 128 bytes at `dst` (row 0 of the warp, a multiple of 8
// rows behind a 1,024-byte boundary), in the 128-byte swizzle; with `sign` 0x80008000
// all of it negated.
template <bool kFp8>
__device__ __forceinline__ void stage_query(const uint4 (&x)[kFp8 ? 4 : 8], uint32_t dst, uint32_t sign,
                                            int lane) {
  constexpr int kLanes = kFp8 ? 4 : 8;
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    const int r = 32 / kLanes * i + lane / kLanes;
    const uint32_t at = dst + r * 128;
    if constexpr (kFp8) {
      const int piece = 2 * (lane & 3);
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[k] = bf16x2_of(f.x, f.y) ^ sign;
      }
      st_shared_16(at + ((piece ^ (r & 7)) << 4), v[0], v[1], v[2], v[3]);
      st_shared_16(at + (((piece + 1) ^ (r & 7)) << 4), v[4], v[5], v[6], v[7]);
    } else {
      st_shared_16(at + (((lane & 7) ^ (r & 7)) << 4), x[i].x ^ sign, x[i].y ^ sign, x[i].z ^ sign,
                   x[i].w ^ sign);
    }
  }
}
// A lane's own row of it, as bf16 pairs.
__device__ __forceinline__ void own_query(uint32_t src, int lane, uint32_t* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[4 * i]), "=r"(v[4 * i + 1]), "=r"(v[4 * i + 2]), "=r"(v[4 * i + 3])
                 : "r"(src + lane * 128 + ((i ^ (lane & 7)) << 4))
                 : "memory");
}

// A warp's 32 query rows: dims 256 h .. 256 h + 255 to tensor memory (a row a lane),
// by way of 4 KB of shared memory; with h = 0 the rotated ones to shared memory.
template <bool kFp8>
__device__ __forceinline__ void load_queries(const void* q, int64_t row0, int live, int h,
                                             uint32_t sign, uint32_t via, uint32_t tmem,
                                             uint32_t rotated, int lane) {
  constexpr int kRowBytes = kQkDim * (kFp8 ? 1 : 2), kChunkBytes = kRowBytes / kChunks;
  constexpr int kLanes = kFp8 ? 4 : 8;
  const uint8_t* rows = static_cast<const uint8_t*>(q) + row0 * kRowBytes;
  if (lane < live) {
    // all lines of the lane's row, so that the chunks behind the first one wait less
#pragma unroll
    for (int i = 0; i < 5; ++i)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(rows + lane * kRowBytes +
                                                    (i < 4 ? 4 * h + i : 8) * kChunkBytes));
  }
  const uint8_t* src = rows + lane / kLanes * kRowBytes + lane % kLanes * 16 + 4 * h * kChunkBytes;
  // (a chunk ahead)
  uint4 x[2][kLanes];
  fetch_query<kFp8>(src, live, lane, x[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t v[32];
    if (c < 3 || h == 0)
      fetch_query<kFp8>(src + (c < 3 ? c + 1 : 8) * kChunkBytes, live, lane, x[(c + 1) & 1]);
    stage_query<kFp8>(x[c & 1], via, sign, lane);
    __syncwarp();
    own_query(via, lane, v);
    __syncwarp();
    tmem_st32(tmem + 32 * c, v);
  }
  if (h == 0) {
    stage_query<kFp8>(x[0], rotated, sign, lane);
    fence_proxy_async_smem();
  }
  __syncwarp();
  tmem_wait_st();
}

template <bool kPaired>
__device__ void run_softmax(const PrefixParams& p, Misc* ms, const Place& at, uint32_t smem,
                            uint32_t tmem, int it0, int it1, int h, int warp, int lane) {
  const int row = warp * 32 + lane, item_row = at.half * kSpRows + row;
  const uint32_t lanes = static_cast<uint32_t>(warp) << 21;      // TMEM lane 32 warp
  const uint32_t tq = tmem + lanes + kColQ, ts = tmem + lanes + kColS;
  const uint32_t stage0 = smem + kStageAt + h * kHalfBytes + row * 128, swizzle = row & 7;
  const float qs = p.q_scale != nullptr ? *p.q_scale : 1.0f;
  const float ks = p.kv_scale != nullptr ? *p.kv_scale : 1.0f;
  // A row's maximum is that of its products, so their factor has to be positive: a
  // negative one turns the queries around, and instead of 0 it is the smallest number,
  // with which finite products still come to 0 (2^-21 at most) but -inf, where there is
  // no key, does not become NaN.  (Multiplied as by the decode kernel, whose equal
  // scores are to stay equal.)
  const float factor = qs * ks * (1.0f / 24.0f) * kLog2e;
  const uint32_t sign = factor < 0.0f ? 0x80008000u : 0u;
  const float scale = factor == 0.0f ? __uint_as_float(1u) : fabsf(factor);
  const uint64_t scale2 = pack_f32x2(scale, scale);
  uint32_t tile = 0;
  Turn<Ring<kPaired>::kPTiles> turn;
  Turn<Ring<kPaired>::kStages> side_of;                  // staging buffers
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return all_waited(mbar_wait_poll(smem_u32(bar), parity, p.err, kErrSoftmax));
  };
  for (int it = it0; it < it1; ++it) {
    const PrefixItem w = item_at(p, ms, it, it0);
    const int tiles = tiles_of(w);
    {
      // Queries, a row a lane of tensor memory, by way of the warp's part of its
      // staging buffer 0 (once the last copy from there has landed).
      const int row0 = at.half * kSpRows + warp * 32;
      const int64_t q_row0 = static_cast<int64_t>(w.q_row) + row0;
      const int live = w.rows - row0;
      const uint32_t via = smem + kStageAt + h * kHalfBytes + warp * 4096;
      constexpr uint32_t kStages = Ring<kPaired>::kStages;
      const uint32_t uses = (tile + kStages - 1) / kStages;
      if (uses > 0 && !all_waited(mbar_wait_cluster(smem_u32(&ms->landed[h]), (uses - 1) & 1, p.err,
                                                    kErrSoftmax)))
        return;
      const uint32_t rotated = smem + Ring<kPaired>::kQrAt + warp * 4096;
      if (p.q_fp8)
        load_queries<true>(p.q, q_row0, live, h, sign, via, tq + 128 * h, rotated, lane);
      else
        load_queries<false>(p.q, q_row0, live, h, sign, via, tq + 128 * h, rotated, lane);
      tc_fence_before();
      arrive_at_first<kPaired, true>(at, &ms->q_ready, lane);
    }
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < tiles; ++j, ++tile, turn.next(), side_of.next()) {
      const uint32_t b = tile & 1;
      if (!wait(&ms->s_full[b], (tile >> 1) & 1)) return;
      tc_fence_after();
      // the scores of this half, and the maxima of both
      uint32_t s[64], other[64];
      const uint32_t mine = ts + 128 * b + 64 * h, theirs = ts + 128 * b + 64 * (1 - h);
      float tops[4];
      tops[0] = tmem_ld32_max(mine, s);
      tops[1] = tmem_ld32_max(mine + 32, s + 32);
      tops[2] = tmem_ld32_max(theirs, other);
      tops[3] = tmem_ld32_max(theirs + 32, other + 32);
      tmem_wait_ld();
      tc_fence_before();
      arrive_at_first<kPaired, false>(at, &ms->s_empty[b], lane);
      // The staging buffer is free once its last copy has landed, the value CTA's once
      // its last tile is through PV: looked at here, waited for below.
      const uint32_t buf = 2 * turn.at + h;
      const uint32_t landed_bar = smem_u32(&ms->landed[2 * side_of.at + h]);
      const bool landed = tile < Ring<kPaired>::kStages || mbar_test_cluster(landed_bar, side_of.lap ^ 1);
      const bool taken = tile < Ring<kPaired>::kPTiles ||
                         mbar_test_cluster(smem_u32(&ms->p_empty[buf]), turn.lap ^ 1);
      const int left = w.keys - j * kSpTile;             // keys of this tile
      if (left < kSpTile) {
        tops[0] = tops[1] = tops[2] = tops[3] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          s[i] = 64 * h + i < left ? s[i] : 0xff800000u;
          tops[0] = fmaxf(tops[0], __uint_as_float(s[i]));
          tops[2] = fmaxf(tops[2], 64 * (1 - h) + i < left ? __uint_as_float(other[i]) : -INFINITY);
        }
      }
      const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * scale;
      uint32_t drop = 0;
      if (top > m + kLag) {
        const float d = ceilf(top - m);                  // (the first tile: infinite)
        drop = d < 200.0f ? static_cast<uint32_t>(d) : 200u;
        m = d < 200.0f ? m + d : top;
        l *= factor_of(drop);
      }
      // a row that has seen no score above -inf keeps p = 2^(-inf) = 0
      const float off = m == -INFINITY ? 0.0f : -m;
      const uint64_t off2 = pack_f32x2(off, off);
      uint64_t by2 = scale2;
      if (fabsf(m) >= kFar) {
        by2 = pack_f32x2(1.0f, 1.0f);
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * scale);
      }
      uint64_t sum0 = 0, sum1 = 0;
      uint32_t pk[32];
#pragma unroll
      for (int i = 0; i < 64; i += 4) {
        float x0, x1, x2, x3;
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), by2,
                               off2), x0, x1);
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])),
                               by2, off2), x2, x3);
        x0 = ex2(x0); x1 = ex2(x1); x2 = ex2(x2); x3 = ex2(x3);
        sum0 = add_f32x2(sum0, pack_f32x2(x0, x1));
        sum1 = add_f32x2(sum1, pack_f32x2(x2, x3));
        pk[i / 2] = bf16x2_of(x0, x1);
        pk[i / 2 + 1] = bf16x2_of(x2, x3);
      }
      float u0, u1;
      unpack_f32x2(add_f32x2(sum0, sum1), u0, u1);
      l += u0 + u1;
      if (!all_waited(landed) &&
          !all_waited(mbar_wait_cluster(landed_bar, side_of.lap ^ 1, p.err, kErrSoftmax)))
        return;
      const uint32_t stage = stage0 + side_of.at * 2 * kHalfBytes;
      if (!all_waited(taken) && !all_waited(mbar_wait_cluster(smem_u32(&ms->p_empty[buf]), turn.lap ^ 1,
                                                              p.err, kErrSoftmax)))
        return;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        st_shared_16(stage + ((i ^ swizzle) << 4), pk[4 * i], pk[4 * i + 1], pk[4 * i + 2],
                     pk[4 * i + 3]);
      ms->factor[buf][row] = static_cast<uint8_t>(drop);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->staged[2 * side_of.at + h]));
    }
    // Sums of both halves; 1 / sum (times the values' scale) to the value CTA.  The
    // buffers on both sides are those of the item before the last: its output was
    // written before the first PV of the last item, so before the PV of the tile
    // before this item's last one was through.
    const uint32_t side = (it - it0) & 1;
    if (tile >= 2) {
      Turn<Ring<kPaired>::kPTiles> before = turn;        // (the tile before the last)
      if constexpr (Ring<kPaired>::kPTiles == 3) before.next();
      const uint32_t lap = before.at < turn.at ? turn.lap : turn.lap ^ 1;
      if (!all_waited(mbar_wait_cluster(smem_u32(&ms->p_empty[2 * before.at + h]), lap, p.err,
                                        kErrSoftmax)))
        return;
    }
    if (h == 1) {
      ms->fin[side][row] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->sum_full));
    } else {
      if (!wait(&ms->sum_full, side)) return;
      l += ms->fin[side][row];
      if (item_row < w.rows)
        p.part_lse[(static_cast<int64_t>(w.slot) * Ring<kPaired>::kCtas + at.half) * kSpRows + row] =
            l == 0.0f ? -INFINITY : m + __log2f(l);
      ms->fin[side][row] = l == 0.0f ? 0.0f : ks / l;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms->fin_staged));
    }
  }
}

// What the softmax has staged goes to the value CTA (one thread).
template <bool kPaired>
__device__ void run_sends(const PrefixParams& p, Misc* ms, const Place& at, uint32_t smem, int it0,
                          int it1) {
  const uint32_t peer_p = dsmem_addr(smem + kPAt, at.peer);
  const uint32_t peer_full = dsmem_addr(smem_u32(ms->p_full), at.peer);
  const uint32_t peer_factor = dsmem_addr(smem_u32(ms->factor), at.peer);
  const uint32_t peer_fin = dsmem_addr(smem_u32(ms->fin), at.peer);
  const uint32_t peer_fin_full = dsmem_addr(smem_u32(ms->fin_full), at.peer);
  uint32_t tile = 0;
  Turn<Ring<kPaired>::kPTiles> turn;
  Turn<Ring<kPaired>::kStages> side_of, last;            // staging buffers
  bool ok = true;
  for (int it = it0; it < it1 && ok; ++it) {
    const int tiles = tiles_of(item_at(p, ms, it, it0));
    for (int j = 0; j < tiles && ok; ++j, ++tile, turn.next(), last = side_of, side_of.next()) {
#pragma unroll
      for (uint32_t h = 0; h < 2; ++h) {
        ok = ok && mbar_wait_poll(smem_u32(&ms->staged[2 * side_of.at + h]), side_of.lap, p.err,
                                  kErrSoftmax);
        if (!ok) break;
        const uint32_t buf = 2 * turn.at + h;
        bulk_to_peer(peer_p + buf * kHalfBytes, smem + kStageAt + (2 * side_of.at + h) * kHalfBytes,
                     kPHalfBytes, peer_full + 8 * buf);
        bulk_to_peer(peer_factor + buf * kFactorBytes, smem_u32(ms->factor[buf]), kFactorBytes,
                     peer_full + 8 * buf);
      }
    }
    const uint32_t side = (it - it0) & 1;
    ok = ok && mbar_wait_poll(smem_u32(&ms->fin_staged), side, p.err, kErrSoftmax);
    if (ok)
      bulk_to_peer(peer_fin + side * kFinBytes, smem_u32(ms->fin[side]), kFinBytes,
                   peer_fin_full + 8 * side);
  }
  // what was sent is there before either CTA goes
  // (of two tiles on their way the earlier one before the later one: landed words
  // come in the order of the tiles)
  for (int h = 0; h < 2 && ok && tile > 0; ++h)
    ok = mbar_wait_cluster(smem_u32(&ms->landed[2 * last.at + h]), last.lap, p.err, kErrSoftmax);
  if (!ok) linger();
}

// --------------------------------------------------------------- output
// (false: a wait gave up)
template <bool kPaired>
__device__ bool run_output(const PrefixParams& p, Misc* ms, const Place& at, uint32_t tmem, int it0,
                           int it1, int half, int warp, int lane) {
  const int row = warp * 32 + lane, item_row = at.half * kSpRows + row;
  const uint32_t to = tmem + (static_cast<uint32_t>(warp) << 21) + kColO + 256 * half;
  const uint32_t landed = dsmem_addr(smem_u32(&ms->landed[half]), at.peer);
  uint32_t side_of = 0;                                  // the sender's staging buffer
  const bool speaker = warp == 0 && lane == 0;
  Turn<Ring<kPaired>::kPTiles> turn, last, earlier;      // the two tiles before
  bool second = false;                                   // (there is one)
  for (int it = it0; it < it1; ++it) {
    const PrefixItem w = item_at(p, ms, it, it0);
    const int tiles = tiles_of(w);
    for (int j = 0; j < tiles; ++j) {
      const uint32_t buf = 2 * turn.at + half;
      if (!all_waited(mbar_wait_poll(smem_u32(&ms->p_full[buf]), turn.lap, p.err, kErrDrain)))
        return false;
      if (speaker) {
        // word of it to the sender; and the next one's bytes, which cannot come
        // before this buffer is given back
        mbar_arrive_cluster_relaxed(landed + 16 * side_of);
        mbar_arrive_expect_tx(smem_u32(&ms->p_full[buf]), kPHalfBytes + kFactorBytes);
      }
      const uint32_t drop = ms->factor[buf][row];
      if (j > 0 && __any_sync(0xffffffffu, drop != 0)) {
        const float f = factor_of(drop);
        if (!all_waited(mbar_wait_poll(smem_u32(&ms->pv_done[last.at]), last.lap, p.err, kErrDrain)))
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
      arrive_at_first<kPaired, true>(at, &ms->o_ready[turn.at], lane);
      second = it > it0 || j > 0;
      earlier = last;
      last = turn;
      turn.next();
      side_of = side_of + 1 == Ring<kPaired>::kStages ? 0 : side_of + 1;
    }
    // The last PV; first the one before it, since this half's P may be there before
    // the other half of an earlier tile in the same buffer is through, and the
    // parities of two laps of a barrier are not to be mixed up.
    const uint32_t side = (it - it0) & 1;
    if ((second && !all_waited(mbar_wait_poll(smem_u32(&ms->pv_done[earlier.at]), earlier.lap, p.err,
                                              kErrDrain))) ||
        !all_waited(mbar_wait_poll(smem_u32(&ms->pv_done[last.at]), last.lap, p.err, kErrDrain)) ||
        !all_waited(mbar_wait_poll(smem_u32(&ms->fin_full[side]), ((it - it0) >> 1) & 1, p.err,
                                   kErrDrain)))
      return false;
    tc_fence_after();
    const float inv = ms->fin[side][row];
    // [dims / 8][row][8]: 32 bytes a lane, a kilobyte a warp
    float* dst = p.part_o +
                 (static_cast<int64_t>(w.slot) * Ring<kPaired>::kCtas + at.half) * kSpRows * kVDim +
                 (32 * half * kSpRows + row) * 8;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t o[64];
      __syncwarp();
      tmem_ld32(to + 64 * c, o);
      tmem_ld32(to + 64 * c + 32, o + 32);
      tmem_wait_ld();
      if (item_row < w.rows) {
#pragma unroll
        for (int i = 0; i < 64; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
#pragma unroll
        for (int i = 0; i < 8; ++i) st_global_32(dst + (8 * c + i) * kSpRows * 8, o + 8 * i);
      }
    }
    tc_fence_before();
    // (re-armed for the item after the next)
    if (half == 0 && speaker) mbar_arrive_expect_tx(smem_u32(&ms->fin_full[side]), kFinBytes);
  }
  return true;
}

template <bool kPaired>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ PrefixParams p) {
  using R = Ring<kPaired>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Misc* ms = reinterpret_cast<Misc*>(smem_raw + kSmemBytes);
  const uint32_t smem = smem_u32(smem_raw);
  if ((smem & 1023u) != 0) {         // (the swizzled tiles need it; there is no room to move)
    if (threadIdx.x == 0) atomicOr(p.err, kErrProducer);
    return;
  }
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  Place at;
  at.kind = static_cast<int>(rank) / R::kCtas;
  at.half = static_cast<int>(rank) % R::kCtas;
  at.first = static_cast<uint32_t>(at.kind * R::kCtas);
  at.peer = rank ^ R::kCtas;
  // (the first kernel of its call: behind what the caller has launched; else only the
  // gathered rows are waited for, by the loads)
  if (p.direct) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(smem_u32(&ms->full[i]), 1);
    for (int i = 0; i < 22; ++i) mbar_init(smem_u32(&ms->empty[i]), 1);
    mbar_init(smem_u32(&ms->drain), 1);
    if (at.kind == 0) {
      mbar_init(smem_u32(&ms->q_ready), 8 * R::kCtas);
      mbar_init(smem_u32(&ms->sum_full), 4);
      mbar_init(smem_u32(&ms->fin_staged), 4);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&ms->s_full[i]), 1);
        mbar_init(smem_u32(&ms->s_empty[i]), 8 * R::kCtas);
        mbar_init(smem_u32(&ms->staged[i]), 4);
        mbar_init(smem_u32(&ms->staged[2 + i]), 4);
        mbar_init(smem_u32(&ms->landed[i]), 1);
        mbar_init(smem_u32(&ms->landed[2 + i]), 1);
      }
      for (int b = 0; b < 6; ++b) mbar_init(smem_u32(&ms->p_empty[b]), 1);
    } else {
      for (int i = 0; i < 3; ++i) {
        mbar_init(smem_u32(&ms->o_ready[i]), 8 * R::kCtas);
        mbar_init(smem_u32(&ms->pv_done[i]), 1);
      }
      for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&ms->fin_full[i]), 1);
      for (int b = 0; b < 6; ++b) mbar_init(smem_u32(&ms->p_full[b]), 1);
    }
    fence_mbar_init();
    if (at.kind == 1) {
      for (uint32_t b = 0; b < 2 * R::kPTiles; ++b)
        mbar_arrive_expect_tx(smem_u32(&ms->p_full[b]), kPHalfBytes + kFactorBytes);
      for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(smem_u32(&ms->fin_full[i]), kFinBytes);
    }
  }
  if (warp == 9) {
    if constexpr (kPaired) {
      tmem_alloc_pair(smem_u32(&ms->tmem), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&ms->tmem), 512);
      tmem_relinquish();
    }
  }
  // the cluster's items, all checked before the first is taken up (its CTAs check
  // the same ones)
  const int4 mine = reinterpret_cast<const int4*>(p.clusters)[blockIdx.x / (2 * R::kCtas)];
  bool sound = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp &&
               check_of(CtaItems{mine.x, mine.y, 0u, 0}, p.stamp) == static_cast<uint32_t>(mine.z);
  const int it0 = sound ? mine.x : 0;
  for (int it = it0 + static_cast<int>(threadIdx.x); sound && it < mine.y; it += kThreads) {
    const PrefixItem w = load_item(p.items + it);
    sound = check_of(w, p.stamp) == w.check;
    if (it == it0) ms->first = w;
  }
  sound = __syncthreads_and(sound);
  if (!sound && threadIdx.x == 0) atomicOr(p.err, kErrStale);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                    // the other CTAs' barriers are set up too
  tc_fence_after();
  const uint32_t tmem = uniform(ms->tmem);
  const int first = uniform(it0), last = uniform(sound ? mine.y : it0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp < 8) {
    if (at.kind == 0)
      run_softmax<kPaired>(p, ms, at, smem, tmem, first, last, warp >> 2, warp & 3, lane);
    else if (!run_output<kPaired>(p, ms, at, tmem, first, last, warp >> 2, warp & 3, lane))
      linger();                      // copies on their way land before this CTA goes
  } else if (warp == 9) {
    if (at.half == 0) {
      if (at.kind == 0)
        run_scores<kPaired>(p, ms, at, smem, tmem, first, last);
      else
        run_values<kPaired>(p, ms, at, smem, tmem, first, last);
      // no product may run on after the CTAs have gone
      if (elect_one()) {
        commit<kPaired>(at, &ms->drain);
        mbar_wait_poll(smem_u32(&ms->drain), 0, p.err, kErrDrain);
      }
    }
  } else if (warp == 11) {
    if (lane == 0 && at.kind == 0) run_sends<kPaired>(p, ms, at, smem, first, last);
  } else if (lane == 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");        // the gathered rows are there
    if (at.kind == 0)
      load_keys<kPaired>(p, ms, at, smem + R::kKRingAt, first, last, warp == 8 ? 0 : 1);
    else if (warp == 8)
      load_values<kPaired>(p, ms, at, smem + R::kVRingAt, first, last);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();                    // nothing of the cluster is under way any more
  if (warp == 9) {
    if constexpr (kPaired)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

template <bool kPaired>
cudaError_t configure(cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&attr)[2], int clusters,
                      bool dependent, cudaStream_t stream) {
  constexpr int bytes = kSmemBytes + sizeof(Misc), ctas = 2 * Ring<kPaired>::kCtas;
  cfg->gridDim = dim3(ctas * clusters);
  cfg->blockDim = dim3(kThreads);
  cfg->dynamicSmemBytes = bytes;
  cfg->stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {ctas, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = dependent ? 2 : 1;
  return cudaFuncSetAttribute(prefix_kernel<kPaired>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              bytes);
}
template <bool kPaired>
cudaError_t launch(const PrefixParams& p, int clusters, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  const cudaError_t e = configure<kPaired>(&cfg, attr, clusters, true, stream);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, prefix_kernel<kPaired>, p);
}
template <bool kPaired>
int fitting() {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (configure<kPaired>(&cfg, attr, 1, false, nullptr) != cudaSuccess) return 0;
  return cudaOccupancyMaxActiveClusters(&n, prefix_kernel<kPaired>, &cfg) == cudaSuccess ? n : 0;
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, bool paired, int clusters, cudaStream_t stream) {
  return paired ? launch<true>(p, clusters, stream) : launch<false>(p, clusters, stream);
}
int prefix_clusters(bool paired) { return paired ? fitting<true>() : fitting<false>(); }

}  // namespace mla
