// expand.cu -- expansion of cached rows into keys and values: for every
// cached token t and head h
//     kx[h][t][0:128] = W_UK[h] c_t,   kx[h][t][128:256] = W_UV[h] c_t
// (one matrix product, K = 512, N = 256 a head), and kr[t] = the 64 rotated
// dims.  The rows are gathered through the page table and decoded on the way
// into shared memory; nothing is written back in between.
//
// Bound: 2 x 512 x 256 flops per (token, head) against 512 bytes written; the
// weights (256 KB a head) come from L2.  A pair of CTAs works on two 128-row
// tiles with one product of M = 256, N = 256: each keeps its rows (128 KB of
// bf16) in shared memory and streams half of each head's weights past them.
// On its own a CTA would read 12 KB of operands a product (128 cycles) and
// take in 8 KB of weights, 160 bytes a cycle of a shared memory that gives 128
// (32,845 MXFP4 keys, 16 heads: 121 us; in pairs 93 us).  Rows are read and decoded
// once per pair that meets them; units (two tiles, head) are split evenly over
// the pairs.  Two 256-column accumulators let the epilogue of one head run
// under the products of the next.  Operand reads, weights and outputs still
// take about 125 bytes a cycle at the products' full rate, and new rows of a
// single buffer stop them for about 8,000 cycles a tile pair: the tensor pipe is
// 62 % busy in the long run (1.48 PFLOP/s); 8192 bf16 keys take 32 us (1.07
// PFLOP/s), of which about 8 us pass before the first product (page table, rows
// and weights from memory).
// With the rows in tensor memory (bulk copies, decoded a lane a row, products of
// N = 128) it took 90 / 33 us: faster on long rows, slower on short ones.
//
// Roundings: e4m3 and e2m1 values with their block exponents are exact in
// bf16; the per-tensor scale goes into the fp32 epilogue.  Keys are rounded to
// bf16 once, as operands of the attention's products, values to fp16 where each of
// the 32 rows of a warp has its largest magnitude in [2^-6, 2^15] (three bits
// more, far from fp16's ends: an error below 2^-25 is 2^-19 of that magnitude),
// else to bf16; a flag per 32 rows and head says which.  (Each row, as a query may
// see only the shortest of them; rows past the request's end do not count.)
//
// A value row that is not finite would reach every query through 0 x NaN in
// the attention's product, also those that must not see the token.  Such a
// row's values are written as zeros and its key as NaN: the queries that see
// the token get NaN through their scores, the others nothing.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "prefill.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kExpandThreads = 448;        // 4 epilogue, 8 row, 1 weight, 1 product warps
constexpr uint32_t kAChunk = 128 * 128;    // 128 rows x 64 bf16
constexpr uint32_t kWChunk = 128 * 128;    // this CTA's 128 weight rows x 64 bf16
constexpr int kChunks = kVDim / 64;
constexpr int kWSlots = 4;
constexpr uint32_t kBox = 32 * 128;        // a warp's output box: 32 rows x 64 bf16, two a warp
constexpr uint32_t kExpandSmem = kChunks * kAChunk + kWSlots * kWChunk + 4 * 2 * kBox;
// Row chunks that a thread has in flight from memory.  The proxy fence behind a
// chunk waits for all of the thread's loads, so none is issued between fences:
// the chunks come in batches (registers: four of bf16, all of the others).
constexpr int kFenced = 4;                 // chunks handed over behind one proxy fence
template <int KV>
constexpr int kBatch = KV == MLA_DTYPE_BF16 ? 4 : 8;

// Barriers that the issuing (even) CTA waits on stand there; commits arrive in
// both CTAs.
struct ExpandMisc {
  uint64_t a_full[kChunks], a_peer[kChunks / kFenced], a_empty[kChunks];
  uint64_t w_full[kWSlots], w_empty[kWSlots];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem, ours;
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
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

// 16 consecutive bytes of a stored row: 8 bf16, 16 e4m3 or 32 e2m1 values (a
// block, with its exponent).
template <int KV>
constexpr int kPerLoad = KV == MLA_DTYPE_BF16 ? 8 : KV == MLA_DTYPE_FP8_E4M3 ? 16 : 32;
struct Raw {
  uint4 v;
  uint32_t e;
};

// The g-th 16 bytes of a row.
template <int KV>
__device__ __forceinline__ Raw load_raw(const ExpandParams& p, int64_t row, int g) {
  constexpr int kRow = kQkDim / kPerLoad<KV> * 16;
  Raw r;
  r.v = *reinterpret_cast<const uint4*>(p.kv + row * kRow + g * 16);
  r.e = KV == MLA_DTYPE_MXFP4 ? p.e8m0[row * p.e8m0_stride + g] : 0;
  return r;
}

// Values 8 q .. 8 q + 7 of those, as bf16, exactly (e4m3 without the
// per-tensor scale).
template <int KV>
__device__ __forceinline__ uint4 decode(const Raw& r, int q) {
  if constexpr (KV == MLA_DTYPE_BF16) {
    return r.v;
  } else if constexpr (KV == MLA_DTYPE_FP8_E4M3) {
    auto two = [](uint32_t v) {
      const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(v));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      return bf16x2(f.x, f.y);
    };
    const uint32_t a = q ? r.v.z : r.v.x, b = q ? r.v.w : r.v.y;
    return make_uint4(two(a & 0xffffu), two(a >> 16), two(b & 0xffffu), two(b >> 16));
  } else {
    const uint32_t w = q == 0 ? r.v.x : q == 1 ? r.v.y : q == 2 ? r.v.z : r.v.w;
    const uint32_t s = e8m0_to_bf16x2(r.e);
    uint4 o;
    e2m1x4_to_bf16(w, s, o.x, o.y);
    e2m1x4_to_bf16(w >> 16, s, o.z, o.w);
    return o;
  }
}
// The same with the per-tensor scale, rounded.
__device__ __forceinline__ uint4 scaled(const uint4& v, float sc) {
  auto one = [&](uint32_t u) {
    return bf16x2(__uint_as_float(u << 16) * sc, __uint_as_float(u & 0xffff0000u) * sc);
  };
  return make_uint4(one(v.x), one(v.y), one(v.z), one(v.w));
}

// The tile of this CTA in tile pair `pair`; an odd last pair has an empty one,
// and so does a record that fails its check.
__device__ __forceinline__ ExpandTile tile_of(const ExpandParams& p, int pair, int rank) {
  const int i = 2 * pair + rank;
  const ExpandTile none{0, 0, 0, -1, 0u, {}};
  if (i >= p.num_tiles) return none;
  const int4 a = reinterpret_cast<const int4*>(p.tiles + i)[0];
  const ExpandTile t{a.x, a.y, a.z, a.w, p.tiles[i].check, {}};
  if (check_of(t, p.stamp) == t.check) return t;
  atomicOr(p.err, kErrStale);
  return none;
}

template <int KV>
__device__ void run_rows(const ExpandParams& p, ExpandMisc* ms, uint8_t* a_smem, int u0, int u1,
                         int rank, int tid) {
  // a chunk of a row is kLanes loads; this thread's rows are r0 + kStep i
  constexpr int kLanes = 64 / kPerLoad<KV>, kStep = 256 / kLanes, kRows = kPfTile / kStep;
  constexpr int kPieces = kPerLoad<KV> / 8;  // 16-byte pieces of bf16 that a load becomes
  const int g = tid % kLanes, r0 = tid / kLanes;
  const float sc = KV == MLA_DTYPE_FP8_E4M3 ? *p.kv_scale : 1.0f;
  uint32_t lap = 0;
  for (int u = u0; u < u1; ++lap) {
    const int pair = u / p.heads;
    const ExpandTile t = tile_of(p, pair, rank);
    int64_t row[kRows];
    bool live[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int tok = t.tok0 + r0 + kStep * i;
      live[i] = tok < t.len;
      row[i] = live[i] ? pool_row(p, t.page_base, tok) : 0;
    }
    Raw raw[kBatch<KV>][kRows];
    Raw last[kRows];                         // chunk 8: the rotated dims
    auto fetch = [&](Raw* r, int c) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (live[i]) r[i] = load_raw<KV>(p, row[i], kLanes * c + g);
    };
#pragma unroll
    for (int b = 0; b < kChunks; b += kBatch<KV>) {
#pragma unroll
      for (int k = 0; k < kBatch<KV>; ++k) fetch(raw[k], b + k);
      if (b + kBatch<KV> == kChunks) fetch(last, kChunks);
#pragma unroll
      for (int k = 0; k < kBatch<KV>; ++k) {
        const int c = b + k;
        if (lap > 0 && !mbar_wait(smem_u32(&ms->a_empty[c]), (lap - 1) & 1, p.err, kErrProducer))
          return;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = r0 + kStep * i;
#pragma unroll
          for (int q = 0; q < kPieces; ++q)
            *reinterpret_cast<uint4*>(a_smem + c * kAChunk + r * 128 +
                                      (((g * kPieces + q) ^ (r & 7)) << 4)) =
                live[i] ? decode<KV>(raw[k][i], q) : make_uint4(0, 0, 0, 0);
        }
        if (c % kFenced != kFenced - 1) continue;
        fence_proxy_async_smem();
        __syncwarp();
        if ((tid & 31) == 0)
          for (int d = c - kFenced + 1; d <= c; ++d) mbar_arrive(smem_u32(&ms->a_full[d]));
      }
    }
    if (u % p.heads == 0 && t.out_row >= 0) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        uint4* out = reinterpret_cast<uint4*>(
            p.kr + (static_cast<int64_t>(t.out_row) + r0 + kStep * i) * kRope);
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live[i]) v = decode<KV>(last[i], q);
          if (KV == MLA_DTYPE_FP8_E4M3) v = scaled(v, sc);
          out[g * kPieces + q] = v;
        }
      }
    }
    u = min(u1, (pair + 1) * p.heads);
  }
}

// In the odd CTA: passes the arrival of its rows on to the even one, whose
// products read them.  Ordinary shared memory goes to another CTA, so this is a
// release for the cluster, met by an acquire; a thread that does nothing else
// issues it, once for the chunks behind one proxy fence (with eight relaxed
// arrivals a tile the expansion took as long: 54 us of the ragged fp8 batch, 91
// of 32,845 MXFP4 keys).
__device__ void run_relay(const ExpandParams& p, ExpandMisc* ms, int u0, int u1) {
  uint32_t lap = 0;
  for (int u = u0; u < u1; ++lap) {
    for (int c = 0; c < kChunks; ++c) {
      if (!mbar_wait(smem_u32(&ms->a_full[c]), lap & 1, p.err, kErrProducer)) return;
      if (c % kFenced != kFenced - 1) continue;
      fence_proxy_async_smem();
      mbar_arrive_cluster_release(dsmem_addr(smem_u32(&ms->a_peer[c / kFenced]), 0));
    }
    u = min(u1, (u / p.heads + 1) * p.heads);
  }
}

__device__ void run_weights(const ExpandParams& p, ExpandMisc* ms, uint32_t w_smem, int u0, int u1,
                            int rank) {
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
      if (rank == 0) mbar_arrive_expect_tx(smem_u32(&ms->w_full[s]), 2 * kWChunk);
      tma_load_3d_pair(w_smem + s * kWChunk, &p.map_w, dsmem_addr(smem_u32(&ms->w_full[s]), 0),
                       64 * c, 128 * rank, h, keep);
    }
  }
  if (!ok && rank == 0)   // a wait gave up: no copy may land after the CTAs have gone
    for (uint32_t k = n > kWSlots ? n - kWSlots : 0; k < n; ++k)
      mbar_wait(smem_u32(&ms->w_full[k % kWSlots]), (k / kWSlots) & 1, p.err, kErrProducer);
}

// The whole warp (of the even CTA) walks the units; one lane issues.
__device__ void run_products(const ExpandParams& p, ExpandMisc* ms, uint32_t a_smem,
                             uint32_t w_smem, uint32_t tmem, int u0, int u1) {
  constexpr uint32_t idesc = make_idesc(1, 1, false, false, 256, kWRows);
  const uint64_t ad = smem_desc(a_smem, 16, 1024, kSwizzle128B);
  const uint64_t wd = smem_desc(w_smem, 16, 1024, kSwizzle128B);
  auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
  uint32_t slot = 0, phase = 0, lap = 0, k = 0;
  bool w_ready = false;
  int left = p.heads - uniform(u0 % p.heads);                // units of the present tiles
  bool first = true;                                         // of the tiles, here
  for (int u = u0; u < u1; ++u, ++k) {
    const bool last = u + 1 == u1 || left == 1;
    const uint32_t buf = k & 1;
    if (k >= 2 && !all(mbar_wait_cluster(smem_u32(&ms->acc_empty[buf]), ((k >> 1) - 1) & 1, p.err,
                                         kErrMma)))
      return;
    tc_fence_after();
    const uint32_t d = tmem + buf * kWRows;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (first) {
        if (!all(mbar_wait(smem_u32(&ms->a_full[c]), lap & 1, p.err, kErrMma))) return;
        if (c % kFenced == 0 &&
            !all(mbar_wait_cluster<true>(smem_u32(&ms->a_peer[c / kFenced]), lap & 1, p.err,
                                         kErrMma)))
          return;
      }
      if (!all(w_ready) &&
          !all(mbar_wait_poll(smem_u32(&ms->w_full[slot]), phase, p.err, kErrMma)))
        return;
      tc_fence_after();
      const uint64_t a = ad + ((c * kAChunk) >> 4), w = wd + ((slot * kWChunk) >> 4);
      const uint32_t s = slot;
      if (++slot == kWSlots) {
        slot = 0;
        phase ^= 1;
      }
      w_ready = mbar_test(smem_u32(&ms->w_full[slot]), phase);     // the next chunk's, ahead
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_pair(d, a + 2 * kk, w + 2 * kk, idesc, (c | kk) != 0);
        tc_commit_pair(smem_u32(&ms->w_empty[s]));
        if (last) tc_commit_pair(smem_u32(&ms->a_empty[c]));
      }
    }
    if (elect_one()) tc_commit_pair(smem_u32(&ms->acc_full[buf]));
    if (last) ++lap;
    first = last;
    left = left == 1 ? p.heads : left - 1;
  }
}

// Accumulators to bf16 rows of kx, 64 columns at a time through a box in shared
// memory and a bulk store: rows are 512 bytes apart, and a thread's own stores
// (a sector each) took about 250 cycles an instruction.
__device__ void run_epilogue(const ExpandParams& p, ExpandMisc* ms, uint8_t* boxes, uint32_t tmem,
                             int u0, int u1, int rank, int warp, int lane) {
  const float sc = p.kv_dtype == MLA_DTYPE_FP8_E4M3 ? *p.kv_scale : 1.0f;
  uint8_t* box = boxes + warp * 2 * kBox;
  uint32_t k = 0;
  for (int u = u0; u < u1; ++u, ++k) {
    const uint32_t buf = k & 1;
    const int pair = u / p.heads, h = u - pair * p.heads;
    const ExpandTile tile = tile_of(p, pair, rank);
    const int out_row = tile.out_row;                        // -1: no tile here
    const bool past = tile.tok0 + warp * 32 + lane >= tile.len;
    const bool ok = mbar_wait(smem_u32(&ms->acc_full[buf]), (k >> 1) & 1, p.err, kErrDrain);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after();
    const uint32_t acc = tmem + buf * kWRows + (static_cast<uint32_t>(warp) << 21);
    // 64 columns from x on, scaled and rounded to fp16 or bf16
    auto load = [&](auto half, int x, uint32_t (&v)[32]) {
      uint32_t f[64];
      tmem_ld32(acc + x, f);
      tmem_ld32(acc + x + 32, f + 32);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float lo = __uint_as_float(f[2 * i]) * sc, hi = __uint_as_float(f[2 * i + 1]) * sc;
        v[i] = decltype(half)::value ? half2_of(lo, hi) : bf16x2(lo, hi);
      }
    };
    const auto as_half = std::true_type();
    const auto as_bf16 = std::false_type();
    auto store = [&](int b, int x, const uint32_t (&v)[32]) {
      // the box's last store has read it (one lane keeps the groups)
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
      uint8_t* at = box + b * kBox + lane * 128;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(at + ((i ^ (lane & 7)) << 4)) =
            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (out_row >= 0)
          tma_store_3d(&p.map_kx, smem_u32(box + b * kBox), x, out_row + warp * 32, h);
        bulk_commit();
      }
    };
    // values first: whether they are finite decides what the key becomes, and
    // how large each row's are which type the warp's 32 rows take
    uint32_t v0[32], v1[32];
    load(as_half, kNope, v0);
    load(as_half, kNope + 64, v1);
    __half2 top2 = __floats2half2_rn(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      top2 = __hmax2_nan(top2, __habs2(*reinterpret_cast<const __half2*>(&v0[i])));
      top2 = __hmax2_nan(top2, __habs2(*reinterpret_cast<const __half2*>(&v1[i])));
    }
    // (bits of magnitudes have their order, infinity and NaN above all)
    uint32_t top = *reinterpret_cast<const uint32_t*>(&top2);
    top = max(top & 0x7fffu, (top >> 16) & 0x7fffu);
    bool finite = true;
    const uint32_t off = past ? 0u : top - 0x2400u;          // above 2^-6; below it wraps around
    const bool half = __reduce_max_sync(0xffffffffu, off) <= 0x7800u - 0x2400u;   // 2^15
    if (!half) {                             // not the common size: once more, to bf16
      load(as_bf16, kNope, v0);
      load(as_bf16, kNope + 64, v1);
      __nv_bfloat162 most = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v0[i])));
        most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v1[i])));
      }
      finite = __low2float(most) < INFINITY && __high2float(most) < INFINITY;
    }
    if (lane == 0 && out_row >= 0)
      p.v_half[(static_cast<int64_t>(h) * p.kx_rows + out_row) / kPfGroup + warp] = half ? 1 : 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v0[i] = finite ? v0[i] : 0u;
      v1[i] = finite ? v1[i] : 0u;
    }
    store(0, kNope, v0);
    store(1, kNope + 64, v1);
    load(as_bf16, 0, v0);
    load(as_bf16, 64, v1);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster_relaxed(dsmem_addr(smem_u32(&ms->acc_empty[buf]), 0));
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v0[i] = finite ? v0[i] : 0x7fc07fc0u;
      v1[i] = finite ? v1[i] : 0x7fc07fc0u;
    }
    store(0, 0, v0);
    store(1, 64, v1);
  }
  // the boxes stay until their stores are through, and the stores' rows are
  // there before the kernel counts as ended
  if (lane == 0) bulk_wait_all();
  __syncwarp();
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
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kChunks; ++i) {
      mbar_init(smem_u32(&ms->a_full[i]), 8);             // a warp's arrival each
      mbar_init(smem_u32(&ms->a_empty[i]), 1);
    }
    for (int i = 0; i < kChunks / kFenced; ++i) mbar_init(smem_u32(&ms->a_peer[i]), 1);
    for (int i = 0; i < kWSlots; ++i) {
      mbar_init(smem_u32(&ms->w_full[i]), 1);
      mbar_init(smem_u32(&ms->w_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ms->acc_full[i]), 1);
      mbar_init(smem_u32(&ms->acc_empty[i]), 2 * 4);      // a warp's arrival each
    }
    mbar_init(smem_u32(&ms->drain), 1);
    fence_mbar_init();
    ms->ours = reinterpret_cast<const WsHeader*>(p.err)->stamp == p.stamp ? 1 : 0;
    if (!ms->ours) atomicOr(p.err, kErrStale);
    else if (blockIdx.x == 0) *expanded_word(p.err) = 0;
  }
  if (warp == 13) {
    tmem_alloc_pair(smem_u32(&ms->tmem), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                       // the other CTA's barriers are set up too
  tc_fence_after();
  const uint32_t tmem = uniform(ms->tmem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (ms->ours) {
    const int64_t units = static_cast<int64_t>((p.num_tiles + 1) / 2) * p.heads;
    const int64_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int u0 = static_cast<int>(units * pair / pairs);
    const int u1 = static_cast<int>(units * (pair + 1) / pairs);
    if (warp < 4) {
      run_epilogue(p, ms, smem + kChunks * kAChunk + kWSlots * kWChunk, tmem, u0, u1, rank, warp,
                   lane);
    } else if (warp < 12) {
      run_rows<KV>(p, ms, smem, u0, u1, rank, threadIdx.x - 128);
    } else if (warp == 12) {
      if (lane == 0) run_weights(p, ms, w_smem, u0, u1, rank);
    } else if (rank == 0) {
      run_products(p, ms, a_smem, w_smem, tmem, uniform(u0), uniform(u1));
      // no product may run on after the CTAs have gone
      if (elect_one()) {
        tc_commit_pair(smem_u32(&ms->drain));
        mbar_wait(smem_u32(&ms->drain), 0, p.err, kErrDrain);
      }
    } else {
      if (lane == 0) run_relay(p, ms, u0, u1);
    }
    __syncwarp();
  }
  // Nothing here needs the rotation of the queries (a launch in full stream
  // order, behind everything that the expansion reads); what follows needs both.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();                       // nothing of the pair is under way any more
  if (warp == 13) tmem_dealloc_pair(tmem, 512);
}

template <int KV>
cudaError_t launch(const ExpandParams& p, int pairs, bool dependent, cudaStream_t stream) {
  constexpr int bytes = kExpandSmem + 1024;
  const cudaError_t e =
      cudaFuncSetAttribute(expand_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kExpandThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {2, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, expand_kernel<KV>, p);
}

}  // namespace

cudaError_t launch_expand(const ExpandParams& p, int num_ctas, bool dependent,
                          cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>((p.num_tiles + 1) / 2) * p.heads;
  const int64_t most = num_ctas >= 2 ? num_ctas / 2 : 1;
  const int pairs = static_cast<int>(units < most ? units : most);
  if (p.kv_dtype == MLA_DTYPE_BF16) return launch<MLA_DTYPE_BF16>(p, pairs, dependent, stream);
  if (p.kv_dtype == MLA_DTYPE_FP8_E4M3)
    return launch<MLA_DTYPE_FP8_E4M3>(p, pairs, dependent, stream);
  return launch<MLA_DTYPE_MXFP4>(p, pairs, dependent, stream);
}

}  // namespace mla
