// shared_api.cu -- host side of the shared-prefix decode: validation, the plan
// (the decode kernel's work over the requests' own ends, the prefix kernel's
// over the prefixes), workspace layout, tensor maps and launches.  The C
// declarations and their contracts are in include/mla_decode.h.

#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

#include "plan.h"
#include "shared.h"

using mla::CtaItems;
using mla::ExpandTile;
using mla::MeetJob;
using mla::PrefixItem;

struct mla_shared {
  int32_t bs = 0, groups = 0, q_len = 1, page_size = 0, num_sms = 0;
  int q_dtype = 0, kv_dtype = 0;
  bool paired = false;               // clusters of two score and two value CTAs, 256 rows
  bool direct = false;               // the prefix kernel reads the pool itself
  bool tall = false;                 // a tile's 128 keys stand together there
  bool each = false;                 // the decode kernel reads the prefixes for every request
  int32_t most = 0;                  // partial results of a token, at most
  int32_t blocks = 1;                // of 128 rows in an item
  int32_t num_clusters = 0, num_slots = 0;
  int64_t prefix_tokens = 0, identity_rows = 0;
  mla_plan* own = nullptr;           // over the requests' own ends (and, `each`, their prefixes),
                                     // partial results only
  std::vector<ExpandTile> tiles;
  std::vector<PrefixItem> items;
  std::vector<CtaItems> cluster_items;
  std::vector<MeetJob> jobs;
  size_t off_tiles = 0, off_clusters = 0, off_items = 0, off_jobs = 0, off_own = 0, off_rows = 0,
         off_part_o = 0, off_part_lse = 0, ws_bytes = 0;
  std::vector<uint8_t> table;
  uint64_t stamp = 0;
  mutable void* uploaded_ws = nullptr;
  const void* map_ptr = nullptr;     // rows of the tensor maps
  int64_t map_count = 0;
  CUtensorMap map_k, map_v;
  ~mla_shared() { mla_plan_destroy(own); }
};

namespace {

constexpr int32_t kTokensPerBlock = mla::kSpRows / mla::kHeads;

// What an item costs beside its tiles, in tiles: the queries' way into tensor
// memory, the first scores and the last values without the other half's work
// beside them, and the output take 20,000 cycles.  (256 requests on 8192 tokens:
// 87 us with 2, 85 with 5, 83 with 8.)
constexpr int64_t kItemCost = 8;

struct Block {
  int32_t q_row, rows, key0, keys;   // key0: row or key of the group's first key
  int32_t page_base;
};

// The blocks' key tiles, in order, cut into at most `clusters` ranges of nearly
// equal cost (kItemCost for each item, 1 for each tile).  The smallest largest
// cost that greedy ranges reach is found by bisection.
template <class Emit>
int64_t cut(const std::vector<Block>& blocks, int64_t cap, Emit&& emit) {
  int64_t ranges = 0, left = 0;
  for (size_t k = 0; k < blocks.size(); ++k) {
    const int64_t tiles = (blocks[k].keys + mla::kSpTile - 1) / mla::kSpTile;
    for (int64_t at = 0; at < tiles;) {
      if (left <= kItemCost) {
        left = cap;
        ++ranges;
      }
      const int64_t take = std::min(left - kItemCost, tiles - at);
      emit(k, at, take, ranges - 1);
      left -= kItemCost + take;
      at += take;
    }
  }
  return ranges;
}
int64_t smallest_cost(const std::vector<Block>& blocks, int64_t clusters) {
  int64_t total = 0;
  for (const Block& b : blocks) total += (b.keys + mla::kSpTile - 1) / mla::kSpTile;
  int64_t lo = kItemCost + 1, hi = kItemCost * (1 + static_cast<int64_t>(blocks.size())) + total;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (cut(blocks, mid, [](size_t, int64_t, int64_t, int64_t) {}) <= clusters) hi = mid; else lo = mid + 1;
  }
  return lo;
}
void cut_blocks(mla_shared* P, const std::vector<Block>& blocks, int64_t cost) {
  int64_t last = -1;
  cut(blocks, cost, [&](size_t k, int64_t at, int64_t take, int64_t range) {
    const Block& b = blocks[k];
    if (range != last) {
      const int32_t n = static_cast<int32_t>(P->items.size());
      if (last >= 0) P->cluster_items.back().end = n;
      P->cluster_items.push_back(CtaItems{n, n, 0u, 0});
      last = range;
    }
    PrefixItem w{};
    w.q_row = b.q_row;
    w.rows = b.rows;
    w.key0 = static_cast<int32_t>(b.key0 + at * mla::kSpTile);
    w.keys = static_cast<int32_t>(std::min<int64_t>(take * mla::kSpTile, b.keys - at * mla::kSpTile));
    w.slot = static_cast<int32_t>(P->items.size());       // a block's are consecutive
    w.page_base = b.page_base;
    P->items.push_back(w);
  });
  if (!P->cluster_items.empty()) P->cluster_items.back().end = static_cast<int32_t>(P->items.size());
  P->num_clusters = static_cast<int32_t>(P->cluster_items.size());
  P->num_slots = static_cast<int32_t>(P->items.size());
}

// Cycles of a tile in blocks of 128 and 256 rows.
double tile_cycles(const mla_shared* P, bool paired) {
  return paired ? 2600 : P->direct && P->page_size % mla::kSpTile != 0 ? 3900 : 3300;
}

// The decode kernel's time (us) on a number of CTAs: 9, and for each CTA its share of
// the items' beginnings and ends and of their tiles.  Linear fits to 324 calls of 16 to
// 512 items of up to 1,500 tokens on 8 to 64 CTAs (12% off, all in all).
struct DecodeWork {
  double item, tile, sum;
  explicit DecodeWork(const mla_shared* P) : sum(0) {
    const bool pairs = P->own->rows > mla::kHeads;       // two query tokens an item
    switch (P->kv_dtype) {
      case MLA_DTYPE_BF16: item = 0.8, tile = 4.1; break;
      case MLA_DTYPE_MXFP4: item = 1.5, tile = 2.6; break;
      default:
        if (P->q_dtype == MLA_DTYPE_BF16)
          item = pairs ? 5.0 : 3.5, tile = pairs ? 2.9 : 1.8;
        else
          item = pairs ? 2.7 : 1.2, tile = pairs ? 2.6 : 2.0;
    }
  }
  void add(int64_t items, int64_t tiles) {
    sum += item * static_cast<double>(items) + tile * static_cast<double>(tiles);
  }
  double on(int64_t ctas) const { return 9 + sum / static_cast<double>(ctas); }
};

// How the prefixes' tiles are cut (the largest cost of a cluster), and for how many CTAs
// the requests' own ends.  Those run beside the prefix kernel on the SMs that it leaves
// and are not to last longer than it does: with fewer clusters, where that takes less
// time in all, or else (0) cut for all SMs, to come behind it.  `us`: until both are
// through.  64 requests with 256 own tokens on average behind 32,768: 64 us on 32
// clusters, 73 on 36; 128 behind 4,096: 39 on 24, 47 on 32.  Over 93 calls 11% less
// than with all clusters, and within 1% of the best of six settings of these estimates.
int64_t choose_cut(const mla_shared* P, const std::vector<Block>& blocks, const DecodeWork& own,
                   int32_t* own_ctas, double* us) {
  const double cost_us = tile_cycles(P, P->paired) / 1900;
  const int64_t most = P->num_clusters;
  int64_t best = smallest_cost(blocks, most);
  *own_ctas = 0;
  *us = static_cast<double>(best) * cost_us;
  if (own.sum == 0) return best;
  *us += own.on(P->num_sms);
  const int64_t step = std::max<int64_t>(1, most / 64);
  for (int64_t n = most; n >= std::max<int64_t>(1, most / 2); n -= step) {
    const int64_t idle = P->num_sms - n * (P->paired ? 4 : 2);
    if (idle <= 0) continue;
    const int64_t cost = smallest_cost(blocks, n);
    const double t = std::max(static_cast<double>(cost) * cost_us, own.on(idle));
    if (t >= *us) continue;
    *us = t;
    best = cost;
    *own_ctas = static_cast<int32_t>(idle);
  }
  return best;
}

// Whether to work in blocks of 256 rows, and on how many clusters at most.  A tile of
// 128 keys takes 2,600 cycles on a paired cluster and 3,300 on another (3,900 with boxes
// of 64 keys), but blocks of 256 rows may leave half of one empty, and 36 clusters of
// four have a place where 76 of two have.  64 requests of a 32,768-token prefix: 73 us
// paired, 87 not; 5 to 19 requests of three prefixes: 40 us paired, 39 not.
void choose_blocks(mla_shared* P, const int32_t* group_indptr, const int32_t* prefix_indptr,
                   bool whole_device) {
  int32_t on_device[2] = {P->num_sms / 2, P->num_sms / 4};
  if (whole_device)
    for (int k = 0; k < 2; ++k) {
      const int32_t n = mla::prefix_clusters(k == 1);
      if (n > 0) on_device[k] = std::min(on_device[k], n);
    }
  double time[2] = {0, 0};
  for (int32_t g = 0; g < P->groups; ++g) {
    const int64_t keys = (static_cast<int64_t>(prefix_indptr[g + 1]) - prefix_indptr[g]) * P->page_size;
    const int64_t tokens = static_cast<int64_t>(group_indptr[g + 1] - group_indptr[g]) * P->q_len;
    const int64_t tiles = (keys + mla::kSpTile - 1) / mla::kSpTile;
    for (int k = 0; k < 2; ++k) {
      const int64_t per = (k + 1) * kTokensPerBlock;
      time[k] += static_cast<double>(tiles * ((tokens + per - 1) / per)) * tile_cycles(P, k == 1) /
                 std::max(1, on_device[k]);
    }
  }
  P->paired = on_device[1] > 0 && time[1] < time[0];
  P->blocks = P->paired ? 2 : 1;
  P->tall = !P->paired && (!P->direct || P->page_size % mla::kSpTile == 0);
  P->num_clusters = std::max(1, on_device[P->paired]);
}

mla_status make_plan(mla_shared* P, const int32_t* group_indptr, const int32_t* prefix_indptr,
                     const int32_t* kv_indptr, const int32_t* last_len, mla_shared_form form) {
  const int32_t t = P->q_len, per_block = P->blocks * kTokensPerBlock;
  const int32_t per_request = P->own->bs / P->bs;        // items: query tokens, or pairs
  std::vector<int32_t> each_base(P->bs, 0), each_pages(P->bs, 0);
  DecodeWork own(P);
  for (const mla::WorkItem& w : P->own->items) own.add(w.tok_begin == 0, 0);
  own.add(0, P->own->total_tiles);
  DecodeWork each = own;
  int64_t gathered = 0;
  std::vector<Block> blocks;
  std::vector<int32_t> block_of(P->bs, -1), first_of(P->bs, 0);   // first: the group's first token
  int64_t rows = 0;
  for (int32_t g = 0; g < P->groups; ++g) {
    const int64_t np = static_cast<int64_t>(prefix_indptr[g + 1]) - prefix_indptr[g];
    const int32_t b0 = group_indptr[g], b1 = group_indptr[g + 1];
    if (np < 0 || b1 < b0) return MLA_ERR_INVALID_ARG;
    const int64_t keys = np * P->page_size;
    if (keys == 0) continue;
    if (rows + keys > INT32_MAX - mla::kSpTile) return MLA_ERR_INVALID_ARG;
    if (b1 == b0) continue;
    P->identity_rows = std::max(P->identity_rows,
                                (static_cast<int64_t>(prefix_indptr[g]) + np) * P->page_size);
    P->prefix_tokens += keys;
    for (int32_t b = b0; b < b1; ++b) {
      // every query token sees the whole prefix
      int64_t n = (static_cast<int64_t>(kv_indptr[b + 1]) - kv_indptr[b]) * P->page_size;
      if (n > 0 && last_len != nullptr) n -= P->page_size - last_len[b];
      if (n < t - 1) return MLA_ERR_INVALID_ARG;
      each_base[b] = prefix_indptr[g];
      each_pages[b] = static_cast<int32_t>(np);
      each.add(per_request, per_request * ((keys + mla::kTile - 1) / mla::kTile));
      block_of[b] = static_cast<int32_t>(blocks.size());
      first_of[b] = b0 * t;
    }
    const int64_t tokens = static_cast<int64_t>(b1 - b0) * t;
    for (int64_t a = 0; a < tokens; a += per_block) {
      Block b;
      b.q_row = static_cast<int32_t>((static_cast<int64_t>(b0) * t + a) * mla::kHeads);
      b.rows = static_cast<int32_t>(std::min<int64_t>(per_block, tokens - a) * mla::kHeads);
      b.key0 = P->direct ? 0 : static_cast<int32_t>(rows);
      b.page_base = prefix_indptr[g];
      b.keys = static_cast<int32_t>(keys);
      blocks.push_back(b);
    }
    if (P->direct) continue;
    gathered += keys;
    for (int64_t k = 0; k < keys; k += mla::kSpTile) {
      ExpandTile e{};
      e.page_base = prefix_indptr[g];
      e.tok0 = static_cast<int32_t>(k);
      e.len = static_cast<int32_t>(keys);
      e.out_row = static_cast<int32_t>(rows + k);
      P->tiles.push_back(e);
    }
    rows += (keys + mla::kSpTile - 1) / mla::kSpTile * mla::kSpTile;
  }
  // Whether the prefixes are to be read for every request instead, by the decode
  // kernel, which has no rows to gather and fewer kernels in a row.  (us; fitted to 259
  // calls of both forms: 1 to 5 groups, 2 to 128 requests, prefixes of 64 to 32,768
  // tokens, all types, 1 to 4 query tokens.  The form taken is 0.5% slower than the
  // better one on average, by more than a tenth in 3 of them.  8 requests of 1,024 e4m3
  // tokens: 12.5 us each on its own, 22.7 once for all; 32 of 16,384: 55 and 39; 128 of
  // 16,384: 181 and 68.)
  int32_t own_ctas = 0;
  double once_us = 0;
  const int64_t cost = choose_cut(P, blocks, own, &own_ctas, &once_us);
  once_us += 8 + 0.33e-3 * static_cast<double>(gathered) + 6.0 * P->bs * t / P->num_sms;
  P->each = form == MLA_SHARED_EACH || (form == MLA_SHARED_AUTO && each.on(P->num_sms) + 3 < once_us);
  if (P->each) {
    own_ctas = 0;
    blocks.clear();
    P->tiles.clear();
    block_of.assign(P->bs, -1);
  }
  cut_blocks(P, blocks, cost);
  if (P->each || own_ctas > 0) {
    mla_plan_destroy(P->own);
    P->own = nullptr;
    const mla_plan_options o{0, own_ctas > 0 ? own_ctas : P->num_sms, 0, 0, 1};
    const mla::PrefixPages prefixes{each_base.data(), each_pages.data()};
    const mla_status st = mla::plan_with_prefixes(kv_indptr, last_len, P->bs, t, P->page_size,
                                                  static_cast<mla_dtype>(P->q_dtype),
                                                  static_cast<mla_dtype>(P->kv_dtype), &o,
                                                  P->each ? &prefixes : nullptr, &P->own);
    if (st != MLA_OK) return st;
  }
  // partial results of every block, then of every query token
  std::vector<int32_t> first_slot(blocks.size(), 0), slots(blocks.size(), 0);
  {
    size_t k = 0;
    int64_t left = blocks.empty() ? 0 : blocks[0].keys;
    for (size_t i = 0; i < P->items.size(); ++i) {
      if (slots[k]++ == 0) first_slot[k] = static_cast<int32_t>(i);
      left -= P->items[i].keys;
      if (left == 0 && ++k < blocks.size()) left = blocks[k].keys;
    }
  }
  std::vector<int32_t> own_first, own_count;
  mla::plan_partials_only(P->own, &own_first, &own_count);
  const bool two = P->own->rows == 2 * mla::kHeads;      // tokens of a request in pairs
  for (int32_t b = 0; b < P->bs; ++b)
    for (int32_t i = 0; i < t; ++i) {
      MeetJob j{};
      const int32_t r = two ? b * (t / 2) + i / 2 : b * t + i;
      j.own_first = own_first[r];
      j.own_count = own_count[r];
      j.own_row = two ? i % 2 * mla::kHeads : 0;
      if (block_of[b] >= 0) {
        const int32_t in = b * t + i - first_of[b], k = block_of[b] + in / per_block;
        j.prefix_first = first_slot[k] * P->blocks + in % per_block / kTokensPerBlock;
        j.prefix_count = slots[k];
        j.prefix_row = in % kTokensPerBlock * mla::kHeads;
      }
      P->most = std::max(P->most, j.own_count + j.prefix_count);
      P->jobs.push_back(j);
    }
  size_t off = sizeof(mla::PrefillHeader);
  auto take = [&](size_t bytes) {
    const size_t at = (off + 255) & ~static_cast<size_t>(255);
    off = (at + bytes + 255) & ~static_cast<size_t>(255);
    return at;
  };
  P->off_tiles = take(sizeof(ExpandTile) * P->tiles.size());
  P->off_clusters = take(sizeof(CtaItems) * P->cluster_items.size());
  P->off_items = take(sizeof(PrefixItem) * P->items.size());
  P->off_jobs = take(sizeof(MeetJob) * P->jobs.size());
  P->table.assign(off, 0);
  P->off_own = take(P->own->ws_bytes);
  P->off_rows = take(sizeof(uint16_t) * P->tiles.size() * mla::kSpTile * mla::kQkDim);
  P->off_part_o = take(sizeof(float) * P->num_slots * P->blocks * mla::kSpRows * mla::kVDim);
  P->off_part_lse = take(sizeof(float) * P->num_slots * P->blocks * mla::kSpRows);
  P->ws_bytes = off;
  P->stamp = mla::new_plan_stamp();
  mla::PrefillHeader hdr{};
  hdr.ws.stamp = P->stamp;
  std::memcpy(P->table.data(), &hdr, sizeof(hdr));
  auto put = [&](size_t at, auto& records) {
    for (auto& r : records) r.check = mla::check_of(r, P->stamp);
    if (!records.empty())
      std::memcpy(P->table.data() + at, records.data(), sizeof(records[0]) * records.size());
  };
  put(P->off_tiles, P->tiles);
  put(P->off_clusters, P->cluster_items);
  put(P->off_items, P->items);
  put(P->off_jobs, P->jobs);
  return MLA_OK;
}

// bf16 rows as {64 dims, rows, 9 panels} with the 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* rows, int64_t count, uint32_t box_rows,
              uint32_t box_panels) {
  const mla::TiledEncoder enc = mla::tiled_encoder();
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(count), mla::kQkDim / 64};
  const cuuint64_t strides[2] = {mla::kQkDim * 2, 128};
  const cuuint32_t box[3] = {64, box_rows, box_panels}, one[3] = {1, 1, 1};
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(rows), dims, strides, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

mla_status mla_shared_plan(const int32_t* group_indptr_host, const int32_t* prefix_indptr_host,
                           int32_t num_groups, const int32_t* kv_indptr_host,
                           const int32_t* kv_last_page_len_host, int32_t q_len, int32_t page_size,
                           mla_dtype q_dtype, mla_dtype kv_dtype, int32_t num_sms,
                           mla_shared_form form, mla_shared** plan_out) {
  if (plan_out == nullptr) return MLA_ERR_INVALID_ARG;
  *plan_out = nullptr;
  if (form < MLA_SHARED_AUTO || form > MLA_SHARED_EACH) return MLA_ERR_INVALID_ARG;
  if (group_indptr_host == nullptr || prefix_indptr_host == nullptr || kv_indptr_host == nullptr ||
      num_groups < 1 || num_sms < 0)
    return MLA_ERR_INVALID_ARG;
  if (group_indptr_host[0] != 0 || prefix_indptr_host[0] < 0) return MLA_ERR_INVALID_ARG;
  for (int32_t g = 0; g < num_groups; ++g)
    if (group_indptr_host[g + 1] < group_indptr_host[g]) return MLA_ERR_INVALID_ARG;
  const bool whole_device = num_sms == 0;
  if (whole_device) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return MLA_ERR_CUDA;
  }
  mla_shared* P = nullptr;
  mla_status st = MLA_ERR_INVALID_ARG;
  try {
    P = new mla_shared();
    P->bs = group_indptr_host[num_groups];
    P->groups = num_groups;
    P->q_len = q_len;
    P->page_size = page_size;
    P->num_sms = num_sms;
    P->q_dtype = q_dtype;
    P->kv_dtype = kv_dtype;
    // (its rows are the tensor map's, 64 of them always on one page)
    P->direct = kv_dtype == MLA_DTYPE_BF16 && page_size % 64 == 0;
    // (checks the batch's lengths, query tokens, page size and types)
    const mla_plan_options o{0, num_sms, 0, 0, 1};
    st = mla_decode_plan_ex(kv_indptr_host, kv_last_page_len_host, P->bs, q_len, page_size, q_dtype,
                            kv_dtype, &o, &P->own);
    if (st == MLA_OK) {
      choose_blocks(P, group_indptr_host, prefix_indptr_host, whole_device);
      st = make_plan(P, group_indptr_host, prefix_indptr_host, kv_indptr_host, kv_last_page_len_host,
                     form);
    }
  } catch (...) {   // out of host memory
    st = MLA_ERR_INVALID_ARG;
  }
  if (st != MLA_OK) {
    delete P;
    return st;
  }
  *plan_out = P;
  return MLA_OK;
}

mla_status mla_shared_get_info(const mla_shared* plan, mla_shared_info* info) {
  if (plan == nullptr || info == nullptr) return MLA_ERR_INVALID_ARG;
  info->batch_size = plan->bs;
  info->num_groups = plan->groups;
  info->q_len = plan->q_len;
  info->num_clusters = plan->num_clusters;
  info->block_rows = plan->blocks * mla::kSpRows;
  info->num_items = static_cast<int32_t>(plan->items.size());
  info->prefix_tokens = plan->prefix_tokens;
  info->own_tokens = plan->own->total_tokens;
  info->workspace_bytes = plan->ws_bytes;
  return MLA_OK;
}

void mla_shared_destroy(mla_shared* plan) { delete plan; }

mla_status mla_shared_run(mla_shared* plan, const void* q, const float* q_scale, const void* kv,
                          const float* kv_scale, const uint8_t* kv_e8m0, int64_t kv_e8m0_row_stride,
                          int64_t kv_pool_rows, const int32_t* prefix_indices,
                          const int32_t* kv_indices, void* workspace, size_t workspace_bytes,
                          void* out, float* lse, mla_stream_t stream_) {
  using mla::ptr_aligned;
  if (plan == nullptr || q == nullptr || kv == nullptr || out == nullptr || workspace == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(workspace, 256) || !ptr_aligned(q, 16) || !ptr_aligned(kv, 16) ||
      !ptr_aligned(out, 16) || !ptr_aligned(lse, 4) || !ptr_aligned(q_scale, 4) ||
      !ptr_aligned(kv_scale, 4) || !ptr_aligned(prefix_indices, 4) || !ptr_aligned(kv_indices, 4))
    return MLA_ERR_INVALID_ARG;
  if (kv_pool_rows < 1 || kv_pool_rows > INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (plan->q_dtype == MLA_DTYPE_FP8_E4M3 && q_scale == nullptr) return MLA_ERR_INVALID_ARG;
  if (plan->kv_dtype == MLA_DTYPE_FP8_E4M3 && kv_scale == nullptr) return MLA_ERR_INVALID_ARG;
  if (plan->kv_dtype == MLA_DTYPE_MXFP4) {
    if (kv_e8m0 == nullptr || kv_e8m0_row_stride < 18) return MLA_ERR_INVALID_ARG;
    if (kv_e8m0_row_stride % 2 != 0 || !ptr_aligned(kv_e8m0, 2)) return MLA_ERR_UNSUPPORTED;
  }
  if (workspace_bytes < plan->ws_bytes) return MLA_ERR_WORKSPACE;
  if (prefix_indices == nullptr ? plan->identity_rows > kv_pool_rows
                                : kv_pool_rows % plan->page_size != 0)
    return MLA_ERR_INVALID_ARG;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  // the requests' own ends: everything that can be refused comes before the
  // first launch
  mla::DecodeLaunch own{};
  const mla_status st = mla::decode_prepare(
      plan->own, q, q_scale, kv, kv_scale, kv_e8m0, kv_e8m0_row_stride, kv_pool_rows, kv_indices,
      plan->each ? prefix_indices : nullptr, ws + plan->off_own, plan->own->ws_bytes, out, nullptr,
      stream, &own);
  if (st != MLA_OK) return st;
  if (plan->uploaded_ws != workspace) {
    if (cudaMemcpyAsync(ws, plan->table.data(), plan->table.size(), cudaMemcpyHostToDevice,
                        stream) != cudaSuccess)
      return MLA_ERR_CUDA;
    plan->uploaded_ws = workspace;
  }
  int32_t* err = reinterpret_cast<int32_t*>(ws);
  uint16_t* rows = reinterpret_cast<uint16_t*>(ws + plan->off_rows);
  float* part_o = reinterpret_cast<float*>(ws + plan->off_part_o);
  float* part_lse = reinterpret_cast<float*>(ws + plan->off_part_lse);
  if (plan->num_clusters > 0) {
    const void* map_rows = plan->direct ? kv : rows;
    const int64_t count = plan->direct ? kv_pool_rows
                                       : static_cast<int64_t>(plan->tiles.size()) * mla::kSpTile;
    if (plan->map_ptr != map_rows || plan->map_count != count) {
      plan->map_ptr = nullptr;
      if (!make_map(&plan->map_k, map_rows, count, plan->tall ? 128 : 64, 1) ||
          !make_map(&plan->map_v, map_rows, count, 64, plan->paired ? 2 : 4))
        return MLA_ERR_CUDA;
      plan->map_ptr = map_rows;
      plan->map_count = count;
    }
    mla::GatherParams g{};
    g.tiles = reinterpret_cast<const ExpandTile*>(ws + plan->off_tiles);
    g.num_tiles = static_cast<int32_t>(plan->tiles.size());
    g.kv = static_cast<const uint8_t*>(kv);
    g.e8m0 = kv_e8m0;
    g.e8m0_stride = kv_e8m0_row_stride;
    g.pool_rows = kv_pool_rows;
    g.indices = prefix_indices;
    g.page_size = plan->page_size;
    g.kv_dtype = plan->kv_dtype;
    g.rows = rows;
    g.err = err;
    g.stamp = plan->stamp;
    if (!plan->direct && mla::launch_gather(g, stream) != cudaSuccess) return MLA_ERR_CUDA;
    mla::PrefixParams p{};
    p.map_k = plan->map_k;
    p.map_v = plan->map_v;
    p.items = reinterpret_cast<const PrefixItem*>(ws + plan->off_items);
    p.clusters = reinterpret_cast<const CtaItems*>(ws + plan->off_clusters);
    p.direct = plan->direct ? 1 : 0;
    p.tall = plan->tall ? 1 : 0;
    p.page_size = plan->page_size;
    p.indices = prefix_indices;
    p.pool_rows = kv_pool_rows;
    p.q = q;
    p.q_fp8 = plan->q_dtype == MLA_DTYPE_FP8_E4M3 ? 1 : 0;
    p.q_scale = p.q_fp8 ? q_scale : nullptr;
    p.kv_scale = plan->kv_dtype == MLA_DTYPE_FP8_E4M3 ? kv_scale : nullptr;
    p.part_o = part_o;
    p.part_lse = part_lse;
    p.err = err;
    p.stamp = plan->stamp;
    if (mla::launch_prefix(p, plan->paired, plan->num_clusters, stream) != cudaSuccess)
      return MLA_ERR_CUDA;
    own.stage1.beside = 1;
  } else {
    own.stage1.beside = 2;
  }
  if (mla::decode_launch(plan->own, own, stream) != MLA_OK) return MLA_ERR_CUDA;
  mla::MeetParams m{};
  m.jobs = reinterpret_cast<const MeetJob*>(ws + plan->off_jobs);
  m.tokens = static_cast<int64_t>(plan->bs) * plan->q_len;
  m.own_o = reinterpret_cast<const float*>(ws + plan->off_own + plan->own->off_part_o);
  m.own_lse = reinterpret_cast<const float*>(ws + plan->off_own + plan->own->off_part_lse);
  m.own_rows = plan->own->rows;
  m.blocks = plan->blocks;
  m.most = plan->most;
  m.alone = plan->num_clusters == 0 && plan->own->num_ctas == 0 ? 1 : 0;
  m.prefix_o = part_o;
  m.prefix_lse = part_lse;
  m.out = static_cast<uint16_t*>(out);
  m.lse = lse;
  m.err = err;
  m.stamp = plan->stamp;
  return mla::launch_meet(m, stream) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status mla_shared_check(const mla_shared* plan, void* workspace, mla_stream_t stream_) {
  if (plan == nullptr || workspace == nullptr) return MLA_ERR_INVALID_ARG;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const mla_status own =
      mla_decode_check(plan->own, static_cast<uint8_t*>(workspace) + plan->off_own, stream_);
  int32_t word = 0;
  if (cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, stream) !=
          cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (word == 0) return own;
  if (cudaMemsetAsync(workspace, 0, sizeof(word), stream) != cudaSuccess) return MLA_ERR_CUDA;
  if (word & mla::kErrStale) {
    if (plan->uploaded_ws == workspace) plan->uploaded_ws = nullptr;
    return MLA_ERR_WORKSPACE;
  }
  if (own != MLA_OK) return own;
  return (word & mla::kErrTimeout) ? MLA_ERR_DEVICE_TIMEOUT : MLA_ERR_INVALID_ARG;
}

}  // extern "C"
