// prefill_api.cu -- host side of the expanded form: the plan (expansion
// tiles, attention items and their assignment to CTAs, join jobs), workspace
// layout, argument checks and launches.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <functional>
#include <new>
#include <queue>
#include <vector>

#include "plan.h"
#include "prefill.h"

struct mla_prefill {
  int32_t bs = 0, heads = 0, page_size = 0, kv_dtype = 0, num_sms = 0;
  int32_t num_ctas = 0, num_pairs = 0, num_partials = 0;
  int64_t q_tokens = 0, k_tokens = 0, kx_rows = 0, identity_rows = 0;
  std::vector<mla::ExpandTile> tiles;
  // items of CTAs on their own, then of CTA pairs, each list by CTA or pair
  std::vector<mla::CtaItems> cta_items, pair_items;
  std::vector<mla::AttnItem> items;
  std::vector<uint32_t> item_checks;
  std::vector<mla::JoinJob> jobs;
  size_t off_tiles = 0, off_ctas = 0, off_pairs = 0, off_items = 0, off_checks = 0,
         off_jobs = 0, off_kx = 0, off_kr = 0, off_vh = 0, off_qr = 0, off_part_o = 0, off_part_lse = 0, ws_bytes = 0;
  std::vector<uint8_t> table;
  uint64_t stamp = 0;
  // per-run caches: the workspace holding the table, the tensor maps and what they describe
  mutable void* uploaded_ws = nullptr;
  CUtensorMap map_q, map_qr, map_kx, map_kr, map_kx_out, map_w;
  const void* map_w_ptr = nullptr;
  const void* map_q_ptr = nullptr;
  int64_t map_q_ts = 0, map_q_hs = 0;
  void* map_ws = nullptr;
};

namespace {

using mla::AttnItem;
using mla::CtaItems;
using mla::ExpandTile;
using mla::JoinJob;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Costs of the assignment, in tenths of one 128-key step of an item at full
// width (256 rows on a CTA, 512 on a pair).
constexpr int64_t kStepCost = 10;     // (one query tile at work costs no less: nothing runs
                                      // under its softmax)
constexpr int64_t kItemCost = 15;     // prologue and epilogue of an item
constexpr int64_t kJoinCost = 40;     // a join launch, once
constexpr int64_t kLaunchCost = 40;   // a second attention kernel, once
constexpr int64_t kPairRows = 384;    // a pair's item needs more query rows than this: half of
                                      // its second tile must be there to be worth two CTAs

constexpr int64_t kMaxItems = INT32_MAX / 64;   // whole items of a plan

int64_t item_tiles(const AttnItem& w) {
  return (static_cast<int64_t>(w.kv_end) - w.kv_begin + mla::kPfTile - 1) / mla::kPfTile;
}
int64_t item_steps(const AttnItem& w) {
  return mla::halved(w) ? (item_tiles(w) + 1) / 2 : item_tiles(w);
}
int64_t item_cost(const AttnItem& w) { return kItemCost + item_steps(w) * kStepCost; }

// Number of ranges of at most `limit` steps that an item is cut into, or 0 to
// leave it whole.  At most 128 rows are halved when cut, even into one range.
int64_t parts_of(const AttnItem& w, int64_t limit) {
  const int64_t tiles = item_tiles(w);
  if (tiles <= limit) return 0;
  return w.rows <= mla::kPfTile ? (tiles + 2 * limit - 1) / (2 * limit)
                                : (tiles + limit - 1) / limit;
}

// Longest first, each to the CTA with the least so far: the largest sum, and
// (out != null) the assignment.
int64_t assign(const std::vector<AttnItem>& items, const std::vector<int64_t>& cost, int32_t ctas,
               std::vector<std::vector<int32_t>>* out) {
  std::vector<int32_t> order(items.size());
  for (size_t i = 0; i < order.size(); ++i) order[i] = static_cast<int32_t>(i);
  std::stable_sort(order.begin(), order.end(),
                   [&](int32_t a, int32_t b) { return cost[a] > cost[b]; });
  typedef std::pair<int64_t, int32_t> Load;
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> heap;
  for (int32_t c = 0; c < ctas; ++c) heap.push({0, c});
  int64_t most = 0;
  for (const int32_t i : order) {
    Load l = heap.top();
    heap.pop();
    l.first += cost[i];
    most = std::max(most, l.first);
    if (out != nullptr) (*out)[l.second].push_back(i);
    heap.push(l);
  }
  return most;
}

// The items with every item of more than `limit` key tiles cut into equal ranges.
std::vector<AttnItem> cut_items(const std::vector<AttnItem>& whole, int64_t limit) {
  std::vector<AttnItem> out;
  for (const AttnItem& w : whole) {
    const int64_t n = item_tiles(w), cut = parts_of(w, limit), parts = std::max<int64_t>(cut, 1);
    for (int64_t s = 0; s < parts; ++s) {
      AttnItem v = w;
      v.kv_begin = w.kv_begin + static_cast<int32_t>(n * s / parts) * mla::kPfTile;
      if (s + 1 < parts)
        v.kv_end = w.kv_begin + static_cast<int32_t>(n * (s + 1) / parts) * mla::kPfTile;
      v.slot = cut > 0 ? 0 : -1;
      out.push_back(v);
    }
  }
  return out;
}

std::vector<int64_t> costs_of(const std::vector<AttnItem>& items) {
  std::vector<int64_t> c(items.size());
  for (size_t i = 0; i < items.size(); ++i) c[i] = item_cost(items[i]);
  return c;
}

// A list of items assigned to CTAs (or pairs).
struct Schedule {
  std::vector<AttnItem> items;      // by CTA
  std::vector<CtaItems> of_cta;
  std::vector<JoinJob> jobs;
  int32_t ctas = 0, partials = 0;
  int64_t most = 0;                 // the largest sum of costs
};

// Cuts the items' keys where that ends sooner on `ctas` CTAs (or pairs), gives
// the parts their slots, from `slot0` on, and join jobs and lists the items by
// CTA.
Schedule schedule(const std::vector<AttnItem>& whole, int32_t ctas, int32_t slot0) {
  Schedule S;
  if (whole.empty()) return S;
  // Cut limit: the one whose longest-first assignment ends first.  With many
  // more items than CTAs and none of them long, no cut can help.
  int64_t total = 0, longest = 0, max_tiles = 0;
  for (const AttnItem& w : whole) {
    total += item_cost(w);
    longest = std::max(longest, item_cost(w));
    max_tiles = std::max(max_tiles, item_tiles(w));
  }
  int64_t best_limit = INT32_MAX;
  if (2 * longest > std::max<int64_t>(1, total / ctas)) {
    int64_t best = assign(whole, costs_of(whole), ctas, nullptr), seen = 0;
    for (int64_t k = 2; k <= 128 && (max_tiles + k - 1) / k >= 4; ++k) {
      const int64_t limit = (max_tiles + k - 1) / k;
      if (limit == seen) continue;
      seen = limit;
      const std::vector<AttnItem> cut = cut_items(whole, limit);
      if (cut.size() > whole.size() + 16u * ctas) break;
      const int64_t most = assign(cut, costs_of(cut), ctas, nullptr) + kJoinCost;
      if (most < best) {
        best = most;
        best_limit = limit;
      }
    }
  }
  std::vector<AttnItem> items = cut_items(whole, best_limit);
  // slots, in item order: the parts of a whole item are neighbours
  for (size_t i = 0; i < items.size();) {
    size_t e = i + 1;
    if (items[i].slot >= 0) {
      while (e < items.size() && items[e].q_row == items[i].q_row &&
             items[e].head == items[i].head)
        ++e;
      // slots of a partial result, and partial results of a part
      const int32_t span = (items[i].rows + mla::kPfRows - 1) / mla::kPfRows;
      const int32_t each = mla::halved(items[i]) ? 2 : 1;
      S.jobs.push_back(JoinJob{items[i].q_row, items[i].rows, items[i].head, slot0 + S.partials,
                               static_cast<int32_t>(e - i) * each, items[i].vis0, span, 0u});
      for (size_t j = i; j < e; ++j) {
        items[j].slot = slot0 + S.partials;
        S.partials += span * each;
      }
    }
    i = e;
  }
  S.ctas = static_cast<int32_t>(std::min<size_t>(ctas, items.size()));
  std::vector<std::vector<int32_t>> of(S.ctas);
  S.most = assign(items, costs_of(items), S.ctas, &of) + (S.jobs.empty() ? 0 : kJoinCost);
  for (const std::vector<int32_t>& l : of) {
    const int32_t begin = static_cast<int32_t>(S.items.size());
    for (const int32_t i : l) S.items.push_back(items[i]);
    S.of_cta.push_back(CtaItems{begin, static_cast<int32_t>(S.items.size()), 0u, 0});
  }
  return S;
}

// The items of a request's m query rows on one head each: blocks of 512 rows
// for pairs while more than `pair_rows` are left, then of 256.
void add_items(std::vector<AttnItem>* pairs, std::vector<AttnItem>* singles, int64_t pair_rows,
               int32_t q_row, int64_t m, int64_t n, int64_t kv_row, int32_t heads) {
  for (int64_t r0 = 0; r0 < m;) {
    const bool pair = m - r0 > pair_rows;
    AttnItem w{};
    w.q_row = q_row + static_cast<int32_t>(r0);
    w.rows = static_cast<int32_t>(std::min<int64_t>((pair ? 2 : 1) * mla::kPfRows, m - r0));
    w.kv_row = static_cast<int32_t>(kv_row);
    w.vis0 = static_cast<int32_t>(n - m + 1 + r0);
    w.kv_end = std::max(0, w.vis0 + w.rows - 1);
    w.slot = -1;
    for (int32_t h = 0; h < heads; ++h) {
      w.head = h;
      (pair ? pairs : singles)->push_back(w);
    }
    r0 += w.rows;
  }
}

mla_status make_plan(mla_prefill* P, const int32_t* qo, const int32_t* kvp, const int32_t* last) {
  // every row on CTAs on their own, or blocks of 512 rows on pairs and the rest so
  std::vector<AttnItem> all, pairs, rest;
  for (int32_t b = 0; b < P->bs; ++b) {
    const int64_t m = static_cast<int64_t>(qo[b + 1]) - qo[b];
    const int64_t np = static_cast<int64_t>(kvp[b + 1]) - kvp[b];
    if (m < 0 || np < 0) return MLA_ERR_INVALID_ARG;
    int64_t n = np * P->page_size;
    if (np > 0 && last != nullptr) {
      if (last[b] < 1 || last[b] > P->page_size) return MLA_ERR_INVALID_ARG;
      n -= P->page_size - last[b];
    }
    if (n > INT32_MAX - mla::kPfTile || n - m < -INT32_MAX) return MLA_ERR_INVALID_ARG;
    if (n > 0)
      P->identity_rows =
          std::max(P->identity_rows, static_cast<int64_t>(kvp[b]) * P->page_size + n);
    P->k_tokens += n;
    if (m == 0) continue;
    // (before the lists are built: 2^31 rows of 1024 heads would be 8.6 G items)
    const int64_t blocks = (m + mla::kPfRows - 1) / mla::kPfRows;
    if (static_cast<int64_t>(all.size()) + blocks * P->heads > kMaxItems)
      return MLA_ERR_INVALID_ARG;
    const int64_t kv_row = P->kx_rows;
    for (int64_t t = 0; t < n; t += mla::kPfTile) {
      P->tiles.push_back(ExpandTile{kvp[b], static_cast<int32_t>(t), static_cast<int32_t>(n),
                                    static_cast<int32_t>(P->kx_rows), 0u, {}});
      P->kx_rows += mla::kPfTile;
      if (P->kx_rows > INT32_MAX - mla::kPfTile) return MLA_ERR_INVALID_ARG;
    }
    add_items(nullptr, &all, INT64_MAX, qo[b], m, n, kv_row, P->heads);
    add_items(&pairs, &rest, kPairRows, qo[b], m, n, kv_row, P->heads);
  }
  if (static_cast<int64_t>(P->tiles.size()) * P->heads > INT32_MAX) return MLA_ERR_INVALID_ARG;
  P->q_tokens = qo[P->bs];
  // Pairs take nine tenths of the time of single CTAs for the same rows, but
  // rows of both kinds run one after the other: whichever ends first.
  Schedule single = schedule(all, P->num_sms, 0), pair;
  if (!pairs.empty() && P->num_sms >= 2) {
    Schedule a = schedule(pairs, P->num_sms / 2, 0);
    Schedule b = schedule(rest, P->num_sms, a.partials);
    if (9 * a.most / 10 + b.most + (b.ctas > 0 ? kLaunchCost : 0) < single.most) {
      pair = std::move(a);
      single = std::move(b);
    }
  }
  P->num_ctas = single.ctas;
  P->num_pairs = pair.ctas;
  P->num_partials = single.partials + pair.partials;
  P->items = single.items;
  P->items.insert(P->items.end(), pair.items.begin(), pair.items.end());
  P->cta_items = single.of_cta;
  P->pair_items = pair.of_cta;
  for (CtaItems& c : P->pair_items) {
    c.begin += static_cast<int32_t>(single.items.size());
    c.end += static_cast<int32_t>(single.items.size());
  }
  P->jobs = pair.jobs;
  P->jobs.insert(P->jobs.end(), single.jobs.begin(), single.jobs.end());

  size_t off = align256(sizeof(mla::PrefillHeader));
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  P->off_tiles = take(sizeof(ExpandTile) * P->tiles.size());
  P->off_ctas = take(sizeof(CtaItems) * P->cta_items.size());
  P->off_pairs = take(sizeof(CtaItems) * P->pair_items.size());
  P->off_items = take(sizeof(AttnItem) * P->items.size());
  P->off_checks = take(sizeof(uint32_t) * P->items.size());
  P->off_jobs = take(sizeof(JoinJob) * P->jobs.size());
  P->table.assign(off, 0);
  P->off_kx = take(sizeof(uint16_t) * P->kx_rows * P->heads * mla::kWRows);
  P->off_kr = take(sizeof(uint16_t) * P->kx_rows * mla::kRope);
  P->off_vh = take(static_cast<size_t>(P->kx_rows) / mla::kPfGroup * P->heads);
  P->off_qr = take(sizeof(uint16_t) * P->q_tokens * P->heads * mla::kRope);
  P->off_part_o = take(sizeof(float) * P->num_partials * mla::kPfRows * mla::kVHead);
  P->off_part_lse = take(sizeof(float) * P->num_partials * mla::kPfRows);
  P->ws_bytes = off;
  P->stamp = mla::new_plan_stamp();
  mla::PrefillHeader hdr{};
  hdr.ws.stamp = P->stamp;
  auto put = [&](size_t at, const void* src, size_t bytes) {
    if (bytes > 0) std::memcpy(P->table.data() + at, src, bytes);
  };
  auto put_records = [&](size_t at, auto& records) {
    for (auto& r : records) r.check = mla::check_of(r, P->stamp);
    put(at, records.data(), sizeof(records[0]) * records.size());
  };
  for (const AttnItem& w : P->items) P->item_checks.push_back(mla::check_of(w, P->stamp));
  put(0, &hdr, sizeof(hdr));
  put_records(P->off_tiles, P->tiles);
  put_records(P->off_ctas, P->cta_items);
  put_records(P->off_pairs, P->pair_items);
  put(P->off_items, P->items.data(), sizeof(AttnItem) * P->items.size());
  put(P->off_checks, P->item_checks.data(), sizeof(uint32_t) * P->item_checks.size());
  put_records(P->off_jobs, P->jobs);
  return MLA_OK;
}

// A 3-D tensor of bf16 whose 64-element boxes land in shared memory as rows of
// 128 bytes with the 128-byte swizzle; rows out of bounds are zeros.
bool make_map(CUtensorMap* map, const void* ptr, const cuuint64_t (&dims)[3],
              const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3]) {
  const mla::TiledEncoder enc = mla::tiled_encoder();
  const cuuint32_t one[3] = {1, 1, 1};
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

mla_status mla_prefill_plan(const int32_t* qo_indptr_host, const int32_t* kv_indptr_host,
                            const int32_t* kv_last_page_len_host, int32_t batch_size,
                            int32_t page_size, int32_t heads, mla_dtype kv_dtype, int32_t num_sms,
                            mla_prefill** plan_out) {
  if (plan_out == nullptr) return MLA_ERR_INVALID_ARG;
  *plan_out = nullptr;
  if (qo_indptr_host == nullptr || kv_indptr_host == nullptr || batch_size < 1 || page_size < 1 ||
      heads < 1 || heads > 1024 || num_sms < 0 || kv_dtype < MLA_DTYPE_BF16 ||
      kv_dtype > MLA_DTYPE_MXFP4)
    return MLA_ERR_INVALID_ARG;
  if (qo_indptr_host[0] != 0 || kv_indptr_host[0] < 0) return MLA_ERR_INVALID_ARG;
  if (num_sms == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return MLA_ERR_CUDA;
  }
  mla_prefill* P = nullptr;
  try {
    P = new mla_prefill();
    P->bs = batch_size;
    P->heads = heads;
    P->page_size = page_size;
    P->kv_dtype = kv_dtype;
    P->num_sms = num_sms;
    const mla_status st = make_plan(P, qo_indptr_host, kv_indptr_host, kv_last_page_len_host);
    if (st != MLA_OK) {
      delete P;
      return st;
    }
  } catch (...) {   // out of host memory
    delete P;
    return MLA_ERR_INVALID_ARG;
  }
  *plan_out = P;
  return MLA_OK;
}

mla_status mla_prefill_get_info(const mla_prefill* plan, mla_prefill_info* info) {
  if (plan == nullptr || info == nullptr) return MLA_ERR_INVALID_ARG;
  info->batch_size = plan->bs;
  info->heads = plan->heads;
  info->num_ctas = plan->num_ctas + 2 * plan->num_pairs;
  info->num_items = static_cast<int32_t>(plan->items.size());
  info->num_partials = plan->num_partials;
  info->query_tokens = plan->q_tokens;
  info->key_tokens = plan->k_tokens;
  info->workspace_bytes = plan->ws_bytes;
  return MLA_OK;
}

void mla_prefill_destroy(mla_prefill* plan) { delete plan; }

mla_status mla_prefill_run(mla_prefill* plan, const void* q, int64_t q_token_stride,
                           int64_t q_head_stride, const void* kv, const float* kv_scale,
                           const uint8_t* kv_e8m0, int64_t kv_e8m0_row_stride,
                           int64_t kv_pool_rows, const int32_t* kv_indices, const void* w,
                           float sm_scale, const float* cos_sin, int64_t max_positions,
                           const int32_t* positions, mla_rope rope, void* workspace,
                           size_t workspace_bytes, void* out, float* lse, mla_stream_t stream_) {
  using mla::ptr_aligned;
  if (plan == nullptr || kv == nullptr || w == nullptr || workspace == nullptr)
    return MLA_ERR_INVALID_ARG;
  if (plan->q_tokens > 0 && (q == nullptr || out == nullptr)) return MLA_ERR_INVALID_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(kv, 16) || !ptr_aligned(w, 16) ||
      !ptr_aligned(out, 32) || !ptr_aligned(workspace, 256) || !ptr_aligned(lse, 4) ||
      !ptr_aligned(kv_scale, 4) || !ptr_aligned(kv_indices, 4) || !ptr_aligned(positions, 4))
    return MLA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return MLA_ERR_INVALID_ARG;
  // strides of a tensor map: multiples of 16 bytes below 2^40
  if (q_token_stride < mla::kQHead || q_head_stride < mla::kQHead || q_token_stride % 8 != 0 ||
      q_head_stride % 8 != 0 || q_token_stride >= (1LL << 39) || q_head_stride >= (1LL << 39))
    return MLA_ERR_INVALID_ARG;
  if (kv_pool_rows < 1 || kv_pool_rows > INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (plan->kv_dtype == MLA_DTYPE_FP8_E4M3 && kv_scale == nullptr) return MLA_ERR_INVALID_ARG;
  if (plan->kv_dtype == MLA_DTYPE_MXFP4) {
    if (kv_e8m0 == nullptr || kv_e8m0_row_stride < 18) return MLA_ERR_INVALID_ARG;
    if (kv_e8m0_row_stride % 2 != 0 || !ptr_aligned(kv_e8m0, 2)) return MLA_ERR_UNSUPPORTED;
  }
  const mla::Rotation rot{cos_sin, positions, max_positions, rope == MLA_ROPE_HALF ? 1 : 0};
  if (!mla::rotation_ok(rot, rope, plan->q_tokens)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->ws_bytes) return MLA_ERR_WORKSPACE;
  if (kv_indices == nullptr ? plan->identity_rows > kv_pool_rows
                            : kv_pool_rows % plan->page_size != 0)
    return MLA_ERR_INVALID_ARG;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (plan->uploaded_ws != workspace) {
    if (cudaMemcpyAsync(ws, plan->table.data(), plan->table.size(), cudaMemcpyHostToDevice,
                        stream) != cudaSuccess)
      return MLA_ERR_CUDA;
    plan->uploaded_ws = workspace;
  }
  int32_t* err = reinterpret_cast<int32_t*>(ws);
  uint16_t* kx = reinterpret_cast<uint16_t*>(ws + plan->off_kx);
  uint16_t* kr = reinterpret_cast<uint16_t*>(ws + plan->off_kr);
  uint8_t* v_half = ws + plan->off_vh;
  uint16_t* qr = reinterpret_cast<uint16_t*>(ws + plan->off_qr);
  float* part_o = reinterpret_cast<float*>(ws + plan->off_part_o);
  float* part_lse = reinterpret_cast<float*>(ws + plan->off_part_lse);
  // (a plan without key rows has nothing to expand and no tile to load)
  if (plan->kx_rows > 0 && plan->map_ws != workspace) {
    const cuuint64_t rows = static_cast<cuuint64_t>(plan->kx_rows);
    const cuuint64_t heads = static_cast<cuuint64_t>(plan->heads);
    const cuuint64_t tokens = static_cast<cuuint64_t>(plan->q_tokens);
    plan->map_ws = nullptr;
    if (!make_map(&plan->map_kx, kx, {mla::kWRows, rows, heads},
                  {mla::kWRows * 2, rows * mla::kWRows * 2}, {64, 64, 1}) ||
        !make_map(&plan->map_kx_out, kx, {mla::kWRows, rows, heads},
                  {mla::kWRows * 2, rows * mla::kWRows * 2}, {64, 32, 1}) ||
        !make_map(&plan->map_kr, kr, {mla::kRope, rows, 1},
                  {mla::kRope * 2, rows * mla::kRope * 2}, {64, 64, 1}) ||
        !make_map(&plan->map_qr, qr, {mla::kRope, heads, tokens},
                  {mla::kRope * 2, heads * mla::kRope * 2}, {64, 1, mla::kPfTile}))
      return MLA_ERR_CUDA;
    plan->map_ws = workspace;
  }
  if (!plan->tiles.empty()) {
    if (plan->map_w_ptr != w) {
      plan->map_w_ptr = nullptr;
      if (!make_map(&plan->map_w, w,
                    {mla::kVDim, mla::kWRows, static_cast<cuuint64_t>(plan->heads)},
                    {mla::kVDim * 2, mla::kVDim * mla::kWRows * 2}, {64, 128, 1}))
        return MLA_ERR_CUDA;
      plan->map_w_ptr = w;
    }
    mla::ExpandParams p{};
    p.map_w = plan->map_w;
    p.map_kx = plan->map_kx_out;
    p.tiles = reinterpret_cast<const ExpandTile*>(ws + plan->off_tiles);
    p.num_tiles = static_cast<int32_t>(plan->tiles.size());
    p.heads = plan->heads;
    p.kv = static_cast<const uint8_t*>(kv);
    p.kv_scale = kv_scale;
    p.e8m0 = kv_e8m0;
    p.e8m0_stride = kv_e8m0_row_stride;
    p.pool_rows = kv_pool_rows;
    p.kv_indices = kv_indices;
    p.page_size = plan->page_size;
    p.kv_dtype = plan->kv_dtype;
    p.kr = kr;
    p.v_half = v_half;
    p.kx_rows = plan->kx_rows;
    p.err = err;
    p.stamp = plan->stamp;
    if (rot.cos_sin != nullptr) {
      const mla::RotateParams r{static_cast<const uint16_t*>(q), q_token_stride, q_head_stride,
                                plan->q_tokens, plan->heads, rot, qr, err, plan->stamp};
      if (mla::launch_rotate(r, stream) != cudaSuccess) return MLA_ERR_CUDA;
    }
    if (mla::launch_expand(p, plan->num_sms, rot.cos_sin != nullptr, stream) != cudaSuccess)
      return MLA_ERR_CUDA;
  }
  if (plan->num_ctas > 0 || plan->num_pairs > 0) {
    if (plan->map_q_ptr != q || plan->map_q_ts != q_token_stride ||
        plan->map_q_hs != q_head_stride) {
      plan->map_q_ptr = nullptr;
      if (!make_map(&plan->map_q, q,
                    {mla::kQHead, static_cast<cuuint64_t>(plan->heads),
                     static_cast<cuuint64_t>(plan->q_tokens)},
                    {static_cast<cuuint64_t>(q_head_stride) * 2,
                     static_cast<cuuint64_t>(q_token_stride) * 2},
                    {64, 1, mla::kPfTile}))
        return MLA_ERR_CUDA;
      plan->map_q_ptr = q;
      plan->map_q_ts = q_token_stride;
      plan->map_q_hs = q_head_stride;
    }
    mla::AttnParams p{};
    p.map_q = plan->map_q;
    p.map_qr = rot.cos_sin != nullptr ? plan->map_qr : plan->map_q;
    p.qr_x = rot.cos_sin != nullptr ? 0 : mla::kNope;
    p.map_kx = plan->map_kx;
    p.map_kr = plan->map_kr;
    p.items = reinterpret_cast<const AttnItem*>(ws + plan->off_items);
    p.item_checks = reinterpret_cast<const uint32_t*>(ws + plan->off_checks);
    p.v_half = v_half;
    p.kx_rows = plan->kx_rows;
    p.heads = plan->heads;
    p.scale_log2 = sm_scale * mla::kLog2e;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.part_o = part_o;
    p.part_lse = part_lse;
    p.err = err;
    p.stamp = plan->stamp;
    if (plan->num_pairs > 0) {
      p.ctas = reinterpret_cast<const CtaItems*>(ws + plan->off_pairs);
      if (mla::launch_attn_pairs(p, plan->num_pairs, stream) != cudaSuccess) return MLA_ERR_CUDA;
    }
    if (plan->num_ctas > 0) {
      p.ctas = reinterpret_cast<const CtaItems*>(ws + plan->off_ctas);
      p.after_attn = plan->num_pairs > 0 ? 1 : 0;
      if (mla::launch_attn(p, plan->num_ctas, stream) != cudaSuccess) return MLA_ERR_CUDA;
    }
  }
  if (!plan->jobs.empty()) {
    const mla::JoinParams p{reinterpret_cast<const JoinJob*>(ws + plan->off_jobs),
                            static_cast<int32_t>(plan->jobs.size()), plan->heads, part_o,
                            part_lse, static_cast<uint16_t*>(out), lse, err, plan->stamp};
    if (mla::launch_join(p, stream) != cudaSuccess) return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

mla_status mla_prefill_check(const mla_prefill* plan, void* workspace, mla_stream_t stream_) {
  if (plan == nullptr || workspace == nullptr) return MLA_ERR_INVALID_ARG;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  int32_t word = 0;
  if (cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, stream) !=
          cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (word == 0) return MLA_OK;
  if (cudaMemsetAsync(workspace, 0, sizeof(word), stream) != cudaSuccess) return MLA_ERR_CUDA;
  if (word & mla::kErrStale) {
    if (plan->uploaded_ws == workspace) plan->uploaded_ws = nullptr;
    return MLA_ERR_WORKSPACE;
  }
  return (word & mla::kErrTimeout) ? MLA_ERR_DEVICE_TIMEOUT : MLA_ERR_INVALID_ARG;
}

}  // extern "C"
