// prefill.h -- internal interface between the host side of the expanded form
// (prefill_api.cu) and its kernels (expand.cu, rotate.cu, attn.cu, join.cu).
#pragma once

#include "layer.h"

namespace mla {

constexpr int kPfRows = 256;     // query rows of a CTA's item (two 128-row matrix tiles); a pair's
                                 // item has up to twice as many
constexpr int kPfTile = 128;     // keys of a tile
constexpr int kPfGroup = 32;     // keys whose values share a type: fp16 (flag 1) or bf16 (0)

// The workspace begins with WsHeader and, behind it, `expanded`: 0 from the
// expansion on, 1 once the attention on pairs has found the expansion through.
struct PrefillHeader {
  WsHeader ws;
  int32_t expanded;
  int32_t pad[3];
};
__device__ __forceinline__ int32_t* expanded_word(int32_t* err) {
  return &reinterpret_cast<PrefillHeader*>(err)->expanded;
}

// Every record of the table carries a check word of the plan's stamp and its
// own fields.  A record of another plan, one that something else has overwritten
// in a workspace with the stamp still in place, or half of an upload (a run on a
// second stream that does not wait for it) fails it, is reported as kErrStale
// and stands for no work: nothing is read or written by what it says.
__host__ __device__ inline uint32_t mix(uint32_t h, int32_t v) {
  h = (h ^ static_cast<uint32_t>(v)) * 0x9e3779b1u;
  return h ^ (h >> 15);
}

// 128 consecutive cached tokens of one request, expanded into workspace rows
// out_row .. out_row + 127 (rows past the request's end are written as zeros).
struct ExpandTile {
  int32_t page_base, tok0, len, out_row;   // first page-table entry, first token, request length
  uint32_t check;
  int32_t pad[3];
};
static_assert(sizeof(ExpandTile) == 32, "an expansion tile is two int4");
__host__ __device__ inline uint32_t check_of(const ExpandTile& t, uint64_t stamp) {
  return mix(mix(mix(mix(static_cast<uint32_t>(stamp), t.page_base), t.tok0), t.len), t.out_row);
}

// The items of one CTA (or pair).
struct CtaItems {
  int32_t begin, end;
  uint32_t check;
  int32_t pad;
};
static_assert(sizeof(CtaItems) == 16, "a CTA's range is one int4");
__host__ __device__ inline uint32_t check_of(const CtaItems& c, uint64_t stamp) {
  return mix(mix(static_cast<uint32_t>(stamp), c.begin), c.end);
}

// Query rows q_row .. q_row + rows - 1 of one head against keys
// [kv_begin, kv_end) of their request (kv_begin a multiple of 128).  Row i
// sees the request's first vis0 + i keys.  slot < 0: out and lse are written;
// else a partial result.  Partial items of at most 128 rows are `halved`: their
// rows fill both query tiles, tile 0 against the first half of the keys and
// tile 1 against the second, with partial results slot and slot + 1.
// (Their check words stand in an array of their own: the attention kernel has no
// register left for one.)
struct AttnItem {
  int32_t q_row, rows, head, kv_row;       // kv_row: workspace row of the request's key 0
  int32_t vis0, kv_begin, kv_end, slot;
};
static_assert(sizeof(AttnItem) == 32, "an attention item is two int4");
__host__ __device__ inline uint32_t check_of(const AttnItem& w, uint64_t stamp) {
  const uint32_t h = mix(mix(mix(static_cast<uint32_t>(stamp), w.q_row), w.rows), w.head);
  return mix(mix(mix(mix(mix(h, w.kv_row), w.vis0), w.kv_begin), w.kv_end), w.slot);
}

__host__ __device__ inline bool halved(const AttnItem& w) {
  return w.slot >= 0 && w.rows <= kPfTile;
}
// First key of the second half: whole tiles, the larger half first.
__host__ __device__ inline int32_t middle_key(const AttnItem& w) {
  const int32_t tiles = (w.kv_end - w.kv_begin + kPfTile - 1) / kPfTile;
  const int32_t mid = w.kv_begin + (tiles + 1) / 2 * kPfTile;
  return mid < w.kv_end ? mid : w.kv_end;
}

// Join of `count` consecutive partials, of `span` slots of 256 rows each, of
// the same query rows and head.
struct JoinJob {
  int32_t q_row, rows, head, first, count, vis0, span;
  uint32_t check;
};
static_assert(sizeof(JoinJob) == 32, "a join job is two int4");
__host__ __device__ inline uint32_t check_of(const JoinJob& j, uint64_t stamp) {
  const uint32_t h = mix(mix(mix(static_cast<uint32_t>(stamp), j.q_row), j.rows), j.head);
  return mix(mix(mix(mix(h, j.first), j.count), j.vis0), j.span);
}

struct ExpandParams {
  CUtensorMap map_w;           // {512, 256, heads}, boxes {64, 128, 1}
  CUtensorMap map_kx;          // {256, kx_rows, heads}, boxes {64, 32, 1}: keys' dims, then values'
  const ExpandTile* tiles;
  int32_t num_tiles, heads;
  const uint8_t* kv;
  const float* kv_scale;
  const uint8_t* e8m0;
  int64_t e8m0_stride;
  int64_t pool_rows;
  const int32_t* kv_indices;   // null: identity
  int32_t page_size;
  int32_t kv_dtype;
  uint16_t* kr;                // [kx_rows][64]: the keys' rotated dims
  uint8_t* v_half;             // [heads][kx_rows / 32]: type of the values of 32 rows
  int64_t kx_rows;
  int32_t* err;                // workspace header
  uint64_t stamp;
};

struct RotateParams {
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride, q_tokens;
  int32_t heads;
  Rotation rot;
  uint16_t* qr;                // [q_tokens][heads][64]
  int32_t* err;
  uint64_t stamp;
};

struct AttnParams {
  CUtensorMap map_q;           // {192, heads, tokens}, boxes {64, 1, 128}
  CUtensorMap map_qr;          // the rotated query dims, from x = qr_x on: {64, heads, tokens}
                               // (workspace), or map_q itself without a rotation
  CUtensorMap map_kx;          // {256, kx_rows, heads}, boxes {64, 64, 1}
  CUtensorMap map_kr;          // {64, kx_rows, 1}, boxes {64, 64, 1}
  const AttnItem* items;
  const uint32_t* item_checks;
  const CtaItems* ctas;        // [CTAs] or [pairs]
  const uint8_t* v_half;       // [heads][kx_rows / 32]
  int64_t kx_rows;
  int32_t heads;
  int32_t qr_x;
  int32_t after_attn;          // 1: launched behind another attention kernel of the call
  float scale_log2;            // sm_scale * log2(e)
  uint16_t* out;
  float* lse;
  float* part_o;               // [partials][256][128]
  float* part_lse;             // [partials][256], log2 domain
  int32_t* err;
  uint64_t stamp;
};

struct JoinParams {
  const JoinJob* jobs;
  int32_t num_jobs, heads;
  const float* part_o;
  const float* part_lse;
  uint16_t* out;
  float* lse;
  int32_t* err;
  uint64_t stamp;
};

// The kernels of a call are programmatic dependents of one another, in the
// order rotate, expand, attention (pairs, then single CTAs), join; the first
// one launched is not (`dependent` for the expansion: the rotation precedes it).
cudaError_t launch_expand(const ExpandParams& p, int num_ctas, bool dependent, cudaStream_t stream);
cudaError_t launch_rotate(const RotateParams& p, cudaStream_t stream);
cudaError_t launch_attn(const AttnParams& p, int num_ctas, cudaStream_t stream);
cudaError_t launch_attn_pairs(const AttnParams& p, int num_pairs, cudaStream_t stream);
cudaError_t launch_join(const JoinParams& p, cudaStream_t stream);

}  // namespace mla
