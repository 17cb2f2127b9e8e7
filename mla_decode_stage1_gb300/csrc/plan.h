// plan.h -- the host-side plan object behind the opaque mla_plan handle
// (internal to libmla_decode).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "kernels.h"
#include "mla_decode.h"

struct mla_plan {
  int32_t bs = 0, page_size = 0, num_splits = 0;   // bs: rows of q (requests x q_len)
  int32_t q_len = 1;                                 // query tokens per request
  int32_t nreq = 0;                                  // requests of the batch
  int32_t rows = 16;                                 // output rows per planned request (16 x tokens it holds)
  int q_dtype = 0, kv_dtype = 0, qmode = 0;
  int32_t num_ctas = 0, num_partials = 0;
  int32_t max_parts = 0;   // most partials of one request (stage 2 goes wide above 4)
  int32_t unit_tokens = mla::kTile;   // tokens between the planner's possible cut points
  int32_t item_cost = 1;              // cost of an extra item in a CTA (balanced plan)
  int32_t num_sms = 0;                // CTAs the balanced plan was cut for
  int32_t exact_q = 0;                // see Stage1Params
  int32_t cluster = 0;                // CTAs per cluster merging a request inside stage 1 (0: stage 2)
  int64_t total_tokens = 0, total_tiles = 0;
  int64_t identity_rows = 0;   // pool rows the requests reach without a page table
  std::vector<int32_t> cta_indptr;
  std::vector<mla::WorkItem> items;
  std::vector<mla::MergeJob> jobs;
  // workspace layout (byte offsets)
  size_t off_err = 0, off_indptr = 0, off_items = 0, off_jobs = 0, off_part_o = 0,
         off_part_lse = 0, ws_bytes = 0;
  std::vector<uint8_t> table;  // image of [0, off_part_o) uploaded once per workspace
  uint64_t stamp = 0;          // unique per plan; written into the table header and CTA heads
  // per-run caches (the upload cache is reset by mla_decode_check when a
  // kernel found another plan's table in the workspace)
  mutable void* uploaded_ws = nullptr;
  CUtensorMap tmap;
  const void* tmap_ptr = nullptr;
  int64_t tmap_rows = -1;
  int32_t tmap_box_rows = -1;
  cudaEvent_t ev_before = nullptr, ev_after = nullptr;
  mutable int cluster_dev = -1;       // device whose cluster fit was checked (cluster_fits)
  mutable bool cluster_fits = false;
};

namespace mla {
// Device address of the library's own workspace array on the current device
// (noalloc.cu), looked up once per device.
mla_status static_workspace(void** out);
constexpr size_t kStaticWorkspaceBytes = size_t(16) << 20;

// The two steps of mla_decode_run (api.cu).
struct DecodeLaunch {
  Stage1Params stage1;
  Stage2Params stage2;
  bool merge;
};
mla_status decode_prepare(mla_plan* plan, const void* q, const float* q_scale, const void* kv,
                          const float* kv_scale, const uint8_t* kv_e8m0,
                          int64_t kv_e8m0_row_stride, int64_t kv_pool_rows,
                          const int32_t* kv_indices, const int32_t* prefix_indices,
                          void* workspace, size_t workspace_bytes, void* out, float* lse,
                          cudaStream_t stream, DecodeLaunch* launch);
mla_status decode_launch(const mla_plan* plan, const DecodeLaunch& launch, cudaStream_t stream);

// What the other host files take from api.cu: a process-wide unique stamp for
// a new plan, and the driver's cuTensorMapEncodeTiled (null if not found).
uint64_t new_plan_stamp();
typedef CUresult (*TiledEncoder)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
TiledEncoder tiled_encoder();
// mla_decode_plan_ex for requests that have pages in front of their own as well, which
// all their query tokens see whole: prefix_pages[b] entries from prefix_base[b] on of
// another page table (prefix_indices).  A part of either kind is an item of its own, so
// every request's items write partial results: for plan_partials_only.
struct PrefixPages {
  const int32_t *base, *pages;
};
mla_status plan_with_prefixes(const int32_t* kv_indptr_host, const int32_t* kv_last_page_len_host,
                              int32_t batch_size, int32_t q_len, int32_t page_size,
                              mla_dtype q_dtype, mla_dtype kv_dtype,
                              const mla_plan_options* options, const PrefixPages* prefixes,
                              mla_plan** plan_out);
// Turns a new plan into one whose every item writes a partial result and whose
// run merges nothing: request b's are slots first[b] .. first[b] + count[b] - 1.
// Its run splits a bf16 query without loss where the decode call rounds it a
// little (a log-sum-exp of few tokens was 3e-4 off).
void plan_partials_only(mla_plan* P, std::vector<int32_t>* first, std::vector<int32_t>* count);
}  // namespace mla
