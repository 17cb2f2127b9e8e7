// shared.h -- internal interface between the host side of the shared-prefix
// decode (shared_api.cu) and its kernels (gather.cu, prefix.cu, meet.cu).
#pragma once

#include "prefill.h"

namespace mla {

// A launch as a programmatic dependent of the kernel before it in the stream: the
// kernel begins while that one ends, and waits for its end before it touches memory
// (a trip less between the kernels of a step: 1 to 3 us a call).  What the kernel before
// may have written is read with plain loads, not with those for memory that stays the
// same while a kernel runs.
template <class Params>
cudaError_t launch_dependent(void (*kernel)(const Params), dim3 grid, int threads, size_t smem,
                             cudaStream_t stream, const Params& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

__device__ __forceinline__ uint4 ld_na_v4(const void* ptr) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(ptr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_u8(const uint8_t* ptr) {
  uint16_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=h"(v) : "l"(ptr) : "memory");
  return v;
}

constexpr int kSpRows = 128;     // query rows of a CTA: 8 tokens x 16 heads
constexpr int kSpTile = 128;     // keys of a tile

// Query rows q_row .. q_row + rows - 1 (row = token * 16 + head) of one group, up
// to 128 or (paired) 256, against `keys` of its prefix's rows from key0 on: a row of
// the workspace, or a key of the group, whose page table begins at page_base.
struct PrefixItem {
  int32_t q_row, rows, key0, keys, slot, page_base;   // slot: of the partial result
  uint32_t check;
  int32_t pad;
};
static_assert(sizeof(PrefixItem) == 32, "a prefix item is two int4");
__host__ __device__ inline uint32_t check_of(const PrefixItem& w, uint64_t stamp) {
  const uint32_t h = mix(mix(mix(static_cast<uint32_t>(stamp), w.q_row), w.rows), w.key0);
  return mix(mix(mix(h, w.keys), w.slot), w.page_base);
}

// The partial results of one query token: `own_count` of the decode kernel from
// own_first on (its 16 heads from row own_row of each), prefix_count of the
// prefix kernel from block prefix_first on, a block of 128 rows in each slot (from
// row prefix_row of it).
struct MeetJob {
  int32_t own_first, own_count, own_row, prefix_first, prefix_count, prefix_row;
  uint32_t check;
  int32_t pad;
};
static_assert(sizeof(MeetJob) == 32, "a meeting is two int4");
__host__ __device__ inline uint32_t check_of(const MeetJob& j, uint64_t stamp) {
  const uint32_t h = mix(mix(mix(static_cast<uint32_t>(stamp), j.own_first), j.own_count), j.own_row);
  return mix(mix(mix(h, j.prefix_first), j.prefix_count), j.prefix_row);
}

struct GatherParams {
  const ExpandTile* tiles;     // 128 rows each
  int32_t num_tiles;
  const uint8_t* kv;
  const uint8_t* e8m0;
  int64_t e8m0_stride;
  int64_t pool_rows;
  const int32_t* indices;      // page table of the prefixes, or null: identity
  int32_t page_size;
  int32_t kv_dtype;
  uint16_t* rows;              // [tiles * 128][576] bf16
  int32_t* err;                // workspace header
  uint64_t stamp;
};

struct PrefixParams {
  CUtensorMap map_k;           // {64, rows, 9} of the rows, boxes {64, 64, 1} or (tall) {64, 128, 1}
  CUtensorMap map_v;           // the same, boxes {64, 64, 4} or (paired) {64, 64, 2}
  const PrefixItem* items;
  const CtaItems* clusters;
  int32_t direct;              // 1: the rows are a bf16 pool's, in pages of a multiple of 64
  int32_t tall;                // 1: tiles of 128 keys stand together (not paired)
  int32_t page_size;
  const int32_t* indices;      // page table of the prefixes, or null: identity
  int64_t pool_rows;
  const void* q;               // [tokens * 16][576], bf16 or e4m3
  int32_t q_fp8;
  const float* q_scale;        // device [1], or null: 1
  const float* kv_scale;       // device [1], or null: 1
  float* part_o;               // [slots][blocks][64][128][8] fp32, normalised: dim / 8, row, dim % 8
  float* part_lse;             // [slots][blocks][128], log2 domain
  int32_t* err;
  uint64_t stamp;
};

struct MeetParams {
  const MeetJob* jobs;
  int64_t tokens;
  const float* own_o;          // [partials][own_rows][512]
  const float* own_lse;
  int32_t own_rows;
  int32_t blocks;              // of 128 rows in a slot of the prefix kernel
  int32_t most;                // partial results of a token, at most
  int32_t alone;               // 1: the only kernel of its call (nothing is cached)
  const float* prefix_o;       // [slots][blocks][64][128][8]
  const float* prefix_lse;
  uint16_t* out;
  float* lse;
  int32_t* err;
  uint64_t stamp;
};

// The kernels of a call are chained as programmatic dependents, in the order
// gather, prefix, the decode kernel over the own ends, meet.  The first one waits
// for the end of what the caller has launched before it touches memory.  The prefix
// kernel waits for the gathered rows only before it loads them; the decode kernel
// reads nothing of the others and runs on the SMs that they leave; each ends after
// the one before it, so that the last one waits for all.
cudaError_t launch_gather(const GatherParams& p, cudaStream_t stream);
cudaError_t launch_prefix(const PrefixParams& p, bool paired, int clusters, cudaStream_t stream);
// Clusters of the prefix kernel that the current device holds at a time (0: unknown).
int prefix_clusters(bool paired);
cudaError_t launch_meet(const MeetParams& p, cudaStream_t stream);

}  // namespace mla
