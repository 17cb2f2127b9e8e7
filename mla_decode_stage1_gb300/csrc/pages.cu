// pages.cu -- choosing the pages that a query attends to: the bounds of every
// page's rows, the score of each page for each query, and the best pages as the
// page table of a decode call.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "layer.h"
#include "ptx.cuh"

namespace mla {
namespace {

__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void report(int32_t* err, int32_t bits) {
  if (err != nullptr) atomicOr(err, bits);
}

// ------------------------------------------------------------------- bounds
//
// For page p with the rows x_t (the stored values, without an e4m3 pool's
// scale): lo[d] = min_t x_t[d], hi[d] = max_t x_t[d], both as bf16, which holds
// every stored value.  A dim with a value that is not finite gets NaN for both.
// A page that had rows before goes on from its bounds, so a step reads its new
// rows only.
//
// Bound: memory, one pass over the new rows; latency for a step of one token.

constexpr uint32_t kPosInf2 = 0x7f807f80u, kNegInf2 = 0xff80ff80u, kNan2 = 0x7fff7fffu;
constexpr int kBoundThreads = 288;

struct BoundsParams {
  const uint8_t* kv;
  const uint8_t* e8m0;
  int64_t e8m0_stride;
  int64_t pool_rows;
  uint16_t* bounds;             // [pages][2][576]
  int64_t pages;
  const int32_t* table;
  int64_t table_stride;
  int32_t table_pages;
  const int32_t* old_lens;
  const int32_t* new_lens;      // null: one new token per request
  int32_t page_size;
  int32_t* err;
};

template <int KV>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const BoundsParams p) {
  constexpr int kPieces = KV == MLA_DTYPE_BF16 ? 72 : KV == MLA_DTYPE_FP8_E4M3 ? 36 : 18;
  constexpr int kRows = kBoundThreads / kPieces;        // rows at a time
  constexpr int kWords = kQkDim / 2 / kPieces;          // bf16 pairs of a piece
  constexpr int kAhead = KV == MLA_DTYPE_MXFP4 ? 2 : 4;
  __shared__ uint32_t part[2][kRows][kQkDim / 2];
  const int b = blockIdx.x;
  int64_t old_len = p.old_lens[b], new_len = p.new_lens != nullptr ? p.new_lens[b] : 1;
  if (old_len < 0 || new_len < 0) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(p.err, kErrBadLength);
    old_len = old_len < 0 ? 0 : old_len;
    new_len = new_len < 0 ? 0 : new_len;
  }
  if (new_len == 0) return;
  const int64_t len = old_len + new_len;
  const int64_t first = old_len / p.page_size, end = (len + p.page_size - 1) / p.page_size;
  if (end > p.table_pages && threadIdx.x == 0 && blockIdx.y == 0) report(p.err, kErrCapacity);
  const int piece = threadIdx.x % kPieces, group = threadIdx.x / kPieces;
  for (int64_t j = first + blockIdx.y; j < end && j < p.table_pages; j += gridDim.y) {
    const int64_t page = p.table[b * p.table_stride + j];
    if (page < 0 || page >= p.pages || (page + 1) * p.page_size > p.pool_rows) {
      if (threadIdx.x == 0) report(p.err, kErrBadPage);
      continue;
    }
    const int r0 = static_cast<int>(j == first ? old_len % p.page_size : 0);
    const int r1 = static_cast<int>(len - j * p.page_size < p.page_size ? len - j * p.page_size
                                                                        : p.page_size);
    uint32_t lo[kWords], hi[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) lo[i] = kPosInf2, hi[i] = kNegInf2;
    const int64_t row0 = page * p.page_size;
    for (int r = r0 + group; r < r1; r += kRows * kAhead) {
      uint4 v[kAhead];
      uint32_t e[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        // (past the end: this thread's first row again)
        const int64_t row = row0 + (r + u * kRows < r1 ? r + u * kRows : r);
        v[u] = ld_nc_na_v4(p.kv + (row * kPieces + piece) * 16);
        if constexpr (KV == MLA_DTYPE_MXFP4)
          e[u] = ld_nc_u8_early(p.e8m0 + row * p.e8m0_stride + piece);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t x[kWords];
        if constexpr (KV == MLA_DTYPE_BF16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = w[i];
        } else if constexpr (KV == MLA_DTYPE_FP8_E4M3) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            const __nv_bfloat162 o = __floats2bfloat162_rn(f.x, f.y);
            x[i] = *reinterpret_cast<const uint32_t*>(&o);
          }
        } else {
          const uint32_t scale = e8m0_to_bf16x2(e[u]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e2m1x4_to_bf16(w[i], scale, x[4 * i], x[4 * i + 1]);
            e2m1x4_to_bf16(w[i] >> 16, scale, x[4 * i + 2], x[4 * i + 3]);
          }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          lo[i] = min_nan_bf16x2(lo[i], x[i]);
          hi[i] = max_nan_bf16x2(hi[i], x[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      part[0][group][piece * kWords + i] = lo[i];
      part[1][group][piece * kWords + i] = hi[i];
    }
    __syncthreads();
    // a thread per pair of dims
    uint32_t* out = reinterpret_cast<uint32_t*>(p.bounds + page * 2 * kQkDim) + threadIdx.x;
    uint32_t a = r0 > 0 ? out[0] : kPosInf2, c = r0 > 0 ? out[kQkDim / 2] : kNegInf2;
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      a = min_nan_bf16x2(a, part[0][g][threadIdx.x]);
      c = max_nan_bf16x2(c, part[1][g][threadIdx.x]);
    }
    // both bounds NaN where either is not finite
#pragma unroll
    for (int s = 0; s < 32; s += 16)
      if (((a >> s) & 0x7f80u) == 0x7f80u || ((c >> s) & 0x7f80u) == 0x7f80u) {
        a = (a & ~(0xffffu << s)) | (kNan2 & (0xffffu << s));
        c = (c & ~(0xffffu << s)) | (kNan2 & (0xffffu << s));
      }
    out[0] = a;
    out[kQkDim / 2] = c;
    __syncthreads();
  }
}

// ------------------------------------------------------------------- scores
//
// For query token r with heads h and page p:
//     score[r,p] = scale max_h sum_d max(q[h,d] lo[d], q[h,d] hi[d])
//                = scale max_h (q+[h] . hi + q-[h] . lo),
// with q+ = max(q, 0), q- = min(q, 0): a product of 16 rows (the heads, the M of
// a matrix instruction) and 1,152 columns for every page.  No score of a token
// of the page exceeds it.
//
// Bound: memory, 2,304 bytes a page.  A warp holds 8 kTiles pages; a lane loads
// 16 bytes (8 dims) of a page's bounds, which are its share of two instructions:
// the order of the sum over d is free, so lane c of a quad takes dims
// 8 c .. 8 c + 7 of 32, for the queries as well.

constexpr int kScoreWarps = 4;
constexpr int kQPitch = kQkDim + 8;           // bf16 elements: rows start 4 banks apart

struct ScoresParams {
  const void* q;
  int32_t q_fp8;
  const float* q_scale;
  const float* kv_scale;
  const uint16_t* bounds;
  int64_t pages;
  const int32_t* table;
  int64_t table_stride;
  int32_t columns;              // of the table and the scores that are used
  const int32_t* lens;
  int32_t page_size, q_len;
  float* scores;
  int64_t scores_stride;
  int32_t chunks;               // CTAs of a row
  int32_t* err;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Tokens that query token t of a request with n cached tokens sees.
__device__ __forceinline__ int64_t seen_by(int64_t n, int q_len, int t) {
  const int64_t s = n - q_len + 1 + t;
  return s < 0 ? 0 : s;
}

template <int kTiles>
__global__ void __launch_bounds__(32 * kScoreWarps) page_scores_kernel(const ScoresParams p) {
  __shared__ __align__(16) uint16_t qs[kHeads * kQPitch];
  const int b = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks, t = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(b) * p.q_len + t;
  int64_t n = p.lens[b];
  const bool first_cta = chunk == 0 && t == 0 && threadIdx.x == 0;
  if (n < 0) {
    if (first_cta) report(p.err, kErrBadLength);
    n = 0;
  }
  int64_t pages = (seen_by(n, p.q_len, t) + p.page_size - 1) / p.page_size;
  if (pages > p.columns) {
    if (first_cta) report(p.err, kErrCapacity);
    pages = p.columns;
  }
  float* out = p.scores + row * p.scores_stride;
  const int64_t cta0 = static_cast<int64_t>(chunk) * (kScoreWarps * 8 * kTiles);
  if (cta0 >= pages) {
    for (int i = threadIdx.x; i < kScoreWarps * 8 * kTiles; i += 32 * kScoreWarps)
      if (cta0 + i < p.columns) out[cta0 + i] = -INFINITY;
    return;
  }
  for (int i = threadIdx.x; i < kHeads * kQkDim / 16; i += 32 * kScoreWarps) {
    const int h = i / (kQkDim / 16), d = i % (kQkDim / 16) * 16;
    uint32_t v[8];
    if (p.q_fp8) {
      const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) +
                                                      (row * kHeads + h) * kQkDim + d);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t f16 = e4m3x2_to_f16x2(static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f16));
        const __nv_bfloat162 o = __floats2bfloat162_rn(f.x, f.y);
        v[k] = *reinterpret_cast<const uint32_t*>(&o);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                        (row * kHeads + h) * kQkDim + d);
      const uint4 x = src[0], y = src[1];
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    }
    uint4* dst = reinterpret_cast<uint4*>(qs + h * kQPitch + d);
    dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
    dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
  __syncthreads();
  const int64_t page0 = cta0 + warp * (8 * kTiles);
  const int g = lane >> 2, c = lane & 3;
  const uint4* src[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    // (columns past the last: its page again)
    const int64_t col = page0 + 8 * i + g;
    int64_t page = p.table[b * p.table_stride + (col < pages ? col : pages - 1)];
    if (page < 0 || page >= p.pages) {
      if (c == 0 && col < pages) report(p.err, kErrBadPage);
      page = 0;
    }
    src[i] = reinterpret_cast<const uint4*>(p.bounds + page * 2 * kQkDim) + c;
  }
  // The instruction's own sums round towards zero: 12 in a row, then one rounded
  // addition (72 in a row were 1.2e-6 off, against 2e-7).
  float sum[kTiles][4], acc[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[i][k] = acc[i][k] = 0.0f;
  const uint16_t* qa = qs + g * kQPitch + 8 * c;
#pragma unroll 3
  for (int d = 0; d < kQkDim / 32; ++d) {
    uint4 lo[kTiles], hi[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      lo[i] = ld_nc_na_v4(src[i] + 4 * d);
      hi[i] = ld_nc_na_v4(src[i] + kQkDim / 8 + 4 * d);
    }
    const uint4 x = *reinterpret_cast<const uint4*>(qa + 32 * d);
    const uint4 y = *reinterpret_cast<const uint4*>(qa + 8 * kQPitch + 32 * d);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
    uint32_t xp[4], xn[4], yp[4], yn[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      xp[k] = max_nan_bf16x2(xs[k], 0u); xn[k] = min_nan_bf16x2(xs[k], 0u);
      yp[k] = max_nan_bf16x2(ys[k], 0u); yn[k] = min_nan_bf16x2(ys[k], 0u);
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      mma_16816(acc[i], xp[0], yp[0], xp[1], yp[1], hi[i].x, hi[i].y);
      mma_16816(acc[i], xp[2], yp[2], xp[3], yp[3], hi[i].z, hi[i].w);
      mma_16816(acc[i], xn[0], yn[0], xn[1], yn[1], lo[i].x, lo[i].y);
      mma_16816(acc[i], xn[2], yn[2], xn[3], yn[3], lo[i].z, lo[i].w);
      if (d % 3 == 2)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sum[i][k] += acc[i][k];
          acc[i][k] = 0.0f;
        }
    }
  }
  float scale = 1.0f / 24.0f;
  if (p.q_scale != nullptr) scale *= *p.q_scale;
  if (p.kv_scale != nullptr) scale *= *p.kv_scale;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    // columns 2 c and 2 c + 1 of the tile, the best of all heads
    float s0 = max_nan(sum[i][0], sum[i][2]), s1 = max_nan(sum[i][1], sum[i][3]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      s0 = max_nan(s0, __shfl_xor_sync(0xffffffffu, s0, o));
      s1 = max_nan(s1, __shfl_xor_sync(0xffffffffu, s1, o));
    }
    const int64_t col = page0 + 8 * i + 2 * c;
    if (g == 0) {
      if (col < p.columns) out[col] = col < pages ? s0 * scale : -INFINITY;
      if (col + 1 < p.columns) out[col + 1] = col + 1 < pages ? s1 * scale : -INFINITY;
    }
  }
}

// ------------------------------------------------------------------- select
//
// Row r sees n pages.  All of them are kept if n <= top, else the first
// `first`, the last `last` and the top - first - last with the largest scores
// between them: ties go to the lower column, NaN counts as the largest, -0 as 0.
// Kept pages are written in ascending order, from the sum of the earlier rows'
// counts on.
//
// The smallest kept score is found by its 32 bits, 8 at a time from the top: a
// histogram of the scores that agree with what is known so far says which byte
// comes next.  A thread holds consecutive columns, so that one scan of the
// threads' counts places every kept page.  Latency-bound: 4 histograms, 2 scans.

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;

struct SelectParams {
  const float* scores;
  int64_t scores_stride;
  const int32_t* table;
  int64_t table_stride;
  int32_t columns;
  const int32_t* lens;
  int32_t page_size, q_len;
  int64_t rows;
  int32_t top, first, last;
  int32_t* kv_indptr;
  int32_t* last_page;
  int32_t* kv_indices;
  int64_t max_indices;
  int32_t* kept_columns;        // [rows][top] or null
  int32_t* err;
};

// Larger scores have larger keys.
__device__ __forceinline__ uint32_t key_of(float s) {
  if (s != s) return 0xffffffffu;
  const uint32_t u = __float_as_uint(s + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelectShared {
  uint32_t hist[256];
  uint32_t warp_sum[2][kSelWarps];
  uint32_t byte, above;
  int64_t before;
};

// Pages that row r sees, with what is wrong with its length.
__device__ __forceinline__ int64_t pages_of_row(const SelectParams& p, int64_t r, int64_t* seen,
                                                int32_t* bad) {
  int64_t n = p.lens[r / p.q_len];
  *bad = 0;
  if (n < 0) {
    *bad = kErrBadLength;
    n = 0;
  }
  int64_t s = seen_by(n, p.q_len, static_cast<int>(r % p.q_len));
  int64_t pages = (s + p.page_size - 1) / p.page_size;
  if (pages > p.columns) {
    *bad = kErrCapacity;
    pages = p.columns;
    s = pages * p.page_size;
  }
  *seen = s;
  return pages;
}

// Exclusive sums over the CTA of two counts, and their totals.
__device__ __forceinline__ void scan2(SelectShared& sh, uint32_t a, uint32_t b, uint32_t& ea,
                                      uint32_t& eb, uint32_t& ta, uint32_t& tb) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia += x, ib += y;
  }
  __syncthreads();
  if (lane == 31) sh.warp_sum[0][warp] = ia, sh.warp_sum[1][warp] = ib;
  __syncthreads();
  ta = tb = 0;
  ea = ia - a;
  eb = ib - b;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    if (w < warp) ea += sh.warp_sum[0][w], eb += sh.warp_sum[1][w];
    ta += sh.warp_sum[0][w];
    tb += sh.warp_sum[1][w];
  }
}

__global__ void __launch_bounds__(kSelThreads) page_select_kernel(const SelectParams p) {
  __shared__ SelectShared sh;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  int64_t seen;
  int32_t bad;
  const int64_t n = pages_of_row(p, r, &seen, &bad);
  if (bad && tid == 0) report(p.err, bad);
  const int64_t kept = n < p.top ? n : p.top;
  // entries of the rows before
  if (tid == 0) sh.before = 0;
  __syncthreads();
  {
    int64_t mine = 0;
    for (int64_t i = tid; i < r; i += kSelThreads) {
      int64_t s;
      int32_t w;
      const int64_t m = pages_of_row(p, i, &s, &w);
      mine += m < p.top ? m : p.top;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if ((tid & 31) == 0 && mine)
      atomicAdd(reinterpret_cast<unsigned long long*>(&sh.before), static_cast<unsigned long long>(mine));
  }
  __syncthreads();
  const int64_t before = sh.before;
  if (tid == 0) {
    if (r == 0) p.kv_indptr[0] = 0;
    p.kv_indptr[r + 1] = static_cast<int32_t>(before + kept);
    p.last_page[r] = static_cast<int32_t>(n > 0 ? seen - (n - 1) * p.page_size : 0);
    if (before + kept > p.max_indices) report(p.err, kErrCapacity);
  }
  const float* scores = p.scores + r * p.scores_stride;
  const int32_t* table = p.table + r / p.q_len * p.table_stride;
  int32_t* cols = p.kept_columns != nullptr ? p.kept_columns + r * p.top : nullptr;
  auto put = [&](int64_t rank, int64_t col) {
    if (before + rank < p.max_indices) p.kv_indices[before + rank] = table[col];
    if (cols != nullptr) cols[rank] = static_cast<int32_t>(col);
  };
  if (cols != nullptr)
    for (int64_t i = kept + tid; i < p.top; i += kSelThreads) cols[i] = -1;
  if (n <= p.top) {
    for (int64_t i = tid; i < n; i += kSelThreads) put(i, i);
    return;
  }
  const int64_t lo = p.first, hi = n - p.last;
  uint32_t need = static_cast<uint32_t>(p.top - p.first - p.last);     // of the columns between
  uint32_t prefix = 0;
  for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int64_t i = lo + tid; i < hi; i += kSelThreads) {
      const uint32_t k = key_of(scores[i]);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    // byte v: fewer than `need` scores lie above it, at least `need` from it on
    uint32_t ea, eb, ta, tb;
    const uint32_t mine = sh.hist[255 - tid];              // thread t: byte 255 - t
    scan2(sh, mine, 0, ea, eb, ta, tb);
    if (ea < need && ea + mine >= need) {
      sh.byte = 255 - tid;
      sh.above = ea;
    }
    __syncthreads();
    prefix |= sh.byte << shift;
    need -= sh.above;
    __syncthreads();
  }
  // `need` of the columns with the key `prefix` are kept, and all above it
  // (need 0 from the start: none)
  const bool none = p.top == p.first + p.last;
  uint32_t run_above = 0, run_equal = 0;
  for (int64_t base = 0; base < n; base += kSelThreads) {
    const int64_t i = base + tid;
    uint32_t above = 0, equal = 0;
    if (i < n) {
      if (i < lo || i >= hi) {
        above = 1;
      } else if (!none) {
        const uint32_t k = key_of(scores[i]);
        above = k > prefix;
        equal = k == prefix;
      }
    }
    uint32_t ea, eb, ta, tb;
    scan2(sh, above, equal, ea, eb, ta, tb);
    ea += run_above;
    eb += run_equal;
    if (above || (equal && eb < need)) put(ea + (eb < need ? eb : need), i);
    run_above += ta;
    run_equal += tb;
  }
}

}  // namespace
}  // namespace mla

namespace {
bool table_ok(const int32_t* table, int64_t stride, int32_t columns, int32_t batch, int32_t page) {
  return batch >= 1 && page >= 1 && columns >= 0 && stride >= columns &&
         (table != nullptr || columns == 0) && mla::ptr_aligned(table, 4);
}
}  // namespace

extern "C" mla_status mla_page_bounds(const void* kv, mla_dtype kv_dtype, const uint8_t* kv_e8m0,
                                      int64_t kv_e8m0_row_stride, int64_t kv_pool_rows,
                                      int32_t page_size, const int32_t* old_lens,
                                      const int32_t* new_lens, int32_t batch_size,
                                      const int32_t* block_table, int64_t table_stride,
                                      int32_t table_pages, void* bounds, int64_t num_pages,
                                      int32_t* err, mla_stream_t stream_) {
  if (!table_ok(block_table, table_stride, table_pages, batch_size, page_size) || old_lens == nullptr ||
      kv == nullptr || bounds == nullptr || num_pages < 1 || kv_pool_rows < 1 ||
      kv_pool_rows > INT32_MAX || kv_dtype < MLA_DTYPE_BF16 || kv_dtype > MLA_DTYPE_MXFP4)
    return MLA_ERR_INVALID_ARG;
  if (kv_dtype == MLA_DTYPE_MXFP4 && (kv_e8m0 == nullptr || kv_e8m0_row_stride < 18))
    return MLA_ERR_INVALID_ARG;
  if (!mla::ptr_aligned(kv, 16) || !mla::ptr_aligned(bounds, 16) || !mla::ptr_aligned(old_lens, 4) ||
      !mla::ptr_aligned(new_lens, 4) || !mla::ptr_aligned(err, 4))
    return MLA_ERR_INVALID_ARG;
  if (table_pages == 0) table_stride = 0;
  mla::BoundsParams p{static_cast<const uint8_t*>(kv), kv_e8m0, kv_e8m0_row_stride, kv_pool_rows,
                      static_cast<uint16_t*>(bounds), num_pages, block_table, table_stride,
                      table_pages, old_lens, new_lens, page_size, err};
  const int32_t slices = std::max(1, std::min(table_pages, 1216 / std::min(batch_size, 1216)));
  const dim3 grid(batch_size, slices);
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (kv_dtype == MLA_DTYPE_BF16)
    mla::page_bounds_kernel<MLA_DTYPE_BF16><<<grid, mla::kBoundThreads, 0, stream>>>(p);
  else if (kv_dtype == MLA_DTYPE_FP8_E4M3)
    mla::page_bounds_kernel<MLA_DTYPE_FP8_E4M3><<<grid, mla::kBoundThreads, 0, stream>>>(p);
  else
    mla::page_bounds_kernel<MLA_DTYPE_MXFP4><<<grid, mla::kBoundThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_page_scores(const void* q, mla_dtype q_dtype, const float* q_scale,
                                      const float* kv_scale, const void* bounds, int64_t num_pages,
                                      const int32_t* lens, int32_t batch_size, int32_t q_len,
                                      int32_t page_size, const int32_t* block_table,
                                      int64_t table_stride, int32_t table_pages, float* scores,
                                      int64_t scores_stride, int32_t* err, mla_stream_t stream_) {
  if (!table_ok(block_table, table_stride, table_pages, batch_size, page_size) || lens == nullptr ||
      q == nullptr || bounds == nullptr || num_pages < 1 || q_len < 1 || q_len > MLA_MAX_Q_LEN ||
      (scores == nullptr && table_pages > 0) || scores_stride < table_pages)
    return MLA_ERR_INVALID_ARG;
  if (q_dtype != MLA_DTYPE_BF16 && q_dtype != MLA_DTYPE_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  if (q_dtype == MLA_DTYPE_FP8_E4M3 && q_scale == nullptr) return MLA_ERR_INVALID_ARG;
  if (!mla::ptr_aligned(q, 16) || !mla::ptr_aligned(bounds, 16) || !mla::ptr_aligned(lens, 4) ||
      !mla::ptr_aligned(scores, 4) || !mla::ptr_aligned(q_scale, 4) ||
      !mla::ptr_aligned(kv_scale, 4) || !mla::ptr_aligned(err, 4))
    return MLA_ERR_INVALID_ARG;
  if (table_pages == 0) return MLA_OK;
  mla::ScoresParams p{q, q_dtype == MLA_DTYPE_FP8_E4M3 ? 1 : 0, q_dtype == MLA_DTYPE_FP8_E4M3 ? q_scale : nullptr,
                      kv_scale, static_cast<const uint16_t*>(bounds), num_pages, block_table,
                      table_stride, table_pages, lens, page_size, q_len, scores, scores_stride, 0, err};
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  constexpr int32_t kPages = mla::kScoreWarps * 8;
  const int64_t rows = static_cast<int64_t>(batch_size) * q_len;
  const bool wide = rows * table_pages >= 152 * 8 * kPages;
  p.chunks = (table_pages - 1) / (wide ? 4 * kPages : kPages) + 1;
  if (static_cast<int64_t>(p.chunks) * batch_size > INT32_MAX) return MLA_ERR_INVALID_ARG;
  const dim3 grid(p.chunks * batch_size, q_len);
  if (wide)
    mla::page_scores_kernel<4><<<grid, 32 * mla::kScoreWarps, 0, stream>>>(p);
  else
    mla::page_scores_kernel<1><<<grid, 32 * mla::kScoreWarps, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" mla_status mla_page_select(const float* scores, int64_t scores_stride,
                                      const int32_t* lens, int32_t batch_size, int32_t q_len,
                                      int32_t page_size, const int32_t* block_table,
                                      int64_t table_stride, int32_t table_pages, int32_t top_pages,
                                      int32_t first_pages, int32_t last_pages, int32_t* kv_indptr,
                                      int32_t* kv_last_page_len, int32_t* kv_indices,
                                      int64_t max_indices, int32_t* columns, int32_t* err,
                                      mla_stream_t stream_) {
  if (!table_ok(block_table, table_stride, table_pages, batch_size, page_size) || lens == nullptr ||
      (scores == nullptr && table_pages > 0) || scores_stride < table_pages || q_len < 1 ||
      q_len > MLA_MAX_Q_LEN || top_pages < 1 || first_pages < 0 || last_pages < 1 ||
      static_cast<int64_t>(first_pages) + last_pages > top_pages || kv_indptr == nullptr ||
      kv_last_page_len == nullptr || max_indices < 0 || (kv_indices == nullptr && max_indices > 0))
    return MLA_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(batch_size) * q_len;
  if (rows * std::min(top_pages, table_pages) > INT32_MAX || rows > INT32_MAX) return MLA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(scores), static_cast<const void*>(lens),
                        static_cast<const void*>(kv_indptr), static_cast<const void*>(kv_last_page_len),
                        static_cast<const void*>(kv_indices), static_cast<const void*>(columns),
                        static_cast<const void*>(err)})
    if (!mla::ptr_aligned(x, 4)) return MLA_ERR_INVALID_ARG;
  mla::SelectParams p{scores, scores_stride, block_table, table_stride, table_pages, lens,
                      page_size, q_len, rows, top_pages, first_pages, last_pages, kv_indptr,
                      kv_last_page_len, kv_indices, max_indices, columns, err};
  mla::page_select_kernel<<<static_cast<unsigned>(rows), mla::kSelThreads, 0,
                            reinterpret_cast<cudaStream_t>(stream_)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
