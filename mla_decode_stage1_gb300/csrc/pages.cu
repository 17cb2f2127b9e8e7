// pages.cu -- choosing the pages that a query attends to: the bounds of every
// page's rows, the score of each page for each query, and the best pages as the
// page table of a decode call.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "layer.h"
#include "ptx.cuh"
#include "shared.h"

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
// These kernels are launched while the one before them in the stream ends: all that
// they read and write is touched behind this wait for its end.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
// Bound: memory, one pass over the new rows; latency for a step of one token.  The
// pages of all requests are one list (every CTA adds up the requests' counts, from
// L2), handed out to the CTAs in turn, so that requests of any lengths are even work.
// bf16 rows in pages of 32, 34 MB, take 8.9 us (3.8 TB/s; 0.8 more with 4 rows of a thread
// ahead instead of 8); a row for each of 256 requests 4.8 (1.5 more with 8 e4m3 rows
// ahead).

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
  int32_t bs, page_size;
  int32_t* err;
};

template <int KV>
__global__ void __launch_bounds__(kBoundThreads, KV == MLA_DTYPE_BF16 ? 4 : 3)
    page_bounds_kernel(const BoundsParams p) {
  constexpr int kPieces = KV == MLA_DTYPE_BF16 ? 72 : KV == MLA_DTYPE_FP8_E4M3 ? 36 : 18;
  constexpr int kRows = kBoundThreads / kPieces;        // rows at a time
  constexpr int kWords = kQkDim / 2 / kPieces;          // bf16 pairs of a piece
  constexpr int kAhead = KV == MLA_DTYPE_BF16 ? 8 : KV == MLA_DTYPE_FP8_E4M3 ? 4 : 2;
  __shared__ uint32_t part[2][kRows][kQkDim / 2];
  __shared__ uint32_t ends[kBoundThreads];               // pages of the requests up to each
  __shared__ uint32_t warp_sum[kBoundThreads / 32];
  const int piece = threadIdx.x % kPieces, group = threadIdx.x / kPieces;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t page_size = p.page_size;
  auto lengths = [&](int b, uint32_t& old_len, uint32_t& new_len) {
    const int32_t o = p.old_lens[b], n = p.new_lens != nullptr ? p.new_lens[b] : 1;
    old_len = o < 0 ? 0 : o;
    new_len = n < 0 ? 0 : n;
    return o < 0 || n < 0 ? kErrBadLength : 0;
  };
  wait_for_stream();
  uint32_t mine = blockIdx.x;                            // the next page of the list to do
  uint32_t before = 0;                                   // pages of the chunks before
  for (int b0 = 0; b0 < p.bs; b0 += kBoundThreads) {
    uint32_t count = 0, old_len, new_len;
    if (b0 + static_cast<int>(threadIdx.x) < p.bs) {
      int32_t bad = lengths(b0 + threadIdx.x, old_len, new_len);
      // (their sum may be beyond 31 bits, not beyond 32)
      const uint32_t end = (old_len + new_len - 1) / page_size + 1;
      if (new_len > 0) {
        if (end > static_cast<uint32_t>(p.table_pages)) bad |= kErrCapacity;
        const uint32_t first = old_len / page_size, last = min(end, static_cast<uint32_t>(p.table_pages));
        count = last > first ? last - first : 0;
      }
      if (bad && blockIdx.x == 0) report(p.err, bad);
    }
    uint32_t sum = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += warp_sum[w];
    ends[threadIdx.x] = sum;
    __syncthreads();
    const uint32_t total = ends[kBoundThreads - 1];
    for (; mine - before < total; mine += gridDim.x) {
      // request and column of the page
      uint32_t at = 0;
#pragma unroll
      for (uint32_t step = 256; step > 0; step >>= 1)
        if (at + step <= kBoundThreads && ends[at + step - 1] <= mine - before) at += step;
      const int b = b0 + static_cast<int>(at);
      lengths(b, old_len, new_len);
      const uint32_t first = old_len / page_size;
      const uint32_t j = first + mine - before - (at > 0 ? ends[at - 1] : 0);
      const int64_t page = p.table[b * p.table_stride + j];
      if (page < 0 || page >= p.pages || (page + 1) * p.page_size > p.pool_rows) {
        if (threadIdx.x == 0) report(p.err, kErrBadPage);
        continue;
      }
      const int r0 = static_cast<int>(j == first ? old_len % page_size : 0);
      const int r1 = static_cast<int>(min(old_len + new_len - j * page_size, page_size));
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
          v[u] = ld_na_v4(p.kv + (row * kPieces + piece) * 16);
          if constexpr (KV == MLA_DTYPE_MXFP4)
            e[u] = ld_u8(p.e8m0 + row * p.e8m0_stride + piece);
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
      // a thread per pair of dims for what the page has
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
    before += total;
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
// Bound: memory, 2,304 bytes a page.  A warp holds 8 kTiles pages; a lane loads 32
// bytes (16 dims) of a page's bounds, a quad whole lines, kAhead steps of 64 dims
// ahead of their use.  They are its share of four instructions: the order of the sum over d is
// free, so lane c of a quad takes dims 16 c .. 16 c + 15 of 64, for the queries as
// well.  32,768 pages, 78 MB with all else, take 13.4 us (5.8 TB/s, of 6.8 that a copy
// reaches).

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

// 32 bytes, not kept in L1 (read once).
__device__ __forceinline__ void ld_na_32(const void* ptr, uint32_t (&v)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                 "=r"(v[7])
               : "l"(ptr));
}

// Tokens that query token t of a request with n cached tokens sees.
__device__ __forceinline__ int64_t seen_by(int64_t n, int q_len, int t) {
  const int64_t s = n - q_len + 1 + t;
  return s < 0 ? 0 : s;
}

template <int kTiles, int kAhead>
__global__ void __launch_bounds__(32 * kScoreWarps) page_scores_kernel(const ScoresParams p) {
  __shared__ __align__(16) uint16_t qs[kHeads * kQPitch];
  const int b = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks, t = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(b) * p.q_len + t;
  const int64_t cta0 = static_cast<int64_t>(chunk) * (kScoreWarps * 8 * kTiles);
  const int64_t page0 = cta0 + warp * (8 * kTiles);
  const int g = lane >> 2, c = lane & 3;
  wait_for_stream();
  // (read beside the length; what is behind it is not looked at)
  int32_t entry[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
    entry[i] = p.table[b * p.table_stride + min(page0 + 8 * i + g, static_cast<int64_t>(p.columns - 1))];
  int64_t n = p.lens[b];
  // (later query tokens see more)
  const bool first_cta = chunk == 0 && threadIdx.x == 0;
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
  if (cta0 >= pages) {
    for (int i = threadIdx.x; i < kScoreWarps * 8 * kTiles; i += 32 * kScoreWarps)
      if (cta0 + i < p.columns) out[cta0 + i] = -INFINITY;
    return;
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    // (columns past the last: page 0)
    if (page0 + 8 * i + g >= pages) entry[i] = 0;
    if (entry[i] < 0 || entry[i] >= p.pages) {
      if (c == 0) report(p.err, kErrBadPage);
      entry[i] = 0;
    }
  }
  const uint16_t* bounds = p.bounds + 16 * c;
  uint32_t lo[kAhead][kTiles][8], hi[kAhead][kTiles][8];
  auto fetch = [&](int d, int at) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint16_t* src = bounds + static_cast<int64_t>(entry[i]) * (2 * kQkDim) + 64 * d;
      ld_na_32(src, lo[at][i]);
      ld_na_32(src + kQkDim, hi[at][i]);
    }
  };
#pragma unroll
  for (int d = 0; d < kAhead; ++d) fetch(d, d);
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
  // The instruction's own sums round towards zero: 8 in a row, then one rounded
  // addition (72 in a row were 1.2e-6 off, against 1e-7).
  float sum[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[i][k] = 0.0f;
  const uint16_t* qa = qs + g * kQPitch + 16 * c;
#pragma unroll
  for (int d = 0; d < kQkDim / 64; ++d) {
    const int at = d % kAhead;
    float acc[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 x = *reinterpret_cast<const uint4*>(qa + 64 * d + 8 * half);
      const uint4 y = *reinterpret_cast<const uint4*>(qa + 8 * kQPitch + 64 * d + 8 * half);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
      uint32_t xp[4], xn[4], yp[4], yn[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        xp[k] = max_nan_bf16x2(xs[k], 0u); xn[k] = min_nan_bf16x2(xs[k], 0u);
        yp[k] = max_nan_bf16x2(ys[k], 0u); yn[k] = min_nan_bf16x2(ys[k], 0u);
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const uint32_t* h = hi[at][i] + 4 * half;
        const uint32_t* l = lo[at][i] + 4 * half;
        mma_16816(acc[i], xp[0], yp[0], xp[1], yp[1], h[0], h[1]);
        mma_16816(acc[i], xp[2], yp[2], xp[3], yp[3], h[2], h[3]);
        mma_16816(acc[i], xn[0], yn[0], xn[1], yn[1], l[0], l[1]);
        mma_16816(acc[i], xn[2], yn[2], xn[3], yn[3], l[2], l[3]);
      }
    }
    if (d + kAhead < kQkDim / 64) fetch(d + kAhead, at);
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[i][k] += acc[i][k];
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
// A CTA per row.  Up to 256 columns: every score's rank by comparison with all
// others (in shared memory), which takes fewer steps than anything with a barrier
// between them.  Beyond: the range of the keys that holds the smallest kept one is
// cut into 2,048 bins again and again, the scores in it counted, until what is in a
// bin is kept whole or has one key (2 rounds for scores that are spread, 3 at most).
// A thread then holds consecutive columns, so that one scan of the threads' counts
// places every kept column, in the pages' place; their pages come last, with all
// loads of them under way at once.
//
// Bound: latency, of loads that wait for one another above all: the scores (and for
// short rows the pages) are read beside the lengths.  256 rows of 128 columns 2.7 us,
// one of 16,384 13 us, of 32,768 20.  The keys of longer rows do not fit in shared
// memory, and every round reads the scores again: one of 32,769 35 us, of 65,536 64, of
// 131,072 150.

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

// Pages that row r sees, with what is wrong with its length.
__device__ __forceinline__ uint32_t pages_of_row(const SelectParams& p, uint32_t r, uint32_t* seen,
                                                 int32_t* bad) {
  const uint32_t b = r / p.q_len, t = r % p.q_len;
  const int32_t n = p.lens[b];
  *bad = n < 0 ? kErrBadLength : 0;
  uint32_t s = static_cast<uint32_t>(seen_by(n < 0 ? 0 : n, p.q_len, t));
  uint32_t pages = (s + p.page_size - 1) / p.page_size;
  if (pages > static_cast<uint32_t>(p.columns)) {
    *bad = kErrCapacity;
    pages = p.columns;
    s = pages * p.page_size;
  }
  *seen = s;
  return pages;
}

constexpr int kBins = 2048;
template <int kThreads>
struct SelectShared {
  uint32_t warp_sum[2][32];
  // per warp: smallest and largest key, entries of the rows before
  uint32_t least[kThreads / 32], most[kThreads / 32];
  unsigned long long before[kThreads / 32];
  uint32_t bin, above, inside;
};

// Exclusive sums over the CTA of two counts.
template <int kThreads>
__device__ __forceinline__ void scan2(SelectShared<kThreads>& sh, uint32_t a, uint32_t b,
                                      uint32_t& ea, uint32_t& eb) {
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia += x, ib += y;
  }
  if (lane == 31) sh.warp_sum[0][warp] = ia, sh.warp_sum[1][warp] = ib;
  __syncthreads();
  // every warp adds up the warps before it
  uint32_t x = lane < warp ? sh.warp_sum[0][lane] : 0, y = lane < warp ? sh.warp_sum[1][lane] : 0;
  static_assert(kWarps <= 32, "a lane per warp");
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
  ea = x + ia - a;
  eb = y + ib - b;
}

// Columns that the counting form takes.
constexpr uint32_t kCountColumns = 256;
constexpr uint32_t kKeysInShared = 32768;      // 128 KB

template <int kThreads, bool kCount>
__global__ void __launch_bounds__(kThreads) page_select_kernel(const SelectParams p) {
  constexpr uint32_t kEarly = kCount ? kCountColumns / kThreads : 8;
  constexpr int kWarps = kThreads / 32;
  __shared__ SelectShared<kThreads> sh;
  extern __shared__ __align__(16) uint32_t dynamic[];
  uint32_t* hist = dynamic;
  uint32_t* keys = dynamic + (kCount ? 0 : kBins);       // of the columns, while they fit
  const uint32_t r = blockIdx.x;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* scores = p.scores + r * p.scores_stride;
  const int32_t* table = p.table + r / p.q_len * p.table_stride;
  const uint32_t columns = p.columns;
  wait_for_stream();
  // The first columns of a thread, read beside the length: what is behind it is not
  // looked at.
  float early[kEarly];
  int32_t entry[kEarly];
#pragma unroll
  for (uint32_t u = 0; u < kEarly; ++u) {
    const uint32_t i = tid + u * kThreads;
    early[u] = i < columns ? scores[i] : 0.0f;
    if constexpr (kCount) entry[u] = i < columns ? table[i] : 0;
  }
  uint32_t seen;
  int32_t bad;
  const uint32_t n = pages_of_row(p, r, &seen, &bad);
  const uint32_t top = p.top, kept = n < top ? n : top;
  const bool all = n <= top;
  // the columns between (of n > top)
  const uint32_t lo = all ? 0 : p.first, hi = all ? 0 : n - p.last, m = hi - lo;
  if (tid == 0 && bad) report(p.err, bad);
  // entries of the rows before
  {
    uint32_t mine = 0;
    for (uint32_t i = tid; i < r; i += kThreads) {
      uint32_t s;
      int32_t w;
      const uint32_t k = pages_of_row(p, i, &s, &w);
      mine += k < top ? k : top;
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) sh.before[warp] = mine;
  }
  // the keys, and the range of those between
  const bool held = kCount || n <= kKeysInShared;
  if constexpr (kCount) {
#pragma unroll
    for (uint32_t u = 0; u < kEarly; ++u) {
      const uint32_t i = tid + u * kThreads;
      keys[i] = i >= lo && i < hi ? key_of(early[u]) : 0u;    // (no score's key)
    }
  } else {
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    uint32_t least = 0xffffffffu, most = 0;
    auto take = [&](uint32_t i, float s) {
      const uint32_t k = key_of(s);
      if (held && i < n) keys[i] = k;
      if (i >= lo && i < hi) {
        least = min(least, k);
        most = max(most, k);
      }
    };
#pragma unroll
    for (uint32_t u = 0; u < kEarly; ++u) take(tid + u * kThreads, early[u]);
    for (uint32_t i = tid + kEarly * kThreads; i < hi; i += 8 * kThreads) {
      float s[8];
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) s[u] = i + u * kThreads < n ? scores[i + u * kThreads] : 0.0f;
#pragma unroll
      for (uint32_t u = 0; u < 8; ++u) take(i + u * kThreads, s[u]);
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) sh.least[warp] = least, sh.most[warp] = most;
  }
  __syncthreads();
  int64_t before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) before += sh.before[w];
  if (tid == 0) {
    if (r == 0) p.kv_indptr[0] = 0;
    p.kv_indptr[r + 1] = static_cast<int32_t>(before + kept);
    p.last_page[r] = static_cast<int32_t>(n > 0 ? seen - (n - 1) * p.page_size : 0);
    if (before + kept > p.max_indices) report(p.err, kErrCapacity);
  }
  int32_t* cols = p.kept_columns != nullptr ? p.kept_columns + static_cast<int64_t>(r) * top : nullptr;
  if (cols != nullptr)
    for (uint32_t i = kept + tid; i < top; i += kThreads) cols[i] = -1;
  const uint32_t need = top - p.first - p.last;          // of the columns between (n > top)
  if constexpr (kCount) {
    // a column's rank: how many of those between have a larger key, or an equal one and
    // stand before it; 32 columns at a time, which but for a warp's own are all before
    // it or all behind
    uint32_t rank[kEarly];
#pragma unroll
    for (uint32_t u = 0; u < kEarly; ++u) {
      uint32_t part[4] = {0, 0, 0, 0};
      rank[u] = 0;
      const uint32_t own = warp + u * kWarps;
      if (all || 32 * own >= hi || 32 * own + 32 <= lo) continue;
      const uint32_t k = keys[tid + u * kThreads], below = k - 1;
      for (uint32_t g = lo / 32; 32 * g < hi; ++g) {
        const uint4* x = reinterpret_cast<const uint4*>(keys + 32 * g);
        if (g == own) {
#pragma unroll
          for (uint32_t i = 0; i < 32; ++i) part[i % 4] += keys[32 * g + i] > (i < lane ? below : k);
        } else {
          const uint32_t limit = g < own ? below : k;
#pragma unroll
          for (uint32_t i = 0; i < 8; ++i) {
            const uint4 v = x[i];
            part[0] += v.x > limit;
            part[1] += v.y > limit;
            part[2] += v.z > limit;
            part[3] += v.w > limit;
          }
        }
      }
      rank[u] = part[0] + part[1] + part[2] + part[3];
    }
    uint32_t mask[kEarly];
#pragma unroll
    for (uint32_t u = 0; u < kEarly; ++u) {
      const uint32_t i = tid + u * kThreads;
      const bool stays = i < n && (all || i < lo || i >= hi || rank[u] < need);
      mask[u] = __ballot_sync(0xffffffffu, stays);
      if (lane == 0) sh.warp_sum[0][warp + u * kWarps] = __popc(mask[u]);
    }
    __syncthreads();
    // (the 32 columns of a warp stand together: one count for each)
    static_assert(kCountColumns / 32 <= 32, "a lane for 32 columns");
    const uint32_t count = sh.warp_sum[0][lane];
#pragma unroll
    for (uint32_t u = 0; u < kEarly; ++u) {
      const uint32_t i = tid + u * kThreads, w = i / 32;
      const uint32_t at = __reduce_add_sync(0xffffffffu, lane < w ? count : 0u) +
                          __popc(mask[u] & ((1u << lane) - 1));
      if (mask[u] >> lane & 1) {
        if (before + at < p.max_indices) p.kv_indices[before + at] = entry[u];
        if (cols != nullptr) cols[at] = static_cast<int32_t>(i);
      }
    }
    return;
  }
  // Columns first, in the place of the pages (those past max_indices: nowhere).
  auto put = [&](uint32_t rank, uint32_t col) {
    if (before + rank < p.max_indices) p.kv_indices[before + rank] = static_cast<int32_t>(col);
    if (cols != nullptr) cols[rank] = static_cast<int32_t>(col);
  };
  if (all) {
    for (uint32_t i = tid; i < n; i += kThreads) {
      if (before + i < p.max_indices) p.kv_indices[before + i] = table[i];
      if (cols != nullptr) cols[i] = static_cast<int32_t>(i);
    }
    return;
  }
  for (uint32_t i = tid; i < lo; i += kThreads) put(i, i);
  for (uint32_t i = hi + tid; i < n; i += kThreads) put(top - n + i, i);
  if (need > 0) {
    auto key = [&](uint32_t i) { return held ? keys[i] : key_of(scores[i]); };
    // All keys above b are kept, and `left` of those in [a, b].
    uint32_t a = __reduce_min_sync(0xffffffffu, sh.least[lane % kWarps]);
    uint32_t b = __reduce_max_sync(0xffffffffu, sh.most[lane % kWarps]);
    uint32_t left = need;
    bool whole = left == m;                              // those in [a, b] all are
    while (!whole && a < b) {
      const int shift = max(0, 21 - __clz(b - a));       // (b - a) >> shift < 2048
#pragma unroll 8
      for (uint32_t i = lo + tid; i < hi; i += kThreads) {
        const uint32_t k = key(i);
        if (k >= a && k <= b) atomicAdd(&hist[(k - a) >> shift], 1u);
      }
      __syncthreads();
      // bins from the top: thread t holds the t-th part of them
      constexpr int kPer = kBins / kThreads;
      uint32_t c[kPer], sum = 0, above, none;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        uint32_t& bin = hist[kBins - 1 - (kPer * tid + u)];
        c[u] = bin;
        bin = 0;
        sum += c[u];
      }
      scan2(sh, sum, 0, above, none);
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        if (above < left && above + c[u] >= left) {
          sh.bin = kBins - 1 - (kPer * tid + u);
          sh.above = above;
          sh.inside = c[u];
        }
        above += c[u];
      }
      __syncthreads();
      a += sh.bin << shift;
      if (b - a >= (1u << shift)) b = a + (1u << shift) - 1;
      left -= sh.above;
      whole = sh.inside == left;
      __syncthreads();
    }
    // Kept: keys above b, and in [a, b] all, or the first `left` of one key.
    uint32_t run_above = 0, run_in = 0;
    for (uint32_t base = lo; base < hi; base += kThreads * 32) {
      // consecutive columns of a thread, an odd number (banks)
      const uint32_t count = min(hi - base, static_cast<uint32_t>(kThreads * 32));
      const uint32_t per = min(((count + kThreads - 1) / kThreads) | 1u, 33u);
      const uint32_t i0 = base + per * tid, i1 = min(i0 + per, base + count);
      uint32_t na = 0, ni = 0;
      const uint32_t* part = keys;
      if (!held) {
        // (whole lines, to where a thread can walk along them)
        __syncthreads();
#pragma unroll 8
        for (uint32_t i = tid; i < count; i += kThreads) keys[i] = key_of(scores[base + i]);
        __syncthreads();
        part = keys - base;
      }
#pragma unroll 4
      for (uint32_t i = i0; i < i1; ++i) {
        const uint32_t k = part[i];
        na += k > b;
        ni += k >= a && k <= b;
      }
      uint32_t ea, ei;
      scan2(sh, na, ni, ea, ei);
      ea += run_above;
      ei += run_in;
#pragma unroll 4
      for (uint32_t i = i0; i < i1; ++i) {
        const uint32_t k = part[i];
        const bool in = k >= a && k <= b;
        if (k > b || (in && ei < left)) put(lo + ea + min(ei, left), i);
        ea += k > b;
        ei += in;
      }
      if (base + count < hi) {
        // totals, for the next part
        __syncthreads();
        if (tid == kThreads - 1) sh.above = ea, sh.inside = ei;
        __syncthreads();
        run_above = sh.above;
        run_in = sh.inside;
      }
    }
  }
  // then their pages
  __syncthreads();
  const int64_t room = p.max_indices - before;
  const int64_t written = min(room, static_cast<int64_t>(kept));
  int32_t* out = p.kv_indices + before;
  for (int64_t i = tid; i < written; i += 4 * kThreads) {
    int32_t c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) c[u] = i + u * kThreads < written ? out[i + u * kThreads] : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) c[u] = table[c[u]];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * kThreads < written) out[i + u * kThreads] = c[u];
  }
}

template <int kThreads, bool kCount>
cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  const uint32_t columns = p.columns;
  constexpr uint32_t kBinWords = kCount ? 0 : kBins;
  const uint32_t bytes = 4 * (kCount ? kCountColumns : kBinWords + std::min(columns, kKeysInShared));
  if (bytes > 32768) {
    const cudaError_t e = cudaFuncSetAttribute(page_select_kernel<kThreads, kCount>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               4 * (kBinWords + kKeysInShared));
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(page_select_kernel<kThreads, kCount>, dim3(static_cast<unsigned>(p.rows)), kThreads,
                bytes, stream, p);
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
  if (!mla::ptr_aligned(kv, 16) || !mla::ptr_aligned(bounds, 32) || !mla::ptr_aligned(old_lens, 4) ||
      !mla::ptr_aligned(new_lens, 4) || !mla::ptr_aligned(err, 4))
    return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(batch_size) * table_pages > INT32_MAX) return MLA_ERR_INVALID_ARG;
  if (table_pages == 0) table_stride = 0;
  mla::BoundsParams p{static_cast<const uint8_t*>(kv), kv_e8m0, kv_e8m0_row_stride, kv_pool_rows,
                      static_cast<uint16_t*>(bounds), num_pages, block_table, table_stride,
                      table_pages, old_lens, new_lens, batch_size, page_size, err};
  // (at most 8 CTAs an SM; the number of pages is known on the device only)
  const int64_t most = static_cast<int64_t>(batch_size) * std::max(table_pages, 1);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(most, 1216)));
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  auto* kernel = kv_dtype == MLA_DTYPE_BF16       ? mla::page_bounds_kernel<MLA_DTYPE_BF16>
                 : kv_dtype == MLA_DTYPE_FP8_E4M3 ? mla::page_bounds_kernel<MLA_DTYPE_FP8_E4M3>
                                                  : mla::page_bounds_kernel<MLA_DTYPE_MXFP4>;
  const cudaError_t e = mla::launch_dependent(kernel, grid, mla::kBoundThreads, 0, stream, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
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
  if (!mla::ptr_aligned(q, 16) || !mla::ptr_aligned(bounds, 32) || !mla::ptr_aligned(lens, 4) ||
      !mla::ptr_aligned(scores, 4) || !mla::ptr_aligned(q_scale, 4) ||
      !mla::ptr_aligned(kv_scale, 4) || !mla::ptr_aligned(err, 4))
    return MLA_ERR_INVALID_ARG;
  if (table_pages == 0) return MLA_OK;
  const bool fp8 = q_dtype == MLA_DTYPE_FP8_E4M3;
  mla::ScoresParams p{q, fp8 ? 1 : 0, fp8 ? q_scale : nullptr, kv_scale,
                      static_cast<const uint16_t*>(bounds), num_pages, block_table, table_stride,
                      table_pages, lens, page_size, q_len, scores, scores_stride, 0, err};
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  constexpr int32_t kPages = mla::kScoreWarps * 8;
  const int64_t rows = static_cast<int64_t>(batch_size) * q_len;
  // A tile a warp while all CTAs are on the machine at once (4 an SM): 32,768 pages
  // take 18.7 us in 1,024 such CTAs, 16.4 in 256 of four tiles a warp (two an SM; all 255
  // registers, and 24 bytes a thread spilled).
  const bool wide = rows * ((table_pages - 1) / kPages + 1) > 4 * 152;
  p.chunks = (table_pages - 1) / (wide ? 4 * kPages : kPages) + 1;
  if (static_cast<int64_t>(p.chunks) * batch_size > INT32_MAX) return MLA_ERR_INVALID_ARG;
  const dim3 grid(p.chunks * batch_size, q_len);
  auto* kernel = wide ? mla::page_scores_kernel<4, 3> : mla::page_scores_kernel<1, 4>;
  const cudaError_t e = mla::launch_dependent(kernel, grid, 32 * mla::kScoreWarps, 0, stream, p);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
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
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  // Counting: 512 rows of 256 columns 9.6 us (by ranges 10.3), one row 4.2 (6.2); of 512
  // columns 24.3 (10.3).  1,024 threads: a row of 16,384 columns 15.7 us (with 256
  // threads 27.7), of 8,192 12.3 (14.4), but 512 rows of 8,192 41 us (25.7).
  const int32_t few = rows > 152 ? 8192 : 4096;
  const cudaError_t e = table_pages <= static_cast<int32_t>(mla::kCountColumns)
                            ? mla::launch_select<256, true>(p, stream)
                        : table_pages <= few ? mla::launch_select<256, false>(p, stream)
                                             : mla::launch_select<1024, false>(p, stream);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
