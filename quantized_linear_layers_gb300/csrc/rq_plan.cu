// rq_plan.cu -- cache slots, positions and page-table entries of a pass's new
// tokens, from the lengths of its sequences (sm_103a).
//
// Sequence b with n cached and c new tokens holds ceil(n / ps) pages and needs
// ceil((n + c) / ps); its first new page is number sum_{a < b} need_a of the
// pass, its first row number sum_{a < b} span_a (span: c, or new_tokens in the
// padded layout).  Both are exclusive sums over the batch.
//
// Every CTA takes kRows rows and forms the sums over the batch by itself, as
// far as its rows need them: 8 bytes a sequence from L2 cost less than a
// second launch or a wait between CTAs.  A sequence marks its first row inside
// the CTA; a running maximum over the marks tells each row its sequence.  New
// page i's first token sits at an offset of 0, so that token's row writes the
// table entry, and rows read the stack, not the entries written here: nothing
// passes between CTAs.
#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {

namespace {

__device__ unsigned int g_plan_error = 0;  // bit 1: an index outside its array

constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPer = 4;                      // sequences and rows a thread takes at a time
constexpr int kRows = kPlanThreads * kPer;   // rows of a CTA
constexpr int kPlaceMax = 0x7FFFFFFF;

struct PlanArgs {
  const int32_t *length, *count;
  int batch, new_tokens, lg_page;
  int32_t* page_table;
  int max_pages;
  const int32_t* free_pages;
  int free_capacity;
  const int32_t* free_count;
  int32_t* free_left;
  int64_t* slot;
  int32_t *position, *sequence;
  int rows;
  int32_t *row_start, *next_length;
};

// What a row needs of its sequence.
struct Seq {
  int b, length, count;
  int have;        // pages that hold its cached tokens
  int64_t start;   // its first row
  int64_t page0;   // its first new page, counted over the pass
};

__device__ __forceinline__ int64_t warp_scan64(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) batch_plan_kernel(const PlanArgs a) {
  __shared__ Seq seq[kRows];              // at a sequence's first row inside the CTA
  __shared__ int mark[kRows];             // that row, or -1
  __shared__ int64_t part[2][2][kPlanWarps];
  __shared__ int warp_top[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r0 = (int64_t)blockIdx.x * kRows;
  const int64_t r1 = r0 + kRows < a.rows ? r0 + kRows : a.rows;
  const bool lead = blockIdx.x == 0;  // also writes what there is once per sequence
  bool bad = false;

  for (int i = tid; i < kRows; i += kPlanThreads) mark[i] = -1;
  pdl_wait();
  pdl_trigger();
  const int stack = *a.free_count;
  const int top = min(max(stack, 0), a.free_capacity);  // valid entries
  if (stack != top) bad = true;
  __syncthreads();

  // the sums over the batch
  int64_t rows = 0, pages = 0;  // of the sequences before this round's
  for (int b0 = 0, round = 0; b0 < a.batch; b0 += kRows, round ^= 1) {
    int n[kPer], c[kPer], need[kPer], have[kPer];
    int64_t my_rows = 0, my_pages = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = b0 + tid * kPer + i;
      n[i] = b < a.batch ? a.length[b] : -1;
      c[i] = b < a.batch ? (a.count != nullptr ? a.count[b] : a.new_tokens) : 0;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = b0 + tid * kPer + i;
      if (n[i] < 0 || c[i] < 0) c[i] = 0;
      if (a.new_tokens > 0 && c[i] > a.new_tokens) {
        c[i] = a.new_tokens;
        bad = true;
      }
      const int64_t end = (int64_t)max(n[i], 0) + c[i];
      const int64_t ps = (int64_t)1 << a.lg_page;
      have[i] = (int)((max(n[i], 0) + ps - 1) >> a.lg_page);
      const int64_t all = (end + ps - 1) >> a.lg_page;
      need[i] = max((int)(all < a.max_pages ? all : a.max_pages) - have[i], 0);
      my_rows += b >= a.batch ? 0 : a.new_tokens > 0 ? a.new_tokens : c[i];
      my_pages += c[i] > 0 ? need[i] : 0;
    }
    const int64_t scan_r = warp_scan64(my_rows, lane), scan_p = warp_scan64(my_pages, lane);
    if (lane == 31) {
      part[round][0][warp] = scan_r;
      part[round][1][warp] = scan_p;
    }
    __syncthreads();
    int64_t row = rows + scan_r - my_rows, page = pages + scan_p - my_pages;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      if (w < warp) {
        row += part[round][0][w];
        page += part[round][1][w];
      }
      rows += part[round][0][w];
      pages += part[round][1][w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = b0 + tid * kPer + i;
      if (b < a.batch) {
        const int span = a.new_tokens > 0 ? a.new_tokens : c[i];
        const int64_t first = row > r0 ? row : r0;
        if (first < r1 && row + span > first) {
          const int at = (int)(first - r0);
          seq[at] = Seq{b, n[i], c[i], have[i], row, page};
          mark[at] = at;
        }
        if (lead) {
          const int64_t end = (int64_t)n[i] + c[i];
          if (end > kPlaceMax) bad = true;
          if (a.next_length != nullptr)
            a.next_length[b] = (int)(end < kPlaceMax ? end : kPlaceMax);
          if (a.row_start != nullptr) a.row_start[b] = (int)(row < a.rows ? row : a.rows);
        }
        row += span;
        page += c[i] > 0 ? need[i] : 0;
      }
    }
    if (!lead && rows >= r1) break;  // (the same for every thread)
  }
  if (lead && tid == 0) {
    const int64_t left = (int64_t)top - pages;
    *a.free_left = (int)(left > -kPlaceMax ? left : -kPlaceMax);
    if (a.row_start != nullptr) a.row_start[a.batch] = (int)(rows < a.rows ? rows : a.rows);
    if (rows > a.rows) bad = true;
  }
  __syncthreads();

  // the rows: the last mark at or before each
  int at[kPer];
  int last = -1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    last = max(last, mark[tid * kPer + i]);
    at[i] = last;
  }
  int scan = last;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan = max(scan, x);
  }
  if (lane == 31) warp_top[warp] = scan;
  int before = __shfl_up_sync(0xFFFFFFFFu, scan, 1);
  if (lane == 0) before = -1;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = max(before, warp_top[w]);

#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t r = r0 + tid * kPer + i;
    if (r >= r1) break;
    const int m = max(at[i], before);
    int64_t slot = -1;
    int position = 0, b = -1;
    if (m >= 0) {
      const Seq s = seq[m];
      const int64_t k = r - s.start;
      if (k < s.count) {
        const int64_t place = s.length + k;
        const int64_t pg = place >> a.lg_page;
        const int off = (int)(place & ((1 << a.lg_page) - 1));
        b = s.b;
        position = (int)(place < kPlaceMax ? place : kPlaceMax);
        if (pg < a.max_pages) {
          int32_t* entry = a.page_table + (int64_t)s.b * a.max_pages + pg;
          int page;
          if (pg < s.have) {
            page = *entry;
          } else {
            const int64_t i_free = top - 1 - (s.page0 + pg - s.have);
            page = i_free >= 0 ? a.free_pages[i_free] : -1;
            if (off == 0) *entry = page;
          }
          if (page >= 0) slot = ((int64_t)page << a.lg_page) + off;
        }
        if (slot < 0) bad = true;
      }
    }
    a.slot[r] = slot;
    a.position[r] = position;
    if (a.sequence != nullptr) a.sequence[r] = b;
  }
  if (bad) atomicOr(&g_plan_error, 2u);
}

}  // namespace

rq_status launch_batch_plan(const int32_t* length, const int32_t* count, int batch,
                            int new_tokens, int page_size, int32_t* page_table, int max_pages,
                            const int32_t* free_pages, int free_capacity,
                            const int32_t* free_count, int32_t* free_left, int64_t* slot,
                            int32_t* position, int32_t* sequence, int rows, int32_t* row_start,
                            int32_t* next_length, cudaStream_t st) {
  int lg = 0;
  while ((1 << lg) < page_size) ++lg;
  const PlanArgs a = {length,     count,      batch,         new_tokens, lg,
                      page_table, max_pages,  free_pages,    free_capacity, free_count,
                      free_left,  slot,       position,      sequence,   rows,
                      row_start,  next_length};
  const int64_t ctas = ((int64_t)rows + kRows - 1) / kRows;
  return launch_kernel(batch_plan_kernel, dim3((unsigned)(ctas < 1 ? 1 : ctas)),
                       dim3(kPlanThreads), 0, st, a);
}

rq_status read_and_clear_plan_error() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_plan_error, sizeof(v)) != cudaSuccess) return RQ_ERR_CUDA;
  if (v == 0) return RQ_OK;
  const unsigned int zero = 0;
  if (cudaMemcpyToSymbol(g_plan_error, &zero, sizeof(zero)) != cudaSuccess) return RQ_ERR_CUDA;
  return RQ_ERR_INDEX;
}

}  // namespace rq
