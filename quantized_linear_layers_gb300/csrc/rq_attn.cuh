// rq_attn.cuh -- what the attention kernels share: their arguments, how work
// is cut between CTAs, and the exact conversion of cache codes (sm_103a).
#pragma once

#include <cuda_bf16.h>

#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {

constexpr int kMaxItems = 1024;  // (sequence, row tile) pairs that a launch cuts by length

struct SharedSegment;
struct AttnArgs {
  const void* q;
  void* out;
  int64_t q_stride, q_bytes;
  const uint8_t *k, *v;
  const float *ks, *vs;
  const int32_t *table, *length;
  const unsigned long long* tree;
  int batch, new_tokens, q_heads, kv_heads, group, rows, row_tiles;
  Divisor by_heads, by_group, by_tiles;  // kv_heads, group, row_tiles
  int max_pages, lg_page;
  int64_t pages;
  float scale_log2;
  int dtype;
  int direct;  // whole segments only
  float* part;
  unsigned int* counter;
  SharedSegment* shares;  // per CTA: the segment it begins for several (null: no join)
  float4* flushed;        // per CTA: sums of output rows taken out of TMEM
  unsigned int* error;  // bit 1: an index outside its array
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (a, b) as an f16 pair and, in `lo`, what the rounding left over.
__device__ __forceinline__ uint32_t split_half2(float a, float b, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  lo = pack_half2(a - f.x, b - f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Codes as f16 pairs, exactly.  E4M3 has a conversion; 8-bit integers, biased
// by 128, become the low mantissa bits of 1024 + b, less 1152.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
  return h;
}

// Four E4M3 codes, its NaN (0x7F, 0xFF) made zero.  A V row that some query
// rows see and others do not takes part in the product with weights of 0 for
// these, and 0 * NaN is not 0.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  const uint32_t t = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // a byte's top bit: NaN
  return w & ~(t | (t - (t >> 7)));
}

__device__ __forceinline__ uint32_t minus_1152(uint32_t h) {
  const uint32_t bias = 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h),
                            *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Bytes (0, 1) and (2, 3) of a word.
template <bool I8>
__device__ __forceinline__ void codes_in_order(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (I8) {
    const uint32_t u = w ^ 0x80808080u;
    a = minus_1152(__byte_perm(u, 0x64646464u, 0x4140));
    b = minus_1152(__byte_perm(u, 0x64646464u, 0x4342));
  } else {
    a = e4m3_pair(w & 0xFFFFu);
    b = e4m3_pair(w >> 16);
  }
}

// Bytes (0, 2) and (1, 3).
template <bool I8>
__device__ __forceinline__ void codes_across(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (I8) {
    const uint32_t u = w ^ 0x80808080u;
    a = minus_1152(__byte_perm(u, 0x64646464u, 0x4240));
    b = minus_1152(__byte_perm(u, 0x64646464u, 0x4341));
  } else {
    const uint32_t x = e4m3_pair(w & 0xFFFFu), y = e4m3_pair(w >> 16);
    a = __byte_perm(x, y, 0x5410);
    b = __byte_perm(x, y, 0x7632);
  }
}

// (v, mx, sum) joined with another partial row: its output piece, and its
// maximum and sum.
__device__ __forceinline__ void merge(float4& v, float& mx, float& sum, const float4& ov,
                                      const float2& ml, float c) {
  const float mn = fmaxf(mx, ml.x);
  if (mn == -INFINITY) {
    sum += ml.y;  // 0, or the NaN of a row whose scores all are
    return;
  }
  const float f0 = ex2((mx - mn) * c), f1 = ex2((ml.x - mn) * c);
  v.x = v.x * f0 + ov.x * f1;
  v.y = v.y * f0 + ov.y * f1;
  v.z = v.z * f0 + ov.z * f1;
  v.w = v.w * f0 + ov.w * f1;
  sum = sum * f0 + ml.y * f1;
  mx = mn;
}

// Fetch what the launch reads first and only once, q and the page table, into
// L2 while the lengths are on their way.
__device__ __forceinline__ void prefetch_l2(const void* base, int64_t bytes) {
  const int64_t line = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 128;
  if (line < bytes)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(base) + line));
}

// The page of place `place` of sequence b; page 0 where the table's entry
// lies outside the cache.
__device__ __forceinline__ int page_of(const AttnArgs& a, int b, int64_t place) {
  const int64_t page = a.table[(int64_t)b * a.max_pages + (place >> a.lg_page)];
  if (page >= 0 && page < a.pages) return (int)page;
  atomicOr(a.error, 2u);
  return 0;
}

// A segment's part in a CTA's work: units [first, end) of it.
struct Segment {
  int item, head, first, end;
  int kv;        // places its rows may see, 0: an unused sequence
  int left;      // cost (kRun) or segments (else) of the CTA's work after it
};

// A segment that several CTAs share, as its first one notes it.
struct SharedSegment {
  int parts;          // how many, 0: found from the rest
  int segment;        // item * kv_heads + head, -1: none
  int second;         // the first one's part lies in its second set of rows
  int ctas;
  int last, cost;  // the last sharer is the CTA ((last + 1) ctas - 1) / cost
};

struct CutShared {
  int warp_sum[32], warp_most[32];
  int cut, split, ctas;
  int cost;                       // of all segments
  int each, over;                 // cost / ctas, cost % ctas
  int item_start[kMaxItems + 1];  // cost of the items before each, for one kv head
  int length[kMaxItems];          // the sequences' lengths
};

// Work is the sequence of segments (sequence, row tile of ROWS rows, kv
// head), each a run of units of KEYS keys, of which a CTA takes STEP in a
// round.  How it is cut follows from the lengths, which only the device
// knows:
//   kParts: every segment in up to `split` equal parts, one CTA each;
//   kWhole: a run of whole segments per CTA;
//   kRun: an equal run of cost per CTA, wherever segments begin or end; a
//     unit is its CTA's in whose run it begins.
// A unit costs WHOLE, or PART in a row tile of at most ROWS / 2 rows, and a
// segment BEGIN before its first unit.  Joining
// a segment over CTAs costs as much as about ROUNDS rounds, and so does
// beginning another one: no part is made smaller than that, segments that
// short stay whole, and a run may begin and end inside segments only where
// that evens out more.
template <int ROWS, int KEYS, int STEP, int ROUNDS, int WHOLE = 1, int PART = 1, int BEGIN = 0>
struct Cutter {
  enum { kParts, kWhole, kRun };
  static constexpr int kLeast = ROUNDS * STEP * WHOLE;  // cost of the smallest part

  // Host: whether a launch is cut by length.  Costs are 32-bit numbers; where
  // the page table has room for more, or there are more items, each CTA takes
  // one whole segment.
  static bool cuts(const AttnArgs& a, int64_t items) {
    const int64_t units = (((int64_t)a.max_pages << a.lg_page) + KEYS - 1) / KEYS;
    return items <= kMaxItems && (units * WHOLE + BEGIN) * items <= 0x7FFFFFFF / a.kv_heads;
  }
  const AttnArgs& a;
  CutShared& sh;

  __device__ __forceinline__ Cutter(const AttnArgs& args, CutShared& shared)
      : a(args), sh(shared) {}

  __device__ __forceinline__ int sequence(int item) const {
    return (int)quotient((uint32_t)item, a.by_tiles);
  }

  // Places that row tile rt of a sequence of n cached tokens may see.  Up to
  // 64 new tokens every tile takes them all: a chain is then cut as a tree of
  // one branch is, and gives its bits.
  __device__ __forceinline__ int places(int n, int rt) const {
    if (n < 0) return 0;
    const int64_t limit = (int64_t)a.max_pages << a.lg_page;
    int64_t kv = (int64_t)n + a.new_tokens;
    if (kv > limit) {
      atomicOr(a.error, 2u);
      kv = limit;
    }
    if (a.new_tokens > 64) {
      int last = (rt + 1) * ROWS;
      last = (last < a.rows ? last : a.rows) - 1;
      const int64_t end = (int64_t)n + quotient((uint32_t)last, a.by_group) + 1;
      kv = end < kv ? end : kv;
    }
    return (int)(kv < 0x7FFFFF00 ? kv : 0x7FFFFF00);
  }

  __device__ __forceinline__ int units_of(int kv) const {
    return kv < 1 ? 1 : (kv + KEYS - 1) / KEYS;
  }
  __device__ __forceinline__ int cost_of(int rt) const {  // of a unit
    return WHOLE == PART || a.rows - rt * ROWS > ROWS / 2 ? WHOLE : PART;
  }
  // x / c rounded up, c a unit's cost
  __device__ __forceinline__ static uint32_t units_in(uint32_t x, uint32_t c) {
    return WHOLE == PART || c == WHOLE ? (x + WHOLE - 1u) / WHOLE : (x + PART - 1u) / PART;
  }
  __device__ __forceinline__ int tile(const Segment& g) const {
    return g.item - sequence(g.item) * a.row_tiles;
  }

  __device__ __forceinline__ int length(int b) const { return a.direct ? a.length[b] : sh.length[b]; }

  // Reads the lengths and chooses the cut (all threads of the CTA; THREADS a
  // multiple of 32).
  template <int THREADS>
  __device__ __forceinline__ void choose() {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int items = a.batch * a.row_tiles, grid = (int)gridDim.x;
    if (a.direct) {
      if (tid == 0) {
        sh.cut = kWhole;
        sh.split = 1;
      }
      __syncthreads();
      return;
    }
    int carry = 0, most = 1;
    for (int base = 0; base < items; base += THREADS) {
      const int i = base + tid;
      int n = 0;
      if (i < items) {
        const int b = sequence(i), rt = i - b * a.row_tiles;
        const int len = a.length[b];
        if (rt == 0) sh.length[b] = len;
        n = BEGIN + units_of(places(len, rt)) * cost_of(rt);
      }
      int scan = n, top = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += x;
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      }
      __syncthreads();
      if (lane == 31) {
        sh.warp_sum[warp] = scan;
        sh.warp_most[warp] = top;
      }
      __syncthreads();
      int before = carry;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        const int x = sh.warp_sum[w];
        if (w < warp) before += x;
        carry += x;
        most = max(most, sh.warp_most[w]);
      }
      if (i < items) sh.item_start[i] = before + scan - n;
    }
    if (tid == 0) {
      const int cost = carry * a.kv_heads;
      const int64_t segments = (int64_t)items * a.kv_heads;
      int cut = kWhole, split = 1;
      if (segments <= grid) {
        split = (int)min((uint32_t)grid / (uint32_t)segments, (uint32_t)(most + kLeast - 1) / kLeast);
        // the longest part's rounds against an even share's
        const int64_t longest = ((int64_t)(most - BEGIN) + (int64_t)(BEGIN + 1) * split - 1) * grid;
        cut = longest <= (cost + (int64_t)kLeast * grid) * split ? kParts : kRun;
      } else if (most > kLeast) {
        cut = kRun;
      }
      sh.item_start[items] = carry;
      sh.cost = cost;
      sh.cut = cut;
      sh.split = split;
      // a unit begins in every run: a CTA without one would be counted among
      // a segment's and leave no part
      sh.ctas = min(grid, max(1, cost / (WHOLE + BEGIN)));
      sh.each = cost / sh.ctas;
      sh.over = cost - sh.each * sh.ctas;
    }
    __syncthreads();
  }

  // Sets end and left; item, head, first are set, and left: under kRun the
  // cost from the segment's first unit to the run's end.
  __device__ __forceinline__ void open(Segment& g) const {
    const int b = sequence(g.item), rt = g.item - b * a.row_tiles;
    g.kv = places(length(b), rt);
    const int n = units_of(g.kv);
    g.end = n;
    if (sh.cut == kRun) {
      const int c = cost_of(rt);
      const int all = n * c;
      if (g.left < all) g.end = (int)units_in((uint32_t)g.left, (uint32_t)c);
      g.left -= all + BEGIN;
    } else {
      --g.left;
    }
  }

  __device__ __forceinline__ void next(Segment& g) const {
    if (++g.head == a.kv_heads) {
      g.head = 0;
      ++g.item;
    }
    g.first = 0;
    open(g);
  }

  // kParts: units [first, end) of a segment of n that are part `part` of it,
  // of *parts.
  __device__ __forceinline__ bool part_of(int n, int cost, int part, int* parts, int* first,
                                          int* end) const {
    const uint32_t want =
        min((uint32_t)sh.split, ((uint32_t)n * (uint32_t)cost + kLeast - 1u) / kLeast);
    const uint32_t each = ((uint32_t)n + want - 1u) / want;
    *parts = (int)(((uint32_t)n + each - 1u) / each);
    *first = part * (int)each;
    *end = min(n, *first + (int)each);
    return part < *parts;
  }

  // This CTA's first segment; false if it has no work.
  __device__ __forceinline__ bool begin(Segment& g) const {
    const int grid = (int)gridDim.x, items = a.batch * a.row_tiles;
    g.first = 0;
    if (sh.cut == kRun) {
      if ((int)blockIdx.x >= sh.ctas) return false;
      const int x0 = begin_of(blockIdx.x), x1 = begin_of(blockIdx.x + 1);
      int lo = 0, hi = items - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sh.item_start[mid] * a.kv_heads <= x0)
          lo = mid;
        else
          hi = mid - 1;
      }
      const uint32_t all = (uint32_t)(sh.item_start[lo + 1] - sh.item_start[lo]);
      const uint32_t from = (uint32_t)(x0 - sh.item_start[lo] * a.kv_heads);
      g.item = lo;
      g.head = (int)(from / all);
      const uint32_t rest = from - (uint32_t)g.head * all;
      g.left = x1 - x0 + (int)rest - BEGIN;
      g.first = rest > BEGIN ? (int)units_in(rest - BEGIN, (uint32_t)cost_of(tile(g))) : 0;
      const int skip = g.first;
      open(g);
      if (skip >= g.end) {  // its last unit began in the run before
        if (g.left <= 0) return false;
        next(g);
      }
      return true;
    }
    const int segments = items * a.kv_heads;
    int s0 = (int)blockIdx.x, s1 = s0 + 1;
    if (sh.cut == kParts) {
      s0 = (int)((uint32_t)s0 / (uint32_t)sh.split);
      s1 = s0 + 1;
      if (s0 >= segments) return false;
    } else {
      s0 = (int)((int64_t)segments * blockIdx.x / grid);
      s1 = (int)((int64_t)segments * (blockIdx.x + 1) / grid);
      if (s0 >= s1) return false;
    }
    g.item = (int)quotient((uint32_t)s0, a.by_heads);
    g.head = s0 - g.item * a.kv_heads;
    g.left = s1 - s0;
    open(g);
    if (sh.cut == kParts) {
      int parts;
      return part_of(g.end, cost_of(tile(g)), (int)blockIdx.x - s0 * sh.split, &parts, &g.first,
                     &g.end);
    }
    return true;
  }

  // Whether the segment is all this CTA's, and which of the CTA's two sets of
  // partial rows its part goes to: the second where its work began earlier.
  __device__ __forceinline__ bool whole(const Segment& g) const {
    return g.first == 0 && g.end == units_of(g.kv);
  }
  __device__ __forceinline__ bool second_set(const Segment& g, bool first_of_cta) const {
    return sh.cut == kRun && g.first == 0 && !first_of_cta;
  }

  // Which CTAs share a segment that is not whole: `parts` from CTA cta0 on,
  // of which this is number `part`; second: where the first one's part lies.
  struct Sharers {
    int cta0, parts, part;
    bool second;
  };
  __device__ __forceinline__ int begin_of(uint32_t cta) const {  // of its run: cost * cta / ctas
    return (int)(cta * (uint32_t)sh.each + cta * (uint32_t)sh.over / (uint32_t)sh.ctas);
  }
  __device__ __forceinline__ int owner(int x) const {  // whose run x lies in
    return (int)((((int64_t)x + 1) * sh.ctas - 1) / sh.cost);
  }
  __device__ __forceinline__ Sharers sharers(const Segment& g) const {
    Sharers r = {(int)blockIdx.x, 1, 0, false};
    if (whole(g)) return r;
    if (sh.cut == kRun) {
      const int all = sh.item_start[g.item + 1] - sh.item_start[g.item];
      const int s0 = sh.item_start[g.item] * a.kv_heads + g.head * all;
      r.cta0 = owner(s0 + BEGIN);
      r.parts = owner(s0 + all - cost_of(tile(g))) - r.cta0 + 1;
      r.part = (int)blockIdx.x - r.cta0;
      // the first one's run began in an earlier segment, and had a unit there
      const int x0 = begin_of((uint32_t)r.cta0);
      r.second = x0 < s0 && begins_before(x0, s0, g);
    } else if (sh.cut == kParts) {
      r.part = (int)(blockIdx.x % (uint32_t)sh.split);
      r.cta0 = (int)blockIdx.x - r.part;
      int first, end;
      part_of(units_of(g.kv), cost_of(tile(g)), r.part, &r.parts, &first, &end);
    }
    return r;
  }

  // What a join after the launch has to know of the segment that this CTA
  // begins and others finish.  (Left to it: the division that finds the last
  // of them, which would cost the kernel's roles registers.)
  __device__ __forceinline__ SharedSegment note(const Segment& g, bool first_of_cta) const {
    SharedSegment r = {0, g.item * a.kv_heads + g.head, second_set(g, first_of_cta) ? 1 : 0,
                       sh.ctas, 0, sh.cost};
    if (sh.cut == kRun) {
      const int all = sh.item_start[g.item + 1] - sh.item_start[g.item];
      r.last = sh.item_start[g.item] * a.kv_heads + (g.head + 1) * all - cost_of(tile(g));
    } else if (sh.cut == kParts) {
      int first, end;
      part_of(units_of(g.kv), cost_of(tile(g)), 0, &r.parts, &first, &end);
    }
    return r;
  }

 private:
  // Whether a unit begins in [x, s0), s0 being where segment g begins: the
  // last unit before s0 does unless it began before x.
  __device__ __forceinline__ bool begins_before(int x, int s0, const Segment& g) const {
    const int item = g.head > 0 ? g.item : g.item - 1;
    const int rt = item - sequence(item) * a.row_tiles;
    return s0 - cost_of(rt) >= x;
  }
};

// rq_attn_rows.cu: the kernel for many query rows per sequence, and the bytes
// of scratch that it needs at most.
size_t attention_rows_scratch();
rq_status launch_attention_rows(AttnArgs a, int head_dim, bool i8, AttnScratch* scratch,
                                cudaStream_t st);

}  // namespace rq
