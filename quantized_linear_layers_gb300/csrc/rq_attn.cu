// rq_attn.cu -- attention of new tokens over the paged quantized K/V cache
// (sm_103a).
//
// With codes k8, v8 and row scales ks, vs of the cache, a query row q sees
//   x_j = (q . k8_j) ks_j,   out = sum_j p_j vs_j v8_j / sum_j p_j,
//   p_j = 2^(c (x_j - max x)),  c = scale log2(e),
// in one pass over the keys with the running maximum and sum.  Codes of both
// formats are exact in f16, so the two products run on f16 tensor
// instructions with f32 sums: an f32 operand (q, p vs) is split into a high
// and a low f16 part, 22 bits in all, which occupy two rows of the tile.

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "rq_attn.cuh"

namespace rq {

namespace {

// bit 0: a pipeline wait ran out; bit 1: an index outside its array
__device__ unsigned int g_attn_error = 0;

constexpr int kKeys = 16;            // keys of a unit: one warp's step
constexpr int kRows = 8;             // query rows of a segment
constexpr int kJoin = 8;             // neighbouring partials that are joined first
// The tensor cores cut their sums off towards zero, by an amount that grows
// with the additions: f32 rows' sums leave the instruction's registers every
// kFlush units of a warp, for a rounded one in shared memory.  Relative error of
// 1025 sequences of 60000 tokens, which are not cut, at head sizes 64, 128 and
// 256: 3.9e-7, 4.1e-7 and 5.6e-7 (7.8e-6, 1.1e-5 and 1.7e-5 without); one token
// over 131000 takes 33.4 us (32.6 without).
constexpr int kFlush = 16;

// rq_attn_rows.cu's kernel runs from kManyRows query rows per kv head on, for
// launches of at least kManyWork: rows times keys (the places that the page
// table has room for: the lengths are on the device), and kBeginning keys more
// a row for what beginning its 8 rows costs here.  It costs about 20 us before
// and after its products and then hardly more for 112 rows than for 8, this
// file's kernel 8 us and then a pass over the cache for every 8 rows.
// Measured, that / this (28 query heads, 4 kv heads of 128, bf16, tables that
// fit, cold L2, microseconds with the events' own 6): 8 sequences of 8000
// tokens, 21 rows 59 / 45, 28 rows 59 / 55, 42 rows 61 / 68, 112 rows 61 / 133;
// of 2000 tokens, 42 rows (3.3e6) 37 / 33, 56 rows (4.4e6) 37 / 35; one of
// 8000, 84 rows (2.8e6) 35 / 29, 112 rows (3.8e6) 35 / 37; prompts of 100
// tokens behind 50 (1.7e6) 23 / 18, 200 behind 10 (3.7e6) 25 / 27, 400 behind
// 100 (10e6) 29 / 57.  f32 takes that kernel 4 to 10 us more and this one the
// same.  Where the table has room to spare the choice can be the dearer one: 8
// tokens behind 500 take 14 us with a table of 9 pages and 31 with one of 2048.
constexpr int kManyRows = 32;
constexpr int kBeginning = 400;
constexpr double kManyWork = 3.4e6;

template <int D, bool WIDE>
struct Geometry {
  static constexpr int kPanel = D < 128 ? D : 128;  // bytes of a row in one swizzled panel
  static constexpr int kPanels = D / kPanel;
  static constexpr int kBytes = kKeys * D;          // codes of K (or V) in a unit
  // As many warps on an SM as the registers hold: the output rows alone are
  // D / 2 registers a thread, the query rows D / 4.  WIDE: in one CTA, for
  // launches of no more segments than SMs, where a CTA has one part of one
  // segment (one token over 500 cached ones 8.6 us against 10.9 in two, over
  // 131000 33.3 against 40.1).  Otherwise in two, so that one streams while
  // the other begins or joins a segment (64 sequences of up to 8192 tokens
  // 155 us, 165 in one).
  static constexpr int kCtas = WIDE ? 1 : 2;
  static constexpr int kWarps = (D == 64 ? 16 : D == 128 ? 12 : 8) / kCtas;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = D == 256 ? 2 : 3;  // units in flight per warp
  static constexpr int kRing = kWarps * kStages * 2 * kBytes;
};

// Shared memory after the ring.
template <int D, bool WIDE>
struct Tail {
  static constexpr int kWarps = Geometry<D, WIDE>::kWarps;
  static constexpr int kStages = Geometry<D, WIDE>::kStages;
  float scale[kWarps][kStages][2][kKeys];  // ks, vs of the units in flight
  float o[kWarps][kRows][D + 4];
  float m[kWarps][kRows], l[kWarps][kRows];
  float c[kRows];
  int flag;
  CutShared cut;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a panel of rows of PANEL bytes:
// eight rows' chunks of one column lie in different banks.
template <int PANEL>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  if constexpr (PANEL == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the newest N groups of copies have landed.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A unit's 16 rows, which lie one after another, into its panels: lane l
// takes 16-byte pieces l, l + 32, ...  The swizzle's terms of the lane and of
// the piece fall on separate bits, so each piece's place is `dst` (the
// lane's, of the first piece) with constants.
template <int D>
__device__ __forceinline__ void copy_rows(uint32_t dst, const uint8_t* src) {
  constexpr int kPieces = kKeys * D / 512;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    constexpr int kRowsPer = 512 / D;  // rows that a warp's pieces span
    const uint32_t to = D == 64 ? dst + i * 512
                                : (dst ^ (((i * kRowsPer) & 7) << 4)) + i * kRowsPer * 128;
    copy16(to, src + i * 512);
  }
}

// ------------------------------------------------------------ the kernel --
//
// How the work is cut between CTAs: Cutter.  A segment cut between CTAs is
// joined by the last of them to finish, in part order, from partial (max,
// sum, output) rows in scratch.  A round of its warps takes about 0.6 us,
// joining or beginning a segment 2.5 us.
//
// Within a CTA the warps take units in turn, each with its own ring of units
// in flight (asynchronous copies, on into the next segment) and a softmax of
// its own, so that nothing is exchanged inside the loop; their results are
// joined when the segment ends.  A warp's 16-row tile holds the
// high f16 parts of 8 query rows and below them their low parts: an f32 row
// costs no product more than an f16 one would.
template <int D, bool I8, bool WIDE>
__global__ void __launch_bounds__(Geometry<D, WIDE>::kThreads, Geometry<D, WIDE>::kCtas)
attn_kernel(const AttnArgs a) {
  using G = Geometry<D, WIDE>;
  using TailT = Tail<D, WIDE>;
  constexpr int W = G::kWarps, S = G::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  TailT& tail = *reinterpret_cast<TailT*>(smem + G::kRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem) + warp * (S * 2 * G::kBytes);

  pdl_wait();
  pdl_trigger();

  prefetch_l2(a.q, a.q_bytes);
  prefetch_l2(a.table, (int64_t)a.batch * a.max_pages * 4);
  Cutter<kRows, kKeys, W, 6> cutter(a, tail.cut);
  cutter.template choose<G::kThreads>();
  Segment seg;
  if (!cutter.begin(seg)) return;

  // -------- the warp's loads, S - 1 units ahead of its products
  Segment ahead = seg;
  int unit = seg.first + warp;         // next unit to load
  int in_window = 0, pages_of = 0;     // lane i: page of the window's unit i, W units apart
  int ld_stage = 0;
  auto page_window = [&]() {  // (looked at when they are used)
    in_window = 0;
    const int64_t u = unit + (int64_t)lane * W;
    pages_of = 0;
    if (u < ahead.end && u * kKeys < ahead.kv)
      pages_of = a.table[(int64_t)cutter.sequence(ahead.item) * a.max_pages +
                         ((u * kKeys) >> a.lg_page)];
  };
  page_window();
  const int page_mask = (1 << a.lg_page) - 1;
  // where this lane's first piece of a unit goes
  const int piece_row = lane * 16 / D, piece_chunk = lane * 16 % D / 16;
  const uint32_t piece = (piece_chunk / (G::kPanel / 16)) * (kKeys * G::kPanel) +
                         swizzled<G::kPanel>(piece_row, piece_chunk % (G::kPanel / 16));
  auto load_one = [&]() {  // starts copying the warp's next unit, if there is one
    while (unit >= ahead.end && ahead.left > 0) {
      cutter.next(ahead);
      unit = warp;
      in_window = 32;
    }
    if (unit < ahead.end && ahead.kv > 0) {
      if (in_window == 32) page_window();
      int page = __shfl_sync(0xFFFFFFFFu, pages_of, in_window);
      ++in_window;
      if (page < 0 || page >= a.pages) {
        if (lane == 0) atomicOr(a.error, 2u);
        page = 0;
      }
      const int64_t row = ((int64_t)(page * a.kv_heads + ahead.head) << a.lg_page) +
                          ((unit * kKeys) & page_mask);
      const uint32_t to = ring + ld_stage * (2 * G::kBytes) + piece;
      copy_rows<D>(to, a.k + row * D + lane * 16);
      copy_rows<D>(to + G::kBytes, a.v + row * D + lane * 16);
      if (lane < 8)
        copy16(smem_u32(&tail.scale[warp][ld_stage][0][0]) + lane * 16,
               (lane < 4 ? a.ks : a.vs - 16) + row + lane * 4);
    }
    copy_commit();  // a group for every unit, there or not
    ld_stage = ld_stage == S - 1 ? 0 : ld_stage + 1;
    unit += W;
  };

  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t matrix =
      swizzled<G::kPanel>(((lane >> 3) & 1) * 8 + (lane & 7), lane >> 4);
  int st = 0;  // ring stage of the next unit
  for (int nseg = 0;; ++nseg) {
    const int b = cutter.sequence(seg.item), rt = seg.item - b * a.row_tiles;
    const int kv = seg.kv;
    // this thread's row: g
    const int row_of = rt * kRows + g;
    const bool live = row_of < a.rows;
    const int tok = live ? (int)quotient((uint32_t)row_of, a.by_group) : 0;
    unsigned long long bits = 0;
    if (live && a.tree != nullptr) bits = a.tree[(int64_t)b * a.new_tokens + tok];
    float c;  // powers of two per unit of the raw score x = (q . k8) ks
    uint32_t qa[D / 16][4];
    {
      const int64_t off = ((int64_t)b * a.new_tokens + tok) * a.q_stride +
                          (int64_t)(seg.head * a.group + (live ? row_of - tok * a.group : 0)) * D;
      // the first loads of keys and values go out while q is on its way (or
      // before it, where its raw values would not stay in registers)
      if (nseg == 0 && D == 256)
        for (int i = 0; i < S - 1; ++i) load_one();
      float x[D / 16][4];
      uint32_t top = 0u;  // largest magnitude, as bits: a NaN counts as above infinity
      if (a.dtype == RQ_F32) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + off +
                                                            16 * i + 4 * t4);
          x[i][0] = v.x;
          x[i][1] = v.y;
          x[i][2] = v.z;
          x[i][3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + off +
                                                          16 * i + 4 * t4);
          x[i][0] = __uint_as_float(v.x);  // unpacked below
          x[i][1] = __uint_as_float(v.y);
        }
      }
      if (nseg == 0 && D < 256)
        for (int i = 0; i < S - 1; ++i) load_one();
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        if (a.dtype != RQ_F32) {
          const uint32_t lo = __float_as_uint(x[i][0]), hi = __float_as_uint(x[i][1]);
          if (a.dtype == RQ_F16) {
            const float2 f0 = half_pair(lo), f1 = half_pair(hi);
            x[i][0] = f0.x;
            x[i][1] = f0.y;
            x[i][2] = f1.x;
            x[i][3] = f1.y;
          } else {
            x[i][0] = __uint_as_float(lo << 16);
            x[i][1] = __uint_as_float(lo & 0xFFFF0000u);
            x[i][2] = __uint_as_float(hi << 16);
            x[i][3] = __uint_as_float(hi & 0xFFFF0000u);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (!live) x[i][k] = 0.0f;
          top = max(top, __float_as_uint(x[i][k]) & 0x7FFFFFFFu);
        }
      }
      // the row times a power of two, so that its f16 parts lie well inside
      // f16's range: largest entry in [2^13, 2^14).  A row that is not finite
      // becomes NaN, and so do its scores; c stays finite, so that what the
      // row does not see weighs 0 all the same.
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      int e = 0;
      if (top > 0u) {
        e = 13 - (int)(top >> 23) + 127;
        e = e < -126 ? -126 : e > 100 ? 100 : e;
      }
      const float up = top < 0x7F800000u ? __uint_as_float((uint32_t)(e + 127) << 23) : NAN;
      c = fmaxf(a.scale_log2 / up, 0x1p-126f);  // (of a NaN: 2^-126)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        qa[i][0] = split_half2(x[i][0] * up, x[i][1] * up, qa[i][1]);
        qa[i][2] = split_half2(x[i][2] * up, x[i][3] * up, qa[i][3]);
      }
    }

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;
    const int n_all = cutter.length(b);
    const int len = n_all < 0 ? 0 : n_all < kv ? n_all : kv;  // places cached before
    // places that every row sees: without a tree also the new ones up to the
    // first row's own
    const int sure =
        a.tree == nullptr
            ? min(kv, len + (int)quotient((uint32_t)(rt * kRows), a.by_group) + 1)
            : len;
    float m = -INFINITY, l = 0.0f;
    float vref = 0x1p-112f;  // power of two at or above every vs that the row has seen
    // The output's sum so far, with what shared memory holds of it: `sum_max` is
    // the maximum that is relative to (-inf: nothing is there).
    float sum_max = -INFINITY;
    auto fold = [&]() {
      const float back = vref * 0x1p-14f;
      const float f = ex2((sum_max - (m == -INFINITY ? 0.0f : m)) * c);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        // dims 16 i + 4 t4 ..: the even tile's two columns and the odd tile's
        float4* const at = reinterpret_cast<float4*>(&tail.o[warp][g][16 * i + 4 * t4]);
        float4 v = make_float4(
            (o[2 * i][0] + o[2 * i][2]) * back, (o[2 * i + 1][0] + o[2 * i + 1][2]) * back,
            (o[2 * i][1] + o[2 * i][3]) * back, (o[2 * i + 1][1] + o[2 * i + 1][3]) * back);
        if (sum_max != -INFINITY) {
          const float4 s = *at;
          v = make_float4(fmaf(s.x, f, v.x), fmaf(s.y, f, v.y), fmaf(s.z, f, v.z),
                          fmaf(s.w, f, v.w));
        }
        *at = v;
      }
    };
    int until = a.dtype == RQ_F32 ? kFlush : 0x7FFFFFFF;

    for (int u = seg.first + warp, end = seg.end; u < end; u += W) {
      copy_wait<S - 2>();
      __syncwarp();
      const int first = u * kKeys;  // place of the first key
      const bool all = first + kKeys <= sure;
      const uint32_t kd = ring + st * (2 * G::kBytes), vd = kd + G::kBytes;
      // ldmatrix's matrix lane / 8: keys 0-7 or 8-15, 16 dims i or i + 1 (i
      // even, so that it only flips bits of the swizzled place)
      auto matrix_at = [&](uint32_t base, int i) -> uint32_t {
        constexpr int kChunks = G::kPanel / 16;
        return ((base + matrix) ^ ((i % kChunks) << 4)) + (i / kChunks) * (kKeys * G::kPanel);
      };
      // ---- scores
      float s[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; i += 2) {
        uint32_t w[4];
        ldsm4(w, matrix_at(kd, i));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t b0, b1;
          codes_in_order<I8>(w[k], b0, b1);
          mma(s[k & 1], qa[i + (k >> 1)], b0, b1);
        }
      }
      // the unit S - 1 ahead goes into the stage that the last one left, while
      // the products are under way
      load_one();
      // ---- scales: this thread's keys are 2 t4, 2 t4 + 1 and 8 more
      const float* sc = &tail.scale[warp][st][0][0];
      const float2 ka = *reinterpret_cast<const float2*>(sc + 2 * t4);
      const float2 kb = *reinterpret_cast<const float2*>(sc + 8 + 2 * t4);
      const float2 va = *reinterpret_cast<const float2*>(sc + kKeys + 2 * t4);
      const float2 vb = *reinterpret_cast<const float2*>(sc + kKeys + 8 + 2 * t4);
      float x[4] = {(s[0][0] + s[0][2]) * ka.x, (s[0][1] + s[0][3]) * ka.y,
                    (s[1][0] + s[1][2]) * kb.x, (s[1][1] + s[1][3]) * kb.y};
      float vv[4] = {va.x, va.y, vb.x, vb.y};
      if (!all) {
        // what a row does not see: no scores; V's codes there may be anything,
        // and 0 * NaN is not 0: zeros past the last place, no NaN before it
        if (!I8 || first + kKeys > kv) {
          const int keys = kv > first ? kv - first : 0;
          for (int i = (I8 ? keys * (D / 16) : 0) + lane; i < kKeys * (D / 16); i += 32) {
            const int r = i / (D / 16), ch = i % (D / 16);
            const uint32_t at = vd + (ch / (G::kPanel / 16)) * (kKeys * G::kPanel) +
                                swizzled<G::kPanel>(r, ch % (G::kPanel / 16));
            uint32_t v[4] = {0u, 0u, 0u, 0u};
            if (!I8 && r < keys) {
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                           : "r"(at)
                           : "memory");
#pragma unroll
              for (int k = 0; k < 4; ++k) v[k] = without_nan(v[k]);
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]),
                         "r"(v[1]), "r"(v[2]), "r"(v[3])
                         : "memory");
          }
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int place = first + 8 * (k >> 1) + 2 * t4 + (k & 1);
          const int draft = place - len;
          bool see = place < kv;
          if (draft >= 0)
            see = see && (a.tree == nullptr ? draft <= tok
                                            : (draft < 64 && ((bits >> draft) & 1ull) != 0ull));
          if (!see) {
            x[k] = -INFINITY;
            vv[k] = 0.0f;
          }
        }
      }
      // ---- running maximum, and the values' scales relative to theirs; both
      // seldom move, so that most units pay one vote for them
      const float xm = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      if (__any_sync(0xFFFFFFFFu,
                     xm > m || fmaxf(fmaxf(vv[0], vv[1]), fmaxf(vv[2], vv[3])) > vref)) {
        float mn = fmaxf(xm, __shfl_xor_sync(0xFFFFFFFFu, xm, 1));
        mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 2));
        mn = fmaxf(mn, m);
        uint32_t vt = 0u;  // bits of what is not negative are in its order
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (vv[k] >= 0.0f && vv[k] <= 1e37f) vt = max(vt, __float_as_uint(vv[k]));  // no NaN, Inf
        // of this row alone: another row's keys may be hidden from it
        vt = max(vt, __shfl_xor_sync(0xFFFFFFFFu, vt, 1));
        vt = max(vt, __shfl_xor_sync(0xFFFFFFFFu, vt, 2));
        const float al = m == -INFINITY ? 0.0f : ex2((m - mn) * c);
        float f = al;
        const uint32_t vbits = __float_as_uint(vref);
        if (vt > vbits) {  // four times the next power of two: rarely passed again
          const uint32_t vnew = (vt & 0x7F800000u) + (2u << 23);
          vref = __uint_as_float(vnew);
          // times old / new, a power of two (0 where that is below f32's)
          const int e = (int)(vbits >> 23) - (int)(vnew >> 23) + 127;
          f *= e > 0 ? __uint_as_float((uint32_t)e << 23) : 0.0f;
        }
        l *= al;
        m = mn;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][k] *= f;
      }
      // 2^14 / vref: the weights p vs / vref lie below 2^14, well inside f16
      const float inv = __uint_as_float((268u << 23) - __float_as_uint(vref));
      const float mr = m == -INFINITY ? 0.0f : m;
      float w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float p = ex2((x[k] - mr) * c);
        l += p;
        w[k] = p * (vv[k] * inv);
      }
      uint32_t pa[4];
      pa[0] = split_half2(w[0], w[1], pa[1]);
      pa[2] = split_half2(w[2], w[3], pa[3]);
      // ---- output
#pragma unroll
      for (int i = 0; i < D / 16; i += 2) {
        uint32_t v[4];
        ldsm4t(v, matrix_at(vd, i));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t e0, e1, o0, o1;
          codes_across<I8>(v[2 * k], e0, o0);
          codes_across<I8>(v[2 * k + 1], e1, o1);
          mma(o[2 * (i + k)], pa, e0, e1);
          mma(o[2 * (i + k) + 1], pa, o0, o1);
        }
      }
      if (--until == 0) {
        fold();
        sum_max = m;
        until = kFlush;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;
      }
      __syncwarp();
      st = st == S - 1 ? 0 : st + 1;
    }

    // ---- join the warps: every lane of a row's four holds part of its sum
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
    l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
    if (t4 == 0) {
      tail.m[warp][g] = m;
      tail.l[warp][g] = l;
      tail.c[g] = c;  // the same from every warp
    }
    fold();
    __syncthreads();

    const auto share = cutter.sharers(seg);
    const int cta0 = share.cta0;
    const int parts = share.parts, part = share.part;
    const bool second = share.second;
    constexpr int kVec = D / 4;
    constexpr int kPartRow = D + 4;  // output, then max and sum
    // A partial row set of this segment, by part number.
    auto part_at = [&](int p) -> int { return (cta0 + p) * 2 + (p == 0 && second ? 1 : 0); };
    // Join this thread's piece of `count` partials, `step` parts apart from
    // part p0 on, several loads in flight at a time (four of two CTAs' threads,
    // whose registers eight would spill); in part order.
    constexpr int kLoads = WIDE ? 8 : 4;
    auto join = [&](int p0, int step, int count, int r, int d, float4& v, float& mx,
                    float& sum) {
      const float cr = tail.c[r];
      for (int q0 = 0; q0 < count; q0 += kLoads) {
        float4 ov[kLoads];
        float2 ml[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          ml[k] = make_float2(-INFINITY, 0.0f);
          ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (q0 + k < count) {
            const float* part = a.part + ((int64_t)part_at(p0 + (q0 + k) * step) * kRows + r) * kPartRow;
            ov[k] = __ldcg(reinterpret_cast<const float4*>(part + d));
            ml[k] = __ldcg(reinterpret_cast<const float2*>(part + D));
          }
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) merge(v, mx, sum, ov[k], ml[k], cr);
      }
    };
    auto arrive = [&](unsigned int* ctr, unsigned int of) -> bool {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned int old = atomicAdd(ctr, 1u);
        tail.flag = old == of - 1u;
        if (tail.flag) *ctr = 0u;
      }
      __syncthreads();
      const bool is_last = tail.flag != 0;
      __threadfence();
      return is_last;
    };
    auto store_part = [&](int slot, int r, int d, const float4& v, float mx, float sum) {
      float* part = a.part + ((int64_t)slot * kRows + r) * kPartRow;
      __stcg(reinterpret_cast<float4*>(part + d), v);
      if (d == 0) __stcg(reinterpret_cast<float2*>(part + D), make_float2(mx, sum));
    };
    constexpr int kPieces = (kRows * kVec + G::kThreads - 1) / G::kThreads;
    float4 v[kPieces];
    float mx[kPieces], sum[kPieces];
    bool mine[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int i = tid + k * G::kThreads, r = i / kVec, d = (i % kVec) * 4;
      mine[k] = i < kRows * kVec && rt * kRows + r < a.rows;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      mx[k] = -INFINITY;
      sum[k] = 0.0f;
      if (!mine[k]) continue;
      float mw[W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        mw[w] = tail.m[w][r];
        mx[k] = fmaxf(mx[k], mw[w]);
      }
      const float cr = tail.c[r], base = mx[k] == -INFINITY ? 0.0f : mx[k];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = ex2((mw[w] - base) * cr);
        const float4 ov = *reinterpret_cast<const float4*>(&tail.o[w][r][d]);
        v[k].x = fmaf(ov.x, f, v[k].x);
        v[k].y = fmaf(ov.y, f, v[k].y);
        v[k].z = fmaf(ov.z, f, v[k].z);
        v[k].w = fmaf(ov.w, f, v[k].w);
        // a warp whose scores are all NaN has no maximum, but its sum counts
        sum[k] += mw[w] == -INFINITY ? tail.l[w][r] : tail.l[w][r] * f;
      }
    }
    bool last = true;
    if (parts > 1) {
      // Two levels, so that no CTA reads more than a few dozen partials: the
      // last of each kJoin neighbours joins theirs, the last of those joins
      // the groups.
      const int first_of = part / kJoin * kJoin;
      const int members = min(parts - first_of, kJoin);
      const int groups = (parts + kJoin - 1) / kJoin;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int i = tid + k * G::kThreads, r = i / kVec, d = (i % kVec) * 4;
        if (mine[k]) store_part(part_at(part), r, d, v[k], mx[k], sum[k]);
      }
      const int slot = part_at(first_of);
      last = arrive(a.counter + slot, (unsigned int)members);
      for (int level = 0; last && level < 2; ++level) {
        if (level == 1) {
          if (groups == 1) break;
          // (a CTA is the first of one shared segment at most)
          last = arrive(a.counter + 2 * gridDim.x + part_at(0), (unsigned int)groups);
          if (!last) break;
        }
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          const int i = tid + k * G::kThreads, r = i / kVec, d = (i % kVec) * 4;
          if (!mine[k]) continue;
          v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          mx[k] = -INFINITY;
          sum[k] = 0.0f;
          if (level == 0)
            join(first_of, 1, members, r, d, v[k], mx[k], sum[k]);
          else
            join(0, kJoin, groups, r, d, v[k], mx[k], sum[k]);
        }
        if (level == 0 && groups > 1) {
          // the joined row takes the place of the group's first member, whose
          // maximum and sum every thread of the row has read by now
          __syncthreads();
#pragma unroll
          for (int k = 0; k < kPieces; ++k) {
            const int i = tid + k * G::kThreads, r = i / kVec, d = (i % kVec) * 4;
            if (mine[k]) store_part(slot, r, d, v[k], mx[k], sum[k]);
          }
        }
      }
    }
    if (last) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int i = tid + k * G::kThreads, r = i / kVec, d = (i % kVec) * 4;
        const int row = rt * kRows + r;
        if (!mine[k]) continue;
        // nothing seen: zeros (a NaN sum stays a NaN)
        const float r1 = sum[k] == 0.0f ? 0.0f : 1.0f / sum[k];
        const float4 y = make_float4(v[k].x * r1, v[k].y * r1, v[k].z * r1, v[k].w * r1);
        const int tk = (int)quotient((uint32_t)row, a.by_group);
        const int64_t dst = (((int64_t)b * a.new_tokens + tk) * a.q_heads + seg.head * a.group +
                             row - tk * a.group) * D + d;
        if (a.dtype == RQ_F32) {
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + dst) = y;
        } else if (a.dtype == RQ_F16) {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + dst) =
              make_uint2(pack_half2(y.x, y.y), pack_half2(y.z, y.w));
        } else {
          const __nv_bfloat162 h0 = __floats2bfloat162_rn(y.x, y.y);
          const __nv_bfloat162 h1 = __floats2bfloat162_rn(y.z, y.w);
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + dst) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&h0),
                         *reinterpret_cast<const uint32_t*>(&h1));
        }
      }
    }
    if (seg.left <= 0) break;
    __syncthreads();  // the joined rows are read before the next segment's are written
    cutter.next(seg);
  }
}

// ------------------------------------------------------------- host side --

int lg(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

template <int D, bool I8, bool WIDE>
rq_status launch_kind(const AttnArgs& a, unsigned grid, cudaStream_t st) {
  using G = Geometry<D, WIDE>;
  constexpr int bytes = G::kRing + (int)sizeof(Tail<D, WIDE>);
  static_assert(bytes <= 232448 && G::kCtas * (bytes + 1024) <= 233472, "shared memory of an SM");
  static bool ready = false;
  if (!ready) {
    if (cudaFuncSetAttribute(attn_kernel<D, I8, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes) != cudaSuccess)
      return RQ_ERR_CUDA;
    ready = true;
  }
  return launch_kernel(attn_kernel<D, I8, WIDE>, dim3(grid), dim3(G::kThreads), (size_t)bytes, st,
                       a);
}

template <int D>
rq_status launch_d(const AttnArgs& a, bool i8, bool wide, unsigned grid, cudaStream_t st) {
  if (wide)
    return i8 ? launch_kind<D, true, true>(a, grid, st) : launch_kind<D, false, true>(a, grid, st);
  return i8 ? launch_kind<D, true, false>(a, grid, st) : launch_kind<D, false, false>(a, grid, st);
}

}  // namespace

rq_status launch_cache_attention(const AttnCall& call, AttnScratch* scratch, cudaStream_t st) {
  const rq_kv_cache& c = *call.cache;
  AttnArgs a = {};
  static void* word = nullptr;
  if (word == nullptr && cudaGetSymbolAddress(&word, g_attn_error) != cudaSuccess)
    return RQ_ERR_CUDA;
  a.error = static_cast<unsigned int*>(word);
  a.q = call.q;
  a.out = call.out;
  a.q_stride = call.q_stride;
  a.q_bytes = (((int64_t)call.batch * call.new_tokens - 1) * call.q_stride +
               (int64_t)call.q_heads * c.head_dim) * (call.dtype == RQ_F32 ? 4 : 2);
  a.k = static_cast<const uint8_t*>(c.k);
  a.v = static_cast<const uint8_t*>(c.v);
  a.ks = c.k_scale;
  a.vs = c.v_scale;
  a.table = call.page_table;
  a.length = call.length;
  a.tree = reinterpret_cast<const unsigned long long*>(call.tree);
  a.batch = call.batch;
  a.new_tokens = call.new_tokens;
  a.q_heads = call.q_heads;
  a.kv_heads = c.kv_heads;
  a.group = call.q_heads / c.kv_heads;
  a.rows = call.new_tokens * a.group;
  a.row_tiles = (a.rows + kRows - 1) / kRows;
  a.by_heads = divisor((uint32_t)a.kv_heads);
  a.by_group = divisor((uint32_t)a.group);
  a.by_tiles = divisor((uint32_t)a.row_tiles);
  a.max_pages = call.max_pages;
  a.lg_page = lg(c.page_size);
  a.pages = c.pages;
  a.scale_log2 = (float)((double)call.scale * 1.4426950408889634);
  a.dtype = call.dtype;

  const double work = ((double)call.max_pages * c.page_size + kBeginning) * c.kv_heads *
                      call.batch * a.rows;
  if (a.rows >= kManyRows && work >= kManyWork && c.head_dim <= 128) {
    ++scratch->many_rows;
    return launch_attention_rows(a, c.head_dim, c.format == RQ_KV_I8, scratch, st);
  }
  ++scratch->few_rows;

  const int64_t items = (int64_t)call.batch * a.row_tiles;
  const int64_t segments = items * c.kv_heads;
  const bool wide = segments <= device_sm_count();
  int64_t grid = (int64_t)(wide ? 1 : 2) * device_sm_count();
  a.direct = !Cutter<kRows, kKeys, 1, 6>::cuts(a, items);
  if (a.direct) {
    grid = segments;
    if (grid > 0x7FFFFFFF) return RQ_ERR_SHAPE;
  } else {
    const rq_status s = scratch->reserve(st);
    if (s != RQ_OK) return s;
    a.part = reinterpret_cast<float*>(scratch->part);
    a.counter = scratch->counter;
  }
  const unsigned g = (unsigned)grid;
  const bool i8 = c.format == RQ_KV_I8;
  switch (c.head_dim) {
    case 64: return launch_d<64>(a, i8, wide, g, st);
    case 128: return launch_d<128>(a, i8, wide, g, st);
    default: return launch_d<256>(a, i8, wide, g, st);
  }
}

// Two sets of partial rows of the largest head for each of at most two CTAs an
// SM, or what the other kernel needs; a counter of arrivals for every set of
// rows, and one for the groups of the segment that begins with it.
rq_status AttnScratch::reserve(cudaStream_t st) {
  if (part != nullptr) return RQ_OK;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &capture) != cudaSuccess) {
    cudaGetLastError();  // (the legacy stream while another one is captured)
    return RQ_ERR_ALLOC;
  }
  if (capture != cudaStreamCaptureStatusNone) return RQ_ERR_ALLOC;
  const size_t ctas = 2 * (size_t)device_sm_count();
  const size_t few = sizeof(float) * 2 * ctas * kRows * (256 + 4);
  const size_t bytes = ((std::max(few, attention_rows_scratch()) + 255) & ~(size_t)255);
  const size_t words = sizeof(unsigned int) * 4 * ctas;
  void* p = nullptr;
  if (cudaMalloc(&p, bytes + words) != cudaSuccess) {
    cudaGetLastError();
    return RQ_ERR_ALLOC;
  }
  // Every launch leaves its counters at zero again.  (Waited for, so that the
  // next call may be on another stream.)
  uint8_t* const at = static_cast<uint8_t*>(p);
  if (cudaMemsetAsync(at + bytes, 0, words, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess) {
    cudaFree(p);
    return RQ_ERR_CUDA;
  }
  part = at;
  counter = reinterpret_cast<unsigned int*>(at + bytes);
  return RQ_OK;
}

void AttnScratch::release() {
  if (part) cudaFree(part);
  *this = AttnScratch();
}

rq_status read_and_clear_attn_error() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(v)) != cudaSuccess) return RQ_ERR_CUDA;
  if (v == 0) return RQ_OK;
  const unsigned int zero = 0;
  if (cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(zero)) != cudaSuccess) return RQ_ERR_CUDA;
  return (v & 1u) ? RQ_ERR_TIMEOUT : RQ_ERR_INDEX;
}

}  // namespace rq
