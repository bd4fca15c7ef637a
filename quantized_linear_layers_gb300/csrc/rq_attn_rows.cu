// rq_attn_rows.cu -- attention of many query rows over the paged quantized
// cache on tcgen05 (sm_103a): drafted trees and prompts, whose heads of one kv
// head and tokens of one sequence make up tiles of 128 rows.
//
// The mathematics is that of rq_attn.cu.  Per CTA up to two tiles of 128 rows
// share 64 keys at a time:
//   warps 0-3, 4-7   softmax of tile 0 and 1: a thread owns a row
//   warps 8-15       codes of K and V to f16 in shared memory, two units deep
//   warps 16, 18     a thread of each issues the products of tile 0 and 1;
//                    warp 16 allocates TMEM
//   warp 17          the scales; asks codes into L2, three units ahead; notes
//                    for the join which segment goes on in other CTAs
//   warp 19          idle
// S = Q K^T (A = Q from shared memory) lands in one of two TMEM buffers per
// row tile; its softmax writes P over it, as f16 high and low parts for f32
// rows (64 + 64 keys in S's 64 columns), and P V takes A = P from TMEM and
// adds to O in TMEM.  While a row tile's softmax runs, the tensor cores work
// on its next scores and on the other tile.  f32 rows take both products
// twice (Q high and low, P high and low), 16-bit rows once: their P is rounded
// to f16, 11 bits, which is finer than a bf16 output and as fine as an f16 one,
// and a second product would cost them 0.3 us a unit.
//
// Measured (28 query, 4 kv heads of 128): trees of 48 over 8 sequences of 8000
// tokens, f32, 118 us (291 TFLOP/s, each product counted once); two prompts of
// 1500 tokens behind 600, bf16, 110 us (498 TFLOP/s).  A unit of 256 rows takes
// 1.4 us in bf16, 1.7 in f32, of which the tensor pipe works 0.6 and 1.25.  No
// pipe is full: what bounds it is the way from scores over softmax, barrier,
// products and barrier back to scores (all exponentials, scales and maxima
// left out of a copy, it still took 1.35 us), and around the units the
// prologue (4 us), the first query rows (4), the change of segments (5) and
// the join (about 6).
#include "rq_attn.cuh"

namespace rq {

namespace {

constexpr int kKeys = 64;                 // keys of a unit
constexpr int kTileRows = 128;            // rows of one accumulator
constexpr int kRows = 2 * kTileRows;      // rows of a segment
constexpr int kSoft = 256;                // softmax threads
constexpr int kConvert = 256;             // conversion threads
constexpr int kThreads = kSoft + kConvert + 128;
// Registers a thread: 256 x 144 + 256 x 64 + 128 x 64 = 640 x 96, the
// launch's own.
constexpr int kSoftRegs = 144, kConvertRegs = 64, kIssueRegs = 64;
constexpr int kIssueWarp = (kSoft + kConvert) / 32;
constexpr int kScales = 4;                // units whose scales are kept
constexpr int kAhead = 3;                 // units that codes are asked into L2 ahead of use
constexpr float kLazy = 8.0f;             // a maximum is kept while scores pass it by less than 2^8
// The tensor cores cut their sums off towards zero.  With f32 rows, whose
// products are carried to 21 bits, the output's sum therefore leaves TMEM every
// kFlush units for one with rounded additions, in the CTA's own scratch (in
// L2).  Relative error over 8000 keys, and trees of 48 over 8 such sequences:
// 5.7e-6, 107 us without; 2.4e-6 every 16 units; 1.4e-6, 116 us every 8;
// 1.1e-6, 118 us every 6; 0.9e-6, 124 us every 4.  (f32 sums in plain form:
// 1.5e-6 there, 0.9e-6 over 2000 keys.)
constexpr int kFlush = 6;
constexpr float kUp = 128.0f;             // weights p vs / vref are kept 2^7 times larger in f16

template <int D, bool SPLIT>
struct Layout {
  static constexpr int kPanels = D / 64;                      // 128-byte panels of an f16 row
  static constexpr int kQPanel = kTileRows * 128;
  static constexpr int kQTile = kPanels * kQPanel;            // one part of one row tile
  static constexpr int kQ = 2 * (SPLIT ? 2 : 1) * kQTile;
  static constexpr int kPanel = kKeys * 128;
  static constexpr int kB = kPanels * kPanel;                 // K (or V) of a unit
  static constexpr int kTail = kQ + 4 * kB;                   // two units of K and V
};

template <int D>
constexpr int kPartRow = D + 4;  // a partial row: output, reference, sum

template <bool W>
struct Flag {
  static constexpr bool value = W;
};

// (a unit takes 1.4 to 1.7 us, in a half row tile 1.1 to 1.3, and the change from
// one segment to the next 5.5)
using Cutting = Cutter<kRows, kKeys, 1, 8, 8, 6, 28>;

struct RowsTail {
  // vs relative to vref, times kUp, and vr as they are
  float ks[kScales][kKeys], vs[kScales][kKeys], vr[kScales][kKeys];
  float vref[kScales];   // of all keys so far; negative: a scale is out of range
  float vmost[kScales];  // largest scale of the unit
  uint64_t q_full[2], k_full[2], k_free[2], v_full[2], v_free[2], sc_full[kScales];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2], drained[2];
  uint32_t tmem;
  CutShared cut;
};

// ------------------------------------------------------------ PTX wrappers --

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Matrix descriptors, 128-byte swizzle.  K-major (rows of 128 bytes along the
// product's inner dimension, 8-row groups 1024 bytes apart) for Q and K;
// N-major for V (rows of 128 bytes along the output's columns, one per key:
// 8-key groups 1024 bytes apart, 64-column panels `panel` bytes apart).  The
// upper word is one constant (stride 1024, version 1, swizzle 128 bytes), the
// lower one the address and the leading offset, in 16-byte units: steps inside
// a tile are additions to it.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k_major(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | 1u << 16;
}
__device__ __forceinline__ uint32_t desc_n_major(uint32_t addr, uint32_t panel) {
  return ((addr & 0x3FFFFu) >> 4) | (panel >> 4) << 16;
}

// kind::f16: D = f32 (bit 4), A = B = f16 (0), B's major-ness at bit 16,
// N >> 3 at bits 17-22, M >> 4 at bits 24-28.
constexpr uint32_t instr(int n, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(kTileRows >> 4) << 24;
}

// One thread of the warp.  Branching on this rather than on a lane number
// lets the operands of the products stay in uniform registers: measured, a
// 128 x 64 x 16 product then issues every 48 cycles instead of 95, a
// 128 x 128 x 16 one every 64, which is what they take.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0u;
}

template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "n"(ADD ? 1 : 0)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "r"(add)
      : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// The wait is part of the load: until it, the registers named as results do
// not hold them, and nothing may be made of them, a spill to the stack least.
__device__ __forceinline__ void tmem_ld64(uint32_t addr, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "{\n\t.reg .b32 a;\n\tadd.u32 a, %64, 32;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [a];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]),
        "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]),
        "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31]), "=r"(u[32]), "=r"(u[33]), "=r"(u[34]),
        "=r"(u[35]), "=r"(u[36]), "=r"(u[37]), "=r"(u[38]), "=r"(u[39]), "=r"(u[40]), "=r"(u[41]),
        "=r"(u[42]), "=r"(u[43]), "=r"(u[44]), "=r"(u[45]), "=r"(u[46]), "=r"(u[47]), "=r"(u[48]),
        "=r"(u[49]), "=r"(u[50]), "=r"(u[51]), "=r"(u[52]), "=r"(u[53]), "=r"(u[54]), "=r"(u[55]),
        "=r"(u[56]), "=r"(u[57]), "=r"(u[58]), "=r"(u[59]), "=r"(u[60]), "=r"(u[61]), "=r"(u[62]),
        "=r"(u[63])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]),
        "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]),
        "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
      "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]),
      "r"(u[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Pairs of f32, one instruction for both.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// The pair w as f16 high parts and, in `lo`, f16 low parts.  The high part is
// w cut to f16's 11 bits, whose conversion is exact, so that the rest w - high
// is as well: 21 bits in all, for one logic operation a value where rounding
// would cost a conversion back.
__device__ __forceinline__ uint32_t cut_half2(float2 w, uint32_t& lo) {
  const float2 h = make_float2(__uint_as_float(__float_as_uint(w.x) & 0xFFFFE000u),
                               __uint_as_float(__float_as_uint(w.y) & 0xFFFFE000u));
  const float2 r = fma2(h, make_float2(-1.0f, -1.0f), w);
  lo = pack_half2(r.x, r.y);
  return pack_half2(h.x, h.y);
}

// Words of a query row as they lie in memory from element `at` on, and value i
// of them (16-bit ones two to a word).
template <int WORDS>
__device__ __forceinline__ void load_q(const void* q, int size, int64_t at, uint32_t (&w)[WORDS]) {
  const uint8_t* p = static_cast<const uint8_t*>(q) + at * size;
  if constexpr (WORDS == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <int E, bool F32, int WORDS>
__device__ __forceinline__ float q_value(bool f16, const uint32_t (&words)[WORDS], int i) {
  if constexpr (F32) return __uint_as_float(words[i]);
  const uint32_t w = words[i / 2 % WORDS];
  if (f16) {
    const float2 f = half_pair(w);
    return (i & 1) ? f.y : f.x;
  }
  return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
}

// Value scales are kept relative to a power of two: four times the next one
// above the largest so far, so that it seldom moves; and kUp over it.
constexpr float kMostScale = 1e37f;  // larger ones, and NaN, do not count
__device__ __forceinline__ float next_scale(float v) {
  return __uint_as_float((__float_as_uint(v) & 0x7F800000u) + (2u << 23));
}
__device__ __forceinline__ float up_over(float vref) {
  return __uint_as_float(((254u + 7u) << 23) - __float_as_uint(vref));
}

// A thread's wait for a barrier phase; after one wait has run out, no further
// one is made, so that every role comes to its end.
__device__ __forceinline__ void wait_one(bool& ok, const uint64_t& bar, uint32_t parity,
                                         unsigned int* error) {
  if (ok) {  // (in line: a call would spill what the roles hold in registers)
    const uint32_t addr = smem_u32(&bar);
    bool done = mbar_try_wait(addr, parity & 1u);
    if (!done) {
      const uint64_t t0 = globaltimer();
      do {
        done = mbar_try_wait(addr, parity & 1u);
      } while (!done && globaltimer() - t0 <= kWaitLimitNs);
      if (!done) atomicOr(error, 1u);
    }
    ok = done;
  }
}

// A warp's.
__device__ __forceinline__ void wait(bool& ok, const uint64_t& bar, uint32_t parity,
                                     unsigned int* error) {
  wait_one(ok, bar, parity, error);
  ok = __all_sync(0xFFFFFFFFu, ok);
}

// The pages of a segment's units, four 16-key boxes each: every lane holds the
// (page, kv head) plane of one box of the present window of 32 boxes (8 units)
// and of the next, so that no fetch waits for the page table.
struct PageWindow {
  int cur, nxt, window;
  __device__ __forceinline__ int load(const AttnArgs& a, const Segment& g, int w, int lane) const {
    const int64_t place = ((int64_t)w * 32 + lane) * 16;
    return place < g.kv ? page_of(a, (int)quotient((uint32_t)g.item, a.by_tiles), place) * a.kv_heads + g.head : 0;
  }
  __device__ __forceinline__ void open(const AttnArgs& a, const Segment& g, int u, int lane) {
    window = u >> 3;
    cur = load(a, g, window, lane);
    nxt = load(a, g, window + 1, lane);
  }
  __device__ __forceinline__ void step(const AttnArgs& a, const Segment& g, int u, int lane) {
    if (u >> 3 == window) return;
    window = u >> 3;
    cur = nxt;
    nxt = load(a, g, window + 1, lane);
  }
  __device__ __forceinline__ int plane(int box) const {  // of the present window
    return __shfl_sync(0xFFFFFFFFu, cur, box & 31);
  }
};

// Whether unit u of a segment begins row tile w's output anew: the two tiles in
// turn, so that one works on while the other's sum is taken out.
template <bool SPLIT>
__device__ __forceinline__ bool starts_anew(int u, int w) {
  return u == 0 || (SPLIT && (u + w * (kFlush / 2)) % kFlush == 0);
}

// ------------------------------------------------------------- the kernel --

template <int D, bool I8, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) attn_rows_kernel(const AttnArgs a) {
  using L = Layout<D, SPLIT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  RowsTail& tail = *reinterpret_cast<RowsTail*>(smem + L::kTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_base = smem_u32(smem);
  const uint32_t kv_base = q_base + L::kQ;  // unit u: K at (u & 1) 2 kB, V behind it

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&tail.q_full[i]), 4);
      mbar_init(smem_u32(&tail.k_full[i]), kConvert / 32);
      mbar_init(smem_u32(&tail.v_full[i]), kConvert / 32);
      mbar_init(smem_u32(&tail.k_free[i]), 2);  // of both row tiles
      mbar_init(smem_u32(&tail.v_free[i]), 2);
      mbar_init(smem_u32(&tail.drained[i]), 1);
      mbar_init(smem_u32(&tail.pv_done[i]), 1);
      for (int j = 0; j < 2; ++j) {
        mbar_init(smem_u32(&tail.s_full[i][j]), 1);
        mbar_init(smem_u32(&tail.p_full[i][j]), 4);
      }
    }
    for (int i = 0; i < kScales; ++i) mbar_init(smem_u32(&tail.sc_full[i]), 1);
    mbar_fence_init();
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&tail.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tail.tmem;
  pdl_wait();
  pdl_trigger();
  prefetch_l2(a.q, a.q_bytes);
  prefetch_l2(a.table, (int64_t)a.batch * a.max_pages * 4);
  Cutting cutter(a, tail.cut);
  cutter.template choose<kThreads>();
  Segment seg;
  const bool work = cutter.begin(seg);
  if (!work && tid == 0 && a.shares != nullptr) a.shares[blockIdx.x].segment = -1;
  bool ok = true;

  // Each group of warps moves its registers at the head of its own branch,
  // never before one: what follows is compiled for the count it names.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    if (work) {
    // ------------------------------------------------------- softmax ----
    const int w = warp >> 2, quad = warp & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t s_col = tmem + w * 256 + lanes, o_col = s_col + 128;
    uint32_t units = 0;            // of this row tile so far
    uint32_t all_units = 0;        // of the CTA: the scales' ring
    for (bool first_seg = true;; first_seg = false) {
      const int b = cutter.sequence(seg.item), rt = seg.item - b * a.row_tiles;
      const int row0 = rt * kRows + w * kTileRows;
      const int n_units = seg.end - seg.first;
      float l = 0.0f, ref = -INFINITY, c = 0.0f, vref = 0x1p-112f;
      // what the flushed sum is relative to; it lies column by column of four,
      // the warp's rows one after another
      float ref_kept = -INFINITY, vref_kept = 0.0f;
      bool kept = false;
      auto to_now = [&]() -> float {  // the kept sum's factor
        return ref_kept == -INFINITY ? 0.0f : ex2(ref_kept - ref) * (vref_kept / vref);
      };
      float4* const sum_at = SPLIT ? a.flushed + ((int64_t)blockIdx.x * 8 + warp) * (D * 8) + lane
                                   : nullptr;
      if (row0 < a.rows) {
        // ---- this warp's 32 query rows, to f16 parts in shared memory
        constexpr int E = D / 32;
        const int my_row = row0 + quad * 32 + lane;
        const bool live = my_row < a.rows;
        const int tok = live ? (int)quotient((uint32_t)my_row, a.by_group) : 0;
        const int64_t my_off =
            ((int64_t)b * a.new_tokens + tok) * a.q_stride +
            (int64_t)(seg.head * a.group + (live ? my_row - tok * a.group : 0)) * D;
        const uint32_t q_at = q_base + w * ((SPLIT ? 2 : 1) * L::kQTile) + quad * 32 * 128;
        // eight or sixteen rows at a time, the next ones' loads in flight
        constexpr int kStep = SPLIT ? 8 : 16;
        constexpr int kLg = SPLIT ? 3 : 4;
        constexpr int kWords = SPLIT ? E : E / 2;
        uint32_t raw[kStep][kWords];
        auto load = [&](int r0) {
#pragma unroll
          for (int r = 0; r < kStep; ++r)
            load_q<kWords>(a.q, SPLIT ? 4 : 2, __shfl_sync(0xFFFFFFFFu, my_off, r0 + r) + lane * E,
                           raw[r]);
        };
        load(0);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += kStep) {
          float x[kStep][E];
          // largest magnitudes, as bits: a NaN counts as above infinity.  (A
          // row past the last one stands in for the sequence's first: what it
          // gives is not written.)
          uint32_t top[kStep];
#pragma unroll
          for (int r = 0; r < kStep; ++r) {
            top[r] = 0u;
#pragma unroll
            for (int i = 0; i < E; ++i) {
              x[r][i] = q_value<E, SPLIT>(a.dtype == RQ_F16, raw[r], i);
              top[r] = max(top[r], __float_as_uint(x[r][i]) & 0x7FFFFFFFu);
            }
          }
          if (r0 + kStep < 32) load(r0 + kStep);
          // the rows' maxima, all at once: each step halves the rows that a
          // lane holds; lane bits from 4 down are the row's bits from the top
#pragma unroll
          for (int n = kStep / 2, o = 16; n >= 1; n >>= 1, o >>= 1) {
            const bool up_half = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < n; ++i) {
              const uint32_t keep = up_half ? top[i + n] : top[i];
              const uint32_t give = up_half ? top[i] : top[i + n];
              top[i] = max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
            }
          }
          uint32_t most = max(top[0], __shfl_xor_sync(0xFFFFFFFFu, top[0], 1));
          if (kLg == 3) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
          // times a power of two: the largest entry in [2^13, 2^14); a row
          // that is not finite becomes NaN, and so do its scores
          int e = 0;
          if (most > 0u) {
            e = 13 - (int)(most >> 23) + 127;
            e = e < -126 ? -126 : e > 100 ? 100 : e;
          }
          const float own = most < 0x7F800000u ? __uint_as_float((uint32_t)(e + 127) << 23) : NAN;
#pragma unroll
          for (int r = 0; r < kStep; ++r) {
            int from = 0;  // the row's bits, the top one at lane bit 4
#pragma unroll
            for (int k = 0; k < kLg; ++k) from |= ((r >> (kLg - 1 - k)) & 1) << (4 - k);
            const float up = __shfl_sync(0xFFFFFFFFu, own, from);
            if (lane == r0 + r) c = up;
            const int byte = lane * E * 2;
            const uint32_t at = q_at + (byte >> 7) * L::kQPanel + (r0 + r) * 128 +
                                ((((byte >> 4) & 7) ^ (r & 7)) << 4) + (byte & 15);
            uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
              const float2 v = mul2(make_float2(x[r][2 * i], x[r][2 * i + 1]), make_float2(up, up));
              if (SPLIT)
                hi[i] = cut_half2(v, lo[i]);
              else
                hi[i] = pack_half2(v.x, v.y);
            }
            if constexpr (E == 4) {
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(hi[0]), "r"(hi[1])
                           : "memory");
              if (SPLIT)
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + L::kQTile),
                             "r"(lo[0]), "r"(lo[1])
                             : "memory");
            } else {
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(hi[0]) : "memory");
              if (SPLIT)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + L::kQTile), "r"(lo[0])
                             : "memory");
            }
          }
        }
        // (2^-126 where c is a NaN: what the row does not see weighs 0 all the same)
        c = fmaxf(a.scale_log2 / c, 0x1p-126f);
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tail.q_full[w]));

        unsigned long long bits = 0;
        if (live && a.tree != nullptr) bits = a.tree[(int64_t)b * a.new_tokens + tok];
        const int kv = seg.kv;
        const int n_all = cutter.length(b);
        const int len = n_all < 0 ? 0 : n_all < kv ? n_all : kv;
        // places that all of the warp's rows see: without a tree also the new
        // ones up to its first row's own
        const int sure =
            a.tree == nullptr ? min(kv, len + __shfl_sync(0xFFFFFFFFu, tok, 0) + 1) : len;

        for (int u = 0; u < n_units; ++u) {
          const uint32_t sc = (all_units + u) % kScales;
          const uint32_t buf = units & 1u;
          const bool fresh = starts_anew<SPLIT>(u, w);  // O begins again from zero
          // Scores of a unit mean that the weights of the one two before were
          // taken, so the scales' barrier is past its last turn: a tile that
          // sat out a segment does not mistake an older turn for this one.
          wait(ok, tail.s_full[w][buf], units >> 1, a.error);
          wait(ok, tail.sc_full[sc], (all_units + u) / kScales, a.error);
          fence_after();
          if (SPLIT && fresh && u > 0) {
            const float f = to_now();
            // (waited for after the scores, which came after the turn before)
            wait(ok, tail.pv_done[w], units - 1u, a.error);
            fence_after();
#pragma unroll
            for (int d = 0; d < D; d += 32) {
              float o[32];
              float4 v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                v[i] = kept ? __ldcg(sum_at + (d / 4 + i) * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
              tmem_ld32(o_col + d, o);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                __stcg(sum_at + (d / 4 + i) * 32,
                       make_float4(fmaf(v[i].x, f, o[4 * i]), fmaf(v[i].y, f, o[4 * i + 1]),
                                   fmaf(v[i].z, f, o[4 * i + 2]), fmaf(v[i].w, f, o[4 * i + 3])));
            }
            kept = true;
            ref_kept = ref;
            vref_kept = vref;
          }
          float x[kKeys];
          tmem_ld64(s_col + buf * kKeys, x);
          const float4* ks = reinterpret_cast<const float4*>(tail.ks[sc]);
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < kKeys / 4; ++i) {
            const float4 k4 = ks[i];
            const float2 xa = mul2(make_float2(x[4 * i], x[4 * i + 1]), make_float2(k4.x, k4.y));
            const float2 xb = mul2(make_float2(x[4 * i + 2], x[4 * i + 3]), make_float2(k4.z, k4.w));
            x[4 * i] = xa.x;
            x[4 * i + 1] = xa.y;
            x[4 * i + 2] = xb.x;
            x[4 * i + 3] = xb.y;
          }
          const int p0 = (seg.first + u) * kKeys;
          const bool edge = p0 + kKeys > sure;
          // The row's value scales are kept relative to a power of two above
          // those that it sees: for all rows alike but for those that do not
          // see the unit that raised it.
          float need = tail.vmost[sc];
          if (edge) {
            // bit k: key k of the unit is seen
            const int before = len - p0;  // keys that every row sees
            unsigned long long see =
                before >= 64 ? ~0ull : before > 0 ? (1ull << before) - 1ull : 0ull;
            if (a.tree != nullptr) {
              if (before > -64 && before < 64)
                see |= before >= 0 ? bits << before : bits >> -before;
            } else {
              const int upto = before + tok + 1;
              if (upto > 0) see |= upto >= 64 ? ~0ull : (1ull << upto) - 1ull;
            }
            const int exist = kv - p0;
            if (exist < 64) see &= exist > 0 ? (1ull << exist) - 1ull : 0ull;
            const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (!((s0 >> i) & 1u)) x[i] = -INFINITY;
              if (!((s1 >> i) & 1u)) x[32 + i] = -INFINITY;
            }
            // (looked at one by one only where the unit raises the power of two:
            // a bf16 prompt of 110 us takes 137 with the loop in every such unit)
            const bool raises = __any_sync(0xFFFFFFFFu, need > vref);
            need = 0.0f;
            if (raises) {
#pragma unroll 1
              for (int i = 0; i < kKeys; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(&tail.vr[sc][i]);
                const uint32_t bits4 = (uint32_t)(see >> i);
                if ((bits4 & 1u) && v.x <= kMostScale) need = fmaxf(need, v.x);
                if ((bits4 & 2u) && v.y <= kMostScale) need = fmaxf(need, v.y);
                if ((bits4 & 4u) && v.z <= kMostScale) need = fmaxf(need, v.z);
                if ((bits4 & 8u) && v.w <= kMostScale) need = fmaxf(need, v.w);
              }
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kKeys; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], fmaxf(x[i + k], x[i + k + 4]));
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          // The reference that the row's weights are relative to moves only
          // when a score passes it by 2^8 (f16 has room for that), so that O
          // is seldom scaled anew.
          const float now = mx * c;  // powers of two
          const float vall = fabsf(tail.vref[sc]);
          // (rows past the last one go with the others)
          const float vnow = !live ? vall : need > vref ? next_scale(need) : vref;
          const bool moves = now > ref + kLazy || vnow != vref;
          if (__any_sync(0xFFFFFFFFu, moves)) {
            const float to = now > ref + kLazy ? now : ref;
            const float al = ref == -INFINITY ? 0.0f : ex2(ref - to);
            const float f = al * (vref / vnow);
            l *= al;
            ref = to;
            vref = vnow;
            if (!fresh) {
              wait(ok, tail.pv_done[w], units - 1u, a.error);
              fence_after();
#pragma unroll
              for (int d = 0; d < D; d += 16) {
                float o[16];
                tmem_ld16(o_col + d, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= f;
                tmem_st16(o_col + d, reinterpret_cast<const uint32_t*>(o));
              }
              tmem_st_wait();
            }
          }
          const float base = ref == -INFINITY ? 0.0f : ref;
          // What a row does not see must not reach it: a scale out of range
          // (times a weight of 0 it may be no 0), or one that others' are
          // relative to.  Then the scales are taken as they are.
          const bool rare = __any_sync(0xFFFFFFFFu, vref != vall) || tail.vref[sc] < 0.0f;
          const float4* vs = reinterpret_cast<const float4*>(rare ? tail.vr[sc] : tail.vs[sc]);
          const float inv = up_over(vref);
          const float2 c2 = make_float2(c, c), nb = make_float2(-base, -base);
          float2 l2 = make_float2(0.0f, 0.0f);
          // (two copies of the loop, the rare one with its tests: 2 % of a bf16
          // prompt's time)
          auto weights = [&](auto own) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 v4 = vs[8 * half + i];
                const float* xi = x + 32 * half + 4 * i;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float2 p = fma2(make_float2(xi[2 * k], xi[2 * k + 1]), c2, nb);
                  p.x = ex2(p.x);
                  p.y = ex2(p.y);
                  l2 = add2(l2, p);
                  float2 v2 = k == 0 ? make_float2(v4.x, v4.y) : make_float2(v4.z, v4.w);
                  if constexpr (decltype(own)::value) v2 = mul2(v2, make_float2(inv, inv));
                  float2 wt = mul2(p, v2);
                  if constexpr (decltype(own)::value) {
                    wt.x = p.x == 0.0f ? 0.0f : wt.x;
                    wt.y = p.y == 0.0f ? 0.0f : wt.y;
                  }
                  if constexpr (SPLIT)
                    hi[2 * i + k] = cut_half2(wt, lo[2 * i + k]);
                  else
                    hi[2 * i + k] = pack_half2(wt.x, wt.y);
                }
              }
              tmem_st16(s_col + buf * kKeys + 16 * half, hi);
              if constexpr (SPLIT) tmem_st16(s_col + buf * kKeys + 32 + 16 * half, lo);
            }
          };
          if (rare)
            weights(Flag<true>());
          else
            weights(Flag<false>());
          l += l2.x + l2.y;
          tmem_st_wait();
          fence_before();
          __syncwarp();
          // A barrier's parity tells a turn from the one before only, and a
          // warp can be a unit ahead of the others: the products of the unit
          // before the last are seen to be done while the last ones' cannot be.
          if (u > 0 && u + 1 == n_units) wait(ok, tail.pv_done[w], units - 1u, a.error);
          if (lane == 0) mbar_arrive(smem_u32(&tail.p_full[w][buf]));
          ++units;
        }
        // ---- the segment's output rows
        wait(ok, tail.pv_done[w], units - 1u, a.error);
        fence_after();
      }
      all_units += n_units;

      // a.part holds per CTA two sets of kRows rows of D values, reference
      // and sum (D + 4 floats); the join kernel learns which sets are whose
      const bool whole = cutter.whole(seg);
      if (row0 < a.rows) {
        float* set = a.part + ((int64_t)blockIdx.x * 2 + (cutter.second_set(seg, first_seg) ? 1 : 0)) *
                                  (int64_t)kRows * kPartRow<D>;
        const int my = w * kTileRows + quad * 32;  // the warp's first row of the segment
        const int my_row = rt * kRows + my + lane;
        const bool live = my_row < a.rows;
        const int tok = live ? (int)quotient((uint32_t)my_row, a.by_group) : 0;
        const int64_t my_dst = (((int64_t)b * a.new_tokens + tok) * a.q_heads +
                                seg.head * a.group + (live ? my_row - tok * a.group : 0)) * D;
        const float back = vref * (1.0f / kUp);
        const float f_kept = SPLIT ? to_now() : 0.0f;
        const float r1 = !whole ? back : l == 0.0f ? 0.0f : back / l;
        // A thread holds a row; memory wants a warp to write one.  The rows
        // pass through the warp's part of the query tile, which the segment's
        // products are done with: as wide as a query row there, in 16-byte
        // pieces whose places are exclusive-ored with the row against bank
        // conflicts.
        constexpr int kBytes = (SPLIT ? 2 : 1) * D * 2;
        const uint32_t stage = q_base + w * ((SPLIT ? 2 : 1) * L::kQTile) + quad * 32 * kBytes;
        auto pass = [&](auto wide, int d0) {  // columns from d0 on, as f32 or 16-bit values
          constexpr bool kWide = decltype(wide)::value;
          constexpr int kCols = kBytes / (kWide ? 4 : 2);
#pragma unroll
          for (int d = 0; d < kCols; d += 32) {
            float o[32];
            tmem_ld32(o_col + d0 + d, o);
            if (SPLIT && kept) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 v = __ldcg(sum_at + ((d0 + d) / 4 + i) * 32);
                o[4 * i] = fmaf(v.x, f_kept, o[4 * i]);
                o[4 * i + 1] = fmaf(v.y, f_kept, o[4 * i + 1]);
                o[4 * i + 2] = fmaf(v.z, f_kept, o[4 * i + 2]);
                o[4 * i + 3] = fmaf(v.w, f_kept, o[4 * i + 3]);
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= r1;
            uint32_t h[kWide ? 32 : 16];
            if constexpr (kWide) {
#pragma unroll
              for (int i = 0; i < 32; ++i) h[i] = __float_as_uint(o[i]);
            } else if (a.dtype == RQ_F16) {
#pragma unroll
              for (int i = 0; i < 16; ++i) h[i] = pack_half2(o[2 * i], o[2 * i + 1]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                h[i] = *reinterpret_cast<const uint32_t*>(&t);
              }
            }
#pragma unroll
            for (int i = 0; i < (kWide ? 8 : 4); ++i) {
              const int piece = d / (kWide ? 4 : 8) + i;
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                               stage + lane * kBytes + ((piece ^ (lane & 7)) << 4)),
                           "r"(h[4 * i]), "r"(h[4 * i + 1]), "r"(h[4 * i + 2]), "r"(h[4 * i + 3])
                           : "memory");
            }
          }
          __syncwarp();
          constexpr int kPer = kBytes / 16, kTake = 32 / kPer;  // pieces of a row, rows at once
#pragma unroll 4
          for (int r0 = 0; r0 < 32; r0 += kTake) {
            const int r = r0 + lane / kPer, piece = lane % kPer;
            const int64_t dst = __shfl_sync(0xFFFFFFFFu, my_dst, r);
            uint32_t h[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                         : "r"(stage + r * kBytes + ((piece ^ (r & 7)) << 4))
                         : "memory");
            if (rt * kRows + my + r >= a.rows) continue;
            const uint4 v = make_uint4(h[0], h[1], h[2], h[3]);
            if (!whole)
              __stcg(reinterpret_cast<uint4*>(set + (my + r) * kPartRow<D> + d0) + piece, v);
            else if (kWide)
              *(reinterpret_cast<uint4*>(static_cast<float*>(a.out) + dst) + piece) = v;
            else
              *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + dst) + piece) = v;
          }
          __syncwarp();
        };
        if (SPLIT) {
          pass(Flag<true>(), 0);
        } else if (!whole) {
          pass(Flag<true>(), 0);
          pass(Flag<true>(), D / 2);
        } else {
          pass(Flag<false>(), 0);
        }
        if (!whole && live)
          __stcg(reinterpret_cast<float2*>(set + (my + lane) * kPartRow<D> + D),
                 make_float2(ref, l));
        fence_before();
        // the query tile is all warps' again
        asm volatile("bar.sync %0, 128;" ::"r"(2 + w) : "memory");
      }
      if (seg.left <= 0) break;
      cutter.next(seg);
    }
    }
  } else if (warp < kIssueWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
    if (work) {
    // --------------------------------------------------- conversion ----
    constexpr int kChunks = D / 16;                    // 16-code chunks of a row
    constexpr int N = kKeys * kChunks / kConvert;      // of K (and of V) per thread and unit
    const int t = tid - kSoft;
    const int chunk = t % kChunks, row_a = t / kChunks;
    constexpr int kRowStep = kConvert / kChunks;
    // where chunk `chunk` of row r goes: 32 bytes of an f16 row
    const uint32_t at = (chunk >> 2) * L::kPanel;
    const int c16 = (chunk & 3) * 2;
    uint4 kc[N], vc[N];  // the next unit's codes, on their way into registers
    PageWindow pages;
    const int page_mask = (1 << a.lg_page) - 1, page_bytes = D << a.lg_page;
    int64_t off[N];  // of the next unit's rows, in K and V alike; negative: no such key
    auto find = [&](const Segment& g, int u) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int key = u * kKeys + row_a + n * kRowStep;
        const int plane = pages.plane(key >> 4);
        off[n] = key < g.kv ? (int64_t)plane * page_bytes + ((key & page_mask) * D + chunk * 16) : -1;
      }
    };
    auto fetch = [&](uint4 (&c)[N], const uint8_t* codes) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        c[n] = make_uint4(0u, 0u, 0u, 0u);
        if (off[n] >= 0) c[n] = ldg_nc_v4(codes + off[n]);
      }
    };
    // the segment's places that every row sees come before `seen`
    int seen = cutter.length(cutter.sequence(seg.item));
    auto convert = [&](const uint4 (&codes)[N], uint32_t base, bool drop) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int r = row_a + n * kRowStep;
        uint32_t words[4] = {codes[n].x, codes[n].y, codes[n].z, codes[n].w};
        if (!I8 && drop) {
#pragma unroll
          for (int i = 0; i < 4; ++i) words[i] = without_nan(words[i]);
        }
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) codes_in_order<I8>(words[i], h[2 * i], h[2 * i + 1]);
        const uint32_t to = base + at + r * 128;
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                         to + ((c16 ^ (r & 7)) << 4)),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                     : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                         to + (((c16 + 1) ^ (r & 7)) << 4)),
                     "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                     : "memory");
      }
    };
    pages.open(a, seg, seg.first, lane);
    find(seg, seg.first);
    fetch(kc, a.k);
    fetch(vc, a.v);
    uint32_t units = 0;
    for (int u = seg.first;;) {
      const uint32_t buf = units & 1u, turn = (units >> 1) ^ 1u;
      const uint32_t kb = kv_base + buf * (2 * L::kB);
      wait(ok, tail.k_free[buf], turn, a.error);
      convert(kc, kb, false);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail.k_full[buf]));
      // the next unit's codes are fetched as soon as this one's have left
      // their registers
      const bool drop = (u + 1) * kKeys > seen;  // of V: new tokens' codes
      bool more = true;
      if (++u < seg.end) {
        pages.step(a, seg, u, lane);
      } else {
        more = seg.left > 0;
        if (more) {
          cutter.next(seg);
          u = seg.first;
          seen = cutter.length(cutter.sequence(seg.item));
          pages.open(a, seg, u, lane);
        }
      }
      if (more) {
        find(seg, u);
        fetch(kc, a.k);
      }
      wait(ok, tail.v_free[buf], turn, a.error);
      convert(vc, kb + L::kB, drop);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail.v_full[buf]));
      if (!more) break;
      fetch(vc, a.v);
      ++units;
    }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (work && warp == kIssueWarp + 1) {
    // ------------------------------------------- scales, and codes into L2 --
    uint32_t units = 0;
    bool first_seg = true;
    const int page_mask = (1 << a.lg_page) - 1, page_bytes = D << a.lg_page;
    for (;;) {
      float vref = 0x1p-112f;
      PageWindow pages, ahead;
      pages.open(a, seg, seg.first, lane);
      ahead = pages;
      int asked = seg.first + 1;
      float s[4];
      auto fetch = [&](int u) {  // of keys lane and lane + 32
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int key = lane + 32 * n;
          const int64_t row = ((int64_t)pages.plane(u * 4 + (key >> 4)) << a.lg_page) +
                              ((u * kKeys + key) & page_mask);
          s[2 * n] = s[2 * n + 1] = 0.0f;
          if (u * kKeys + key < seg.kv) {
            s[2 * n] = __ldg(a.ks + row);
            s[2 * n + 1] = __ldg(a.vs + row);
          }
        }
      };
      fetch(seg.first);
      for (int u = seg.first; u < seg.end; ++u, ++units) {
        // codes of the units up to kAhead on: lanes 0-3 the boxes of K, 4-7
        // those of V
        for (; asked <= u + kAhead && asked < seg.end; ++asked) {
          ahead.step(a, seg, asked, lane);
          const int key = (lane & 3) * 16;
          const int plane = ahead.plane(asked * 4 + (lane & 3));
          if (lane < 8 && asked * kKeys + key < seg.kv) {
            const uint8_t* at = (lane < 4 ? a.k : a.v) + (int64_t)plane * page_bytes +
                                ((asked * kKeys + key) & page_mask) * D;
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "n"(16 * D)
                         : "memory");
          }
        }
        // value scales relative to a power of two above all so far
        float vt = fmaxf(s[1] <= kMostScale ? s[1] : 0.0f, s[3] <= kMostScale ? s[3] : 0.0f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) vt = fmaxf(vt, __shfl_xor_sync(0xFFFFFFFFu, vt, o));
        if (vt > vref) vref = next_scale(vt);
        const float inv = up_over(vref);
        // the ring's place is free once the unit two before is done with
        // (its own occupant was the one four before)
        const uint32_t sc = units % kScales;
        wait(ok, tail.v_free[units & 1u], (units >> 1) ^ 1u, a.error);
        tail.ks[sc][lane] = s[0];
        tail.ks[sc][lane + 32] = s[2];
        tail.vs[sc][lane] = s[1] * inv;
        tail.vs[sc][lane + 32] = s[3] * inv;
        tail.vr[sc][lane] = s[1];
        tail.vr[sc][lane + 32] = s[3];
        const bool odd = __any_sync(0xFFFFFFFFu, !(s[1] >= 0.0f && s[1] <= kMostScale &&
                                                   s[3] >= 0.0f && s[3] <= kMostScale));
        if (lane == 0) {
          tail.vref[sc] = odd ? -vref : vref;
          tail.vmost[sc] = vt;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tail.sc_full[sc]));
        if (u + 1 < seg.end) {
          pages.step(a, seg, u + 1, lane);
          fetch(u + 1);
        }
      }
      if (seg.left <= 0) break;
      cutter.next(seg);
      first_seg = false;
    }
    // for the join: the segment that this CTA begins and others go on with, if
    // any -- the last one of its work
    if (a.shares != nullptr && lane == 0) {
      SharedSegment note = {0, -1, 0, 0, 0, 0};
      if (!cutter.whole(seg) && seg.first == 0) note = cutter.note(seg, first_seg);
      a.shares[blockIdx.x] = note;
    }
  } else if (work && warp != kIssueWarp + 3) {
    // ------------------------------------------------------ products ----
    // A thread for each row tile: a warp's votes in the waits would add to the
    // way from one unit's weights to the scores two units on.
    const int w = (warp - kIssueWarp) >> 1;
    constexpr uint32_t kS = instr(kKeys, false), kO = instr(D, true);
    uint32_t units = 0, segs = 0, mine = 0;
    auto scores = [&](uint32_t unit_no, uint32_t my_no) {  // by one thread
      const uint32_t d = tmem + w * 256 + (my_no & 1u) * kKeys;
      const uint32_t qd = desc_k_major(q_base + w * ((SPLIT ? 2 : 1) * L::kQTile));
      const uint32_t kd = desc_k_major(kv_base + (unit_no & 1u) * (2 * L::kB));
      // The low parts first: the tensor cores cut each sum off towards zero,
      // and those of the low parts are small.
#pragma unroll
      for (int i = 0; i < (SPLIT ? 2 : 1) * L::kPanels; ++i) {
        const uint32_t at = qd + (SPLIT ? (i + L::kPanels) % (2 * L::kPanels) : i) * (L::kQPanel >> 4);
        const uint32_t kp = kd + (i % L::kPanels) * (L::kPanel >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (i + k == 0)
            mma_ss<false>(d, at, kp, kS);
          else
            mma_ss<true>(d, at + 2 * k, kp + 2 * k, kS);
        }
      }
      commit(smem_u32(&tail.s_full[w][my_no & 1u]));
      commit(smem_u32(&tail.k_free[unit_no & 1u]));
    };
    if (elect_one())
    for (;;) {
      const int b = cutter.sequence(seg.item), rt = seg.item - b * a.row_tiles;
      const int n = seg.end - seg.first;
      if (rt * kRows + w * kTileRows >= a.rows) {
        // no rows: the codes are the other tile's alone
        for (int u = 0; u < n; ++u) {
          const uint32_t cur = units + u;
          wait_one(ok, tail.k_full[cur & 1u], cur >> 1, a.error);
          mbar_arrive(smem_u32(&tail.k_free[cur & 1u]));
          wait_one(ok, tail.v_full[cur & 1u], cur >> 1, a.error);
          mbar_arrive(smem_u32(&tail.v_free[cur & 1u]));
        }
      } else {
        // the first scores of the segment
        wait_one(ok, tail.k_full[units & 1u], units >> 1, a.error);
        wait_one(ok, tail.q_full[w], segs, a.error);
        ++segs;
        fence_after();
        scores(units, mine);
        for (int u = 0; u < n; ++u) {
          const uint32_t cur = units + u, buf = cur & 1u;
          const uint32_t p = mine++;  // this unit's number of the row tile
          if (u + 1 < n) {
            wait_one(ok, tail.k_full[buf ^ 1u], (cur + 1) >> 1, a.error);
            // The scores go where the weights two units back are: products
            // into different accumulators are not ordered by themselves.
            if (u > 0) wait_one(ok, tail.pv_done[w], p - 1u, a.error);
            fence_after();
            scores(cur + 1, p + 1);
          }
          wait_one(ok, tail.v_full[buf], cur >> 1, a.error);
          wait_one(ok, tail.p_full[w][p & 1u], p >> 1, a.error);
          fence_after();
          const uint32_t d = tmem + w * 256 + 128;
          const uint32_t pa = tmem + w * 256 + (p & 1u) * kKeys;
          const uint32_t vd = desc_n_major(kv_base + buf * (2 * L::kB) + L::kB, L::kPanel);
#pragma unroll
          for (int s = 0; s < (SPLIT ? 2 : 1); ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(d, pa + s * 32 + k * 8, vd + k * (2048 >> 4), kO,
                     (starts_anew<SPLIT>(u, w) ? 0u : 1u) | s | k);
          commit(smem_u32(&tail.pv_done[w]));
          commit(smem_u32(&tail.v_free[buf]));
        }
      }
      units += n;
      if (seg.left <= 0) break;
      cutter.next(seg);
    }
    __syncwarp();
    // every product has completed before TMEM is released
    if (elect_one()) commit(smem_u32(&tail.drained[w]));
    __syncwarp();
    bool drained = true;
    wait(drained, tail.drained[w], 0, a.error);
  }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if ((threadIdx.x >> 5) == kIssueWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tail.tmem)
                 : "memory");
}

// Joins the partial rows of segments that several CTAs share, in part order: a
// thread takes four columns of kJoinRows rows, with kJoinParts parts of each
// in flight.
constexpr int kJoinRows = 2, kJoinParts = 2;
template <int D>
constexpr int kJoinBlock = 256 / (D / 4) * kJoinRows;  // rows of a CTA

template <int D>
__global__ void __launch_bounds__(256) join_rows_kernel(const AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kBlocks = kRows / kJoinBlock<D>;  // CTAs per segment
  constexpr int kAtOnce = kJoinBlock<D> / kJoinRows;
  const int cta0 = (int)(blockIdx.x / kBlocks);
  const SharedSegment share = a.shares[cta0];
  if (share.segment < 0) return;
  const int parts = share.parts > 0
                        ? share.parts
                        : (int)((((int64_t)share.last + 1) * share.ctas - 1) / share.cost) - cta0 + 1;
  const int item = (int)quotient((uint32_t)share.segment, a.by_heads);
  const int head = share.segment - item * a.kv_heads;
  const int b = (int)quotient((uint32_t)item, a.by_tiles), rt = item - b * a.row_tiles;
  const int d = (int)(threadIdx.x % (D / 4)) * 4;
  const int r0 = (int)(blockIdx.x % kBlocks) * kJoinBlock<D> + (int)(threadIdx.x / (D / 4));
  float4 v[kJoinRows];
  float top[kJoinRows], sum[kJoinRows];
#pragma unroll
  for (int k = 0; k < kJoinRows; ++k) {
    v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    top[k] = -INFINITY;
    sum[k] = 0.0f;
  }
  for (int p0 = 0; p0 < parts; p0 += kJoinParts) {
    float4 o[kJoinRows][kJoinParts];
    float2 ml[kJoinRows][kJoinParts];
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k)
#pragma unroll
      for (int p = 0; p < kJoinParts; ++p) {
        const int r = r0 + k * kAtOnce;
        o[k][p] = make_float4(0.f, 0.f, 0.f, 0.f);
        ml[k][p] = make_float2(-INFINITY, 0.0f);
        if (p0 + p < parts && rt * kRows + r < a.rows) {
          const int set = (cta0 + p0 + p) * 2 + (p0 + p == 0 ? share.second : 0);
          const float* row = a.part + ((int64_t)set * kRows + r) * kPartRow<D>;
          o[k][p] = __ldcg(reinterpret_cast<const float4*>(row + d));
          ml[k][p] = __ldcg(reinterpret_cast<const float2*>(row + D));
        }
      }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k)
#pragma unroll
      for (int p = 0; p < kJoinParts; ++p) merge(v[k], top[k], sum[k], o[k][p], ml[k][p], 1.0f);
  }
#pragma unroll
  for (int k = 0; k < kJoinRows; ++k) {
    const int row = rt * kRows + r0 + k * kAtOnce;
    if (row >= a.rows) continue;
    const float r1 = sum[k] == 0.0f ? 0.0f : 1.0f / sum[k];
    const float4 y = make_float4(v[k].x * r1, v[k].y * r1, v[k].z * r1, v[k].w * r1);
    const int tok = (int)quotient((uint32_t)row, a.by_group);
    const int64_t dst = (((int64_t)b * a.new_tokens + tok) * a.q_heads + head * a.group + row -
                         tok * a.group) * D + d;
    if (a.dtype == RQ_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + dst) = y;
    } else if (a.dtype == RQ_F16) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + dst) =
          make_uint2(pack_half2(y.x, y.y), pack_half2(y.z, y.w));
    } else {
      const __nv_bfloat162 h0 = __floats2bfloat162_rn(y.x, y.y);
      const __nv_bfloat162 h1 = __floats2bfloat162_rn(y.z, y.w);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + dst) = make_uint2(
          *reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    }
  }
}

template <int D, bool I8, bool SPLIT>
rq_status launch_rows(const AttnArgs& a, unsigned grid, cudaStream_t st) {
  constexpr int bytes = Layout<D, SPLIT>::kTail + (int)sizeof(RowsTail);
  static_assert(bytes <= 232448, "shared memory of one CTA");
  static bool ready = false;
  if (!ready) {
    if (cudaFuncSetAttribute(attn_rows_kernel<D, I8, SPLIT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return RQ_ERR_CUDA;
    ready = true;
  }
  const rq_status s = launch_kernel(attn_rows_kernel<D, I8, SPLIT>, dim3(grid), dim3(kThreads),
                                    (size_t)bytes, st, a);
  if (s != RQ_OK || a.shares == nullptr) return s;
  return launch_kernel(join_rows_kernel<D>, dim3(grid * (kRows / kJoinBlock<D>)), dim3(256), 0, st, a);
}

// Partial rows, behind them, per CTA, the segment it begins for several, and
// the sums that left TMEM.
size_t part_bytes(size_t grid, int head_dim) {
  return sizeof(float) * 2 * grid * kRows * (head_dim + 4);
}
size_t share_bytes(size_t grid) { return (sizeof(SharedSegment) * grid + 15) & ~(size_t)15; }

}  // namespace

size_t attention_rows_scratch() {
  const size_t grid = (size_t)device_sm_count();
  return part_bytes(grid, 128) + share_bytes(grid) + sizeof(float) * grid * kRows * 128;
}

rq_status launch_attention_rows(AttnArgs a, int head_dim, bool i8, AttnScratch* scratch,
                                cudaStream_t st) {
  a.row_tiles = (a.rows + kRows - 1) / kRows;
  a.by_tiles = divisor((uint32_t)a.row_tiles);
  const int64_t items = (int64_t)a.batch * a.row_tiles;
  const int64_t segments = items * a.kv_heads;
  const int64_t grid = device_sm_count();
  if (segments > 0x7FFFFFFF) return RQ_ERR_SHAPE;
  a.direct = !Cutting::cuts(a, items);
  const bool split = a.dtype == RQ_F32;
  if (!a.direct || split) {
    const rq_status s = scratch->reserve(st);
    if (s != RQ_OK) return s;
    uint8_t* at = scratch->part;
    if (!a.direct) {
      a.part = reinterpret_cast<float*>(at);
      at += part_bytes((size_t)grid, head_dim);
      a.shares = reinterpret_cast<SharedSegment*>(at);
      at += share_bytes((size_t)grid);
    }
    a.flushed = reinterpret_cast<float4*>(at);
  }
  const unsigned g = (unsigned)grid;
  if (head_dim == 64) {
    if (i8)
      return split ? launch_rows<64, true, true>(a, g, st) : launch_rows<64, true, false>(a, g, st);
    return split ? launch_rows<64, false, true>(a, g, st) : launch_rows<64, false, false>(a, g, st);
  }
  if (i8)
    return split ? launch_rows<128, true, true>(a, g, st) : launch_rows<128, true, false>(a, g, st);
  return split ? launch_rows<128, false, true>(a, g, st) : launch_rows<128, false, false>(a, g, st);
}

}  // namespace rq
