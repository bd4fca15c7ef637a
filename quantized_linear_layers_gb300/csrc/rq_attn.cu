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
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdlib>

#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {

namespace {

// bit 0: a pipeline wait ran out; bit 1: an index outside its array
__device__ unsigned int g_attn_error = 0;

constexpr int kTile = 64;            // keys per pipeline stage
constexpr int kWarps = 4;            // consumer warps, 16 keys of a tile each
constexpr int kAttnThreads = (kWarps + 1) * 32;
constexpr int kMaxItems = 2048;

struct AttnArgs {
  const void* q;
  void* out;
  int64_t q_stride;
  const float *ks, *vs;
  const int32_t *table, *length;
  const unsigned long long* tree;
  int batch, new_tokens, q_heads, kv_heads, group, rows, row_tiles;
  int max_pages, lg_page, lg_box;
  int64_t pages;
  float scale_log2;
  int dtype;
  int direct;  // one CTA per segment, no splitting
  float* part;
  unsigned int* counter;
  uint64_t wait_limit_ns;
};

template <int D>
struct Geometry {
  static constexpr int kPanel = D < 128 ? D : 128;     // bytes of a row in one swizzled panel
  static constexpr int kPanels = D / kPanel;
  static constexpr int kBytes = kTile * D;              // codes of K (or V) in a stage
  static constexpr int kStage = 2 * kBytes + 2 * kTile * 4;
  static constexpr int kStages = D == 64 ? 8 : D == 128 ? 4 : 3;
  static constexpr int kStageAlign = (kStage + 1023) / 1024 * 1024;
};

// Shared memory after the stages.
template <int D, int ROWS>
struct Tail {
  static constexpr int kPitch = D + 4;
  float o[kWarps][ROWS][kPitch];
  float m[kWarps][ROWS], l[kWarps][ROWS];
  float c[ROWS];
  uint64_t full[8], empty[8];
  int flag;
  int total;  // tiles of one kv head over all items
  int item_start[kMaxItems + 1];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Four codes of a word as two f16 pairs: (byte 0, byte 2) and (byte 1, byte 3).
// E4M3 codes keep their bits at f16's places, sign | 4 exponent bits | 3
// mantissa bits, which is the code's value times 2^-8 (exponent bias 15 - 7;
// its subnormals are f16 subnormals).  8-bit integers, biased by 128, become
// the low mantissa bits of 1024 + b, from which 1152 is subtracted: exact.
template <bool I8>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& even, uint32_t& odd) {
  if constexpr (!I8) {
    even = ((w << 8) & 0x80008000u) | ((w << 7) & 0x3F803F80u);
    odd = (w & 0x80008000u) | ((w >> 1) & 0x3F803F80u);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t e = (u & 0x00FF00FFu) | 0x64006400u;
    const uint32_t o = ((u >> 8) & 0x00FF00FFu) | 0x64006400u;
    const uint32_t bias = 0x64806480u;  // 1152
    const __half2 eh = __hsub2(*reinterpret_cast<const __half2*>(&e),
                               *reinterpret_cast<const __half2*>(&bias));
    const __half2 oh = __hsub2(*reinterpret_cast<const __half2*>(&o),
                               *reinterpret_cast<const __half2*>(&bias));
    even = *reinterpret_cast<const uint32_t*>(&eh);
    odd = *reinterpret_cast<const uint32_t*>(&oh);
  }
}

// Byte offset of 16-byte chunk c of row r in a panel of rows of kPanel bytes,
// as the tensor map's swizzle lays it down.
template <int PANEL>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  if constexpr (PANEL == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int row,
                                         int plane, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(row), "r"(plane), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

// Places of a sequence that its new tokens may see, over all row tiles; 0 for
// an unused one.  *len: places every row sees.
__device__ __forceinline__ int64_t places(const AttnArgs& a, int b, int64_t* len) {
  const int64_t n = a.length[b];
  if (n < 0) {
    *len = 0;
    return 0;
  }
  const int64_t most = (int64_t)a.max_pages << a.lg_page;
  int64_t kv = n + a.new_tokens;
  if (kv > most) {
    if (threadIdx.x == 0) atomicOr(&g_attn_error, 2u);
    kv = most;
  }
  *len = n < kv ? n : kv;
  return kv;
}

// Last place + 1 that row tile rt may see.
template <int ROWS>
__device__ __forceinline__ int64_t tile_places(const AttnArgs& a, int rt, int64_t len,
                                               int64_t kv) {
  if (a.tree != nullptr || kv == 0) return kv;
  int last = (rt + 1) * ROWS;
  last = (last < a.rows ? last : a.rows) - 1;
  const int64_t end = len + last / a.group + 1;
  return end < kv ? end : kv;
}

// ------------------------------------------------------------ the kernel --
//
// Work is the sequence of segments (sequence, row tile, kv head), each a run
// of 64-key tiles, laid end to end; CTA c of C takes an equal run of it, so
// that ragged lengths load the SMs evenly and a single long sequence spreads
// over all of them.  A segment cut between CTAs is joined by the last of them
// to finish, in CTA order, from partial (max, sum, output) rows in scratch.
//
// Within a CTA a producer thread keeps a ring of tiles in flight by TMA, and
// four warps each take 16 keys of every tile with a softmax of their own (no
// exchange inside the loop); their results are joined when the segment ends.
// A warp's tile of 16 rows holds ROWS = 16 rows of 16-bit activations, or 8
// rows of f32 as high parts (rows 0-7) and low parts (8-15).
template <int D, bool I8, bool F32>
__global__ void __launch_bounds__(kAttnThreads)
attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
            const AttnArgs a) {
  constexpr int ROWS = F32 ? 8 : 16;
  using G = Geometry<D>;
  using TailT = Tail<D, ROWS>;
  constexpr int S = G::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  TailT& tail = *reinterpret_cast<TailT*>(smem + S * G::kStageAlign);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem_base = smem_u32(smem);

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&tail.full[i]), 1);
      mbar_init(smem_u32(&tail.empty[i]), kWarps);
    }
    mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();

  const int items = a.batch * a.row_tiles;
  int64_t u0, u1;  // this CTA's run of tiles
  int64_t units = 0;
  int ctas = (int)gridDim.x;
  if (!a.direct) {
    // tiles before each item (sequence, row tile), for one kv head
    int carry = 0;
    for (int base = 0; base < items; base += kAttnThreads) {
      const int i = base + tid;
      int n = 0;
      if (i < items) {
        int64_t len;
        const int64_t kv = places(a, i / a.row_tiles, &len);
        n = (int)((tile_places<ROWS>(a, i % a.row_tiles, len, kv) + kTile - 1) / kTile);
        if (n < 1) n = 1;
      }
      int scan = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += x;
      }
      __syncthreads();
      if (lane == 31) reinterpret_cast<int*>(tail.o)[warp] = scan;
      __syncthreads();
      int before = carry;
      for (int w = 0; w <= kWarps; ++w) {
        const int x = reinterpret_cast<int*>(tail.o)[w];
        if (w < warp) before += x;
        carry += x;
      }
      if (i < items) tail.item_start[i] = before + scan - n;
    }
    if (tid == 0) tail.item_start[items] = carry;
    units = (int64_t)carry * a.kv_heads;
    // no CTA below two tiles: joining costs more than it saves there
    if (ctas > (units + 1) / 2) ctas = (int)((units + 1) / 2);
    u0 = (int)blockIdx.x < ctas ? units * blockIdx.x / ctas : 0;
    u1 = (int)blockIdx.x < ctas ? units * (blockIdx.x + 1) / ctas : 0;
  } else {
    u0 = 0;
    u1 = 1;
  }
  __syncthreads();
  if (u0 >= u1) return;

  // the first segment: item, head and first tile
  int item, head;
  int64_t tile0;
  if (a.direct) {
    item = (int)(blockIdx.x % (unsigned)items);
    head = (int)(blockIdx.x / (unsigned)items);
    tile0 = 0;
  } else {
    int lo = 0, hi = items - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)tail.item_start[mid] * a.kv_heads <= u0)
        lo = mid;
      else
        hi = mid - 1;
    }
    item = lo;
    const int n = tail.item_start[item + 1] - tail.item_start[item];
    const int64_t rest = u0 - (int64_t)tail.item_start[item] * a.kv_heads;
    head = (int)(rest / n);
    tile0 = rest - (int64_t)head * n;
  }

  int stage = 0;
  uint32_t phase = 0;
  int64_t at = u0;  // position in the run
  bool ok = true;
  int seg = 0;

  while (at < u1) {
    const int b = item / a.row_tiles, rt = item % a.row_tiles;
    int64_t len;
    const int64_t kv_all = places(a, b, &len);
    const int64_t kv = tile_places<ROWS>(a, rt, len, kv_all);
    int64_t n = (kv + kTile - 1) / kTile;
    if (n < 1) n = 1;
    int64_t tile1 = n;
    if (a.direct)
      at = u1;
    else {
      if (tile0 + (u1 - at) < tile1) tile1 = tile0 + (u1 - at);
      at += tile1 - tile0;
    }

    if (warp == kWarps) {
      // ---------------------------------------------------- producer ----
      if (lane == 0 && ok) {
        const int box = 1 << a.lg_box;
        for (int64_t t = tile0; t < tile1; ++t) {
          ok = mbar_wait(smem_u32(&tail.empty[stage]), phase ^ 1u, a.wait_limit_ns, &g_attn_error);
          if (!ok) break;
          const int64_t p0 = t * kTile;
          const uint32_t bar = smem_u32(&tail.full[stage]);
          const uint32_t kd = smem_base + stage * G::kStageAlign;
          const uint32_t vd = kd + G::kBytes, sd = vd + G::kBytes;
          int64_t left = kv - p0;
          if (left > kTile) left = kTile;
          const int boxes = left > 0 ? (int)((left + box - 1) >> a.lg_box) : 0;
          mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * (2 * D + 8)));
          for (int i = 0; i < boxes; ++i) {
            const int64_t p = p0 + i * box;
            int64_t page = a.table[(int64_t)b * a.max_pages + (p >> a.lg_page)];
            if (page < 0 || page >= a.pages) {
              atomicOr(&g_attn_error, 2u);
              page = 0;
            }
            const int off = (int)(p & ((1 << a.lg_page) - 1));
            const int plane = (int)(page * a.kv_heads + head);
            const int64_t row = ((int64_t)plane << a.lg_page) + off;
#pragma unroll
            for (int h = 0; h < G::kPanels; ++h) {
              const uint32_t to = h * kTile * G::kPanel + i * box * G::kPanel;
              tma_rows(kd + to, &map_k, h * G::kPanel, off, plane, bar);
              tma_rows(vd + to, &map_v, h * G::kPanel, off, plane, bar);
            }
            bulk_g2s(sd + i * box * 4, a.ks + row, (uint32_t)(box * 4), bar);
            bulk_g2s(sd + kTile * 4 + i * box * 4, a.vs + row, (uint32_t)(box * 4), bar);
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else {
      // --------------------------------------------------- consumers ----
      const int g = lane >> 2, t4 = lane & 3;
      // rows of this thread's accumulators: g (and g + 8 when 16 rows)
      constexpr int NR = F32 ? 1 : 2;
      int tok[NR];
      unsigned long long bits[NR];
      float c[NR];  // 2^x per unit of the raw score x = acc * ks
      uint32_t qa[D / 16][4];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int row = rt * ROWS + g + 8 * r;
        const bool live = row < a.rows;
        tok[r] = live ? row / a.group : 0;
        bits[r] = 0;
        if (live && a.tree != nullptr) bits[r] = a.tree[(int64_t)b * a.new_tokens + tok[r]];
        const int64_t off = ((int64_t)b * a.new_tokens + tok[r]) * a.q_stride +
                            (int64_t)(head * a.group + (live ? row % a.group : 0)) * D;
        float x[D / 16][4];
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int64_t e = off + 16 * i + 4 * t4;
          if (F32) {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + e);
            x[i][0] = v.x;
            x[i][1] = v.y;
            x[i][2] = v.z;
            x[i][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + e);
            if (a.dtype == RQ_F16) {
              const float2 f0 = half_pair(v.x), f1 = half_pair(v.y);
              x[i][0] = f0.x;
              x[i][1] = f0.y;
              x[i][2] = f1.x;
              x[i][3] = f1.y;
            } else {
              x[i][0] = __uint_as_float(v.x << 16);
              x[i][1] = __uint_as_float(v.x & 0xFFFF0000u);
              x[i][2] = __uint_as_float(v.y << 16);
              x[i][3] = __uint_as_float(v.y & 0xFFFF0000u);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (!live) x[i][k] = 0.0f;
            top = fmaxf(top, fabsf(x[i][k]));
          }
        }
        // the row times a power of two, so that its f16 parts lie well inside
        // f16's range: largest entry in [2^13, 2^14)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        int e = 0;
        if (top > 0.0f && top <= 3.4e38f) {
          e = 13 - (int)((__float_as_uint(top) >> 23) & 0xFFu) + 127;
          e = e < -126 ? -126 : e > 100 ? 100 : e;
        }
        const float up = __uint_as_float((uint32_t)(e + 127) << 23);
        c[r] = fmaxf(a.scale_log2 / up * (I8 ? 1.0f : 256.0f), 0x1p-126f);
        if (!(top <= 3.4e38f)) c[r] = NAN;  // an infinity in q
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const float x0 = x[i][0] * up, x1 = x[i][1] * up, x2 = x[i][2] * up, x3 = x[i][3] * up;
          if (F32) {
            qa[i][0] = split_half2(x0, x2, qa[i][1]);
            qa[i][2] = split_half2(x1, x3, qa[i][3]);
          } else {
            qa[i][r] = pack_half2(x0, x2);
            qa[i][2 + r] = pack_half2(x1, x3);
          }
        }
      }

      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;
      float m[NR], l[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.0f;
      }
      float vref = 0x1p-112f;  // power of two at or above every vs so far
      const int kr = 16 * warp;  // this warp's keys in the tile

      for (int64_t t = tile0; t < tile1; ++t) {
        if (ok) ok = mbar_wait(smem_u32(&tail.full[stage]), phase, a.wait_limit_ns, &g_attn_error);
        ok = __all_sync(0xFFFFFFFFu, ok);
        const int64_t first = t * kTile + kr;  // place of this warp's first key
        if (ok && first < kv) {
          const uint32_t kd = smem_base + stage * G::kStageAlign;
          const uint32_t vd = kd + G::kBytes;
          const float* sc =
              reinterpret_cast<const float*>(smem + stage * G::kStageAlign + 2 * G::kBytes) + kr;
          // ---- scores of 16 keys
          float s[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][k] = 0.0f;
          // matrix lane / 8: keys 0-7 or 8-15, 16 dims i or i + 1
          const int krow = kr + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
          for (int i = 0; i < D / 16; i += 2) {
            const int chunk = i + (lane >> 4);
            uint32_t w[4];
            ldsm4(w, kd + (chunk / (G::kPanel / 16)) * (kTile * G::kPanel) +
                         swizzled<G::kPanel>(krow, chunk % (G::kPanel / 16)));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t b0, b1;
              codes_to_half<I8>(w[k], b0, b1);
              mma(s[k & 1], qa[i + (k >> 1)], b0, b1);
            }
          }
          // ---- their scales, and what is seen
          float2 ks[2], vs[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ks[i] = *reinterpret_cast<const float2*>(sc + 8 * i + 2 * t4);
            vs[i] = *reinterpret_cast<const float2*>(sc + kTile + 8 * i + 2 * t4);
          }
          unsigned int seen[NR];
          const bool all = first + 16 <= len;
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            seen[r] = 0xFu;
            if (!all) {
              seen[r] = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int64_t place = first + 8 * (k >> 1) + 2 * t4 + (k & 1);
                const int64_t draft = place - len;
                bool see = place < kv;
                if (draft >= 0)
                  see = see && (a.tree == nullptr ? draft <= tok[r]
                                                  : (draft < 64 && ((bits[r] >> draft) & 1ull)));
                if (see) seen[r] |= 1u << k;
              }
            }
          }
          float x[NR][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float kk = (k & 1) ? ks[k >> 1].y : ks[k >> 1].x;
            if (F32) {
              x[0][k] = (s[k >> 1][k & 1] + s[k >> 1][2 + (k & 1)]) * kk;
            } else {
#pragma unroll
              for (int r = 0; r < NR; ++r) x[r][k] = s[k >> 1][2 * r + (k & 1)] * kk;
            }
          }
          if (!all)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!((seen[r] >> k) & 1u)) x[r][k] = -INFINITY;
          // ---- running maximum; value scales relative to their own
          float vt = 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float vv = (k & 1) ? vs[k >> 1].y : vs[k >> 1].x;
            const int64_t place = first + 8 * (k >> 1) + 2 * t4 + (k & 1);
            if (place < kv && vv <= 1e37f) vt = fmaxf(vt, vv);  // NaN, Inf left out
          }
          vt = fmaxf(vt, __shfl_xor_sync(0xFFFFFFFFu, vt, 1));
          vt = fmaxf(vt, __shfl_xor_sync(0xFFFFFFFFu, vt, 2));
          float mn[NR];
          bool moved = vt > vref;
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            mn[r] = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
            mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xFFFFFFFFu, mn[r], 1));
            mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xFFFFFFFFu, mn[r], 2));
            mn[r] = fmaxf(mn[r], m[r]);
            moved = moved || mn[r] > m[r];
          }
          if (__any_sync(0xFFFFFFFFu, moved)) {
            float vnew = vref;
            if (vt > vref)  // four times the next power of two: rarely passed again
              vnew = __uint_as_float(((__float_as_uint(vt) & 0x7F800000u) + (2u << 23)));
            const float vdown = vref / vnew;
            vref = vnew;
            float f[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const float al = m[r] == -INFINITY ? 0.0f : ex2((m[r] - mn[r]) * c[r]);
              l[r] *= al;
              m[r] = mn[r];
              f[r] = al * vdown;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][0] *= f[0];
              o[i][1] *= f[0];
              o[i][2] *= f[NR - 1];
              o[i][3] *= f[NR - 1];
            }
          }
          const float inv = __uint_as_float(((254u + 14u) << 23) - (__float_as_uint(vref)));  // 2^14 / vref
          uint32_t pa[4];
          float w[NR][4];
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float mr = m[r] == -INFINITY ? 0.0f : m[r];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float p = ex2((x[r][k] - mr) * c[r]);
              l[r] += p;
              const float vv = (k & 1) ? vs[k >> 1].y : vs[k >> 1].x;
              w[r][k] = p * (vv * inv);
              if (!all && !((seen[r] >> k) & 1u)) w[r][k] = 0.0f;
            }
          }
          if (F32) {
            pa[0] = split_half2(w[0][0], w[0][1], pa[1]);
            pa[2] = split_half2(w[0][2], w[0][3], pa[3]);
          } else {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              pa[r] = pack_half2(w[r][0], w[r][1]);
              pa[2 + r] = pack_half2(w[r][2], w[r][3]);
            }
          }
          // ---- output
          const int vrow = kr + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
          for (int i = 0; i < D / 16; i += 2) {
            const int chunk = i + (lane >> 4);
            uint32_t v[4];
            ldsm4t(v, vd + (chunk / (G::kPanel / 16)) * (kTile * G::kPanel) +
                          swizzled<G::kPanel>(vrow, chunk % (G::kPanel / 16)));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t e0, e1, o0, o1;
              codes_to_half<I8>(v[2 * k], e0, o0);
              codes_to_half<I8>(v[2 * k + 1], e1, o1);
              mma(o[2 * (i + k)], pa, e0, e1);
              mma(o[2 * (i + k) + 1], pa, o0, o1);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tail.empty[stage]));
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }

      // ---- join the four warps
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
        if (t4 == 0) {
          tail.m[warp][g + 8 * r] = m[r];
          tail.l[warp][g + 8 * r] = l[r];
          tail.c[g + 8 * r] = c[r];  // the same from every warp
        }
      }
      const float back = vref * (I8 ? 0x1p-14f : 0x1p-6f);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        // dims 16 i + 4 t4 ..: even tile's two columns and odd tile's two
        if (F32) {
          float4 v;
          v.x = (o[2 * i][0] + o[2 * i][2]) * back;
          v.y = (o[2 * i + 1][0] + o[2 * i + 1][2]) * back;
          v.z = (o[2 * i][1] + o[2 * i][3]) * back;
          v.w = (o[2 * i + 1][1] + o[2 * i + 1][3]) * back;
          *reinterpret_cast<float4*>(&tail.o[warp][g][16 * i + 4 * t4]) = v;
        } else {
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float4 v;
            v.x = o[2 * i][2 * r] * back;
            v.y = o[2 * i + 1][2 * r] * back;
            v.z = o[2 * i][2 * r + 1] * back;
            v.w = o[2 * i + 1][2 * r + 1] * back;
            *reinterpret_cast<float4*>(&tail.o[warp][g + 8 * r][16 * i + 4 * t4]) = v;
          }
        }
      }
      consumer_sync();

      // which CTAs share this segment
      int64_t parts = 1, cta0 = 0, s0 = 0;
      if (!a.direct) {
        s0 = (int64_t)tail.item_start[item] * a.kv_heads + head * n;
        cta0 = ((s0 + 1) * ctas - 1) / units;
        parts = ((s0 + n) * ctas - 1) / units - cta0 + 1;
      }
      bool last = true;
      constexpr int kVec = D / 4;
      constexpr int kPartRow = D + 4;  // output, then max and sum
      if (parts > 1) {
        float* part = a.part + ((int64_t)blockIdx.x * 2 + (seg == 0 ? 0 : 1)) * ROWS * kPartRow;
        for (int i = tid; i < ROWS * kVec; i += kWarps * 32) {
          const int r = i / kVec, d = (i % kVec) * 4;
          if (rt * ROWS + r >= a.rows) continue;
          float mx = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, tail.m[w][r]);
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          float sum = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float mw = tail.m[w][r];
            const float f = mw == -INFINITY ? 0.0f : ex2((mw - mx) * tail.c[r]);
            const float4 ow = *reinterpret_cast<const float4*>(&tail.o[w][r][d]);
            v.x = fmaf(ow.x, f, v.x);
            v.y = fmaf(ow.y, f, v.y);
            v.z = fmaf(ow.z, f, v.z);
            v.w = fmaf(ow.w, f, v.w);
            sum = fmaf(tail.l[w][r], f, sum);
          }
          __stcg(reinterpret_cast<float4*>(part + r * kPartRow + d), v);
          if (d == 0) __stcg(reinterpret_cast<float2*>(part + r * kPartRow + D), make_float2(mx, sum));
        }
        __threadfence();
        consumer_sync();
        if (tid == 0) {
          unsigned int* ctr = a.counter + ((int64_t)item * a.kv_heads + head);
          const unsigned int old = atomicAdd(ctr, 1u);
          tail.flag = old == (unsigned int)(parts - 1);
          if (tail.flag) *ctr = 0u;
        }
        consumer_sync();
        last = tail.flag != 0;
        __threadfence();
      }
      if (last) {
        for (int i = tid; i < ROWS * kVec; i += kWarps * 32) {
          const int r = i / kVec, d = (i % kVec) * 4;
          const int row = rt * ROWS + r;
          if (row >= a.rows) continue;
          const float cr = tail.c[r];
          float mx = -INFINITY, sum = 0.0f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          const int count = parts > 1 ? (int)parts : kWarps;
          for (int p = 0; p < count; ++p) {
            float4 ov;
            float2 ml;
            if (parts > 1) {
              const int64_t cta = cta0 + p;
              const int slot = p == 0 && units * cta / ctas < s0 ? 1 : 0;
              const float* part = a.part + (cta * 2 + slot) * ROWS * kPartRow + r * kPartRow;
              ov = __ldcg(reinterpret_cast<const float4*>(part + d));
              ml = __ldcg(reinterpret_cast<const float2*>(part + D));
            } else {
              ov = *reinterpret_cast<const float4*>(&tail.o[p][r][d]);
              ml = make_float2(tail.m[p][r], tail.l[p][r]);
            }
            const float mn = fmaxf(mx, ml.x);
            if (mn == -INFINITY) {
              sum += ml.y;  // 0, or the NaN of a row whose scores all are
              continue;
            }
            const float f0 = ex2((mx - mn) * cr), f1 = ex2((ml.x - mn) * cr);
            v.x = v.x * f0 + ov.x * f1;
            v.y = v.y * f0 + ov.y * f1;
            v.z = v.z * f0 + ov.z * f1;
            v.w = v.w * f0 + ov.w * f1;
            sum = sum * f0 + ml.y * f1;
            mx = mn;
          }
          // nothing seen: zeros (a NaN sum stays a NaN)
          const float r1 = sum == 0.0f ? 0.0f : 1.0f / sum;
          v.x *= r1;
          v.y *= r1;
          v.z *= r1;
          v.w *= r1;
          const int64_t dst = (((int64_t)b * a.new_tokens + row / a.group) * a.q_heads +
                               head * a.group + row % a.group) * D + d;
          if (F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + dst) = v;
          } else if (a.dtype == RQ_F16) {
            const uint2 h = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + dst) = h;
          } else {
            const __nv_bfloat162 h0 = __floats2bfloat162_rn(v.x, v.y);
            const __nv_bfloat162 h1 = __floats2bfloat162_rn(v.z, v.w);
            const uint2 h = make_uint2(*reinterpret_cast<const uint32_t*>(&h0),
                                       *reinterpret_cast<const uint32_t*>(&h1));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + dst) = h;
          }
        }
      }
      consumer_sync();  // the joined rows are read before the next segment's are written
    }

    ++seg;
    tile0 = 0;
    if (++head == a.kv_heads) {
      head = 0;
      ++item;
    }
  }

  // a producer that gave up: its last copies are waited for before it ends
  if (warp == kWarps && lane == 0 && !ok) {
    for (int i = 0; i < S; ++i) {
      stage = stage == 0 ? S - 1 : stage - 1;
      if (stage == S - 1) phase ^= 1u;
      mbar_wait(smem_u32(&tail.full[stage]), phase, a.wait_limit_ns, &g_attn_error);
    }
  }
}

// ------------------------------------------------------------- host side --

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static bool tried = false;
  if (!tried) {
    tried = true;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// 3-D map over codes [pages * kv_heads][page_size][head_dim], box = one panel
// of `box` rows; coordinates stay below 2^31 however long the cache is.
bool codes_map(CUtensorMap* map, const void* base, const rq_kv_cache& c, int box) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size,
                              (cuuint64_t)(c.pages * c.kv_heads)};
  const cuuint64_t strides[2] = {(cuuint64_t)c.head_dim,
                                 (cuuint64_t)c.head_dim * (cuuint64_t)c.page_size};
  const cuuint32_t panel = c.head_dim < 128 ? 64 : 128;
  const cuuint32_t boxes[3] = {panel, (cuuint32_t)box, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, boxes,
         estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         panel == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

int lg(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

struct Plan {
  int rows, ctas;
  bool direct;
};

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const AttnArgs);

template <int D, bool I8, bool F32>
rq_status kernel_of(Kernel* k, int* smem, int* per_sm) {
  constexpr int ROWS = F32 ? 8 : 16;
  constexpr int bytes =
      Geometry<D>::kStages * Geometry<D>::kStageAlign + (int)sizeof(Tail<D, ROWS>);
  static int resident = 0;
  if (resident == 0) {
    if (cudaFuncSetAttribute(attn_kernel<D, I8, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes) != cudaSuccess)
      return RQ_ERR_CUDA;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_kernel<D, I8, F32>, kAttnThreads,
                                                      bytes) != cudaSuccess ||
        n < 1)
      return RQ_ERR_CUDA;
    resident = n;
  }
  *k = attn_kernel<D, I8, F32>;
  *smem = bytes;
  *per_sm = resident;
  return RQ_OK;
}

template <int D>
rq_status kernel_for(bool i8, bool f32, Kernel* k, int* smem, int* per_sm) {
  if (i8) return f32 ? kernel_of<D, true, true>(k, smem, per_sm)
                     : kernel_of<D, true, false>(k, smem, per_sm);
  return f32 ? kernel_of<D, false, true>(k, smem, per_sm)
             : kernel_of<D, false, false>(k, smem, per_sm);
}

}  // namespace

rq_status launch_cache_attention(const AttnCall& call, AttnScratch* scratch, cudaStream_t st) {
  const rq_kv_cache& c = *call.cache;
  const bool f32 = call.dtype == RQ_F32, i8 = c.format == RQ_KV_I8;
  Kernel kernel = nullptr;
  int smem = 0, per_sm = 0;
  rq_status s = c.head_dim == 64    ? kernel_for<64>(i8, f32, &kernel, &smem, &per_sm)
                : c.head_dim == 128 ? kernel_for<128>(i8, f32, &kernel, &smem, &per_sm)
                                    : kernel_for<256>(i8, f32, &kernel, &smem, &per_sm);
  if (s != RQ_OK) return s;

  AttnArgs a = {};
  a.q = call.q;
  a.out = call.out;
  a.q_stride = call.q_stride;
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
  const int tile_rows = f32 ? 8 : 16;
  a.row_tiles = (a.rows + tile_rows - 1) / tile_rows;
  a.max_pages = call.max_pages;
  a.lg_page = lg(c.page_size);
  a.lg_box = a.lg_page < 6 ? a.lg_page : 6;
  a.pages = c.pages;
  a.scale_log2 = (float)((double)call.scale * 1.4426950408889634);
  a.dtype = call.dtype;
  a.wait_limit_ns = kWaitLimitNs;

  CUtensorMap mk, mv;
  if (!codes_map(&mk, c.k, c, 1 << a.lg_box) || !codes_map(&mv, c.v, c, 1 << a.lg_box))
    return RQ_ERR_ARCH;

  const int64_t items = (int64_t)call.batch * a.row_tiles;
  const int64_t segments = items * c.kv_heads;
  int64_t grid = (int64_t)device_sm_count() * per_sm;
  a.direct = items > kMaxItems;
  if (a.direct) {
    grid = segments;
    if (grid > 0x7FFFFFFF) return RQ_ERR_SHAPE;
  } else {
    const size_t part = sizeof(float) * 2 * (size_t)grid * tile_rows * (c.head_dim + 4);
    s = scratch->reserve(part, (size_t)segments, st);
    if (s != RQ_OK) return s;
    a.part = scratch->part;
    a.counter = scratch->counter;
  }
  return launch_kernel(kernel, dim3((unsigned)grid), dim3(kAttnThreads), (size_t)smem, st, mk, mv,
                       a);
}

rq_status AttnScratch::reserve(size_t part_bytes, size_t counters, cudaStream_t st) {
  if (part_bytes > part_cap) {
    if (part) cudaFree(part);
    part = nullptr;
    part_cap = 0;
    void* p = nullptr;
    if (cudaMalloc(&p, part_bytes) != cudaSuccess) {
      cudaGetLastError();
      return RQ_ERR_ALLOC;
    }
    part = static_cast<float*>(p);
    part_cap = part_bytes;
  }
  if (counters > counter_cap) {
    if (counter) cudaFree(counter);
    counter = nullptr;
    counter_cap = 0;
    void* p = nullptr;
    if (cudaMalloc(&p, counters * sizeof(unsigned int)) != cudaSuccess) {
      cudaGetLastError();
      return RQ_ERR_ALLOC;
    }
    // every launch leaves its counters at zero again
    if (cudaMemsetAsync(p, 0, counters * sizeof(unsigned int), st) != cudaSuccess) {
      cudaFree(p);
      return RQ_ERR_CUDA;
    }
    counter = static_cast<unsigned int*>(p);
    counter_cap = counters;
  }
  return RQ_OK;
}

void AttnScratch::release() {
  if (part) cudaFree(part);
  if (counter) cudaFree(counter);
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
