// rq_kv.cu -- per-head norm and rotation of q and k, and the quantized K/V
// cache's write and read back (sm_103a).
//
// Per head row x of D values (one token, one head):
//   y = x * rsqrt(mean(x^2) + eps) * weight            (rows with a weight)
//   z = y turned by the token's position                (q and k)
//   q, k out: z rounded to the activations' type, or
//   k, v into the cache: A = max |finite z|, A' = max(A, 2^-100),
//     scale = A' / top, code = rn(z * (top * (1 / A'))).
#include <cuda_bf16.h>

#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {

namespace {

__device__ unsigned int g_kv_error = 0;  // bit 1: an index outside its array

constexpr int kRowThreads = 256;
constexpr float kLeastMax = 0x1p-100f;

struct RowsArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  void *q_out, *k_out;
  const float *q_weight, *k_weight, *cos_table, *sin_table;
  const int32_t* position;
  int64_t positions;
  const int64_t* slot;
  uint8_t *kc, *vc;
  float *ks, *vs;
  int64_t slots;
  int lg_page, hkv, format;
  int hq, hk, hv;  // rows of each kind per token (0: that side is left out)
  int tq, tk;      // tasks of q and of k rows per token
  Divisor tasks;   // tasks per token; a warp takes one
  int tokens, rotary, interleaved;
  float eps;
};

// E consecutive values of an activation row as floats, and back.
template <typename T, int E>
__device__ __forceinline__ void load_row(const T* p, float (&x)[E]) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (E == 2) {
      const float2 a = *reinterpret_cast<const float2*>(p);
      x[0] = a.x;
      x[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(p + i);
        x[i] = a.x;
        x[i + 1] = a.y;
        x[i + 2] = a.z;
        x[i + 3] = a.w;
      }
    }
  } else {
    alignas(16) T t[E];
    if constexpr (E == 2)
      *reinterpret_cast<uint32_t*>(t) = *reinterpret_cast<const uint32_t*>(p);
    else if constexpr (E == 4)
      *reinterpret_cast<uint2*>(t) = *reinterpret_cast<const uint2*>(p);
    else
      *reinterpret_cast<uint4*>(t) = *reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = static_cast<float>(t[i]);
  }
}

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
  return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

template <typename T, int E>
__device__ __forceinline__ void store_row(T* p, const float (&x)[E]) {
  alignas(16) T t[E];
#pragma unroll
  for (int i = 0; i < E; ++i) t[i] = from_float<T>(x[i]);
  constexpr int kBytes = E * (int)sizeof(T);
  if constexpr (kBytes == 4)
    *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(t);
  else if constexpr (kBytes == 8)
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(t);
  else
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(t)[i];
}

// N floats of a table row.
template <int N>
__device__ __forceinline__ void load_table(const float* p, float (&x)[N]) {
  if constexpr (N == 1) {
    x[0] = __ldg(p);
  } else if constexpr (N == 2) {
    const float2 a = __ldg(reinterpret_cast<const float2*>(p));
    x[0] = a.x;
    x[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
      x[i] = a.x;
      x[i + 1] = a.y;
      x[i + 2] = a.z;
      x[i + 3] = a.w;
    }
  }
}

// One code byte; what is not finite takes its sign's largest code.
__device__ __forceinline__ uint32_t encode_e4m3(float x, float s) {
  if (non_finite(x)) return saturated_code(x);
  return cvt_e4m3x2(0.0f, __fmul_rn(x, s)) & 0xFFu;
}

__device__ __forceinline__ uint32_t encode_i8(float x, float s) {
  const float y = non_finite(x) ? copysignf(127.0f, x) : __fmul_rn(x, s);
  return (uint32_t)__float2int_rn(fminf(fmaxf(y, -127.0f), 127.0f)) & 0xFFu;
}

// Two code bytes of finite values.  Integers by the addition of 1.5 2^23,
// which rounds to the nearest even one and leaves it in the low bits; the
// product with top / max is at most top but for two roundings, so that no
// limit is needed before rounding.
__device__ __forceinline__ uint32_t encode2(bool e4m3, float lo, float hi, float s) {
  const float a = __fmul_rn(lo, s), b = __fmul_rn(hi, s);
  if (e4m3) return cvt_e4m3x2(b, a);
  return __byte_perm(__float_as_uint(a + 12582912.0f), __float_as_uint(b + 12582912.0f), 0x0040) &
         0xFFFFu;
}

// 1 / sqrt(x): the approximate instruction and one Newton step.
__device__ __forceinline__ float inv_sqrt(float x) {
  const float y = rsqrtf(x);
  const float h = 0.5f * x * y;
  const float r = fmaf(-h, y, 0.5f);
  // (an infinite or zero x leaves r NaN: the instruction's value stands)
  return r == r ? fmaf(y, r, y) : y;
}

// Sums of R rows over the warp: a lane ends with row `R - 1 bits of its lane
// number's top` -- for R = 4, row 2 b4 + b3 of lane bits 4 and 3 -- since each
// of the first steps halves the rows that it holds instead of adding all of
// them five times.
template <int R>
__device__ __forceinline__ float rows_sum(const float (&v)[R], int lane) {
  if constexpr (R == 1) {
    return warp_sum(v[0]);
  } else {
    static_assert(R == 4, "1 or 4 rows a warp");
    const bool b4 = (lane & 16) != 0, b3 = (lane & 8) != 0;
    const float k0 = b4 ? v[2] : v[0], g0 = b4 ? v[0] : v[2];
    const float k1 = b4 ? v[3] : v[1], g1 = b4 ? v[1] : v[3];
    const float a0 = k0 + __shfl_xor_sync(0xFFFFFFFFu, g0, 16);
    const float a1 = k1 + __shfl_xor_sync(0xFFFFFFFFu, g1, 16);
    float b = (b3 ? a1 : a0) + __shfl_xor_sync(0xFFFFFFFFu, b3 ? a0 : a1, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    return b;
  }
}

// A warp takes RPW rows of one kind (q, k or v) and one token: lane l holds
// values [l E, l E + E) of each, E = D / 32.  The rotation's partner values
// are in the lane rotary / 2 / E away (host: rotary % 16 == 0, so that
// distance is a whole number); sums are shuffles, maxima one warp reduction
// of the magnitudes' bits: a row is read once and nothing passes through
// shared memory.  Bound by memory from a few hundred tokens on (4096 tokens
// of 28 + 4 + 4 heads of 128 in f32: 26 us, 5.4 TB/s), by launch and load
// latency below.
template <typename T, int E, int RPW>
__global__ void __launch_bounds__(kRowThreads)
rows_kernel(const RowsArgs a) {
  constexpr int D = 32 * E;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const uint32_t task = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const uint32_t t = quotient(task, a.tasks);
  if (t >= (uint32_t)a.tokens) return;
  const int j = (int)(task - t * a.tasks.d);
  const int d0 = lane * E;

  // the task's rows
  const bool is_q = j < a.tq, is_k = !is_q && j < a.tq + a.tk;
  const int h0 = (is_q ? j : is_k ? j - a.tq : j - a.tq - a.tk) * RPW;
  const int n = min(RPW, (is_q ? a.hq : is_k ? a.hk : a.hv) - h0);
  const T* src = static_cast<const T*>(is_q ? a.q : is_k ? a.k : a.v) +
                 (int64_t)t * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) +
                 (int64_t)h0 * D + d0;
  float x[RPW][E];
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[r][i] = 0.0f;
    if (r < n) load_row<T, E>(src + r * D, x[r]);
  }
  const bool stored = a.slot != nullptr && !is_q;
  int64_t slot = -1;
  if (stored) slot = a.slot[t];

  // the token's turn: cos and sin of this lane's pairs
  const int half = a.rotary >> 1;
  bool turn = a.rotary > 0 && (is_q || is_k);
  float c[E], s[E];
  if (turn) {
    const int64_t at = a.position[t];
    if (at < 0 || at >= a.positions) {
      if (lane == 0) atomicOr(&g_kv_error, 2u);
      turn = false;
    } else if (d0 < a.rotary) {
      if (a.interleaved) {
        float c2[E / 2], s2[E / 2];
        load_table<E / 2>(a.cos_table + at * half + d0 / 2, c2);
        load_table<E / 2>(a.sin_table + at * half + d0 / 2, s2);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          c[i] = c2[i / 2];
          s[i] = (i & 1) ? s2[i / 2] : -s2[i / 2];
        }
      } else {
        const bool second = d0 >= half;
        load_table<E>(a.cos_table + at * half + (second ? d0 - half : d0), c);
        load_table<E>(a.sin_table + at * half + (second ? d0 - half : d0), s);
#pragma unroll
        for (int i = 0; i < E; ++i) s[i] = second ? s[i] : -s[i];
      }
    }
  }

  const float* weight = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
  if (weight != nullptr) {
    float w[E], sq[RPW];
    load_table<E>(weight + d0, w);
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      sq[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) sq[r] = fmaf(x[r][i], x[r][i], sq[r]);
    }
    const float own = inv_sqrt(rows_sum<RPW>(sq, lane) * (1.0f / D) + a.eps);
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      const float inv = RPW == 1 ? own : __shfl_sync(0xFFFFFFFFu, own, (r >> 1) * 16 + (r & 1) * 8);
#pragma unroll
      for (int i = 0; i < E; ++i) x[r][i] = x[r][i] * inv * w[i];
    }
  }
  if (turn) {
    const int hop = half / E;
    const int partner = (d0 < half ? lane + hop : lane - hop) & 31;
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      float o[E];
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = x[r][i ^ 1];
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = __shfl_sync(0xFFFFFFFFu, x[r][i], partner);
      }
      if (d0 < a.rotary) {
#pragma unroll
        for (int i = 0; i < E; ++i) x[r][i] = fmaf(x[r][i], c[i], o[i] * s[i]);
      }
    }
  }

  if (!stored) {
    T* dst = is_q ? static_cast<T*>(a.q_out) + ((int64_t)t * a.hq + h0) * D + d0
                  : static_cast<T*>(a.k_out) + ((int64_t)t * a.hk + h0) * D + d0;
#pragma unroll
    for (int r = 0; r < RPW; ++r)
      if (r < n) store_row<T, E>(dst + r * D, x[r]);
    return;
  }
  if (slot >= a.slots) {
    if (lane == 0) atomicOr(&g_kv_error, 2u);
    slot = -1;
  }
  if (slot < 0) return;
  const bool e4m3 = a.format == RQ_KV_E4M3;
  const float top = e4m3 ? 448.0f : 127.0f;
  const int64_t page = slot >> a.lg_page;
  // heads of a token lie a page's tokens apart
  const int64_t row = ((page * a.hkv + h0) << a.lg_page) + (slot & ((1 << a.lg_page) - 1));
  uint32_t most[RPW], own = 0u;  // largest magnitudes, as bits; lane r keeps row r's
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < E; ++i) m = max(m, __float_as_uint(x[r][i]) & 0x7FFFFFFFu);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    most[r] = m;
    if (m >= 0x7F800000u) {  // something is not finite: the largest of the rest
      m = 0u;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (!non_finite(x[r][i])) m = max(m, __float_as_uint(x[r][i]) & 0x7FFFFFFFu);
      m = __reduce_max_sync(0xFFFFFFFFu, m);
    }
    if (lane == r) own = m;
  }
  // the rows' divisions side by side, a lane each
  const float own_max = fmaxf(__uint_as_float(own), kLeastMax);
  const float own_mul = __fmul_rn(top, __frcp_rn(own_max));
  if (lane < n) (is_k ? a.ks : a.vs)[row + ((int64_t)lane << a.lg_page)] = __fdiv_rn(own_max, top);
  uint8_t* dst = (is_k ? a.kc : a.vc) + row * D + d0;
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
    const float mul = RPW == 1 ? __shfl_sync(0xFFFFFFFFu, own_mul, 0)
                               : __shfl_sync(0xFFFFFFFFu, own_mul, r);
    if (r >= n) break;
    uint32_t code[(E + 3) / 4];
    if (most[r] < 0x7F800000u) {
      code[0] = encode2(e4m3, x[r][0], x[r][1], mul);
#pragma unroll
      for (int i = 2; i < E; i += 2) {
        const uint32_t two = encode2(e4m3, x[r][i], x[r][i + 1], mul);
        code[i / 4] = (i & 3) ? code[i / 4] | two << 16 : two;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint32_t one = e4m3 ? encode_e4m3(x[r][i], mul) : encode_i8(x[r][i], mul);
        code[i / 4] = (i & 3) ? code[i / 4] | one << (8 * (i & 3)) : one;
      }
    }
    uint8_t* to = dst + (((int64_t)r << a.lg_page) * D);
    if constexpr (E == 2)
      *reinterpret_cast<uint16_t*>(to) = (uint16_t)code[0];
    else if constexpr (E == 4)
      *reinterpret_cast<uint32_t*>(to) = code[0];
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
  }
}

template <typename T, int E>
rq_status launch_rows_rpw(RowsArgs a, cudaStream_t st) {
  // One row per warp while that fills no more than the SMs once: a single
  // token's rows then run side by side.  Four rows per warp otherwise, so
  // that cos, sin and the slot are fetched once for four and the loads of
  // four rows are in flight together.
  const int rows = a.hq + a.hk + a.hv;
  const int rpw = (int64_t)a.tokens * rows <= 8 * (int64_t)device_sm_count() ? 1 : 4;
  a.tq = (a.hq + rpw - 1) / rpw;
  a.tk = (a.hk + rpw - 1) / rpw;
  a.tasks = divisor((uint32_t)(a.tq + a.tk + (a.hv + rpw - 1) / rpw));
  const int64_t warps = (int64_t)a.tokens * a.tasks.d;
  const unsigned grid = (unsigned)((warps + kRowThreads / 32 - 1) / (kRowThreads / 32));
  return rpw == 1 ? launch_kernel(rows_kernel<T, E, 1>, grid, kRowThreads, 0, st, a)
                  : launch_kernel(rows_kernel<T, E, 4>, grid, kRowThreads, 0, st, a);
}

template <typename T>
rq_status launch_rows_t(const RowsArgs& a, int head_dim, cudaStream_t st) {
  switch (head_dim) {
    case 64: return launch_rows_rpw<T, 2>(a, st);
    case 128: return launch_rows_rpw<T, 4>(a, st);
    default: return launch_rows_rpw<T, 8>(a, st);
  }
}

rq_status launch_rows(const RowsArgs& a, int dtype, int head_dim, cudaStream_t st) {
  switch (dtype) {
    case RQ_F32: return launch_rows_t<float>(a, head_dim, st);
    case RQ_F16: return launch_rows_t<__half>(a, head_dim, st);
    default: return launch_rows_t<__nv_bfloat16>(a, head_dim, st);
  }
}

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

void set_cache(RowsArgs& a, const rq_kv_cache& c, const int64_t* slot) {
  a.slot = slot;
  a.kc = static_cast<uint8_t*>(c.k);
  a.vc = static_cast<uint8_t*>(c.v);
  a.ks = c.k_scale;
  a.vs = c.v_scale;
  a.slots = c.pages * c.page_size;
  a.lg_page = log2_of(c.page_size);
  a.hkv = c.kv_heads;
  a.format = c.format;
}

// ----------------------------------------------------------- read back --

// A thread takes kReadRuns runs of 8 codes of k and the same of v, 256 runs
// apart, so that the warps' stores stay whole lines and several loads are in
// flight behind each slot's (30000 tokens of 4 heads of 128: 16.1 us, 5.8 TB/s with two
// runs, 18.1 us with one, 16.3 us with four).
constexpr int kReadRuns = 2;
template <typename T>
__global__ void __launch_bounds__(256)
read_kernel(const rq_kv_cache c, const int64_t* __restrict__ slot, int tokens, int lg_page,
            int lg_chunks, const Divisor heads, T* __restrict__ k_out, T* __restrict__ v_out) {
  pdl_wait();
  pdl_trigger();
  const int64_t id0 = (int64_t)blockIdx.x * (256 * kReadRuns) + threadIdx.x;
  uint2 codes[kReadRuns][2];
  float scale[kReadRuns][2];
  bool live[kReadRuns];
#pragma unroll
  for (int u = 0; u < kReadRuns; ++u) {
    const int64_t id = id0 + 256 * u;
    const uint32_t at = (uint32_t)(id >> lg_chunks);  // token * kv_heads + head, below 2^31
    const uint32_t t = quotient(at, heads);
    const int h = (int)(at - t * heads.d);
    live[u] = t < (uint32_t)tokens;
    int64_t s = live[u] ? slot[t] : -1;
    if (s >= c.pages << lg_page) {
      atomicOr(&g_kv_error, 2u);
      s = -1;
    }
    codes[u][0] = codes[u][1] = make_uint2(0u, 0u);
    scale[u][0] = scale[u][1] = 0.0f;
    if (s >= 0) {
      const int64_t src =
          (((s >> lg_page) * c.kv_heads + h) << lg_page) + (s & ((1 << lg_page) - 1));
      const int64_t chunk = (src << lg_chunks) + (id & ((1 << lg_chunks) - 1));
      codes[u][0] = __ldg(static_cast<const uint2*>(c.k) + chunk);
      codes[u][1] = __ldg(static_cast<const uint2*>(c.v) + chunk);
      scale[u][0] = __ldg(c.k_scale + src);
      scale[u][1] = __ldg(c.v_scale + src);
    }
  }
#pragma unroll
  for (int u = 0; u < kReadRuns; ++u) {
    if (!live[u]) continue;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const uint32_t w[2] = {codes[u][o].x, codes[u][o].y};
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint32_t pair = w[i / 4] >> (8 * (i & 3));
        float lo, hi;
        if (c.format == RQ_KV_E4M3) {
          uint32_t h2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((unsigned short)(pair & 0xFFFFu)));
          const float2 f = half_pair(h2);
          lo = f.x;
          hi = f.y;
        } else {
          lo = (float)(int8_t)(pair & 0xFFu);
          hi = (float)(int8_t)((pair >> 8) & 0xFFu);
        }
        x[i] = lo * scale[u][o];
        x[i + 1] = hi * scale[u][o];
      }
      store_row<T, 8>((o == 0 ? k_out : v_out) + (id0 + 256 * u) * 8, x);
    }
  }
}

template <typename T>
rq_status launch_read_t(const rq_kv_cache& c, const int64_t* slot, void* k_out, void* v_out,
                        int tokens, cudaStream_t st) {
  const int lg_chunks = log2_of(c.head_dim / 8);
  const int64_t threads = ((int64_t)tokens * c.kv_heads) << lg_chunks;
  const unsigned grid = (unsigned)((threads + 256 * kReadRuns - 1) / (256 * kReadRuns));
  return launch_kernel(read_kernel<T>, dim3(grid), dim3(256), 0, st, c, slot, tokens,
                       log2_of(c.page_size), lg_chunks, divisor((uint32_t)c.kv_heads),
                       static_cast<T*>(k_out), static_cast<T*>(v_out));
}

}  // namespace

rq_status launch_qkv_rows(const rq_qk_params* p, int dtype, const void* q, int64_t q_stride,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const int32_t* position, void* q_out, void* k_out,
                          const rq_kv_cache* cache, const int64_t* slot, int tokens,
                          cudaStream_t st) {
  RowsArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.k_out = k_out;
  a.position = position;
  a.tokens = tokens;
  int head_dim, hkv;
  if (p != nullptr) {
    a.q_weight = p->q_weight;
    a.k_weight = p->k_weight;
    a.cos_table = p->cos_table;
    a.sin_table = p->sin_table;
    a.positions = p->positions;
    a.rotary = p->rotary_dim;
    a.interleaved = p->interleaved;
    a.eps = p->eps;
    head_dim = p->head_dim;
    hkv = p->kv_heads;
    a.hq = q != nullptr ? p->q_heads : 0;
  } else {
    head_dim = cache->head_dim;
    hkv = cache->kv_heads;
  }
  a.hk = k != nullptr ? hkv : 0;
  a.hv = v != nullptr ? hkv : 0;
  if (cache != nullptr) set_cache(a, *cache, slot);
  return launch_rows(a, dtype, head_dim, st);
}

rq_status launch_kv_read(const rq_kv_cache& cache, int dtype, const int64_t* slot, void* k_out,
                         void* v_out, int tokens, cudaStream_t st) {
  switch (dtype) {
    case RQ_F32: return launch_read_t<float>(cache, slot, k_out, v_out, tokens, st);
    case RQ_F16: return launch_read_t<__half>(cache, slot, k_out, v_out, tokens, st);
    default: return launch_read_t<__nv_bfloat16>(cache, slot, k_out, v_out, tokens, st);
  }
}

rq_status read_and_clear_kv_error() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(v)) != cudaSuccess) return RQ_ERR_CUDA;
  if (v == 0) return RQ_OK;
  const unsigned int zero = 0;
  if (cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(zero)) != cudaSuccess) return RQ_ERR_CUDA;
  return RQ_ERR_INDEX;
}

}  // namespace rq
