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
  int rows, tasks;  // hq + hk + hv, and tasks of RPW rows per token
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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
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

// One warp takes RPW rows of one token at once: lane l holds values
// [l E, l E + E) of each, E = D / 32.  The rotation's partner values are in
// the lane rotary / 2 / E away (host: rotary % 16 == 0, so that distance is a
// whole number), the sums and maxima are shuffles: a row is read once and
// nothing passes through shared memory.
template <typename T, int E, int RPW>
__global__ void __launch_bounds__(kRowThreads)
rows_kernel(const RowsArgs a) {
  constexpr int D = 32 * E;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t task = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = task / a.tasks;
  if (t >= a.tokens) return;
  const int j0 = (int)(task - t * a.tasks) * RPW;
  const int d0 = lane * E;

  float x[RPW][E];
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
    const int j = j0 + r;
    if (j >= a.rows) continue;
    const T* p;
    if (j < a.hq)
      p = static_cast<const T*>(a.q) + t * a.q_stride + (int64_t)j * D;
    else if (j < a.hq + a.hk)
      p = static_cast<const T*>(a.k) + t * a.k_stride + (int64_t)(j - a.hq) * D;
    else
      p = static_cast<const T*>(a.v) + t * a.v_stride + (int64_t)(j - a.hq - a.hk) * D;
    load_row<T, E>(p + d0, x[r]);
  }

  // the token's turn: cos and sin of this lane's pairs
  const int half = a.rotary >> 1;
  bool turn = a.rotary > 0 && j0 < a.hq + a.hk;
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
  const int hop = half / E;
  const int partner = a.interleaved ? lane : (d0 < half ? lane + hop : lane - hop) & 31;

  int64_t slot = -1;
  if (a.slot != nullptr && j0 + RPW > a.hq) {
    slot = a.slot[t];
    if (slot >= a.slots) {
      if (lane == 0) atomicOr(&g_kv_error, 2u);
      slot = -1;
    }
  }

  const int hqk = a.hq + a.hk;
#pragma unroll
  for (int r = 0; r < RPW; ++r) {
    const int j = j0 + r;
    if (j >= a.rows) break;
    const float* weight = j < a.hq ? a.q_weight : j < hqk ? a.k_weight : nullptr;
    if (weight != nullptr) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) sum = fmaf(x[r][i], x[r][i], sum);
      sum = warp_sum(sum);
      const float inv = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
      float w[E];
      load_table<E>(weight + d0, w);
#pragma unroll
      for (int i = 0; i < E; ++i) x[r][i] = x[r][i] * inv * w[i];
    }
    if (turn && j < hqk) {
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
    if (j < a.hq) {
      store_row<T, E>(static_cast<T*>(a.q_out) + (t * a.hq + j) * D + d0, x[r]);
      continue;
    }
    const bool is_v = j >= hqk;
    const int h = is_v ? j - hqk : j - a.hq;
    if (a.slot == nullptr) {
      store_row<T, E>(static_cast<T*>(a.k_out) + (t * a.hk + h) * D + d0, x[r]);
      continue;
    }
    if (slot < 0) continue;
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) m = fmaxf(m, non_finite(x[r][i]) ? 0.0f : fabsf(x[r][i]));
    m = fmaxf(warp_max(m), kLeastMax);
    const float top = a.format == RQ_KV_E4M3 ? 448.0f : 127.0f;
    const float mul = __fmul_rn(top, __frcp_rn(m));
    alignas(8) uint8_t b[E];
    if (a.format == RQ_KV_E4M3) {
#pragma unroll
      for (int i = 0; i < E; ++i) b[i] = (uint8_t)encode_e4m3(x[r][i], mul);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) b[i] = (uint8_t)encode_i8(x[r][i], mul);
    }
    const int64_t page = slot >> a.lg_page;
    const int64_t row = ((page * a.hkv + h) << a.lg_page) + (slot & ((1 << a.lg_page) - 1));
    uint8_t* dst = (is_v ? a.vc : a.kc) + row * D + d0;
    if constexpr (E == 2)
      *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(b);
    else if constexpr (E == 4)
      *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(b);
    else
      *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(b);
    if (lane == 0) (is_v ? a.vs : a.ks)[row] = __fdiv_rn(m, top);
  }
}

template <typename T, int E>
rq_status launch_rows_rpw(RowsArgs a, cudaStream_t st) {
  // One row per warp while that fills no more than the SMs once: a single
  // token's rows then run side by side.  Four rows per warp otherwise, so
  // that cos, sin and the slot are fetched once for four and the loads of
  // four rows are in flight together.
  const int rpw = (int64_t)a.tokens * a.rows <= 8 * (int64_t)device_sm_count() ? 1 : 4;
  a.tasks = (a.rows + rpw - 1) / rpw;
  const int64_t warps = (int64_t)a.tokens * a.tasks;
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

// One thread takes 8 codes of k and the same 8 of v.
template <typename T>
__global__ void __launch_bounds__(256)
read_kernel(const rq_kv_cache c, const int64_t* __restrict__ slot, int tokens, int lg_page,
            int lg_chunks, T* __restrict__ k_out, T* __restrict__ v_out) {
  pdl_wait();
  pdl_trigger();
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id >> lg_chunks;  // token * kv_heads + head
  const int64_t t = row / c.kv_heads;
  if (t >= tokens) return;
  const int h = (int)(row - t * c.kv_heads);
  int64_t s = slot[t];
  if (s >= c.pages << lg_page) {
    atomicOr(&g_kv_error, 2u);
    s = -1;
  }
  float x[2][8] = {};
  if (s >= 0) {
    const int64_t src =
        (((s >> lg_page) * c.kv_heads + h) << lg_page) + (s & ((1 << lg_page) - 1));
    const int64_t chunk = (src << lg_chunks) + (id & ((1 << lg_chunks) - 1));
    const uint2 kb = __ldg(reinterpret_cast<const uint2*>(c.k) + chunk);
    const uint2 vb = __ldg(reinterpret_cast<const uint2*>(c.v) + chunk);
    const float sc[2] = {__ldg(c.k_scale + src), __ldg(c.v_scale + src)};
    const uint32_t w[2][2] = {{kb.x, kb.y}, {vb.x, vb.y}};
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint32_t pair = w[o][i / 4] >> (8 * (i & 3));
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
        x[o][i] = lo * sc[o];
        x[o][i + 1] = hi * sc[o];
      }
  }
  store_row<T, 8>(k_out + id * 8, x[0]);
  store_row<T, 8>(v_out + id * 8, x[1]);
}

template <typename T>
rq_status launch_read_t(const rq_kv_cache& c, const int64_t* slot, void* k_out, void* v_out,
                        int tokens, cudaStream_t st) {
  const int lg_chunks = log2_of(c.head_dim / 8);
  const int64_t threads = ((int64_t)tokens * c.kv_heads) << lg_chunks;
  return launch_kernel(read_kernel<T>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st,
                       c, slot, tokens, log2_of(c.page_size), lg_chunks, static_cast<T*>(k_out),
                       static_cast<T*>(v_out));
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
  a.rows = a.hq + a.hk + a.hv;
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
