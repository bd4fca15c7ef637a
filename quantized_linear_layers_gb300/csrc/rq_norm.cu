// rq_norm.cu -- the norm after a block, the gated and scaled sum with the
// residual stream and the norm before the next block (sm_103a).
//
// Per token, over its width values, in f32:
//   p = y * rsqrt(mean(y^2) + eps) * post_weight     (or y)
//   h' = h + scale * (gate * p)
//   x = h' * rsqrt(mean(h'^2) + eps) * pre_weight    (or h')
//
// A group of threads keeps its token in registers between the two sums: y and
// h are read once and h' and x written once, which is what the operator cannot
// do without.  Bound by memory: 4096 tokens of 3584 f32 values take 36.8 us
// (6.39 TB/s, 95 % of a measured copy), 37.7 with the largest magnitude (calls one
// behind another on three sets of tensors; 41 between other kernels with a cold
// L2); bf16 on an f32 stream 29.8 us (5.90 TB/s), bf16 throughout 23.1 (5.07: there
// a CTA's steps one after another count).  y and h stay as they lie in memory until
// they are used, which lets four CTAs of 224 threads onto an SM (16-bit rows as
// floats: 27.3 us; six CTAs spill registers: 40.9 for f32).  One token: 2.2 us in a
// replayed graph.  Odd widths: 1091 tokens of 6245 f32 values with a gate a
// token 34 us (an element at a time 40).
#include "rq_device.cuh"
#include "rq_elem.cuh"
#include "rq_internal.h"

namespace rq {

namespace {

constexpr int kMaxWarps = 32;

struct NormArgs {
  const void *y, *gate, *h;
  int64_t y_stride, gate_stride, h_stride;
  const float *post_weight, *pre_weight;
  void *h_out, *x_out;
  uint32_t* absmax;
  int width, tokens;
  int post, pre, alone;  // alone: one CTA holds every token
  float eps, scale, inv_width;
};

// Sum over the warps of a token's group.  `part` is written once per launch.
template <bool kOneWarp>
__device__ __forceinline__ float group_sum(float v, float* part) {
  v = warp_sum(v);
  if constexpr (!kOneWarp) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum(lane < warps ? part[lane] : 0.0f);
  }
  return v;
}

// V values as they lie in memory, and as floats.
template <typename T, int V>
struct Raw {
  static constexpr int kWords = V * (int)sizeof(T) / 16;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ float operator[](int j) const {
    constexpr int kPer = 16 / (int)sizeof(T);
    return elem_float(reinterpret_cast<const T*>(&w[j / kPer])[j % kPer]);
  }
  // values [c, c + V) of a row of which some may not be there (zeros)
  __device__ __forceinline__ void load_some(const T* row, int c, int width) {
    alignas(16) T t[V];
#pragma unroll
    for (int j = 0; j < V; ++j)
      t[j] = c + j >= 0 && c + j < width ? row[c + j] : float_elem<T>(0.0f);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(t)[i];
  }
};
template <typename T>
struct Raw<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ void load_some(const T*, int, int) {}
  __device__ __forceinline__ float operator[](int) const { return elem_float(w); }
};

// V values to a row, of which some may not be there.
template <typename T, int V>
__device__ __forceinline__ void store_some(T* row, int c, int width, const float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (c + j >= 0 && c + j < width) row[c + j] = float_elem<T>(x[j]);
}

// T: type of y, gate and x; R: of the residual stream; V: values a thread
// takes at a time; G: how many such groups it holds.  kOneWarp: a token is one
// warp's, several to a CTA; else a CTA's, of at most kThreads threads.  kSkew:
// rows of a width that is no multiple of V, one behind another.  Groups are then
// counted over all of them, so that they are aligned; a row's first and last
// group are its own in part, and weights are read a value at a time.
template <typename T, typename R, int V, int G, bool kOneWarp, bool kSkew, int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) residual_norm_kernel(const NormArgs a) {
  __shared__ float part[2][kMaxWarps];
  __shared__ unsigned int top;
  const int group = kOneWarp ? 32 : (int)blockDim.x;
  const int lane = kOneWarp ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const int64_t t = kOneWarp ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                             : (int64_t)blockIdx.x;
  if (threadIdx.x == 0) top = 0u;
  pdl_wait();
  pdl_trigger();
  float most = 0.0f;
  if (t < a.tokens) {
    const T* yp = static_cast<const T*>(a.y) + t * a.y_stride;
    const R* hp = static_cast<const R*>(a.h) + t * a.h_stride;
    const T* gp = static_cast<const T*>(a.gate) + t * a.gate_stride;
    const int skew = kSkew ? (int)(t * a.width % V) : 0;
    // a thread's group g: its first value, whether it has any, and all
    const auto at = [&](int g) { return (g * group + lane) * V - skew; };
    const auto any = [&](int c) { return c < a.width; };
    const auto whole = [&](int c) { return !kSkew || (c >= 0 && c + V <= a.width); };
    Raw<T, V> y[G];
    Raw<R, V> hr[G];
    // a thread of few values sends for weights and gate with them; one of many
    // keeps its registers for those
    constexpr bool kEarly = G * V <= 8 && !kSkew;
    constexpr int E = kEarly ? G : 1;
    Raw<float, V> post[E], pre[E];
    Raw<T, V> gate[E];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c = at(g);
      if (any(c)) {
        if (whole(c)) {
          if (a.y != nullptr) y[g].load(yp + c);
          hr[g].load(hp + c);
        } else {
          if (a.y != nullptr) y[g].load_some(yp, c, a.width);
          hr[g].load_some(hp, c, a.width);
        }
        if constexpr (kEarly) {
          if (a.post_weight != nullptr) post[g].load(a.post_weight + c);
          if (a.gate != nullptr) gate[g].load(gp + c);
          if (a.pre_weight != nullptr) pre[g].load(a.pre_weight + c);
        }
      }
    }
    float r = a.scale;
    if (a.post) {
      float sum = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (any(at(g))) {
#pragma unroll
          for (int j = 0; j < V; ++j) sum = fmaf(y[g][j], y[g][j], sum);
        }
      sum = group_sum<kOneWarp>(sum, part[0]);
      r = rsqrtf(fmaf(sum, a.inv_width, a.eps));
    }
    float h[G][V];
    float square = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c = at(g);
      if (!any(c)) continue;
#pragma unroll
      for (int j = 0; j < V; ++j) h[g][j] = hr[g][j];
      if (a.y != nullptr) {
        constexpr bool kLate = !kEarly;
        const int e = kEarly ? g : 0;
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = a.post ? y[g][j] * r : y[g][j];
        if (a.post_weight != nullptr) {
          if constexpr (kSkew)
            post[e].load_some(a.post_weight, c, a.width);
          else if constexpr (kLate)
            post[e].load(a.post_weight + c);
#pragma unroll
          for (int j = 0; j < V; ++j) f[j] *= post[e][j];
        }
        if (a.gate != nullptr) {
          if (kSkew && (a.gate_stride == 0 || !whole(c)))
            gate[e].load_some(gp, c, a.width);
          else if constexpr (kLate)
            gate[e].load(gp + c);
#pragma unroll
          for (int j = 0; j < V; ++j) f[j] *= gate[e][j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) h[g][j] = fmaf(a.scale, f[j], h[g][j]);
        if (a.h_out != nullptr) {
          R* ho = static_cast<R*>(a.h_out) + t * a.width;
          if (whole(c))
            store_elems<R, V>(ho + c, h[g]);
          else
            store_some<R, V>(ho, c, a.width, h[g]);
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) square = fmaf(h[g][j], h[g][j], square);
    }
    if (a.x_out != nullptr) {
      r = 1.0f;
      if (a.pre) {
        square = group_sum<kOneWarp>(square, part[1]);
        r = rsqrtf(fmaf(square, a.inv_width, a.eps));
      }
      T* xo = static_cast<T*>(a.x_out) + t * a.width;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int c = at(g);
        if (!any(c)) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) h[g][j] *= r;
        if (a.pre_weight != nullptr) {
          const int e = kEarly ? g : 0;
          if constexpr (kSkew)
            pre[e].load_some(a.pre_weight, c, a.width);
          else if constexpr (!kEarly)
            pre[e].load(a.pre_weight + c);
#pragma unroll
          for (int j = 0; j < V; ++j) h[g][j] *= pre[e][j];
        }
        if (a.absmax != nullptr) {
#pragma unroll
          for (int j = 0; j < V; ++j) most = fmaxf(most, fabsf(h[g][j]));  // (a NaN is passed over)
        }
        if (whole(c))
          store_elems<T, V>(xo + c, h[g]);
        else
          store_some<T, V>(xo, c, a.width, h[g]);
      }
    }
  }
  if (a.absmax != nullptr) {
    // non-negative floats are ordered as their bits
    const unsigned int m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) atomicMax(&top, m);
    __syncthreads();
    if (threadIdx.x == 0) {
      if (a.alone)
        *a.absmax = top;
      else
        atomicMax(a.absmax, top);
    }
  }
}

// The word that the CTAs' maxima go to.  A kernel, not a memset: the next one's
// launch overlaps it.
__global__ void clear_word_kernel(uint32_t* word) {
  pdl_wait();
  pdl_trigger();
  *word = 0u;
}

// Groups of V values that a thread takes of many tokens' rows.
template <int V>
constexpr int kManyGroups = 16 / V < 4 ? 16 / V : 4;

template <typename T, typename R, int V, int G, bool kSkew>
rq_status launch_groups(const NormArgs& a, int threads, int per_cta, cudaStream_t st) {
  const unsigned ctas = (unsigned)((a.tokens + per_cta - 1) / per_cta);
  // (a thread takes another number of groups only where 1024 threads would not
  // hold the row with fewer, and then there are more than 512)
  if constexpr (G == 1 || G == kManyGroups<V>) {
    if (threads == 32)
      return launch_kernel(residual_norm_kernel<T, R, V, G, true, kSkew, 128, 1>, dim3(ctas),
                           dim3(32 * per_cta), 0, st, a);
    if (threads <= 256)
      return launch_kernel(residual_norm_kernel<T, R, V, G, false, kSkew, 256, 4>, dim3(ctas),
                           dim3(threads), 0, st, a);
  }
  return launch_kernel(residual_norm_kernel<T, R, V, G, false, kSkew, 1024, 1>, dim3(ctas),
                       dim3(threads), 0, st, a);
}

// `groups` of V values in a row, G of them a thread.
template <typename T, typename R, int V, bool kSkew>
rq_status launch_width(NormArgs a, cudaStream_t st) {
  constexpr int kMost = 16 / V;  // groups that fit 16 values a thread
  const int groups = (a.width + V - 1 + (kSkew ? V - 1 : 0)) / V;
  // few tokens: as many threads as the row has groups, so that each thread
  // waits for one load; many: as many loads in flight a thread as fit
  const bool few = a.tokens <= 2 * device_sm_count();
  int G = few || groups <= 32 ? 1 : kManyGroups<V>;
  while (G < kMost && (groups + G - 1) / G > 1024) G *= 2;
  const int threads = ((groups + G - 1) / G + 31) / 32 * 32;
  const int per_cta = threads == 32 ? 4 : 1;
  a.alone = a.tokens <= per_cta;
  if (a.absmax != nullptr && !a.alone) {
    const rq_status s = launch_kernel(clear_word_kernel, dim3(1), dim3(1), 0, st, a.absmax);
    if (s != RQ_OK) return s;
  }
  if constexpr (kMost >= 16)
    if (G == 16) return launch_groups<T, R, V, 16, kSkew>(a, threads, per_cta, st);
  if constexpr (kMost >= 8)
    if (G == 8) return launch_groups<T, R, V, 8, kSkew>(a, threads, per_cta, st);
  if constexpr (kMost >= 4)
    if (G == 4) return launch_groups<T, R, V, 4, kSkew>(a, threads, per_cta, st);
  if constexpr (kMost >= 2)
    if (G == 2) return launch_groups<T, R, V, 2, kSkew>(a, threads, per_cta, st);
  return launch_groups<T, R, V, 1, kSkew>(a, threads, per_cta, st);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, typename R>
rq_status launch_types(const NormArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);  // values of 16 bytes of the narrower type
  const auto whole = [](int64_t stride, size_t size) { return stride * size % 16 == 0; };
  const bool rows16 = aligned16(a.y) && aligned16(a.gate) && aligned16(a.h) &&
                      aligned16(a.h_out) && aligned16(a.x_out);
  if (a.width % V == 0 && rows16 && aligned16(a.post_weight) && aligned16(a.pre_weight) &&
      whole(a.y_stride, sizeof(T)) && whole(a.gate_stride, sizeof(T)) &&
      whole(a.h_stride, sizeof(R)))
    return launch_width<T, R, V, false>(a, st);
  // (a row's groups, its own and those it shares, must fit the threads)
  if (rows16 && a.width <= 16384 - 2 * V && a.h_stride == a.width &&
      (a.y == nullptr || a.y_stride == a.width) &&
      (a.gate_stride == 0 || a.gate_stride == a.width))
    return launch_width<T, R, V, true>(a, st);
  return launch_width<T, R, 1, false>(a, st);
}

}  // namespace

rq_status launch_residual_norm(const rq_norm_params& p, int dtype, const void* y,
                               int64_t y_stride, const void* gate, int64_t gate_stride,
                               int h_dtype, const void* h, int64_t h_stride, void* h_out,
                               void* x_out, uint32_t* absmax, int tokens, cudaStream_t st) {
  NormArgs a = {};
  a.y = y;
  a.gate = y != nullptr ? gate : nullptr;
  a.h = h;
  a.y_stride = y != nullptr ? y_stride : 0;
  a.gate_stride = a.gate != nullptr ? gate_stride : 0;
  a.h_stride = h_stride;
  a.post = (p.norms & RQ_NORM_POST) != 0 && y != nullptr;
  a.pre = (p.norms & RQ_NORM_PRE) != 0 && x_out != nullptr;
  a.post_weight = a.post ? p.post_weight : nullptr;
  a.pre_weight = a.pre ? p.pre_weight : nullptr;
  a.h_out = h_out;
  a.x_out = x_out;
  a.absmax = absmax;
  a.width = p.width;
  a.tokens = tokens;
  a.eps = p.eps;
  a.scale = p.scale;
  a.inv_width = 1.0f / (float)p.width;
  if (tokens == 0)
    return absmax == nullptr ? RQ_OK
                             : cuda_status(cudaMemsetAsync(absmax, 0, sizeof(uint32_t), st));
  if (dtype == RQ_F32) return launch_types<float, float>(a, st);
  if (dtype == RQ_F16)
    return h_dtype == RQ_F32 ? launch_types<__half, float>(a, st)
                             : launch_types<__half, __half>(a, st);
  return h_dtype == RQ_F32 ? launch_types<__nv_bfloat16, float>(a, st)
                           : launch_types<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace rq
