// rq_sample.cu -- from logits to a token, or to the probabilities of the
// tokens that temperature, min-p, top-k and top-p leave (sm_103a).
//
// Whole weights W = floor(2^42 e^((l - largest) / T)) make every sum exact:
// where a nucleus ends and which token a random number meets depend on no
// order of summation, however a row is cut up.  42 bits, because a nucleus of
// 10^5 tokens ends at probabilities of 10^-6, so that sums of f32 weights
// (2^-24 each) would move its border; 2^20 tokens of 2^42 still fit 64 bits.
//
// The power.  y = (largest - l) log2(e) / T is carried as a sum of two floats
// (the difference and the products with their rounding errors), and
//   2^-y = 2^-n  2^(-j/256)  e^(-z),   n + j/256 the nearest of 256ths, |z| < 0.0014:
// a table of the 256 powers as sums of two floats, and four terms of the
// series of e^-z, of which only the first needs more than 24 bits.  That is
// about 45 f32 operations per token, relative error about 2^-43.  (64-bit
// floats would need fewer, at 1/64 of the rate.)
//
// Finding where top-k and top-p cut.  Sorting a row is not needed: a histogram
// of y finds the bin that the cut falls in, the bin's tokens (a hundred, say) are
// listed and each counts what stands before it.  A bin of more tokens than the
// list holds is divided again by the bits of its logits; equal logits, however
// many, are cut by counting in order of index.
//
// One cluster of CTAs takes a row and keeps it in shared memory: logits are
// read from memory once.  Every CTA gets the merged histogram and the whole
// list through distributed shared memory and decides by itself, so decisions
// are never sent back.
#include "rq_device.cuh"
#include "rq_elem.cuh"
#include "rq_internal.h"

namespace rq {

namespace {

constexpr int kSThreads = 512;
constexpr int kSWarps = kSThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
constexpr int kList = 512;           // tokens of a bin that are ranked directly
constexpr int kTable = 256;
constexpr float kFar = 43.0f;        // 2^42 2^-y is below 1 from y = 42 on
constexpr int kUnitBits = 42;
constexpr int kCacheMax = 40 * 1024; // logits of a CTA kept in shared memory

// 2^(-j/256) as a sum of two floats.
struct PowerTable {
  float hi[kTable], lo[kTable];
  constexpr PowerTable() : hi(), lo() {
    for (int j = 0; j < kTable; ++j) {
      // e^-x by its series, x < ln 2: the 20th term is below 2^-70
      const double x = 0.693147180559945309417 * j / kTable;
      double term = 1.0, sum = 1.0;
      for (int i = 1; i <= 24; ++i) {
        term *= -x / i;
        sum += term;
      }
      hi[j] = (float)sum;
      lo[j] = (float)(sum - (double)hi[j]);
    }
  }
};
__device__ const PowerTable g_power;

struct Cut {
  uint32_t key;  // tokens of a larger key stay, and those of this key up to
  int index;     // this index
};

struct SampleShared {
  float2 power[kTable];
  unsigned long long merged_w[kBins];
  unsigned long long sums[kMaxCluster * kSWarps];
  unsigned long long list_w[kList];
  unsigned long long tmp_w[kSWarps];
  unsigned long long above_w, total;
  uint32_t count[kBins], lo[kBins], hi[kBins];  // this CTA's part of the row
  uint32_t merged_n[kBins];
  uint32_t list_key[2][kList];  // top-k's and top-p's candidates
  int list_index[2][kList];
  uint32_t tmp_n[kSWarps];
  uint32_t key_min[kMaxCluster], key_max[kMaxCluster];
  float top[kMaxCluster];
  int first[kMaxCluster];
  uint32_t above_n, bin_n, pushed, base;
  int bin, found;
  Cut cut;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ void put_u32(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void put_u64(const void* p, uint32_t rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_rank(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t get_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(p, rank)) : "memory");
  return v;
}

// Floats in order as unsigned integers.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x == 0.0f) x = 0.0f;  // -0 equals +0
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) != 0u ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) != 0u ? 0x80000000u : 0xFFFFFFFFu));
}

template <typename I>
__device__ __forceinline__ I warp_scan_add(I v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

template <typename I>
__device__ __forceinline__ I warp_add(I v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// A row's scale: y = (top - l) (ch + cl).
struct Scale {
  float top;
  // 1, or for a temperature past 2^100 a small power of two that keeps
  // differences of any two floats finite and ch normal
  float pre;
  float near, ch, cl;  // top pre; log2(e) / T / pre
  const float2* power;

  __device__ __forceinline__ void set(float t) {
    const double c = 1.4426950408889634074 / (double)t;
    pre = c < 0x1p-100 ? 0x1p-64f : 1.0f;
    near = top * pre;
    ch = (float)(c / (double)pre);
    cl = (float)(c / (double)pre - (double)ch);
  }

  __device__ __forceinline__ float far(float l) const {
    return l == top ? 0.0f : fmaf(-l, pre, near) * ch;
  }

  __device__ __forceinline__ unsigned long long weight(float l) const {
    if (l == top) return 1ull << kUnitBits;
    // (top - l) pre = s + e exactly
    l *= pre;
    const float s = near - l, t = s - near;
    const float e = (near - (s - t)) - (l + t);
    const float ph = s * ch;
    if (!(ph < kFar)) return 0ull;
    const float pl = fmaf(s, ch, -ph) + fmaf(s, cl, e * ch);
    // the nearest 256th, by the addition of 1.5 2^23
    const float mf = fmaf(ph, 256.0f, 12582912.0f);
    const int m = (int)(__float_as_uint(mf) - 0x4B400000u);
    const float r = fmaf(mf - 12582912.0f, -0x1p-8f, ph);
    // z = (r + pl) ln 2 in two parts, e^-z - 1 = -zh + el
    constexpr float kLn2H = 0.693147182464599609375f, kLn2L = -1.904654299957768e-9f;
    const float zh = r * kLn2H;
    const float zl = fmaf(r, kLn2H, -zh) + fmaf(r, kLn2L, pl * kLn2H);
    const float z = zh + zl;
    const float el = fmaf(z * z, fmaf(z, fmaf(z, 1.0f / 24.0f, -1.0f / 6.0f), 0.5f), -zl);
    // times the table's power, in two parts: v + rest
    const float2 p = power[m & (kTable - 1)];
    const float a = -p.x * zh, b = fmaf(-p.x, zh, -a);
    const float v = p.x + a, ve = a - (v - p.x);
    const float rest = ve + (b + fmaf(-p.y, zh, fmaf(p.x, el, p.y)));
    // v is a multiple of 2^-25 up to 1, |rest| < 2^-18
    const long long f =
        ((long long)__float2int_rz(v * 0x1p30f) << 19) + __float2int_rd(rest * 0x1p49f);
    const int shift = (m >> 8) + 49 - kUnitBits;
    return (unsigned long long)(f >> shift);
  }
};

struct SampleArgs {
  const void* logits;
  int64_t stride;
  const float *temperature, *top_p, *min_p;
  const int32_t* top_k;
  const float* u;
  int32_t* token;
  float* p;
  int vocab;
  int run;     // logits of a warp, a multiple of 4
  int vector;  // rows may be read four logits at a time
};

template <typename T>
__device__ __forceinline__ float4 four(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4*>(p);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const T* t = reinterpret_cast<const T*>(&u);
    return make_float4(elem_float(t[0]), elem_float(t[1]), elem_float(t[2]), elem_float(t[3]));
  }
}

// A NaN counts as -Inf.
__device__ __forceinline__ float plain(float x) { return x == x ? x : -INFINITY; }

// One cluster's row.  Everything but `cache` and the histogram is the same in
// every CTA after each exchange, so that all take the same branches.
template <typename T, bool kCached>
struct RowSampler {
  SampleShared& sh;
  float* cache;            // this CTA's part of the row (kCached)
  const T* row;
  const SampleArgs& a;
  int rank, ranks, tid, lane, warp;
  int begin;               // first token of this warp's run
  Scale scale;
  unsigned long long least;  // weights below it are left out (min-p)
  bool has_cut;
  Cut cut;

  // Four logits of this warp's run at offset i (a multiple of 4); -Inf past it
  // and past the row.
  __device__ __forceinline__ float4 read(int i) const {
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (i >= a.run || begin + i >= a.vocab) return v;
    if constexpr (kCached) return *reinterpret_cast<const float4*>(cache + warp * a.run + i);
    return load(i);
  }
  __device__ __forceinline__ float4 load(int i) const {
    const int at = begin + i;
    float4 v;
    if (a.vector && at + 4 <= a.vocab) {
      v = four<T>(row + at);
    } else {
      v.x = elem_float(row[at]);
      v.y = at + 1 < a.vocab ? elem_float(row[at + 1]) : -INFINITY;
      v.z = at + 2 < a.vocab ? elem_float(row[at + 2]) : -INFINITY;
      v.w = at + 3 < a.vocab ? elem_float(row[at + 3]) : -INFINITY;
    }
    v.x = plain(v.x);
    v.y = plain(v.y);
    v.z = plain(v.z);
    v.w = plain(v.w);
    return v;
  }

  // f(token, logit) over this warp's run, in order of index by rounds.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int i = 4 * lane; i - 4 * lane < a.run; i += 128) {
      const float4 v = read(i);
      f(begin + i, v.x);
      f(begin + i + 1, v.y);
      f(begin + i + 2, v.z);
      f(begin + i + 3, v.w);
    }
  }

  // The row into shared memory, and the row's largest logit.
  __device__ __forceinline__ float fill() {
    float most = -INFINITY;
    constexpr int kAhead = 4;
    for (int i0 = 4 * lane; i0 - 4 * lane < a.run; i0 += 128 * kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + 128 * j;
        v[j] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (i < a.run && begin + i < a.vocab) v[j] = load(i);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = i0 + 128 * j;
        if (kCached && i < a.run) *reinterpret_cast<float4*>(cache + warp * a.run + i) = v[j];
        most = fmaxf(most, fmaxf(fmaxf(v[j].x, v[j].y), fmaxf(v[j].z, v[j].w)));
      }
    }
    const uint32_t k = __reduce_max_sync(0xFFFFFFFFu, key_of(most));
    if (lane == 0) sh.tmp_n[warp] = k;
    __syncthreads();
    const uint32_t best =
        __reduce_max_sync(0xFFFFFFFFu, lane < kSWarps ? sh.tmp_n[lane] : 0u);
    cluster_wait();  // (arrived at the start) every CTA of the cluster runs
    if (tid < ranks) put_u32(&sh.top[rank], (uint32_t)tid, __float_as_uint(float_of(best)));
    cluster_sync();
    most = sh.top[0];
    for (int q = 1; q < ranks; ++q) most = fmaxf(most, sh.top[q]);
    return most;
  }

  // The first token whose logit is the largest.
  __device__ __forceinline__ int likeliest() {
    int at = 0x7FFFFFFF;
    each([&](int v, float l) {
      if (l == scale.top && v < at) at = v;
    });
    at = __reduce_min_sync(0xFFFFFFFFu, at);
    if (lane == 0) sh.tmp_n[warp] = (uint32_t)at;
    __syncthreads();
    const int best = __reduce_min_sync(
        0xFFFFFFFFu, lane < kSWarps ? (int)sh.tmp_n[lane] : 0x7FFFFFFF);
    if (tid < ranks) put_u32(&sh.first[rank], (uint32_t)tid, (uint32_t)best);
    cluster_sync();
    at = sh.first[0];
    for (int q = 1; q < ranks; ++q) at = min(at, sh.first[q]);
    return at;
  }

  __device__ __forceinline__ unsigned long long weight_kept(float l) const {
    const unsigned long long w = scale.weight(l);
    return w >= least ? w : 0ull;
  }

  // A bin's entry; 64-bit sums in two words, the carry passed on by whoever
  // wraps the lower one.
  __device__ __forceinline__ void enter(int bin, unsigned long long w) {
    atomicAdd(&sh.count[bin], 1u);
    const uint32_t lo = (uint32_t)w;
    uint32_t hi = (uint32_t)(w >> 32);
    if (lo != 0u && atomicAdd(&sh.lo[bin], lo) > 0xFFFFFFFFu - lo) ++hi;
    if (hi != 0u) atomicAdd(&sh.hi[bin], hi);
  }

  __device__ __forceinline__ int first_bin(float l) const {
    const float y = scale.far(l);
    return y < kFar ? min((int)(y * (kBins / kFar)), kBins - 1) : -1;
  }

  // The cluster's histogram into every CTA's merged_n / merged_w.
  // bin_of(l): a token's bin, or -1.
  template <typename F>
  __device__ __forceinline__ void histogram(F bin_of, bool weights) {
    for (int i = tid; i < kBins; i += kSThreads) sh.count[i] = sh.lo[i] = sh.hi[i] = 0u;
    __syncthreads();
    each([&](int, float l) {
      const int b = bin_of(l);
      if (b >= 0) enter(b, weights ? weight_kept(l) : 0ull);
    });
    cluster_sync();
    const int per = kBins / ranks;
    for (int i = tid; i < per; i += kSThreads) {
      const int b = rank * per + i;
      uint32_t n = 0;
      unsigned long long w = 0;
      for (int q = 0; q < ranks; ++q) {
        n += get_u32(&sh.count[b], q);
        w += ((unsigned long long)get_u32(&sh.hi[b], q) << 32) + get_u32(&sh.lo[b], q);
      }
      for (int q = 0; q < ranks; ++q) {
        put_u32(&sh.merged_n[b], q, n);
        put_u64(&sh.merged_w[b], q, w);
      }
    }
    cluster_sync();
  }

  // The bin in which the running count reaches `goal` (by_weight: the running
  // weight), after `n0` tokens of weight `w0`: bin (-1: none), above_n, above_w,
  // bin_n.
  __device__ __forceinline__ void find(bool by_weight, unsigned long long goal, uint32_t n0,
                                       unsigned long long w0) {
    constexpr int kPer = kBins / kSThreads;
    uint32_t n[kPer], my_n = 0;
    unsigned long long w[kPer], my_w = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      n[i] = sh.merged_n[tid * kPer + i];
      w[i] = sh.merged_w[tid * kPer + i];
      my_n += n[i];
      my_w += w[i];
    }
    const uint32_t scan_n = warp_scan_add(my_n, lane);
    const unsigned long long scan_w = warp_scan_add(my_w, lane);
    if (lane == 31) {
      sh.tmp_n[warp] = scan_n;
      sh.tmp_w[warp] = scan_w;
    }
    if (tid == 0) sh.bin = -1;
    __syncthreads();
    uint32_t run_n = n0 + scan_n - my_n;
    unsigned long long run_w = w0 + scan_w - my_w;
    for (int q = 0; q < warp; ++q) {
      run_n += sh.tmp_n[q];
      run_w += sh.tmp_w[q];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const unsigned long long before = by_weight ? run_w : run_n;
      if (before < goal && goal <= before + (by_weight ? w[i] : n[i])) {
        sh.bin = tid * kPer + i;
        sh.above_n = run_n;
        sh.above_w = run_w;
        sh.bin_n = n[i];
      }
      run_n += n[i];
      run_w += w[i];
    }
    __syncthreads();
  }

  // Lists the bin's tokens in every CTA and finds the one at which the count
  // (the weight) reaches `goal`.  Sets sh.cut and sh.total, the weight up to it.
  template <typename F>
  __device__ __forceinline__ void resolve(F bin_of, int which, bool by_weight,
                                          unsigned long long goal) {
    const int bin = sh.bin;
    const int n = (int)sh.bin_n;
    if (warp == 0) {
      uint32_t c = lane < ranks ? get_u32(&sh.count[bin], lane) : 0u;
      const uint32_t upto = warp_scan_add(c, lane);
      if (lane == rank) sh.base = upto - c;
      if (lane == 0) sh.pushed = 0u;
    }
    __syncthreads();
    each([&](int v, float l) {
      if (bin_of(l) == bin) {
        const uint32_t at = sh.base + atomicAdd(&sh.pushed, 1u);
        for (int q = 0; q < ranks; ++q) {
          put_u32(&sh.list_key[which][at], q, key_of(l));
          put_u32(&sh.list_index[which][at], q, (uint32_t)v);
        }
      }
    });
    cluster_sync();
    for (int i = tid; i < n; i += kSThreads)
      sh.list_w[i] = weight_kept(float_of(sh.list_key[which][i]));
    __syncthreads();
    // g threads to a candidate
    int g = 1;
    while (g < 32 && 2 * g * n <= kSThreads) g *= 2;
    const int i = tid / g, sub = tid % g;
    uint32_t before_n = 0;
    unsigned long long before_w = 0;
    if (i < n) {
      const uint32_t key = sh.list_key[which][i];
      const int index = sh.list_index[which][i];
      for (int j = sub; j < n; j += g) {
        const uint32_t kj = sh.list_key[which][j];
        if (kj > key || (kj == key && sh.list_index[which][j] < index)) {
          ++before_n;
          before_w += sh.list_w[j];
        }
      }
    }
    for (int o = 1; o < g; o *= 2) {
      before_n += __shfl_xor_sync(0xFFFFFFFFu, before_n, o);
      before_w += __shfl_xor_sync(0xFFFFFFFFu, before_w, o);
    }
    if (i < n && sub == 0) {
      before_w += sh.above_w;
      before_n += sh.above_n;
      const unsigned long long b = by_weight ? before_w : before_n;
      const unsigned long long mine = by_weight ? sh.list_w[i] : 1ull;
      if (b < goal && goal <= b + mine) {
        sh.cut = Cut{sh.list_key[which][i], sh.list_index[which][i]};
        sh.total = before_w + sh.list_w[i];
      }
    }
    __syncthreads();
  }

  // Of more equal logits than the list holds, the one at which the goal is
  // reached: the m-th by index.
  __device__ __forceinline__ void resolve_equal(uint32_t key, bool by_weight,
                                                unsigned long long goal) {
    const float l = float_of(key);
    const unsigned long long w = weight_kept(l);
    const unsigned long long m = by_weight ? (goal - sh.above_w + w - 1) / w : goal - sh.above_n;
    uint32_t mine = 0;
    each([&](int, float x) { mine += x == l ? 1u : 0u; });
    mine = warp_add(mine);
    if (lane < ranks) put_u64(&sh.sums[rank * kSWarps + warp], lane, mine);
    cluster_sync();
    unsigned long long before = 0;
    for (int q = 0; q < rank * kSWarps + warp; ++q) before += sh.sums[q];
    if (before < m && m <= before + mine) {
      // this warp's run holds it
      for (int i = 4 * lane; i - 4 * lane < a.run; i += 128) {
        const float4 v = read(i);
        const float x[4] = {v.x, v.y, v.z, v.w};
        uint32_t c = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) c += x[j] == l ? 1u : 0u;
        const uint32_t scan = warp_scan_add(c, lane);
        unsigned long long run = before + scan - c;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (x[j] == l && ++run == m)
            for (int q = 0; q < ranks; ++q) put_u32(&sh.found, q, (uint32_t)(begin + i + j));
        before += __shfl_sync(0xFFFFFFFFu, scan, 31);
      }
    }
    cluster_sync();
    if (tid == 0) {
      sh.cut = Cut{key, sh.found};
      sh.total = sh.above_w + m * w;
    }
    __syncthreads();
  }

  // Where the running count (weight) reaches the goal, from the row's first
  // histogram on, which `fresh` says is in place (and is no more, if divided
  // further).  False: it does not.
  __device__ __forceinline__ bool search(bool by_weight, unsigned long long goal, bool weights,
                                         bool* fresh) {
    const auto bin0 = [this](float l) { return first_bin(l); };
    if (!*fresh) histogram(bin0, weights);
    *fresh = true;
    find(by_weight, goal, 0u, 0ull);
    if (sh.bin < 0) return false;
    const int which = by_weight ? 1 : 0;
    if (sh.bin_n <= kList) {
      resolve(bin0, which, by_weight, goal);
      return true;
    }
    *fresh = false;
    // the bin's range of logits, then a histogram of its bits, until few are
    // left or all are equal
    int bin = sh.bin;
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    each([&](int, float l) {
      if (first_bin(l) == bin) {
        lo = min(lo, key_of(l));
        hi = max(hi, key_of(l));
      }
    });
    for (;;) {
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      if (lane == 0) {
        sh.tmp_n[warp] = lo;
        sh.tmp_w[warp] = hi;
      }
      __syncthreads();
      for (int q = 0; q < kSWarps; ++q) {
        lo = min(lo, sh.tmp_n[q]);
        hi = max(hi, (uint32_t)sh.tmp_w[q]);
      }
      if (tid < ranks) {
        put_u32(&sh.key_min[rank], (uint32_t)tid, lo);
        put_u32(&sh.key_max[rank], (uint32_t)tid, hi);
      }
      cluster_sync();
      for (int q = 0; q < ranks; ++q) {
        lo = min(lo, sh.key_min[q]);
        hi = max(hi, sh.key_max[q]);
      }
      if (lo == hi) {
        resolve_equal(lo, by_weight, goal);
        return true;
      }
      const uint32_t klo = lo, khi = hi;
      int shift = 0;
      while (((khi - klo) >> shift) >= (uint32_t)kBins) ++shift;
      const auto bits = [=](float l) {
        const uint32_t k = key_of(l);
        return k >= klo && k <= khi ? (int)((khi - k) >> shift) : -1;
      };
      const uint32_t above_n = sh.above_n;
      const unsigned long long above_w = sh.above_w;
      histogram(bits, weights);
      find(by_weight, goal, above_n, above_w);
      if (sh.bin_n <= kList) {
        resolve(bits, which, by_weight, goal);
        return true;
      }
      bin = sh.bin;
      lo = 0xFFFFFFFFu;
      hi = 0u;
      each([&](int, float l) {
        if (bits(l) == bin) {
          lo = min(lo, key_of(l));
          hi = max(hi, key_of(l));
        }
      });
      __syncthreads();  // every thread has read sh.bin and the like
    }
  }

  __device__ __forceinline__ unsigned long long staying(int v, float l) const {
    if (has_cut) {
      const uint32_t k = key_of(l);
      if (k < cut.key || (k == cut.key && v > cut.index)) return 0ull;
    }
    return weight_kept(l);
  }

  // The token that the random number meets.
  __device__ __forceinline__ void draw(float u, int32_t* out) {
    unsigned long long mine = 0;
    each([&](int v, float l) { mine += staying(v, l); });
    mine = warp_add(mine);
    if (lane < ranks) put_u64(&sh.sums[rank * kSWarps + warp], lane, mine);
    cluster_sync();
    unsigned long long before = 0, total = 0;
    for (int q = 0; q < ranks * kSWarps; ++q) {
      const unsigned long long s = sh.sums[q];
      if (q < rank * kSWarps + warp) before += s;
      total += s;
    }
    unsigned int un = 0;
    if (u > 0.0f) un = (unsigned int)fminf(u * 0x1p24f, 16777215.0f);
    const unsigned long long point =
        un * (total >> 24) + ((un * (total & 0xFFFFFFull)) >> 24);
    if (before > point || point >= before + mine) return;
    // in this warp's run
    for (int i = 4 * lane; i - 4 * lane < a.run; i += 128) {
      const float4 v = read(i);
      const float x[4] = {v.x, v.y, v.z, v.w};
      unsigned long long w[4], c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) c += w[j] = staying(begin + i + j, x[j]);
      const unsigned long long scan = warp_scan_add(c, lane);
      unsigned long long run = before + scan - c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (run <= point && point < run + w[j]) *out = begin + i + j;
        run += w[j];
      }
      before += __shfl_sync(0xFFFFFFFFu, scan, 31);
      if (before > point) break;
    }
  }

  // p = weight / total.
  __device__ __forceinline__ void write(float* p) {
    unsigned long long total = sh.total;
    if (!has_cut) {
      unsigned long long mine = 0;
      each([&](int v, float l) { mine += staying(v, l); });
      mine = warp_add(mine);
      if (lane < ranks) put_u64(&sh.sums[rank * kSWarps + warp], lane, mine);
      cluster_sync();
      total = 0;
      for (int q = 0; q < ranks * kSWarps; ++q) total += sh.sums[q];
    }
    const float inv = 1.0f / __ull2float_rn(total);
    each([&](int v, float l) {
      if (v < a.vocab && v < begin + a.run) p[v] = __ull2float_rn(staying(v, l)) * inv;
    });
  }
};

template <typename T, bool kCached, bool kProbs>
__global__ void __launch_bounds__(kSThreads) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(raw);
  float* cache = reinterpret_cast<float*>(raw + (sizeof(SampleShared) + 15) / 16 * 16);
  cluster_arrive();
  const int tid = threadIdx.x;
  for (int i = tid; i < kTable; i += kSThreads)
    sh.power[i] = make_float2(g_power.hi[i], g_power.lo[i]);
  pdl_wait();
  pdl_trigger();
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t r = blockIdx.x / ranks;
  const int warp = tid >> 5, lane = tid & 31;
  RowSampler<T, kCached> s{sh,   cache, static_cast<const T*>(a.logits) + r * a.stride,
                           a,    rank,  ranks,
                           tid,  lane,  warp,
                           (rank * kSWarps + warp) * a.run};
  float t = a.temperature != nullptr ? a.temperature[r] : 1.0f;
  int k = a.top_k != nullptr ? a.top_k[r] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[r] : 1.0f;
  const float min_p = a.min_p != nullptr ? a.min_p[r] : 0.0f;
  if (!(t > 0.0f)) {
    t = 1.0f;
    k = 1;
  }
  s.scale.top = s.fill();
  if (!(s.scale.top > -INFINITY)) {
    // nothing to draw from
    if constexpr (kProbs) {
      s.each([&](int v, float) {
        if (v < a.vocab && v < s.begin + a.run) a.p[r * a.vocab + v] = 0.0f;
      });
    } else if (rank == 0 && tid == 0) {
      a.token[r] = -1;
    }
    return;
  }
  if (k == 1) {
    const int best = s.likeliest();
    if constexpr (kProbs) {
      s.each([&](int v, float) {
        if (v < a.vocab && v < s.begin + a.run) a.p[r * a.vocab + v] = v == best ? 1.0f : 0.0f;
      });
    } else if (rank == 0 && tid == 0) {
      a.token[r] = best;
    }
    return;
  }
  s.scale.set(t);
  s.scale.power = sh.power;
  s.least = 1ull;
  if (min_p > 0.0f) s.least = max(1ull, (unsigned long long)ceil((double)fminf(min_p, 1.0f) * 0x1p42));
  s.has_cut = false;
  const bool nucleus = top_p < 1.0f;
  if (k > 1 || nucleus) {
    bool fresh = false;
    bool cut = k > 1 && s.search(false, (unsigned long long)k, nucleus || kProbs, &fresh);
    if (cut) {
      s.has_cut = true;
      s.cut = sh.cut;
    }
    if (nucleus) {
      unsigned long long total = sh.total;
      if (!cut) {
        if (!fresh) s.histogram([&](float l) { return s.first_bin(l); }, true);
        fresh = true;
        s.find(true, ~0ull, 0u, 0ull);  // (met by no bin: leaves the scan's sums)
        total = 0;
        for (int q = 0; q < kSWarps; ++q) total += sh.tmp_w[q];
      }
      const double goal = ceil((double)fmaxf(top_p, 0.0f) * (double)total);
      __syncthreads();  // sh.total, sh.cut and the scan's sums have been read
      if (s.search(true, max(1ull, (unsigned long long)goal), true, &fresh)) {
        s.has_cut = true;
        s.cut = sh.cut;
      }
    }
  }
  if constexpr (kProbs)
    s.write(a.p + r * a.vocab);
  else
    s.draw(a.u[r], a.token + r);
}

template <typename T, bool kCached, bool kProbs>
rq_status launch_row(const SampleArgs& a, int rows, int ranks, cudaStream_t st) {
  const size_t smem = (sizeof(SampleShared) + 15) / 16 * 16 +
                      (kCached ? (size_t)a.run * kSWarps * sizeof(float) : 0);
  constexpr size_t kMost = (sizeof(SampleShared) + 15) / 16 * 16 + kCacheMax * sizeof(float);
  static_assert(kMost <= 227 * 1024, "shared memory of a CTA");
  auto kernel = sample_kernel<T, kCached, kProbs>;
  static bool ready = false;
  if (!ready) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost) !=
        cudaSuccess)
      return RQ_ERR_CUDA;
    ready = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)rows * (unsigned)ranks);
  cfg.blockDim = dim3(kSThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a));
}

template <typename T>
rq_status launch_type(SampleArgs a, int rows, cudaStream_t st) {
  a.vector = reinterpret_cast<uintptr_t>(a.logits) % (4 * sizeof(T)) == 0 && a.stride % 4 == 0;
  int ranks = kMaxCluster;
  while (ranks > 1 && a.vocab <= 4096 * (ranks / 2)) ranks /= 2;
  const int per = (a.vocab + ranks * kSWarps - 1) / (ranks * kSWarps);
  a.run = (per + 3) / 4 * 4;
  const bool cached = a.run * kSWarps <= kCacheMax;
  if (a.p != nullptr)
    return cached ? launch_row<T, true, true>(a, rows, ranks, st)
                  : launch_row<T, false, true>(a, rows, ranks, st);
  return cached ? launch_row<T, true, false>(a, rows, ranks, st)
                : launch_row<T, false, false>(a, rows, ranks, st);
}

}  // namespace

rq_status launch_sample(const rq_sampling& f, int dtype, const void* logits, int64_t stride,
                        const float* u, int32_t* token, float* p, int rows, int vocab,
                        cudaStream_t st) {
  SampleArgs a = {};
  a.logits = logits;
  a.stride = stride;
  a.temperature = f.temperature;
  a.top_k = f.top_k;
  a.top_p = f.top_p;
  a.min_p = f.min_p;
  a.u = u;
  a.token = token;
  a.p = p;
  a.vocab = vocab;
  if (dtype == RQ_F32) return launch_type<float>(a, rows, st);
  if (dtype == RQ_F16) return launch_type<__half>(a, rows, st);
  return launch_type<__nv_bfloat16>(a, rows, st);
}

}  // namespace rq
