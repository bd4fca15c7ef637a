// rq_sample.cu -- from logits to a token, or to the probabilities of the
// tokens that temperature, min-p, top-k and top-p leave (sm_103a).
//
// Whole weights W = floor(2^42 e^((l - largest) / T)) make every sum exact:
// where a nucleus ends and which token a random number meets depend on no
// order of summation, however a row is cut up.  f32 weights would not do: a
// nucleus of 10^5 tokens ends at probabilities of 10^-6, where sums of
// weights within 2^-24 differ by tokens.  2^20 tokens of 2^42 still fit 64 bits.
//
// The power.  y = 512 log2(e) (largest - l) / T is carried as a sum of two
// floats (the difference and the products with their rounding errors), and
//   2^(-y/512) = 2^-n 2^(-j/512) 2^(-z/512),   512 n + j = rint(y), |z| <= 1/2:
// a table of the 512 powers in 42 bits, less its product with a cubic in z
// that is below 2^-10, so that f32 roundings in it stay below 2^-33 of the
// weight (2^-35.6 on the average, measured).  (64-bit floats would need fewer
// instructions, at 1/64 of the rate.)
//
// Finding where top-k and top-p cut.  Sorting a row is not needed.  Counts of
// tokens in 512 bins of y give top-k's bin, and, since a bin's weights lie
// within 6 % of each other, the few bins that a nucleus can end in.  One pass of
// exact weights then sums what stands before those bins and after them, and
// divides them into 128 finer ones; the few tokens of the bin that the cut
// falls in are listed and each counts what stands before it.  What is not
// divided far enough is divided by the bits of the logits; equal logits,
// however many, are cut by counting in order of index.  A top-k of up to 512
// tokens, with its last bin, lists them all, ranks or sorts them, and needs no
// further look at the row.
//
// One cluster of CTAs takes a row and keeps it in shared memory: logits are
// read from memory once.  Every CTA reads the others' histograms through
// distributed shared memory, receives the whole list and decides by itself:
// one cluster barrier per exchange, and no decision is sent back.
//
// Threads hold consecutive tokens (loads from memory are made in order all
// the same and scattered into shared memory), so that a warp's scan of its
// lanes' sums is a scan by index.
//
// No one thing bounds it: 64 rows of 131072 f32 logits with mixed filters fill 35 %
// of the issue slots, and warps wait at barriers most; 256 rows of 50001 with a
// nucleus fill 50 %.  64 rows without filters take 35 us, of which reading them is
// 5, and reading, the maximum and the barriers are 20 (the likeliest token alone);
// the exact pass issues 45 instructions a token.  With top-k 50 34 us, with a
// nucleus of 0.9 63 us (196 with a histogram of exact weights over the whole row).
// One row: 13, 15 and 23 us, about 8 us of which are 5 to 7 barriers and what
// follows them (with cold inputs, launch and events included); clusters of 16 CTAs
// made that 13, 15 and 24.  What a larger top-k leaves is marked in a word of bits a
// thread, and later passes look at marked tokens only.
#include <type_traits>

#include "rq_device.cuh"
#include "rq_elem.cuh"
#include "rq_internal.h"

namespace rq {

namespace {

constexpr int kSThreads = 512;
constexpr int kSWarps = kSThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kParts = kMaxCluster * kSWarps;
constexpr int kBins = 512;           // one a thread
constexpr int kFine = 128;           // of what is divided further
constexpr int kList = 128;           // tokens that are ranked one by one
constexpr int kSort = kSThreads;     // tokens that top-k leaves and that are sorted
constexpr int kTable = 512;
constexpr float kFar = 43.0f * kTable;  // 2^42 2^-y/512 is below 1 from 42 octaves on
constexpr int kCacheBytes = 176 * 1024;  // of a row's part, at most

// 2^(42 - j/512).
struct PowerTable {
  unsigned long long t[kTable];
  constexpr PowerTable() : t() {
    for (int j = 0; j < kTable; ++j) {
      // e^-x by its series, x < ln 2: the 24th term is below 2^-90
      const double x = 0.693147180559945309417 * j / kTable;
      double term = 1.0, sum = 1.0;
      for (int i = 1; i <= 24; ++i) {
        term *= -x / i;
        sum += term;
      }
      t[j] = (unsigned long long)(sum * 4398046511104.0 + 0.5);
    }
  }
};
__device__ const PowerTable g_power;

// A bin of a CTA's histogram as the others read it.
struct __align__(16) Bin {
  unsigned long long w;
  unsigned int n, unused;
};

struct SampleShared {
  unsigned long long power[kTable];
  // this CTA's histograms: of the row (the last: tokens of no bin), and of what
  // is divided
  unsigned int count[kBins + 1], count_fine[kFine];
  Bin bins[kFine];
  // sums of the weights' bits 0 .. 13, 14 .. 27 and 28 .. 42: up to 2^18 - 1
  // tokens a CTA do not wrap them, and nothing is carried between atomics
  unsigned int weight[3][kFine];
  unsigned long long sums[2][kParts];
  // this CTA's tokens of the lists: those that are ranked for top-k's and the
  // nucleus' cut, and those that are sorted
  unsigned long long found[2 * kList + kSort];
  unsigned long long list[kSort], list_w[kSort];
  unsigned long long cut;              // tokens from this order on stay
  unsigned long long tmp_w[kSWarps];
  unsigned long long above_w, total, goal;
  unsigned int tmp_n[kSWarps];
  unsigned int key_min[kMaxCluster], key_max[kMaxCluster];
  float top[kMaxCluster];
  float tmp_f[2][kSWarps];
  int first[kMaxCluster];
  unsigned int above_n, bin_n;
  unsigned int pushed[3];
  int bin, bin_last, equal;
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
// (After a cluster barrier; no clobber, so that several are in flight.)
__device__ __forceinline__ uint32_t get_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(p, rank)));
  return v;
}
__device__ __forceinline__ unsigned long long get_u64(const void* p, uint32_t rank) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_rank(p, rank)));
  return v;
}
__device__ __forceinline__ Bin get_bin(const Bin* p, uint32_t rank) {
  Bin b;
  asm volatile("{.reg .b32 u; ld.shared::cluster.v4.b32 {%0, %1, %2, u}, [%3];}"
               : "=r"(reinterpret_cast<unsigned int*>(&b.w)[0]),
                 "=r"(reinterpret_cast<unsigned int*>(&b.w)[1]), "=r"(b.n)
               : "r"(map_rank(p, rank)));
  return b;
}
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
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

// Tokens in order as unsigned integers: larger logits, then smaller indices.
__device__ __forceinline__ unsigned long long order_of(int v, float l) {
  return (unsigned long long)key_of(l) << 32 | (0xFFFFFFFFu - (unsigned int)v);
}
__device__ __forceinline__ int index_of(unsigned long long order) {
  return (int)(0xFFFFFFFFu - (unsigned int)order);
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

// A row's scale: y = (top - l) (ch + cl).
struct Scale {
  float top;
  // 1, or for a temperature past 2^90 a small power of two that keeps
  // differences of any two floats finite and ch normal
  float pre;
  float near, ch, cl;  // top pre; 512 log2(e) / T / pre
  const unsigned long long* power;

  __device__ __forceinline__ void set(float t) {
    if (top == INFINITY) {
      // next to +Inf nothing finite weighs anything: near - l pre is -Inf for
      // it, y 0, and beyond kFar for all others
      pre = 0.5f;
      near = 3.0e38f;
      ch = 1.0f;
      cl = 0.0f;
      return;
    }
    pre = t > 0x1p90f ? 0x1p-64f : 1.0f;
    near = top * pre;
    // 512 log2(e) as a sum of two floats, over t
    const float kh = t > 0x1p90f ? 738.65985107421875f * 0x1p64f : 738.65985107421875f;
    const float kl = t > 0x1p90f ? 9.860930513e-6f * 0x1p64f : 9.860930513e-6f;
    ch = __fdiv_rn(kh, t);
    cl = t < INFINITY ? __fdiv_rn(fmaf(-ch, t, kh) + kl, t) : 0.0f;
  }

  // y's larger part, 0 .. kFar (never rises with l); a NaN gives kFar.  (Products
  // that decide a bin are rounded by themselves: fused into what follows them in
  // one pass and not in another, a token would be counted in one bin and listed
  // in its neighbour.)
  __device__ __forceinline__ float far(float l) const {
    return fmaxf(fminf(__fmul_rn(fmaf(-l, pre, near), ch), kFar), 0.0f);
  }

  // W, and far(l).
  __device__ __forceinline__ unsigned long long weight(float l, float& ph) const {
    // (top - l) pre = s + e exactly
    const float lp = l * pre;
    const float s = fmaf(-l, pre, near), t = s - near;
    const float e = (near - (s - t)) - (lp + t);
    const float yh = __fmul_rn(s, ch);
    const float pl = fmaf(e, ch, fmaf(s, cl, fmaf(s, ch, -yh)));
    // (-Inf and NaN: kFar, weight 0, whatever the rest below)
    ph = fmaxf(fminf(yh, kFar), 0.0f);
    // the nearest whole number, by the addition of 1.5 2^23
    const float mf = ph + 12582912.0f;
    const unsigned int m = __float_as_uint(mf) - 0x4B400000u;
    const float z = (ph - (mf - 12582912.0f)) + pl;
    // 1 - 2^(-z/512) = z (k1 - z (k2 - z k3)), k_i = (ln 2 / 512)^i / i!
    constexpr float k1 = 1.35380308703114e-3f, k2 = 9.16391399231e-7f, k3 = 4.1353784e-10f;
    const float q = z * fmaf(-z, fmaf(-z, k3, k2), k1);
    const unsigned long long p = power[m & (kTable - 1)];
    // 2^31 2^(-j/512) to 2^-25 of itself
    const float pf = __uint2float_rn((unsigned int)(p >> 11));
    const int d = __float2int_rn(pf * (q * 0x1p10f));  // halves: 31 bits (a NaN: 0)
    return (p - 2ll * d) >> (m / kTable);
  }

  // 2^-42 W.  Up to kWhole octaves, where W's fraction is below 2^-26 of it, from
  // the special function unit: its power of two is within 2^-22 and the correction
  // rounds once.  Beyond, W itself.
  static constexpr int kWhole = 16;
  __device__ __forceinline__ float share(float l) const {
    const float lp = l * pre;
    const float s = fmaf(-l, pre, near), t = s - near;
    const float e0 = (near - (s - t)) - (lp + t);
    const float yh = __fmul_rn(s, ch);
    const float pl = fmaf(e0, ch, fmaf(s, cl, fmaf(s, ch, -yh)));
    const float ph = fmaxf(fminf(yh, kFar), 0.0f);
    if (ph >= (float)(kWhole * kTable)) {
      float y;
      return __ull2float_rn(weight(l, y)) * 0x1p-42f;
    }
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(ph * (-1.0f / kTable)));
    // (pl is no number where y is none)
    return ph > 0.0f ? fmaf(e, pl * -1.35380308703114e-3f, e) : 1.0f;
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
  int groups;       // 16-byte groups of logits that a thread holds
  int pitch;        // groups between two threads' in shared memory: odd
  Divisor by;       // groups
};

// One cluster's row.  The row is read in aligned 16-byte groups: place 0 is the
// first logit of the group that holds token 0, and token v stands at place
// v + skew.  Everything but the row's parts is the same in every CTA after each
// exchange, so that all take the same branches.
template <typename T, bool kCached>
struct RowSampler {
  static constexpr int kPer = 16 / (int)sizeof(T);  // logits of a group
  SampleShared& sh;
  uint4* cache;            // this CTA's part of the row (kCached)
  const T* row;
  const SampleArgs& a;
  int rank, ranks, tid, lane, warp;
  int skew;
  int first;               // this thread's first place, in groups
  Scale scale;
  unsigned long long least;  // weights below it are left out (min-p)
  bool marked;               // `marks` are this thread's tokens that may stay
  unsigned long long marks;
  bool has_cut;
  float cut_l;             // tokens of a larger logit stay, and of this one
  int cut_v;               // those up to this index

  // A group from memory; -Inf where the row is not.
  __device__ __forceinline__ uint4 load(int group) const {
    const int v0 = group * kPer - skew;
    if (v0 >= 0 && v0 + kPer <= a.vocab) return *reinterpret_cast<const uint4*>(row + v0);
    alignas(16) T t[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      t[i] = v0 + i >= 0 && v0 + i < a.vocab ? row[v0 + i] : float_elem<T>(-INFINITY);
    return *reinterpret_cast<const uint4*>(t);
  }

  __device__ __forceinline__ uint4 read(int i) const {
    if constexpr (kCached) return cache[(warp * 32 + lane) * a.pitch + i];
    return load(first + i);
  }

  // f(token, logit) over this thread's tokens, in order; outside the row the
  // logit is -Inf.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int i = 0; i < a.groups; ++i) {
      const uint4 g = read(i);
      const T* t = reinterpret_cast<const T*>(&g);
      const int v = (first + i) * kPer - skew;
#pragma unroll
      for (int j = 0; j < kPer; ++j) f(v + j, elem_float(t[j]));
    }
  }

  // f over the tokens that are marked, which are few; over all of them where
  // none are marked yet or a thread has more than there are marks.
  template <typename F>
  __device__ __forceinline__ void some(F f) const {
    if (!marked) {
      each(f);
    } else {
      for (unsigned long long m = marks; m != 0ull; m &= m - 1ull) {
        const int i = __ffsll((long long)m) - 1;
        f(first * kPer - skew + i, one(lane, i));
      }
    }
  }
  __device__ __forceinline__ bool can_mark() const { return a.groups * kPer <= 64; }
  // A token's mark.
  __device__ __forceinline__ unsigned long long mark_of(int v) const {
    return 1ull << ((v + skew - first * kPer) & 63);
  }

  // One logit of this warp's thread q.
  __device__ __forceinline__ float one(int q, int i) const {
    if constexpr (kCached) {
      const T* t = reinterpret_cast<const T*>(cache + (warp * 32 + q) * a.pitch);
      return elem_float(t[i]);
    } else {
      const int v = (first + (q - lane) * a.groups) * kPer + i - skew;
      return v >= 0 && v < a.vocab ? elem_float(row[v]) : -INFINITY;
    }
  }

  // The row into shared memory, with the table's power of this thread, and the
  // row's largest logit.
  __device__ __forceinline__ float fill(unsigned long long power) {
    const int mine = first - lane * a.groups;  // the warp's first group
    if constexpr (kCached) {
      for (int i = lane; i < 32 * a.groups; i += 32) {
        const int q = (int)quotient((uint32_t)i, a.by);
        uint4* to = cache + (warp * 32 + q) * a.pitch + (i - q * a.groups);
        const int v0 = (mine + i) * kPer - skew;
        if (v0 >= 0 && v0 + kPer <= a.vocab)
          copy16(to, row + v0);
        else
          *to = load(mine + i);
      }
      sh.power[tid] = power;
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    } else {
      sh.power[tid] = power;
    }
    float most = -INFINITY;
    each([&](int, float l) { most = fmaxf(most, l); });  // (a NaN is passed over)
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
      if (l == scale.top) at = min(at, v);
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
    float y;
    const unsigned long long w = scale.weight(l, y);
    return least > 1ull && w < least ? 0ull : w;
  }

  // A token's place in the first histogram: bin (int)place(l), kBins (or
  // more by a rounding) for tokens of no weight.
  __device__ __forceinline__ static float place_of(float far) {
    return __fmul_rn(far, kBins / kFar);
  }
  __device__ __forceinline__ float place(float l) const { return place_of(scale.far(l)); }
  // Its bin in one that divides the bins [b0, b0 + kFine / step) finer.
  __device__ __forceinline__ static int finer(float x, int b0, float step) {
    return min((int)__fmul_rn(__fsub_rn(x, (float)b0), step), kFine - 1);
  }

  __device__ __forceinline__ void enter(int bin, unsigned long long w) const {
    atomicAdd(&sh.count_fine[bin], 1u);
    atomicAdd(&sh.weight[0][bin], (unsigned int)w & 0x3FFFu);
    atomicAdd(&sh.weight[1][bin], (unsigned int)(w >> 14) & 0x3FFFu);
    atomicAdd(&sh.weight[2][bin], (unsigned int)(w >> 28));
  }

  // The finer histogram; seen by the cluster after its barrier, and cleared
  // again only after another one that follows every CTA's last look at it.
  __device__ __forceinline__ void clear() const {
    if (tid < kFine)
      sh.count_fine[tid] = sh.weight[0][tid] = sh.weight[1][tid] = sh.weight[2][tid] = 0u;
    __syncthreads();
  }
  // (before the barrier, where weights were entered)
  __device__ __forceinline__ void gather() const {
    __syncthreads();
    if (tid < kFine)
      sh.bins[tid] = Bin{sh.weight[0][tid] + ((unsigned long long)sh.weight[1][tid] << 14) +
                             ((unsigned long long)sh.weight[2][tid] << 28),
                         sh.count_fine[tid], 0u};
  }

  // f(rank), each CTA beginning with its own, so that not all read one at a time.
  template <typename F>
  __device__ __forceinline__ void each_rank(F f) const {
    int q = rank;
#pragma unroll 4
    for (int i = 0; i < ranks; ++i) {
      f(q);
      q = q + 1 < ranks ? q + 1 : 0;
    }
  }

  // Counts of the row's tokens by place.
  __device__ __forceinline__ void count_places() const {
    sh.count[tid] = 0u;
    __syncthreads();
    each([&](int, float l) { atomicAdd(&sh.count[min((int)place(l), kBins)], 1u); });
    cluster_sync();
  }

  // The bin of the row's counts, or of the finer histogram, in which the
  // running count reaches `goal` (by_weight: the running weight), after n0
  // tokens of weight w0: bin (-1: none), bin_n, above_n, above_w.
  __device__ __forceinline__ void find(bool fine, bool by_weight, unsigned long long goal,
                                       uint32_t n0, unsigned long long w0) {
    uint32_t n = 0;
    unsigned long long w = 0;
    if (fine && tid >= kFine)
      ;  // (no such bin)
    else if (by_weight)
      each_rank([&](int q) {
        const Bin b = get_bin(&sh.bins[tid], q);
        n += b.n;
        w += b.w;
      });
    else {
      const unsigned int* c = fine ? &sh.count_fine[tid] : &sh.count[tid];
      each_rank([&](int q) { n += get_u32(c, q); });
    }
    const uint32_t scan_n = warp_scan_add(n, lane);
    const unsigned long long scan_w = by_weight ? warp_scan_add(w, lane) : 0ull;
    if (lane == 31) {
      sh.tmp_n[warp] = scan_n;
      sh.tmp_w[warp] = scan_w;
    }
    if (tid == 0) sh.bin = -1;
    __syncthreads();
    uint32_t run_n = n0 + scan_n - n;
    unsigned long long run_w = w0 + scan_w - w;
    for (int q = 0; q < warp; ++q) {
      run_n += sh.tmp_n[q];
      run_w += sh.tmp_w[q];
    }
    const unsigned long long before = by_weight ? run_w : run_n;
    if (before < goal && goal <= before + (by_weight ? w : n)) {
      sh.bin = tid;
      sh.above_n = run_n;
      sh.above_w = run_w;
      sh.bin_n = n;
    }
    __syncthreads();
  }

  // The bins [bin, bin_last] of the counts in which a nucleus of top_p ends.
  // kSure: in which it can end at all, between bounds of the weights before each
  // bin, its own from its edges, a thousandth for roundings on either side
  // (about a tenth of the tokens).  Else where it ends if every token weighs
  // its bin's mean, and the neighbour that is nearer than a quarter of a bin: a
  // bin or two, and if the exact sums say otherwise the search is repeated.
  // `last` is top-k's bin.
  template <bool kSure>
  __device__ __forceinline__ void bracket(float top_p, int last) {
    uint32_t n = 0;
    each_rank([&](int q) { n += get_u32(&sh.count[tid], q); });
    constexpr float kOctaves = kFar / (kBins * kTable);
    const float upper = exp2f(-kOctaves * (float)tid) * (kSure ? 1.001f : 0.9712f);
    const float lower = kSure ? exp2f(-kOctaves * (float)(tid + 1)) * 0.999f : upper;
    const float floor = __ull2float_rn(least) * 0x1p-42f;
    const float most = tid <= last && upper >= floor ? (float)n * upper : 0.0f;
    const float fewest =
        tid <= last - (kSure ? 1 : 0) && lower >= floor ? (float)n * lower : 0.0f;
    float run_most = warp_scan_add(most, lane), run_fewest = warp_scan_add(fewest, lane);
    if (lane == 31) {
      sh.tmp_f[0][warp] = run_most;
      sh.tmp_f[1][warp] = run_fewest;
    }
    if (tid == 0) {
      sh.bin = kBins - 1;
      sh.bin_last = 0;
    }
    __syncthreads();
    float all_most = 0.0f, all_fewest = 0.0f;
    for (int q = 0; q < kSWarps; ++q) {
      if (q == warp) {
        run_most += all_most;
        run_fewest += all_fewest;
      }
      all_most += sh.tmp_f[0][q];
      all_fewest += sh.tmp_f[1][q];
    }
    const float p = fmaxf(top_p, 0.0f);
    if constexpr (kSure) {
      if (run_most * 1.001f >= p * all_fewest) atomicMin(&sh.bin, tid);
      if ((run_fewest - fewest) * 0.999f < p * all_most * 1.001f) atomicMax(&sh.bin_last, tid);
    } else {
      const float goal = p * all_most;
      if (run_most + 0.25f * most >= goal) atomicMin(&sh.bin, tid);
      if (run_most - 1.25f * most < goal) atomicMax(&sh.bin_last, tid);
    }
    __syncthreads();
  }

  // Lists in every CTA the n tokens for which in_list(l) holds, and their
  // weights.  (A CTA's own part is read by the others until their next cluster
  // barrier.)
  template <typename F>
  __device__ __forceinline__ void list(F in_list, int which, int n) {
    some([&](int v, float l) {
      if (in_list(l))
        sh.found[which * kList + atomicAdd(&sh.pushed[which], 1u)] = order_of(v, l);
    });
    cluster_sync();
    const uint32_t mine = lane < ranks ? get_u32(&sh.pushed[which], lane) : 0u;
    int i = tid, q = 0;
    for (int x = 0; x < ranks - 1; ++x) {
      const int c = (int)__shfl_sync(0xFFFFFFFFu, mine, x);
      if (q == x && i >= c) {
        i -= c;
        ++q;
      }
    }
    if (tid < n) {
      const unsigned long long o = get_u64(&sh.found[which * kList + i], q);
      sh.list[tid] = o;
      sh.list_w[tid] = weight_kept(float_of((uint32_t)(o >> 32)));
    }
    __syncthreads();
  }

  // Of n listed tokens, the one at which the count (the weight) reaches
  // `goal`, after above_n tokens of weight above_w: sh.cut, and sh.total, the
  // weight up to it.
  __device__ __forceinline__ void rank_list(int n, bool by_weight, unsigned long long goal,
                                            uint32_t above_n, unsigned long long above_w) {
    constexpr int g = kSThreads / kList;  // threads to a token
    const int i = tid / g;
    uint32_t before_n = 0;
    unsigned long long before_w = 0;
    if (i < n) {
      const unsigned long long o = sh.list[i];
#pragma unroll 4
      for (int j = tid % g; j < n; j += g) {
        const bool before = sh.list[j] > o;
        before_n += before ? 1u : 0u;
        before_w += before ? sh.list_w[j] : 0ull;
      }
    }
#pragma unroll
    for (int o = 1; o < g; o *= 2) {
      before_n += __shfl_xor_sync(0xFFFFFFFFu, before_n, o);
      before_w += __shfl_xor_sync(0xFFFFFFFFu, before_w, o);
    }
    if (i < n && tid % g == 0) {
      before_w += above_w;
      before_n += above_n;
      const unsigned long long b = by_weight ? before_w : before_n;
      const unsigned long long mine = by_weight ? sh.list_w[i] : 1ull;
      if (b < goal && goal <= b + mine) {
        sh.cut = sh.list[i];
        sh.total = before_w + sh.list_w[i];
      }
    }
    __syncthreads();
  }

  // Of more equal logits than the list holds, the one at which the goal is
  // reached: the m-th by index.
  __device__ __forceinline__ void rank_equal(uint32_t key, bool by_weight,
                                             unsigned long long goal) {
    const float l = float_of(key);
    const unsigned long long w = weight_kept(l);
    const unsigned long long m = by_weight ? (goal - sh.above_w + w - 1) / w : goal - sh.above_n;
    uint32_t mine = 0;
    each([&](int, float x) { mine += x == l ? 1u : 0u; });
    const uint32_t upto = warp_scan_add(mine, lane);
    exchange(__shfl_sync(0xFFFFFFFFu, upto, 31));
    unsigned long long all, before = parts_before(0, &all);
    before += upto - mine;
    if (before < m && m <= before + mine) {
      each([&](int v, float x) {
        if (x == l && ++before == m)
          for (int q = 0; q < ranks; ++q) put_u32(&sh.equal, q, (uint32_t)v);
      });
    }
    cluster_sync();
    if (tid == 0) {
      sh.cut = order_of(sh.equal, l);
      sh.total = sh.above_w + m * w;
    }
    __syncthreads();
  }

  // Every warp's sum to every CTA.
  __device__ __forceinline__ void exchange(unsigned long long sum) {
    if (lane < ranks) put_u64(&sh.sums[0][rank * kSWarps + warp], lane, sum);
    cluster_sync();
  }
  // The sums of the warps before this one, and of all.
  __device__ __forceinline__ unsigned long long parts_before(int which,
                                                             unsigned long long* all) const {
    constexpr int kEach = kParts / 32;
    const int me = rank * kSWarps + warp;
    unsigned long long before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int q = lane + 32 * i;
      const unsigned long long s = q < ranks * kSWarps ? sh.sums[which][q] : 0ull;
      total += s;
      before += q < me ? s : 0ull;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
      before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    }
    *all = total;
    return before;
  }

  // Where the running count (weight) reaches the goal within `bin` of a
  // histogram by bin_of, of which sh.bin_n tokens are in that bin after
  // sh.above_n of weight sh.above_w: sh.cut, and sh.total, the weight up to it.
  // (Divided further in the same buffer: the exchange of the range stands
  // between the last look at it and the next use.)
  template <typename F>
  __device__ __forceinline__ void resolve(F bin_of, bool by_weight, unsigned long long goal) {
    const int which = by_weight ? 1 : 0;
    const int bin = sh.bin;
    const int n = (int)sh.bin_n;
    if (n <= kList) {
      list([&](float l) { return bin_of(l) == bin; }, which, n);
      rank_list(n, by_weight, goal, sh.above_n, sh.above_w);
      return;
    }
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    some([&](int, float l) {
      if (bin_of(l) == bin) {
        lo = min(lo, key_of(l));
        hi = max(hi, key_of(l));
      }
    });
    for (;;) {
      // the range of what is left; none of its tokens may be this warp's
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
        rank_equal(lo, by_weight, goal);
        return;
      }
      const uint32_t klo = lo, khi = hi;
      int shift = 0;
      while (((khi - klo) >> shift) >= (uint32_t)kFine) ++shift;
      const auto bits = [=](float l) {
        const uint32_t k = key_of(l);
        return k >= klo && k <= khi ? (int)((khi - k) >> shift) : -1;
      };
      const uint32_t above_n = sh.above_n;
      const unsigned long long above_w = sh.above_w;
      clear();
      some([&](int, float l) {
        const int x = bits(l);
        if (x < 0) return;
        if (by_weight)
          enter(x, weight_kept(l));
        else
          atomicAdd(&sh.count_fine[x], 1u);
      });
      if (by_weight) gather();
      cluster_sync();
      find(true, by_weight, goal, above_n, above_w);
      const int b = sh.bin;
      const int left = (int)sh.bin_n;
      if (left <= kList) {
        list([&](float l) { return bits(l) == b; }, which, left);
        rank_list(left, by_weight, goal, sh.above_n, sh.above_w);
        return;
      }
      lo = 0xFFFFFFFFu;
      hi = 0u;
      some([&](int, float l) {
        if (bits(l) == b) {
          lo = min(lo, key_of(l));
          hi = max(hi, key_of(l));
        }
      });
    }
  }

  // Top-k's cut, in bin b of the counts.
  __device__ __forceinline__ void cut_count(int b, unsigned long long k) {
    const auto bin_of = [this, b](float l) {
      const float x = place(l);
      return (int)x == b ? finer(x, b, (float)kFine) : -1;
    };
    const uint32_t above_n = sh.above_n;
    clear();
    marks = 0;
    each([&](int v, float l) {
      const float x = place(l);
      if ((int)x <= b) marks |= mark_of(v);
      if ((int)x == b) atomicAdd(&sh.count_fine[finer(x, b, (float)kFine)], 1u);
    });
    marked = can_mark();
    cluster_sync();
    find(true, false, k, above_n, 0ull);
    resolve(bin_of, false, k);
  }

  // The nucleus' cut among the bins [b0, b1] of the counts, or false.  *mine:
  // this thread's weight of the bins before b0.
  __device__ __forceinline__ bool cut_weight(int b0, int b1, float top_p,
                                             unsigned long long* mine) {
    const float step = (float)kFine / (float)(b1 - b0 + 1);
    const auto bin_of = [=](float l) {
      const float x = place(l);
      const int b = (int)x;
      return b >= b0 && b <= b1 ? finer(x, b0, step) : -1;
    };
    clear();
    unsigned long long above = 0, all = 0, ends = 0;
    const auto take = [&](int v, float l, auto plain) {
      float y;
      unsigned long long w = scale.weight(l, y);
      if (!plain.value && (w < least || (has_cut && !before_cut(v, l)))) w = 0ull;
      const float x = place_of(y);
      const int b = (int)x;
      all += w;
      above += b < b0 ? w : 0ull;
      if (b >= b0 && b <= b1) {
        enter(finer(x, b0, step), w);
        ends |= mark_of(v);
      }
    };
    if (has_cut || least > 1ull)
      some([&](int v, float l) { take(v, l, std::false_type()); });
    else
      each([&](int v, float l) { take(v, l, std::true_type()); });
    unsigned long long rest = all - above;
    gather();
    *mine = above;
    above = __shfl_sync(0xFFFFFFFFu, warp_scan_add(above, lane), 31);
    rest = __shfl_sync(0xFFFFFFFFu, warp_scan_add(rest, lane), 31);
    if (lane < ranks) put_u64(&sh.sums[1][rank * kSWarps + warp], lane, rest);
    exchange(above);
    unsigned long long before, others;
    parts_before(0, &before);
    parts_before(1, &others);
    if (tid == 0)
      sh.goal = max(1ull, (unsigned long long)ceil((double)fmaxf(top_p, 0.0f) *
                                                   (double)(before + others)));
    __syncthreads();
    const unsigned long long goal = sh.goal;
    find(true, true, goal, 0u, before);
    if (sh.bin < 0) return false;
    marks = ends;
    marked = can_mark();
    resolve(bin_of, true, goal);
    return true;
  }

  // The nucleus' cut, top-k's in bin `last` (or none).  Returns this thread's
  // weight of what stays.
  __device__ __forceinline__ unsigned long long cut_nucleus(float top_p, int last, bool draws) {
    bracket<false>(top_p, last);
    int b0 = sh.bin, b1 = max(sh.bin, sh.bin_last);
    unsigned long long mine;
    if (!cut_weight(b0, b1, top_p, &mine)) {
      cluster_sync();  // (the finer histogram has been read)
      bracket<true>(top_p, last);
      b0 = sh.bin;
      b1 = max(sh.bin, sh.bin_last);
      if (!cut_weight(b0, b1, top_p, &mine)) {
        // (not reached while the bounds' thousandth covers their roundings)
        cluster_sync();
        b0 = 0;
        b1 = kBins - 1;
        cut_weight(b0, b1, top_p, &mine);
      }
    }
    take_cut();
    if (draws)
      some([&](int v, float l) {
        const int b = (int)place(l);
        if (b >= b0 && b <= b1) mine += staying(v, l);
      });
    return mine;
  }

  __device__ __forceinline__ bool before_cut(int v, float l) const {
    return l > cut_l || (l == cut_l && v <= cut_v);
  }
  __device__ __forceinline__ unsigned long long staying(int v, float l) const {
    if (has_cut && !before_cut(v, l)) return 0ull;
    return weight_kept(l);
  }
  __device__ __forceinline__ void take_cut() {
    has_cut = true;
    cut_l = float_of((uint32_t)(sh.cut >> 32));
    cut_v = index_of(sh.cut);
  }
  // This thread's weight of what stays.
  __device__ __forceinline__ unsigned long long sum() const {
    unsigned long long mine = 0;
    if (has_cut || least > 1ull)
      some([&](int v, float l) { mine += staying(v, l); });
    else
      each([&](int, float l) {
        float y;
        mine += scale.weight(l, y);
      });
    return mine;
  }

  __device__ __forceinline__ static unsigned long long point_of(float u,
                                                                unsigned long long total) {
    unsigned int un = 0;
    if (u > 0.0f) un = (unsigned int)fminf(u * 0x1p24f, 16777215.0f);
    return un * (total >> 24) + ((un * (total & 0xFFFFFFull)) >> 24);
  }

  // The token that the random number meets; `mine` is this thread's weight of
  // the tokens that stay.
  __device__ __forceinline__ void draw(float u, int32_t* out, unsigned long long mine) {
    const unsigned long long upto = warp_scan_add(mine, lane);
    const unsigned long long sum = __shfl_sync(0xFFFFFFFFu, upto, 31);
    exchange(sum);
    unsigned long long total, before = parts_before(0, &total);
    const unsigned long long point = point_of(u, total);
    if (before > point || point >= before + sum) return;
    // in this warp's part: the thread that holds it, whose tokens the warp
    // then takes one each
    const int q = __ffs((int)__ballot_sync(0xFFFFFFFFu, before + upto > point)) - 1;
    before += __shfl_sync(0xFFFFFFFFu, upto - mine, q);
    const int v0 = (first + (q - lane) * a.groups) * kPer - skew;
    for (int i = 0; i < a.groups * kPer; i += 32) {
      const int at = i + lane;
      const float l = at < a.groups * kPer ? one(q, at) : -INFINITY;
      const unsigned long long w = staying(v0 + at, l);
      const unsigned long long run = before + warp_scan_add(w, lane);
      if (run - w <= point && point < run) *out = v0 + at;
      before = __shfl_sync(0xFFFFFFFFu, run, 31);
      if (before > point) break;
    }
  }

  // The same among n listed tokens, those up to the cut.
  __device__ __forceinline__ void draw_listed(int n, float u, int32_t* out) const {
    const unsigned long long point = point_of(u, sh.total), cut = sh.cut;
    constexpr int g = kSThreads / kList;
    const int i = tid / g;
    unsigned long long before = 0, mine = 0;
    int index = 0;
    if (i < n) {
      const unsigned long long o = sh.list[i];
      index = index_of(o);
      mine = o >= cut ? sh.list_w[i] : 0ull;
#pragma unroll 4
      for (int j = tid % g; j < n; j += g) {
        const unsigned long long oj = sh.list[j];
        before += oj >= cut && index_of(oj) < index ? sh.list_w[j] : 0ull;
      }
    }
#pragma unroll
    for (int o = 1; o < g; o *= 2) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    if (i < n && tid % g == 0 && before <= point && point < before + mine) *out = index;
  }

  // Sorts a value a thread over the first m threads (a power of two), largest
  // first: a bitonic network, by shuffles within a warp.
  __device__ __forceinline__ unsigned long long sorted(unsigned long long v, int m) const {
    for (int size = 2; size <= m; size *= 2)
      for (int stride = size / 2; stride > 0; stride /= 2) {
        unsigned long long other;
        if (stride < 32) {
          other = __shfl_xor_sync(0xFFFFFFFFu, v, stride);
        } else {
          sh.list[tid] = v;
          __syncthreads();
          other = sh.list[tid ^ stride];
          __syncthreads();
        }
        const bool larger = ((tid & stride) == 0) == ((tid & size) == 0);
        v = larger == (v > other) ? v : other;
      }
    return v;
  }

  // This thread's part of a running sum over the CTA, and the sum of all.
  __device__ __forceinline__ unsigned long long sum_before(unsigned long long w,
                                                           unsigned long long* all) {
    const unsigned long long scan = warp_scan_add(w, lane);
    __syncthreads();
    if (lane == 31) sh.tmp_w[warp] = scan;
    __syncthreads();
    unsigned long long before = scan - w, total = 0;
    for (int q = 0; q < kSWarps; ++q) {
      before += q < warp ? sh.tmp_w[q] : 0ull;
      total += sh.tmp_w[q];
    }
    *all = total;
    return before;
  }

  // Of n listed tokens, among which all of top-k's are: both cuts (sh.cut, and
  // sh.total, the weight of what stays), and for `draws` the token that the random
  // number meets.
  __device__ __forceinline__ void sort_list(int n, int k, float top_p, bool draws, float u,
                                            int32_t* out) {
    int m = 32;
    while (m < n) m *= 2;
    const unsigned long long o = sorted(tid < n ? sh.list[tid] : 0ull, m);
    unsigned long long w = tid < n && tid < k ? weight_kept(float_of((uint32_t)(o >> 32))) : 0ull;
    unsigned long long total;
    const unsigned long long before = sum_before(w, &total);
    if (tid == 0)
      sh.goal = top_p < 1.0f
                    ? max(1ull, (unsigned long long)ceil((double)fmaxf(top_p, 0.0f) *
                                                         (double)total))
                    : total;
    __syncthreads();
    const unsigned long long goal = sh.goal;
    if (before < goal && goal <= before + w) {
      sh.cut = o;
      sh.total = before + w;
    }
    if (!draws) {
      __syncthreads();
      return;
    }
    // by index
    if (before >= goal) w = 0ull;
    sh.list_w[tid] = w;
    const unsigned long long by_index = sorted(
        w != 0ull ? (o << 32 | (unsigned long long)tid) | 1ull << 63 : 0ull, m);
    __syncthreads();
    w = by_index != 0ull ? sh.list_w[(unsigned int)by_index] : 0ull;
    const unsigned long long run = sum_before(w, &total);
    const unsigned long long point = point_of(u, total);
    if (run <= point && point < run + w)
      *out = (int)(0x7FFFFFFFu - ((unsigned int)(by_index >> 32) & 0x7FFFFFFFu));
  }

  // p = weight / total; consecutive tokens by consecutive threads.  What a cut
  // leaves is likely, and nearly all of it takes share's short way (256 rows of
  // 50001, nuclei: 95.8 us, 102 by whole weights); in a whole row both ways meet in
  // most warps, and whole weights are faster (64 rows of 131072: 56.4 us, 66 by
  // share, 55.4 if share took its short way for every token, 12 % off where W is 1).
  __device__ __forceinline__ void write(float* p, bool summed) {
    unsigned long long total = sh.total;
    if (!summed) {
      exchange(__shfl_sync(0xFFFFFFFFu, warp_scan_add(sum(), lane), 31));
      parts_before(0, &total);
    }
    // 1 / total, rounded once: what the total's and the quotient's roundings left
    // out is put back
    const float whole = __ull2float_rn(total), q = __frcp_rn(whole);
    const float rest = __ll2float_rn((long long)(total - (unsigned long long)whole)) * q;
    const float inv = fmaf(q, fmaf(-whole, q, 1.0f) - rest, q);
    if (least > 1ull)
      each_place([&](int v, float l) { p[v] = __ull2float_rn(staying(v, l)) * inv; });
    else if (has_cut)
      each_place([&](int v, float l) {
        p[v] = before_cut(v, l) ? scale.share(l) * (0x1p42f * inv) : 0.0f;
      });
    else
      each_place([&](int v, float l) {
        float y;
        p[v] = __ull2float_rn(scale.weight(l, y)) * inv;
      });
  }

  // f(token, logit) over the warp's tokens, neighbours by neighbouring threads.
  template <typename F>
  __device__ __forceinline__ void each_place(F f) const {
    const int mine = (first - lane * a.groups) * kPer - skew;
    const int width = a.groups * kPer;
    for (int i = lane; i < 32 * width; i += 32) {
      const int v = mine + i;
      if (v < 0 || v >= a.vocab) continue;
      float l;
      if constexpr (kCached) {
        const int q = (int)quotient((uint32_t)(i / kPer), a.by);
        const T* t = reinterpret_cast<const T*>(cache + (warp * 32 + q) * a.pitch);
        l = elem_float(t[i - q * width]);
      } else {
        l = elem_float(row[v]);
      }
      f(v, l);
    }
  }
};

template <typename T, bool kCached, bool kProbs>
__global__ void __launch_bounds__(kSThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  SampleShared& sh = *reinterpret_cast<SampleShared*>(raw);
  uint4* cache = reinterpret_cast<uint4*>(raw + (sizeof(SampleShared) + 15) / 16 * 16);
  const int tid = threadIdx.x;
  if (tid < 3) sh.pushed[tid] = 0u;
  static_assert(kTable == kSThreads, "a power a thread");
  const unsigned long long power = g_power.t[tid];
  cluster_arrive();
  pdl_wait();
  pdl_trigger();
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t r = blockIdx.x / ranks;
  const int warp = tid >> 5, lane = tid & 31;
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  RowSampler<T, kCached> s{sh,   cache, row,  a,    rank, ranks, tid, lane, warp,
                           (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T)),
                           ((rank * kSWarps + warp) * 32 + lane) * a.groups};
  // (looked at after the row is on its way)
  float t = a.temperature != nullptr ? a.temperature[r] : 1.0f;
  int k = a.top_k != nullptr ? a.top_k[r] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[r] : 1.0f;
  const float min_p = a.min_p != nullptr ? a.min_p[r] : 0.0f;
  s.scale.top = s.fill(power);
  if (!(t > 0.0f)) k = 1;
  t = fmaxf(t, 0x1p-116f);  // (ch stays finite)
  float* p = a.p + r * a.vocab;
  if (!(s.scale.top > -INFINITY) || k == 1) {
    // nothing to draw from, or one token
    const int best = s.scale.top > -INFINITY ? s.likeliest() : -1;
    if constexpr (kProbs) {
      s.each_place([&](int v, float) { p[v] = v == best ? 1.0f : 0.0f; });
    } else if (rank == 0 && tid == 0) {
      a.token[r] = best;
    }
    return;
  }
  s.scale.set(t);
  s.scale.power = sh.power;
  s.least = 1ull;
  if (min_p > 0.0f)
    s.least = max(1ull, (unsigned long long)ceilf(fminf(min_p, 1.0f) * 0x1p42f));
  s.has_cut = false;
  s.marked = false;
  const bool nucleus = top_p < 1.0f;
  int last = kBins - 1;  // top-k's bin
  if (k > 1 || nucleus) s.count_places();
  if (k > 1) {
    s.find(false, false, (unsigned long long)k, 0u, 0ull);
    const int b = sh.bin;
    const int n = b < 0 ? kSort + 1 : (int)(sh.above_n + sh.bin_n);
    if (n <= kSort) {
      // all of what top-k leaves can be listed
      s.list([&](float l) { return (int)s.place(l) <= b; }, 2, n);
      cluster_arrive();  // (the lists' parts have been read)
      // few are ranked by comparing all pairs, more are sorted (64 rows of
      // 131072, top-k 50: 35 us by pairs, 37 sorted; one row, top-k 250,
      // nucleus and min-p: 21 us sorted, 24 by the searches below)
      const bool few = n <= kList;
      if (few) {
        s.rank_list(n, false, (unsigned long long)k, 0u, 0ull);
        if (nucleus) {
          if (tid == 0)
            sh.goal = max(1ull, (unsigned long long)ceil((double)fmaxf(top_p, 0.0f) *
                                                         (double)sh.total));
          __syncthreads();
          s.rank_list(n, true, sh.goal, 0u, 0ull);
        }
      }
      if constexpr (kProbs) {
        if (!few) s.sort_list(n, k, top_p, false, 0.0f, nullptr);
        s.take_cut();
        s.write(p, true);
      } else if (rank == 0) {
        if (few)
          s.draw_listed(n, a.u[r], a.token + r);
        else
          s.sort_list(n, k, top_p, true, a.u[r], a.token + r);
      }
      cluster_wait();
      return;
    }
    if (b >= 0) {
      last = b;
      s.cut_count(b, (unsigned long long)k);
      s.take_cut();
    }
    __syncthreads();  // (what was found has been read by every thread)
  }
  if (nucleus) {
    const unsigned long long mine = s.cut_nucleus(top_p, last, !kProbs);
    if constexpr (kProbs) {
      cluster_arrive();  // (the lists' parts have been read)
      s.write(p, true);
      cluster_wait();
    } else {
      s.draw(a.u[r], a.token + r, mine);
    }
    return;
  }
  if constexpr (!kProbs) {
    s.draw(a.u[r], a.token + r, s.sum());
  }
  if constexpr (kProbs)
    s.write(p, false);
}

template <typename T, bool kCached, bool kProbs>
rq_status launch_row(const SampleArgs& a, int rows, int ranks, cudaStream_t st) {
  constexpr size_t kShared = (sizeof(SampleShared) + 15) / 16 * 16;
  static_assert(kShared + kCacheBytes <= 227 * 1024, "shared memory of a CTA");
  const size_t smem = kShared + (kCached ? (size_t)a.pitch * kSThreads * 16 : 0);
  auto kernel = sample_kernel<T, kCached, kProbs>;
  static bool ready = false;
  if (!ready) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kShared + kCacheBytes)) != cudaSuccess)
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
  constexpr int kPer = 16 / (int)sizeof(T);
  // groups of a row, whatever its skew
  const int all = (a.vocab + 2 * (kPer - 1)) / kPer;
  // As many CTAs as two to an SM, at most 64 logits a thread (as many as are
  // marked), at least two groups: a larger cluster pays its barriers more
  // often (256 rows of 50001 16-bit logits, nucleus: 66 us with clusters of 2,
  // 84 with 4, 233 with 8; 64 rows of 131072: 100 with 8, 126 with 4).
  const auto groups_of = [&](int n) { return (all + n * kSThreads - 1) / (n * kSThreads); };
  int ranks = 1;
  while (ranks < kMaxCluster &&
         ((int64_t)rows * ranks < 2 * device_sm_count() || groups_of(ranks) * kPer > 64) &&
         groups_of(ranks) > 2)
    ranks *= 2;
  a.groups = (all + ranks * kSThreads - 1) / (ranks * kSThreads);
  a.pitch = a.groups | 1;
  a.by = divisor((uint32_t)a.groups);
  static_assert((1 << 20) / kMaxCluster + 64 * kSThreads < 1 << 18, "tokens of a CTA");
  const bool cached = (size_t)a.pitch * kSThreads * 16 <= (size_t)kCacheBytes;
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
