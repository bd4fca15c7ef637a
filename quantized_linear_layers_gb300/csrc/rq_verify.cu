// rq_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers (sm_103a).
//
// A draw from weights w: W_v = floor(min(w_v, 1) 2^36) as 64-bit integers,
// Z = sum W_v, point = floor(U Z / 2^24) with U = floor(u 2^24), and the token
// is the first v whose running sum exceeds the point.  Integers make the sum
// associative: the draw is the same however a row is cut up, and the scan
// over 10^5 entries neither drifts nor depends on the launch.  36 bits keep
// weights down to 1.5e-11 of 1 apart from zero while 2^20 of them still fit
// 64 bits.
//
// One cluster of 8 CTAs takes a sequence: each of its 128 warps sums its part
// of the row, every CTA receives all 128 sums through distributed shared
// memory, and finds the token by itself in the part that holds the point: one
// cluster barrier per draw, no scratch, no atomics across CTAs, one launch;
// the walk down a tree is a loop of draws inside it.
//
// Bound by steps one after another: 32 chains of 7 drafts take 5 us over 1000
// entries already (the drafts' test, the sum, the cluster barrier, and two
// searches by one warp that reads its part of the row again), and 10.5 over
// 131072, of which reading the rows is the rest (in a replayed graph; 11.4 with
// cold inputs and the host's call).  A tree's draws follow one another, about 3
// us each (6 trees of 40 drafts over 50001 entries, up to four draws: 13.2 us).
#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {

namespace {

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVCluster = 8;
constexpr int kMaxTree = 1024;

constexpr int kVParts = kVCluster * kVWarps;  // parts of a row, one a warp

struct VerifyShared {
  long long sums[2][kVParts];  // by draw parity and part
  int found[2];
  int first;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ unsigned int warp_sum_u(unsigned int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// What the next token is drawn from: p, max(p - q, 0), or p without one entry.
struct Row {
  const float* p;
  const float* q;  // null: no draft distribution
  int drop;        // entry counted as zero (-1: none)
};

// floor(min(w, 1) 2^36) in two halves of 18 bits, each as the bits of 2^23 + half:
// additions rounded towards zero cut the fraction off, and the rest t - half
// is exact.  (A conversion to 64-bit integers runs at a quarter of an
// addition's rate or less.)
constexpr unsigned int kHalfBase = 0x4B000000u;
__device__ __forceinline__ void halves(float w, unsigned int& hi, unsigned int& lo) {
  const float t = fminf(fmaxf(w, 0.0f), 1.0f) * 0x1p18f;  // a NaN becomes 0
  const float a = __fadd_rz(t, 0x1p23f);
  const float b = __fadd_rz((t - (a - 0x1p23f)) * 0x1p18f, 0x1p23f);
  hi = __float_as_uint(a);
  lo = __float_as_uint(b);
}

__device__ __forceinline__ float weight_of(const Row& row, int v) {
  const float p = __ldg(row.p + v);
  const float w = row.q != nullptr ? __fsub_rn(p, __ldg(row.q + v)) : p;
  return v == row.drop ? 0.0f : w;
}

__device__ __forceinline__ long long weight(const Row& row, int v) {
  unsigned int hi, lo;
  halves(weight_of(row, v), hi, lo);
  return ((long long)(hi - kHalfBase) << 18) + (long long)(lo - kHalfBase);
}

// A warp's sum of the weights of entries [v0, v1), sixteen loads a lane in
// flight.  A lane meets at most 2^20 / 128 / 32 entries and the padding of the
// last round: the sums of halves stay below 2^27, so that 32-bit sums of the
// raw bits, wrapping, still hold them.
template <bool Q>
__device__ __forceinline__ long long part_sum(const Row& row, int v0, int v1) {
  constexpr int kBatch = 16;
  unsigned int hi = 0u, lo = 0u, n = 0u;
  for (int v = v0 + (int)(threadIdx.x & 31); v - (int)(threadIdx.x & 31) < v1; v += 32 * kBatch) {
    float p[kBatch], q[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int x = v + 32 * i;
      p[i] = x < v1 ? __ldg(row.p + x) : 0.0f;
      q[i] = Q && x < v1 ? __ldg(row.q + x) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      float w = Q ? __fsub_rn(p[i], q[i]) : p[i];
      if (!Q && v + 32 * i == row.drop) w = 0.0f;
      unsigned int a, b;
      halves(w, a, b);
      hi += a;
      lo += b;
    }
    n += kBatch;
  }
  hi = warp_sum_u(hi - n * kHalfBase);  // below 2^32 over a warp's 8192 entries of 2^18
  lo = warp_sum_u(lo - n * kHalfBase);
  return ((long long)hi << 18) + (long long)lo;
}

__device__ __forceinline__ unsigned int unit24(float u) {
  if (!(u > 0.0f)) return 0u;
  return (unsigned int)fminf(u * 0x1p24f, 16777215.0f);
}

__device__ __forceinline__ int part_begin(int vocab, int part) {
  return (int)((long long)vocab * part / kVParts);
}

__device__ __forceinline__ long long warp_scan(long long s, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += x;
  }
  return s;
}

// One draw by the whole cluster; every thread of every CTA returns the token
// in *token, and whether the row has any weight.  `d` counts the draws of
// this launch: its parity picks the exchange buffers, which a CTA writes again
// only after the cluster barrier of draw d + 1, and every CTA reaches that
// one after its last read of draw d.
__device__ bool draw(VerifyShared& sh, const Row& row, float u, int vocab, int d, int* token) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = (int)cluster_rank() * kVWarps + warp;
  const int v0 = part_begin(vocab, part), v1 = part_begin(vocab, part + 1);
  const long long sum =
      row.q != nullptr ? part_sum<true>(row, v0, v1) : part_sum<false>(row, v0, v1);
  if (lane < kVCluster) {
    const uint32_t dst = map_rank(smem_u32(&sh.sums[d & 1][part]), (uint32_t)lane);
    asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(dst), "l"(sum) : "memory");
  }
  cluster_sync();
  if (warp == 0) {
    // the part that holds the point: lanes scan four parts each
    constexpr int kPer = kVParts / 32;
    long long s[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s[i] = sh.sums[d & 1][lane * kPer + i];
      mine += s[i];
    }
    const long long scan = warp_scan(mine, lane);
    const long long total = __shfl_sync(0xFFFFFFFFu, scan, 31);
    const long long un = unit24(u);
    const long long point = un * (total >> 24) + ((un * (total & 0xFFFFFF)) >> 24);
    int found = -1;
    if (total > 0) {
      const int at = __ffs((int)__ballot_sync(0xFFFFFFFFu, scan > point)) - 1;
      long long run = __shfl_sync(0xFFFFFFFFu, scan - mine, at);
      int p = at * kPer;
#pragma unroll
      for (int i = 0; i < kPer - 1; ++i) {
        const long long x = __shfl_sync(0xFFFFFFFFu, s[i], at);
        if (p == at * kPer + i && run + x <= point) {
          run += x;
          ++p;
        }
      }
      // narrow [a, b) to one entry: 32 runs of entries, one a lane, each time
      int a = part_begin(vocab, p), b = part_begin(vocab, p + 1);
      while (b - a > 1) {
        const int len = (b - a + 31) / 32;
        const int x0 = min(a + lane * len, b), x1 = min(x0 + len, b);
        long long w = 0;
#pragma unroll 8
        for (int x = x0; x < x1; ++x) w += weight(row, x);
        const long long sc = warp_scan(w, lane);
        const int l = __ffs((int)__ballot_sync(0xFFFFFFFFu, run + sc > point)) - 1;
        run += __shfl_sync(0xFFFFFFFFu, sc - w, l);
        const int na = min(a + l * len, b);
        b = min(na + len, b);
        a = na;
      }
      found = a;
    }
    if (lane == 0) sh.found[d & 1] = found;
  }
  __syncthreads();
  *token = sh.found[d & 1];
  return *token >= 0;
}

__global__ void __cluster_dims__(kVCluster, 1, 1) __launch_bounds__(kVThreads)
verify_chain_kernel(const int32_t* __restrict__ token, const float* __restrict__ p,
                    const float* __restrict__ q, const float* __restrict__ u,
                    int32_t* __restrict__ accepted, int32_t* __restrict__ next, int drafts,
                    int vocab) {
  __shared__ VerifyShared sh;
  pdl_wait();
  pdl_trigger();
  const int64_t b = blockIdx.x / kVCluster;
  const float* pb = p + b * (drafts + 1) * vocab;
  const float* qb = q + b * drafts * vocab;
  const float* ub = u + b * (drafts + 1);
  if (threadIdx.x == 0) sh.first = drafts;
  __syncthreads();
  for (int i = threadIdx.x; i < drafts; i += kVThreads) {
    const int x = token[b * drafts + i];
    bool keep = x >= 0 && x < vocab;
    if (keep) {
      const float px = __ldg(pb + (int64_t)i * vocab + x);
      const float t = q != nullptr ? __fmul_rn(ub[i], __ldg(qb + (int64_t)i * vocab + x)) : ub[i];
      keep = t < px;
    }
    if (!keep) atomicMin(&sh.first, i);
  }
  cluster_sync();  // also: every CTA of the cluster runs before the first remote store
  const int n = sh.first;
  Row row = {pb + (int64_t)n * vocab, nullptr, -1};
  if (n < drafts) {
    const int x = token[b * drafts + n];
    if (x >= 0 && x < vocab) {
      if (q != nullptr)
        row.q = qb + (int64_t)n * vocab;
      else
        row.drop = x;
    }
  }
  int y;
  const bool plain = row.q == nullptr && row.drop < 0;
  if (!draw(sh, row, ub[drafts], vocab, 0, &y) && !plain) {
    row.q = nullptr;
    row.drop = -1;
    draw(sh, row, ub[drafts], vocab, 1, &y);
  }
  if (threadIdx.x == 0 && cluster_rank() == 0) {
    accepted[b] = n;
    next[b] = y;
  }
}

__global__ void __cluster_dims__(kVCluster, 1, 1) __launch_bounds__(kVThreads)
verify_tree_kernel(const int32_t* __restrict__ token, const int32_t* __restrict__ parent,
                   const float* __restrict__ p, const float* __restrict__ u,
                   int32_t* __restrict__ accepted, int32_t* __restrict__ next,
                   int32_t* __restrict__ path, int drafts, int vocab) {
  __shared__ VerifyShared sh;
  __shared__ int tok[kMaxTree], par[kMaxTree];
  pdl_wait();
  pdl_trigger();
  const int64_t b = blockIdx.x / kVCluster;
  const float* pb = p + b * (drafts + 1) * vocab;
  const float* ub = u + b * (drafts + 1);
  for (int i = threadIdx.x; i < drafts; i += kVThreads) {
    tok[i] = token[b * drafts + i];
    const int pa = parent[b * drafts + i];
    par[i] = pa >= -1 && pa < i ? pa : -2;  // -2: never reached
  }
  cluster_sync();
  const bool lead = threadIdx.x == 0 && cluster_rank() == 0;
  int node = -1, count = 0, y = -1;
  for (int d = 0; d <= drafts; ++d) {
    const Row row = {pb + (int64_t)(node + 1) * vocab, nullptr, -1};
    if (!draw(sh, row, ub[node + 1], vocab, d, &y)) break;
    if (threadIdx.x == 0) sh.first = drafts;
    __syncthreads();
    for (int i = node + 1 + threadIdx.x; i < drafts; i += kVThreads)
      if (par[i] == node && tok[i] == y) atomicMin(&sh.first, i);
    __syncthreads();
    const int child = sh.first;
    if (child == drafts) break;
    if (lead) path[b * drafts + count] = child;
    node = child;
    ++count;
    __syncthreads();  // sh.first is read before it is set again
  }
  if (lead) {
    accepted[b] = count;
    next[b] = y;
  }
  if (cluster_rank() == 0)
    for (int i = count + threadIdx.x; i < drafts; i += kVThreads) path[b * drafts + i] = -1;
}

}  // namespace

rq_status launch_verify_chain(const int32_t* token, const float* p, const float* q,
                              const float* u, int32_t* accepted, int32_t* next, int batch,
                              int drafts, int vocab, cudaStream_t st) {
  return launch_kernel(verify_chain_kernel, dim3((unsigned)(batch * kVCluster)), dim3(kVThreads),
                       0, st, token, p, q, u, accepted, next, drafts, vocab);
}

rq_status launch_verify_tree(const int32_t* token, const int32_t* parent, const float* p,
                             const float* u, int32_t* accepted, int32_t* next, int32_t* path,
                             int batch, int drafts, int vocab, cudaStream_t st) {
  return launch_kernel(verify_tree_kernel, dim3((unsigned)(batch * kVCluster)), dim3(kVThreads),
                       0, st, token, parent, p, u, accepted, next, path, drafts, vocab);
}

}  // namespace rq
