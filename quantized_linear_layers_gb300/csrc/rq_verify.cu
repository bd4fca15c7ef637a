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
// One cluster of 8 CTAs takes a sequence: each CTA sums an eighth of the row,
// the eight sums cross through distributed shared memory, and the CTA that
// holds the point finds the token in its part.  No scratch, no atomics, one
// launch; the walk down a tree is a loop of draws inside it.
#include "rq_device.cuh"
#include "rq_internal.h"

namespace rq {

namespace {

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVCluster = 8;
constexpr int kMaxTree = 1024;

struct VerifyShared {
  long long totals[2][kVCluster];  // by draw parity and CTA
  int found[2];
  long long warp_sum[kVWarps];
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

__device__ __forceinline__ long long warp_sum_ll(long long v) {
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

__device__ __forceinline__ long long weight(const Row& row, int v) {
  float w = __ldg(row.p + v);
  if (row.q != nullptr) w = __fsub_rn(w, __ldg(row.q + v));
  if (v == row.drop || !(w > 0.0f)) return 0;
  return __float2ll_rz(fminf(w, 1.0f) * 0x1p36f);
}

__device__ __forceinline__ unsigned int unit24(float u) {
  if (!(u > 0.0f)) return 0u;
  return (unsigned int)fminf(u * 0x1p24f, 16777215.0f);
}

// One draw by the whole cluster; every thread of every CTA returns the token
// in *token, and whether the row has any weight.  `d` counts the draws of
// this launch (its parity picks the exchange buffers: a CTA writes buffer
// d & 1 again only after the cluster barrier of draw d + 1, which every CTA
// reaches after its last read of draw d).
__device__ bool draw(VerifyShared& sh, const Row& row, float u, int vocab, int d, int* token) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  // this warp's part: 32-entry chunks [c0, c1) of the row
  const int chunks = (vocab + 31) / 32;
  const int part = (int)rank * kVWarps + warp, parts = kVCluster * kVWarps;
  const int c0 = (int)((long long)chunks * part / parts);
  const int c1 = (int)((long long)chunks * (part + 1) / parts);
  long long sum = 0;
#pragma unroll 8
  for (int c = c0; c < c1; ++c) {
    const int v = c * 32 + lane;
    if (v < vocab) sum += weight(row, v);
  }
  sum = warp_sum_ll(sum);
  if (lane == 0) sh.warp_sum[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    const long long cta = warp_sum_ll(lane < kVWarps ? sh.warp_sum[lane] : 0);
    if (lane < kVCluster) {
      const uint32_t dst =
          map_rank(smem_u32(&sh.totals[d & 1][rank]), (uint32_t)lane);
      asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(dst), "l"(cta) : "memory");
    }
  }
  cluster_sync();
  long long before = 0, total = 0;
#pragma unroll
  for (int r = 0; r < kVCluster; ++r) {
    const long long s = sh.totals[d & 1][r];
    if (r < (int)rank) before += s;
    total += s;
  }
  const long long un = unit24(u);
  const long long point = un * (total >> 24) + ((un * (total & 0xFFFFFF)) >> 24);
  for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
  if (total > 0 && before <= point && point < before + sh.warp_sum[warp]) {
    // the token is in this warp's part (of one warp of the cluster)
    long long run = before;
    int found = -1;
    for (int c = c0; c < c1 && found < 0; ++c) {
      const int v = c * 32 + lane;
      long long s = v < vocab ? weight(row, v) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += x;
      }
      const unsigned int past = __ballot_sync(0xFFFFFFFFu, run + s > point);
      if (past != 0u) found = c * 32 + __ffs((int)past) - 1;
      run += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane < kVCluster) {
      const uint32_t dst = map_rank(smem_u32(&sh.found[d & 1]), (uint32_t)lane);
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(dst), "r"(found) : "memory");
    }
  }
  cluster_sync();
  *token = total > 0 ? sh.found[d & 1] : -1;
  return total > 0;
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
