// rq_api.cu -- the C ABI of librq.so: validation, context, caches, routing.
//
// Host-side counterpart of realizar 0.8.4 cublas_prefill/gemm.rs
// (get_or_cache_fp8_weight, cublas_prefill_fp8_gemm with its activation
// reuse, cublas_prefill_gemm's FP8 branch), cublas_prefill/mod.rs
// (cublas_gemm_threshold, gpu_absmax_device) and q6k_gemv_indexed.rs
// (null-pointer guard before any launch).  Every argument is checked here,
// before anything is launched; kernels never trap.
#include <cstdlib>
#include <cstring>
#include <map>
#include <tuple>
#include <vector>

#include "rq_internal.h"

namespace rq {

bool pdl_enabled() {
  static const bool on = [] {
    const char* e = std::getenv("RQ_PDL");
    return e == nullptr || std::atoi(e) != 0;
  }();
  return on;
}

int device_sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        n < 1)
      n = 1;
    cached[dev] = n;
  }
  return cached[dev];
}

}  // namespace rq

using namespace rq;

namespace {

bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

struct WeightKey {
  const void* w;
  int qtype, N, K;
  bool operator<(const WeightKey& o) const {
    return std::tie(w, qtype, N, K) < std::tie(o.w, o.qtype, o.N, o.K);
  }
};

struct WeightEntry {
  uint8_t* fp8 = nullptr;  // [N x K] E4M3, followed (256-aligned) by the scale
  float* deq = nullptr;
  size_t bytes = 0;
};

// FP8 weights of a group of linears that share an input, concatenated by
// rows: member i's rows start at starts[i]; its dequant scale is deq[i].
struct GroupEntry {
  uint8_t* fp8 = nullptr;
  float* deq = nullptr;
  int starts[RQ_MAX_GROUP + 1] = {0};
  size_t bytes = 0;
};

rq_status check_quant_shape(int qtype, int N, int K) {
  if (qtype != RQ_Q4K && qtype != RQ_Q6K) return RQ_ERR_QTYPE;
  if (N < 1 || K < 256 || K % 256 != 0) return RQ_ERR_SHAPE;
  return RQ_OK;
}

}  // namespace

// E4M3 codes of one activation, followed (256-aligned) by their scale, and what
// they were made of.
struct ActScratch {
  uint8_t* codes = nullptr;
  float* deq = nullptr;
  size_t cap = 0;
  bool valid = false;
  const float* x = nullptr;
  int M = 0, K = 0;
  uint64_t gen = 0;
  unsigned long long capture = 0;  // the capture that records the quantization
};

struct TraceSlot {
  cudaEvent_t start = nullptr, stop = nullptr;
  int kind = 0;
  int kernels = 1;  // kernels launched between the two events
};

struct rq_ctx {
  int device = 0;
  // kernel tracing
  bool trace_on = false;
  unsigned int trace_mask = (1u << RQ_TRACE_KINDS) - 1u;  // kinds that are traced
  int trace_cap = 0, trace_used = 0;
  std::vector<TraceSlot> trace;
  int threshold = 4;
  std::map<WeightKey, WeightEntry> weights;
  std::map<std::vector<WeightKey>, GroupEntry> groups;
  int64_t weight_bytes = 0;
  // Activation scratch of calls that run at once, and of captured ones: a
  // replay rewrites its codes at a time that the host does not see, so the two
  // share none.  Buffers that captured graphs may use live until destroy.
  ActScratch act[2];
  std::vector<uint8_t*> act_kept;
  uint32_t* absmax = nullptr;  // device word
  bool fused_ok = true;           // RQ_ONE_PASS_QUANT=0 keeps the two-kernel path
  int64_t fused_min = 1 << 20;    // fewer elements: two kernels (RQ_ONE_PASS_MIN)
  // at most this many elements: one cluster, one launch (RQ_CLUSTER_QUANT_MAX;
  // measured on GB300, the 16-SM cluster beats the two grid-wide kernels on
  // the 57 K elements of 16 tokens x 3584 and loses from ~230 K on)
  int64_t cluster_max = 1 << 17;
  uint32_t* slots = nullptr;      // per-CTA partial maxima of the two-kernel path
  unsigned long long* fused = nullptr;        // one-pass quantization barrier word
  unsigned long long* fused_slots = nullptr;  // and its per-CTA words (SM count)
  uint64_t gen = 1;  // activation cache generation
  int64_t hits = 0, misses = 0;
  AttnScratch attn;  // partial rows of split sequences
};

namespace {

cudaError_t record(cudaEvent_t ev, cudaStream_t st) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cs) == cudaSuccess && cs == cudaStreamCaptureStatusActive)
    return cudaEventRecordWithFlags(ev, st, cudaEventRecordExternal);
  return cudaEventRecord(ev, st);
}

// Brackets one kernel launch with a trace slot's events while tracing is on.
class TraceScope {
 public:
  TraceScope(rq_ctx* ctx, int kind, cudaStream_t st) : st_(st) {
    if (ctx != nullptr && ctx->trace_on && ((ctx->trace_mask >> kind) & 1u) != 0 &&
        ctx->trace_used < ctx->trace_cap) {
      slot_ = &ctx->trace[ctx->trace_used++];
      slot_->kind = kind;
      slot_->kernels = 1;
      record(slot_->start, st_);
    }
  }
  // the scope launches n kernels (default 1)
  void kernels(int n) {
    if (slot_ != nullptr) slot_->kernels = n;
  }
  ~TraceScope() {
    if (slot_ != nullptr) record(slot_->stop, st_);
  }
  TraceScope(const TraceScope&) = delete;
  TraceScope& operator=(const TraceScope&) = delete;

 private:
  TraceSlot* slot_ = nullptr;
  cudaStream_t st_;
};

}  // namespace

extern "C" {

int rq_abi_version(void) { return RQ_ABI_VERSION; }

const char* rq_status_string(rq_status s) {
  switch (s) {
    case RQ_OK: return "ok";
    case RQ_ERR_NULL: return "null pointer";
    case RQ_ERR_SHAPE: return "invalid shape or alignment";
    case RQ_ERR_QTYPE: return "unsupported quantization type";
    case RQ_ERR_NOT_CACHED: return "weight not cached";
    case RQ_ERR_ALLOC: return "allocation failed";
    case RQ_ERR_CUDA: return "CUDA error";
    case RQ_ERR_TIMEOUT: return "device pipeline wait timed out";
    case RQ_ERR_ARCH: return "device lacks sm_103 features";
    case RQ_ERR_INDEX: return "index outside its array on the device";
  }
  return "unknown status";
}

rq_status rq_ctx_create(rq_ctx** out) {
  if (out == nullptr) return RQ_ERR_NULL;
  *out = nullptr;
  rq_ctx* c = new (std::nothrow) rq_ctx();
  if (c == nullptr) return RQ_ERR_ALLOC;
  if (cudaGetDevice(&c->device) != cudaSuccess) {
    delete c;
    return RQ_ERR_CUDA;
  }
  const char* env = std::getenv("RQ_GEMM_THRESHOLD");
  if (env != nullptr) {
    const int v = std::atoi(env);
    if (v >= 1) c->threshold = v;
  }
  void* p = nullptr;
  if (cudaMalloc(&p, 256) != cudaSuccess) {
    delete c;
    return RQ_ERR_ALLOC;
  }
  c->absmax = static_cast<uint32_t*>(p);
  c->fused = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(p) + 192);
  if (cudaMemset(p, 0, 256) != cudaSuccess) {
    cudaFree(p);
    delete c;
    return RQ_ERR_CUDA;
  }
  const char* one_pass = std::getenv("RQ_ONE_PASS_QUANT");
  if (one_pass != nullptr && std::atoi(one_pass) == 0) c->fused_ok = false;
  // a small activation goes through the two plain kernels: measured on
  // GB300, the cooperative one-pass launch costs more than it saves there
  // (the 28-layer stack at 16 tokens: 2.32 ms per pass one-pass, 2.10 ms
  // with two kernels)
  if (const char* e = std::getenv("RQ_ONE_PASS_MIN")) c->fused_min = std::atoll(e);
  if (const char* e = std::getenv("RQ_CLUSTER_QUANT_MAX")) c->cluster_max = std::atoll(e);
  void* sl = nullptr;
  if (cudaMalloc(&sl, sizeof(uint32_t) * (size_t)act_quant_slots()) != cudaSuccess) {
    cudaFree(p);
    delete c;
    return RQ_ERR_ALLOC;
  }
  c->slots = static_cast<uint32_t*>(sl);
  void* fs = nullptr;
  const size_t fs_bytes = sizeof(unsigned long long) * (size_t)device_sm_count();
  if (cudaMalloc(&fs, fs_bytes) != cudaSuccess) {
    cudaFree(sl);
    cudaFree(p);
    delete c;
    return RQ_ERR_ALLOC;
  }
  if (cudaMemset(fs, 0, fs_bytes) != cudaSuccess) {
    cudaFree(fs);
    cudaFree(sl);
    cudaFree(p);
    delete c;
    return RQ_ERR_CUDA;
  }
  c->fused_slots = static_cast<unsigned long long*>(fs);
  *out = c;
  return RQ_OK;
}

void rq_ctx_destroy(rq_ctx* ctx) {
  if (ctx == nullptr) return;
  for (auto& t : ctx->trace) {
    if (t.start) cudaEventDestroy(t.start);
    if (t.stop) cudaEventDestroy(t.stop);
  }
  for (auto& kv : ctx->weights) cudaFree(kv.second.fp8);
  for (auto& kv : ctx->groups) cudaFree(kv.second.fp8);
  for (auto& a : ctx->act)
    if (a.codes) cudaFree(a.codes);
  for (uint8_t* p : ctx->act_kept) cudaFree(p);
  if (ctx->absmax) cudaFree(ctx->absmax);
  if (ctx->slots) cudaFree(ctx->slots);
  if (ctx->fused_slots) cudaFree(ctx->fused_slots);
  ctx->attn.release();
  delete ctx;
}

rq_status rq_ctx_set_gemm_threshold(rq_ctx* ctx, int m_threshold) {
  if (ctx == nullptr) return RQ_ERR_NULL;
  if (m_threshold < 1) return RQ_ERR_SHAPE;
  ctx->threshold = m_threshold;
  return RQ_OK;
}

int rq_ctx_get_gemm_threshold(const rq_ctx* ctx) {
  return ctx == nullptr ? -1 : ctx->threshold;
}

rq_status rq_ctx_get_stats(const rq_ctx* ctx, int64_t* act_hits_host,
                           int64_t* act_misses_host, int64_t* weights_host,
                           int64_t* weight_bytes_host) {
  if (ctx == nullptr) return RQ_ERR_NULL;
  if (act_hits_host) *act_hits_host = ctx->hits;
  if (act_misses_host) *act_misses_host = ctx->misses;
  if (weights_host) *weights_host = (int64_t)(ctx->weights.size() + ctx->groups.size());
  if (weight_bytes_host) *weight_bytes_host = ctx->weight_bytes;
  return RQ_OK;
}

rq_status rq_absmax(const float* x, int64_t n, uint32_t* absmax_bits, rq_stream_t stream) {
  if (absmax_bits == nullptr || (x == nullptr && n > 0)) return RQ_ERR_NULL;
  if (n < 0 || !aligned(absmax_bits, 4)) return RQ_ERR_SHAPE;
  return launch_absmax(x, n, absmax_bits, reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_quant_e4m3(const float* x, int64_t n, const uint32_t* absmax_bits,
                        uint8_t* out, float* dequant_out, rq_stream_t stream) {
  if (absmax_bits == nullptr || dequant_out == nullptr) return RQ_ERR_NULL;
  if (n > 0 && (x == nullptr || out == nullptr)) return RQ_ERR_NULL;
  if (n < 0 || !aligned(absmax_bits, 4) || !aligned(dequant_out, 4)) return RQ_ERR_SHAPE;
  return launch_quant(x, n, n, absmax_bits, out, dequant_out,
                      reinterpret_cast<cudaStream_t>(stream));
}

static rq_status check_gemv(const void* w, const float* x, const float* y, int M, int N,
                            int K, uintptr_t w_align) {
  if (w == nullptr || x == nullptr || y == nullptr) return RQ_ERR_NULL;
  if (M < 1 || M > 8 || N < 1 || K < 256 || K % 256 != 0) return RQ_ERR_SHAPE;
  if (!aligned(w, w_align) || !aligned(x, 16) || !aligned(y, 4)) return RQ_ERR_SHAPE;
  // the per-CTA sums of x must fit in shared memory
  if ((int64_t)M * K > 57344 * 8) return RQ_ERR_SHAPE;
  return RQ_OK;
}

rq_status rq_q4k_gemv(const void* w, const float* x, float* y, int M, int N, int K,
                      rq_stream_t stream) {
  rq_status s = check_gemv(w, x, y, M, N, K, 16);
  if (s != RQ_OK) return s;
  return launch_q4k_gemv(static_cast<const uint8_t*>(w), x, y, M, N, K,
                         reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_q6k_gemv(const void* w, const float* x, float* y, int M, int N, int K,
                      rq_stream_t stream) {
  rq_status s = check_gemv(w, x, y, M, N, K, 4);
  if (s != RQ_OK) return s;
  return launch_q6k_gemv(static_cast<const uint8_t*>(w), x, y, M, N, K,
                         reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_fp8_weight_cache(rq_ctx* ctx, rq_qtype qtype, const void* w, int N, int K,
                              const uint8_t** w_fp8, const float** w_dequant,
                              rq_stream_t stream) {
  if (ctx == nullptr || w == nullptr || w_fp8 == nullptr || w_dequant == nullptr)
    return RQ_ERR_NULL;
  rq_status s = check_quant_shape(qtype, N, K);
  if (s != RQ_OK) return s;
  if (!aligned(w, qtype == RQ_Q4K ? 16 : 4)) return RQ_ERR_SHAPE;
  const WeightKey key{w, (int)qtype, N, K};
  auto it = ctx->weights.find(key);
  if (it == ctx->weights.end()) {
    const size_t body = (size_t)N * (size_t)K;
    const size_t bytes = (body + 255) / 256 * 256 + 256;
    void* p = nullptr;
    if (cudaMalloc(&p, bytes) != cudaSuccess) {
      cudaGetLastError();
      return RQ_ERR_ALLOC;
    }
    WeightEntry e;
    e.fp8 = static_cast<uint8_t*>(p);
    e.deq = reinterpret_cast<float*>(e.fp8 + (body + 255) / 256 * 256);
    e.bytes = bytes;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const uint8_t* wb = static_cast<const uint8_t*>(w);
    s = cuda_status(cudaMemsetAsync(ctx->absmax, 0, sizeof(uint32_t), st));
    if (s == RQ_OK) s = launch_dequant_absmax(qtype, wb, N, K, ctx->absmax, st);
    if (s == RQ_OK)
      s = launch_dequant_encode(qtype, wb, N, K, ctx->absmax, e.fp8, e.deq, st);
    // A product that finds this entry loads its first tiles before the launch ahead
    // of it is done.  That launch must not be the encoding: what is no kernel waits
    // for it, and the product for that.
    if (s == RQ_OK) s = cuda_status(cudaMemsetAsync(ctx->absmax, 0, sizeof(uint32_t), st));
    if (s != RQ_OK) {
      cudaFree(p);
      return s;
    }
    it = ctx->weights.emplace(key, e).first;
    ctx->weight_bytes += (int64_t)bytes;
  }
  *w_fp8 = it->second.fp8;
  *w_dequant = it->second.deq;
  return RQ_OK;
}

rq_status rq_fp8_gemm(const uint8_t* x_fp8, const float* x_dequant, const uint8_t* w_fp8,
                      const float* w_dequant, float* y, int M, int N, int K,
                      rq_stream_t stream) {
  if (x_fp8 == nullptr || x_dequant == nullptr || w_fp8 == nullptr ||
      w_dequant == nullptr || y == nullptr)
    return RQ_ERR_NULL;
  if (M < 1 || N < 1 || K < 128 || K % 128 != 0) return RQ_ERR_SHAPE;
  if (!aligned(x_fp8, 16) || !aligned(w_fp8, 16) || !aligned(y, 4) ||
      !aligned(x_dequant, 4) || !aligned(w_dequant, 4))
    return RQ_ERR_SHAPE;
  return launch_fp8_gemm(x_fp8, x_dequant, w_fp8, w_dequant, y, M, N, K,
                         reinterpret_cast<cudaStream_t>(stream));
}

// The capture that `st` is in, 0 if none.
static rq_status capture_of(cudaStream_t st, unsigned long long* id) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  *id = 0;
  if (cudaStreamGetCaptureInfo(st, &status, id) != cudaSuccess) {
    cudaGetLastError();  // (the legacy stream while another one is captured)
    return RQ_ERR_CUDA;
  }
  if (status == cudaStreamCaptureStatusInvalidated) return RQ_ERR_CUDA;
  if (status == cudaStreamCaptureStatusNone) *id = 0;
  return RQ_OK;
}

// Room for `need` codes.  What ran at once is done with its buffer when it is
// freed; a captured graph's stays, and the next is at least twice as large, so
// that all of them together hold less than twice the last.
static rq_status grow(rq_ctx* ctx, ActScratch* a, size_t need, bool captured) {
  if (need <= a->cap) return RQ_OK;
  if (captured && need < 2 * a->cap) need = 2 * a->cap;
  const size_t body = (need + 255) / 256 * 256;
  if (!captured && a->codes) {
    cudaFree(a->codes);
    *a = ActScratch();
  }
  // (an allocation is no work of the stream: it is made at once, and legal
  // while the thread's captures are of the relaxed kind)
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (captured && cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return RQ_ERR_CUDA;
  void* p = nullptr;
  const cudaError_t e = cudaMalloc(&p, body + 256);
  if (captured) cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return RQ_ERR_ALLOC;
  }
  if (a->codes) ctx->act_kept.push_back(a->codes);
  *a = ActScratch();
  a->codes = static_cast<uint8_t*>(p);
  a->deq = reinterpret_cast<float*>(a->codes + body);
  a->cap = need;
  return RQ_OK;
}

// rq_fp8_act_cache; `anew`: without a look at the cache, and nothing is left in
// it, since the caller of such a call does not say when x changes.
static rq_status act_codes(rq_ctx* ctx, const float* x, int M, int K, bool anew,
                           const uint8_t** x_fp8, const float** x_dequant, cudaStream_t st) {
  unsigned long long capture = 0;
  rq_status s = capture_of(st, &capture);
  if (s != RQ_OK) return s;
  ActScratch& a = ctx->act[capture != 0 ? 1 : 0];
  const bool hit = !anew && a.valid && a.x == x && a.M == M && a.K == K && a.gen == ctx->gen &&
                   a.capture == capture;
  if (hit) {
    ++ctx->hits;
  } else {
    const int m_pad = (M + 15) / 16 * 16;
    const size_t need = (size_t)m_pad * (size_t)K;
    s = grow(ctx, &a, need, capture != 0);
    if (s != RQ_OK) return s;
    const int64_t n = (int64_t)M * K;
    s = RQ_ERR_SHAPE;
    if (n <= ctx->cluster_max) {
      // a few tokens: one cluster reads x twice (the second time from L2)
      TraceScope ts(ctx, RQ_TRACE_QUANT, st);
      s = launch_act_quant_cluster(x, n, (int64_t)need, a.codes, ctx->absmax, a.deq, st);
      if (s == RQ_ERR_SHAPE) ts.kernels(0);
    } else if (ctx->fused_ok && n >= ctx->fused_min && act_quant_fused_fits(x, n, a.codes)) {
      TraceScope ts(ctx, RQ_TRACE_QUANT, st);
      s = launch_act_quant_fused(x, n, (int64_t)need, a.codes, ctx->absmax, a.deq, ctx->fused,
                                 ctx->fused_slots, device_sm_count(), st);
      if (s == RQ_ERR_SHAPE) ts.kernels(0);
    }
    // RQ_ERR_SHAPE from the one-cluster or one-pass launcher: nothing was
    // launched
    if (s == RQ_ERR_SHAPE) {
      // two kernels: per-CTA maxima into slots, then the encoding
      TraceScope ts(ctx, RQ_TRACE_QUANT, st);
      ts.kernels(2);
      s = launch_act_quant_two_pass(x, n, (int64_t)need, a.codes, ctx->slots, ctx->absmax, a.deq,
                                    st);
    }
    if (s != RQ_OK) {
      a.valid = false;
      return s;
    }
    a.valid = !anew;
    a.x = x;
    a.M = M;
    a.K = K;
    a.gen = ctx->gen;
    a.capture = capture;
    ++ctx->misses;
  }
  *x_fp8 = a.codes;
  *x_dequant = a.deq;
  return RQ_OK;
}

rq_status rq_fp8_act_cache(rq_ctx* ctx, const float* x, int M, int K,
                           const uint8_t** x_fp8, const float** x_dequant,
                           rq_stream_t stream) {
  if (ctx == nullptr || x == nullptr || x_fp8 == nullptr || x_dequant == nullptr)
    return RQ_ERR_NULL;
  if (M < 1 || K < 1 || !aligned(x, 16)) return RQ_ERR_SHAPE;
  return act_codes(ctx, x, M, K, false, x_fp8, x_dequant, reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_linear(rq_ctx* ctx, rq_qtype qtype, const void* w, const float* x, float* y,
                    int M, int N, int K, rq_stream_t stream) {
  if (ctx == nullptr || w == nullptr || x == nullptr || y == nullptr) return RQ_ERR_NULL;
  rq_status s = check_quant_shape(qtype, N, K);
  if (s != RQ_OK) return s;
  if (M < 1) return RQ_ERR_SHAPE;
  if (!aligned(w, qtype == RQ_Q4K ? 16 : 4) || !aligned(x, 16) || !aligned(y, 4))
    return RQ_ERR_SHAPE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);

  if (M < ctx->threshold) {
    // GEMV straight from the packed weight: Q4_K one launch per token, Q6_K
    // up to 8 tokens per launch
    const int per = qtype == RQ_Q4K ? 1 : 8;
    for (int m0 = 0; m0 < M; m0 += per) {
      const int mc = M - m0 < per ? M - m0 : per;
      TraceScope ts(ctx, RQ_TRACE_GEMV, st);
      s = qtype == RQ_Q4K
              ? rq_q4k_gemv(w, x + (size_t)m0 * K, y + (size_t)m0 * N, mc, N, K, stream)
              : rq_q6k_gemv(w, x + (size_t)m0 * K, y + (size_t)m0 * N, mc, N, K, stream);
      if (s != RQ_OK) return s;
    }
    return RQ_OK;
  }

  const uint8_t* wq = nullptr;
  const float* wdeq = nullptr;
  const bool miss = ctx->weights.find(WeightKey{w, (int)qtype, N, K}) == ctx->weights.end();
  {
    TraceScope ts(miss ? ctx : nullptr, RQ_TRACE_WCACHE, st);
    ts.kernels(2);  // decode + absmax, decode + encode
    s = rq_fp8_weight_cache(ctx, qtype, w, N, K, &wq, &wdeq, stream);
  }
  if (s != RQ_OK) return s;

  const uint8_t* xq = nullptr;
  const float* xdeq = nullptr;
  s = rq_fp8_act_cache(ctx, x, M, K, &xq, &xdeq, stream);
  if (s != RQ_OK) return s;
  TraceScope ts(ctx, RQ_TRACE_GEMM, st);
  // a cached weight built by an earlier call was complete before the launch
  // preceding this GEMM began, so its first tiles may load early
  return launch_fp8_gemm(xq, xdeq, wq, wdeq, y, M, N, K, st, !miss);
}

rq_status rq_linear_group(rq_ctx* ctx, int count, const rq_qtype* qtypes, const void* const* w,
                          const float* x, float* const* y, const int* N, int M, int K,
                          rq_stream_t stream) {
  if (ctx == nullptr || qtypes == nullptr || w == nullptr || x == nullptr || y == nullptr ||
      N == nullptr)
    return RQ_ERR_NULL;
  if (count < 1 || count > RQ_MAX_GROUP || M < 1) return RQ_ERR_SHAPE;
  for (int i = 0; i < count; ++i) {
    if (w[i] == nullptr || y[i] == nullptr) return RQ_ERR_NULL;
    rq_status s = check_quant_shape(qtypes[i], N[i], K);
    if (s != RQ_OK) return s;
    if (!aligned(w[i], qtypes[i] == RQ_Q4K ? 16 : 4) || !aligned(y[i], 4)) return RQ_ERR_SHAPE;
  }
  if (!aligned(x, 16)) return RQ_ERR_SHAPE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (count == 1) return rq_linear(ctx, qtypes[0], w[0], x, y[0], M, N[0], K, stream);

  if (M < ctx->threshold) {
    // GEMV route, one token at a time: the Q4_K members in one launch,
    // joined by the Q6_K member when there is exactly one
    int starts[RQ_MAX_GROUP + 1];
    const uint8_t* ws[RQ_MAX_GROUP];
    int idx4[RQ_MAX_GROUP];
    int n4 = 0, i6 = -1, n6 = 0;
    starts[0] = 0;
    for (int i = 0; i < count; ++i) {
      if (qtypes[i] == RQ_Q4K) {
        ws[n4] = static_cast<const uint8_t*>(w[i]);
        idx4[n4] = i;
        starts[n4 + 1] = starts[n4] + N[i];
        ++n4;
      } else {
        i6 = i;
        ++n6;
      }
    }
    for (int m = 0; m < M; ++m) {
      const float* xm = x + (size_t)m * K;
      float* ys[RQ_MAX_GROUP];
      for (int j = 0; j < n4; ++j) ys[j] = y[idx4[j]] + (size_t)m * N[idx4[j]];
      bool grouped = false, dual = false;
      if (n4 >= 1 && n6 == 1 && std::getenv("RQ_GEMV_NO_DUAL") == nullptr) {
        TraceScope ts(ctx, RQ_TRACE_GEMV, st);
        const rq_status s = launch_gemv_m1_dual(n4, starts, ws, ys,
                                                static_cast<const uint8_t*>(w[i6]),
                                                y[i6] + (size_t)m * N[i6], N[i6], xm, K, st);
        if (s != RQ_OK && s != RQ_ERR_SHAPE) return s;
        grouped = dual = s == RQ_OK;
      }
      if (!grouped && n4 >= 2) {
        TraceScope ts(ctx, RQ_TRACE_GEMV, st);
        const rq_status s = launch_q4k_gemv_group(n4, starts, ws, ys, xm, K, st);
        if (s != RQ_OK && s != RQ_ERR_SHAPE) return s;
        grouped = s == RQ_OK;
      }
      for (int i = 0; i < count; ++i) {
        if (grouped && qtypes[i] == RQ_Q4K) continue;
        if (dual && i == i6) continue;
        const rq_status s =
            rq_linear(ctx, qtypes[i], w[i], xm, y[i] + (size_t)m * N[i], 1, N[i], K, stream);
        if (s != RQ_OK) return s;
      }
    }
    return RQ_OK;
  }

  // FP8 route: the group's weights, concatenated by rows, cached once
  std::vector<WeightKey> key;
  for (int i = 0; i < count; ++i) key.push_back(WeightKey{w[i], (int)qtypes[i], N[i], K});
  auto it = ctx->groups.find(key);
  const bool hit = it != ctx->groups.end();
  if (!hit) {
    GroupEntry e;
    e.starts[0] = 0;
    for (int i = 0; i < count; ++i) e.starts[i + 1] = e.starts[i] + N[i];
    for (int i = count; i < RQ_MAX_GROUP; ++i) e.starts[i + 1] = e.starts[count];
    const size_t body = (size_t)e.starts[count] * (size_t)K;
    const size_t bytes = (body + 255) / 256 * 256 + 256;
    void* p = nullptr;
    if (cudaMalloc(&p, bytes) != cudaSuccess) {
      cudaGetLastError();
      return RQ_ERR_ALLOC;
    }
    e.fp8 = static_cast<uint8_t*>(p);
    e.deq = reinterpret_cast<float*>(e.fp8 + (body + 255) / 256 * 256);
    e.bytes = bytes;
    rq_status s = RQ_OK;
    {
      TraceScope ts(ctx, RQ_TRACE_WCACHE, st);
      ts.kernels(2 * count);
      for (int i = 0; i < count && s == RQ_OK; ++i) {
        const uint8_t* wb = static_cast<const uint8_t*>(w[i]);
        s = cuda_status(cudaMemsetAsync(ctx->absmax, 0, sizeof(uint32_t), st));
        if (s == RQ_OK) s = launch_dequant_absmax(qtypes[i], wb, N[i], K, ctx->absmax, st);
        if (s == RQ_OK)
          s = launch_dequant_encode(qtypes[i], wb, N[i], K, ctx->absmax,
                                    e.fp8 + (size_t)e.starts[i] * K, e.deq + i, st);
      }
    }
    if (s != RQ_OK) {
      cudaFree(p);
      return s;
    }
    it = ctx->groups.emplace(key, e).first;
    ctx->weight_bytes += (int64_t)bytes;
  }
  const uint8_t* xq = nullptr;
  const float* xdeq = nullptr;
  rq_status s = rq_fp8_act_cache(ctx, x, M, K, &xq, &xdeq, stream);
  if (s != RQ_OK) return s;
  const float* deqs[RQ_MAX_GROUP];
  for (int i = 0; i < count; ++i) deqs[i] = it->second.deq + i;
  TraceScope ts(ctx, RQ_TRACE_GEMM, st);
  // a group cache built by an earlier call may be loaded early (as in rq_linear)
  return launch_fp8_gemm_group(xq, xdeq, it->second.fp8, count, it->second.starts, y, deqs, M,
                               K, st, hit);
}

static rq_status check_dtype(int dtype) {
  return dtype == RQ_F32 || dtype == RQ_F16 || dtype == RQ_BF16 ? RQ_OK : RQ_ERR_QTYPE;
}

static int width_of(int dtype) { return dtype == RQ_F32 ? 4 : 2; }

// ---------------------------------- FP8 product with a fused epilogue --

static bool stride_ok(int64_t stride, int64_t row) {
  return stride >= row && stride <= (int64_t)1 << 40;
}

static rq_status check_epilogue(const rq_epilogue& e, int dtype, const void* y, int64_t y_stride,
                                int N) {
  rq_status s = check_dtype(dtype);
  if (s != RQ_OK) return s;
  if (e.act < RQ_ACT_NONE || e.act > RQ_ACT_RELU) return RQ_ERR_QTYPE;
  const int w = width_of(dtype);
  if (!aligned(y, w) || !aligned(e.mul, w) || !aligned(e.residual, w) || !aligned(e.bias, 4) ||
      !stride_ok(y_stride, N) || (e.mul != nullptr && !stride_ok(e.mul_stride, N)) ||
      (e.residual != nullptr && !stride_ok(e.residual_stride, N)))
    return RQ_ERR_SHAPE;
  // an operand in y's place has y's stride
  if ((e.mul == y && e.mul_stride != y_stride) ||
      (e.residual == y && e.residual_stride != y_stride))
    return RQ_ERR_SHAPE;
  return RQ_OK;
}

rq_status rq_fp8_gemm_epilogue(const uint8_t* x_fp8, const float* x_dequant,
                               const uint8_t* w_fp8, const float* w_dequant,
                               const rq_epilogue* epilogue, int dtype, void* y, int64_t y_stride,
                               int M, int N, int K, rq_stream_t stream) {
  if (x_fp8 == nullptr || x_dequant == nullptr || w_fp8 == nullptr || w_dequant == nullptr ||
      y == nullptr)
    return RQ_ERR_NULL;
  const rq_epilogue none = {};
  const rq_epilogue& e = epilogue != nullptr ? *epilogue : none;
  const rq_status s = check_epilogue(e, dtype, y, y_stride, N);
  if (s != RQ_OK) return s;
  if (M < 1 || N < 1 || K < 128 || K % 128 != 0 || !aligned(x_fp8, 16) || !aligned(w_fp8, 16) ||
      !aligned(x_dequant, 4) || !aligned(w_dequant, 4))
    return RQ_ERR_SHAPE;
  return launch_fp8_gemm_epilogue(x_fp8, x_dequant, w_fp8, w_dequant, e, dtype, y, y_stride, M, N,
                                  K, reinterpret_cast<cudaStream_t>(stream), false);
}

rq_status rq_linear_epilogue(rq_ctx* ctx, rq_qtype qtype, const void* w, const float* x,
                             const rq_epilogue* epilogue, int dtype, void* y, int64_t y_stride,
                             int M, int N, int K, rq_stream_t stream) {
  if (ctx == nullptr || w == nullptr || x == nullptr || y == nullptr) return RQ_ERR_NULL;
  rq_status s = check_quant_shape(qtype, N, K);
  if (s != RQ_OK) return s;
  const rq_epilogue none = {};
  const rq_epilogue& e = epilogue != nullptr ? *epilogue : none;
  s = check_epilogue(e, dtype, y, y_stride, N);
  if (s != RQ_OK) return s;
  if (M < 1 || !aligned(w, qtype == RQ_Q4K ? 16 : 4) || !aligned(x, 16)) return RQ_ERR_SHAPE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const uint8_t* wq = nullptr;
  const float* wdeq = nullptr;
  const bool miss = ctx->weights.find(WeightKey{w, (int)qtype, N, K}) == ctx->weights.end();
  {
    TraceScope ts(miss ? ctx : nullptr, RQ_TRACE_WCACHE, st);
    ts.kernels(2);  // decode + absmax, decode + encode
    s = rq_fp8_weight_cache(ctx, qtype, w, N, K, &wq, &wdeq, stream);
  }
  if (s != RQ_OK) return s;
  const uint8_t* xq = nullptr;
  const float* xdeq = nullptr;
  // below the threshold rq_linear reads x itself, and so its callers invalidate
  // nothing there
  s = act_codes(ctx, x, M, K, M < ctx->threshold, &xq, &xdeq, st);
  if (s != RQ_OK) return s;
  TraceScope ts(ctx, RQ_TRACE_GEMM, st);
  return launch_fp8_gemm_epilogue(xq, xdeq, wq, wdeq, e, dtype, y, y_stride, M, N, K, st, !miss);
}

// --------------------------------------- norms between a layer's blocks --

rq_status rq_residual_norm(const rq_norm_params* params, int dtype, const void* y,
                           int64_t y_stride, const void* gate, int64_t gate_stride, int h_dtype,
                           const void* h, int64_t h_stride, void* h_out, void* x_out,
                           uint32_t* absmax_bits, int tokens, rq_stream_t stream) {
  if (params == nullptr ||
      (tokens != 0 && (h == nullptr || (h_out == nullptr && x_out == nullptr) ||
                       (y == nullptr && (h_out != nullptr || gate != nullptr)) ||
                       (absmax_bits != nullptr && x_out == nullptr))))
    return RQ_ERR_NULL;
  rq_status s = check_dtype(dtype);
  if (s != RQ_OK) return s;
  if ((h_dtype != dtype && h_dtype != RQ_F32) || (absmax_bits != nullptr && dtype != RQ_F32))
    return RQ_ERR_QTYPE;
  const int64_t n = params->width;
  const int w = width_of(dtype), wh = width_of(h_dtype);
  if (n < 1 || n > 16384 || tokens < 0 || (params->norms & ~(RQ_NORM_POST | RQ_NORM_PRE)) != 0 ||
      !(params->eps >= 0.0f) || !(params->scale - params->scale == 0.0f) ||
      !aligned(params->post_weight, 4) || !aligned(params->pre_weight, 4))
    return RQ_ERR_SHAPE;
  if (!aligned(y, w) || !aligned(gate, w) || !aligned(h, wh) || !aligned(h_out, wh) ||
      !aligned(x_out, w) || !aligned(absmax_bits, 4) || !stride_ok(h_stride, n) ||
      (y != nullptr && !stride_ok(y_stride, n)) ||
      (gate != nullptr && gate_stride != 0 && !stride_ok(gate_stride, n)))
    return RQ_ERR_SHAPE;
  // in place where the input is dense; the two outputs are apart
  if ((h_out != nullptr && h_out == h && h_stride != n) || (x_out != nullptr && x_out == y && y_stride != n) ||
      (h_out != nullptr && h_out == x_out) || (x_out != nullptr && (x_out == h || x_out == gate)) ||
      (h_out != nullptr && (h_out == y || h_out == gate)))
    return RQ_ERR_SHAPE;
  return launch_residual_norm(*params, dtype, y, y_stride, gate, gate_stride, h_dtype, h, h_stride,
                              h_out, x_out, absmax_bits, tokens,
                              reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------ the places of a pass --

rq_status rq_batch_plan(const int32_t* length, const int32_t* count, int batch, int new_tokens,
                        int page_size, int32_t* page_table, int max_pages,
                        const int32_t* free_pages, int free_capacity, const int32_t* free_count,
                        int32_t* free_left, int64_t* slot, int32_t* position, int32_t* sequence,
                        int rows, int32_t* row_start, int32_t* next_length, rq_stream_t stream) {
  if (free_count == nullptr || free_left == nullptr ||
      (batch != 0 && (length == nullptr || page_table == nullptr)) ||
      (free_capacity != 0 && free_pages == nullptr) ||
      (rows != 0 && (slot == nullptr || position == nullptr)) ||
      (new_tokens == 0 && batch != 0 && count == nullptr))
    return RQ_ERR_NULL;
  if (batch < 0 || batch > 65536 || new_tokens < 0 || max_pages < 1 || free_capacity < 0 ||
      rows < 0 || (new_tokens > 0 && (int64_t)batch * new_tokens != rows) ||
      (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 &&
       page_size != 256))
    return RQ_ERR_SHAPE;
  if (!aligned(length, 4) || !aligned(count, 4) || !aligned(page_table, 4) ||
      !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(free_left, 4) ||
      !aligned(slot, 8) || !aligned(position, 4) || !aligned(sequence, 4) ||
      !aligned(row_start, 4) || !aligned(next_length, 4) || free_left == free_count ||
      (next_length != nullptr && (next_length == length || next_length == count)) ||
      (row_start != nullptr && (row_start == length || row_start == count)))
    return RQ_ERR_SHAPE;
  return launch_batch_plan(length, count, batch, new_tokens, page_size, page_table, max_pages,
                           free_pages, free_capacity, free_count, free_left, slot, position,
                           sequence, rows, row_start, next_length,
                           reinterpret_cast<cudaStream_t>(stream));
}

// ------------------------------------------------- quantized K/V cache --

static bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

static rq_status check_cache(const rq_kv_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->k_scale == nullptr ||
      c->v_scale == nullptr)
    return RQ_ERR_NULL;
  if (c->format != RQ_KV_E4M3 && c->format != RQ_KV_I8) return RQ_ERR_QTYPE;
  if (!head_dim_ok(c->head_dim) || c->kv_heads < 1 || c->pages < 1 ||
      c->pages > 0x7FFFFFFFLL / c->kv_heads)
    return RQ_ERR_SHAPE;
  const int p = c->page_size;
  if (p != 16 && p != 32 && p != 64 && p != 128 && p != 256) return RQ_ERR_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16))
    return RQ_ERR_SHAPE;
  return RQ_OK;
}

// Rows of `heads` heads per token: pointer and token stride.
static rq_status check_rows(const void* p, int64_t stride, int heads, int head_dim, int dtype) {
  const int w = width_of(dtype);
  if (!aligned(p, 16) || stride < (int64_t)heads * head_dim || stride % (16 / w) != 0 ||
      stride > (int64_t)1 << 40)
    return RQ_ERR_SHAPE;
  return RQ_OK;
}

static rq_status check_qk(const rq_qk_params* p, const int32_t* position) {
  if (p == nullptr) return RQ_ERR_NULL;
  if (!head_dim_ok(p->head_dim) || p->q_heads < 0 || p->kv_heads < 0 || p->rotary_dim < 0 ||
      p->rotary_dim > p->head_dim || p->rotary_dim % 16 != 0)
    return RQ_ERR_SHAPE;
  if (p->rotary_dim > 0) {
    if (p->cos_table == nullptr || p->sin_table == nullptr || position == nullptr)
      return RQ_ERR_NULL;
    if (p->positions < 1 || !aligned(p->cos_table, 16) || !aligned(p->sin_table, 16) ||
        !aligned(position, 4))
      return RQ_ERR_SHAPE;
  }
  if (!aligned(p->q_weight, 16) || !aligned(p->k_weight, 16) || !(p->eps >= 0.0f))
    return RQ_ERR_SHAPE;
  return RQ_OK;
}

// At most one row a warp, and warps are numbered in 31 bits.
static bool tokens_ok(int tokens, int rows) {
  return tokens >= 0 && rows >= 1 && (int64_t)tokens * rows < 0x7FFFFF00LL;
}

rq_status rq_qk_norm_rope(const rq_qk_params* params, int dtype, const void* q, int64_t q_stride,
                          const void* k, int64_t k_stride, const int32_t* position, void* q_out,
                          void* k_out, int tokens, rq_stream_t stream) {
  rq_status s = check_qk(params, position);
  if (s != RQ_OK) return s;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) ||
      (q == nullptr && k == nullptr))
    return RQ_ERR_NULL;
  s = check_dtype(dtype);
  if (s != RQ_OK) return s;
  if ((q != nullptr && params->q_heads < 1) || (k != nullptr && params->kv_heads < 1) ||
      !tokens_ok(tokens, (q ? params->q_heads : 0) + (k ? params->kv_heads : 0)))
    return RQ_ERR_SHAPE;
  if (q != nullptr) s = check_rows(q, q_stride, params->q_heads, params->head_dim, dtype);
  if (s == RQ_OK && k != nullptr)
    s = check_rows(k, k_stride, params->kv_heads, params->head_dim, dtype);
  if (s != RQ_OK) return s;
  if (!aligned(q_out, 16) || !aligned(k_out, 16)) return RQ_ERR_SHAPE;
  if (tokens == 0) return RQ_OK;
  return launch_qkv_rows(params, dtype, q, q_stride, k, k_stride, nullptr, 0, position, q_out,
                         k_out, nullptr, nullptr, tokens, reinterpret_cast<cudaStream_t>(stream));
}

static rq_status check_store(const rq_kv_cache* cache, int dtype, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const int64_t* slot, int tokens) {
  rq_status s = check_cache(cache);
  if (s != RQ_OK) return s;
  if (k == nullptr || v == nullptr || slot == nullptr) return RQ_ERR_NULL;
  s = check_dtype(dtype);
  if (s != RQ_OK) return s;
  if (!aligned(slot, 8) || !tokens_ok(tokens, 2 * cache->kv_heads)) return RQ_ERR_SHAPE;
  s = check_rows(k, k_stride, cache->kv_heads, cache->head_dim, dtype);
  if (s == RQ_OK) s = check_rows(v, v_stride, cache->kv_heads, cache->head_dim, dtype);
  return s;
}

rq_status rq_qkv_to_cache(const rq_qk_params* params, int dtype, const void* q, int64_t q_stride,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const int32_t* position, void* q_out, const rq_kv_cache* cache,
                          const int64_t* slot, int tokens, rq_stream_t stream) {
  rq_status s = check_qk(params, position);
  if (s != RQ_OK) return s;
  s = check_store(cache, dtype, k, k_stride, v, v_stride, slot, tokens);
  if (s != RQ_OK) return s;
  if ((q == nullptr) != (q_out == nullptr)) return RQ_ERR_NULL;
  if (params->kv_heads != cache->kv_heads || params->head_dim != cache->head_dim)
    return RQ_ERR_SHAPE;
  if (q != nullptr) {
    if (params->q_heads < 1 || !aligned(q_out, 16) ||
        !tokens_ok(tokens, params->q_heads + 2 * params->kv_heads))
      return RQ_ERR_SHAPE;
    s = check_rows(q, q_stride, params->q_heads, params->head_dim, dtype);
    if (s != RQ_OK) return s;
  }
  if (tokens == 0) return RQ_OK;
  return launch_qkv_rows(params, dtype, q, q_stride, k, k_stride, v, v_stride, position, q_out,
                         nullptr, cache, slot, tokens, reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_kv_write(const rq_kv_cache* cache, int dtype, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const int64_t* slot, int tokens,
                      rq_stream_t stream) {
  rq_status s = check_store(cache, dtype, k, k_stride, v, v_stride, slot, tokens);
  if (s != RQ_OK || tokens == 0) return s;
  return launch_qkv_rows(nullptr, dtype, nullptr, 0, k, k_stride, v, v_stride, nullptr, nullptr,
                         nullptr, cache, slot, tokens, reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_kv_read(const rq_kv_cache* cache, int dtype, const int64_t* slot, void* k_out,
                     void* v_out, int tokens, rq_stream_t stream) {
  rq_status s = check_cache(cache);
  if (s != RQ_OK) return s;
  if (slot == nullptr || k_out == nullptr || v_out == nullptr) return RQ_ERR_NULL;
  s = check_dtype(dtype);
  if (s != RQ_OK) return s;
  if (!aligned(slot, 8) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
      !tokens_ok(tokens, cache->kv_heads))
    return RQ_ERR_SHAPE;
  if (tokens == 0) return RQ_OK;
  return launch_kv_read(*cache, dtype, slot, k_out, v_out, tokens,
                        reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_cache_attention(rq_ctx* ctx, const rq_kv_cache* cache, int dtype, const void* q,
                             int64_t q_stride, void* out, int batch, int new_tokens, int q_heads,
                             const int32_t* page_table, int max_pages, const int32_t* length,
                             const uint64_t* tree, float scale, rq_stream_t stream) {
  if (ctx == nullptr) return RQ_ERR_NULL;
  rq_status s = check_cache(cache);
  if (s != RQ_OK) return s;
  if (q == nullptr || out == nullptr || page_table == nullptr || length == nullptr)
    return RQ_ERR_NULL;
  s = check_dtype(dtype);
  if (s != RQ_OK) return s;
  if (batch < 0 || new_tokens < 1 || q_heads < 1 || q_heads % cache->kv_heads != 0 ||
      max_pages < 1 || (tree != nullptr && new_tokens > 64) ||
      (int64_t)new_tokens * q_heads > 0x7FFFFFFFLL || !(scale > 0.0f) || !(scale < 1e30f))
    return RQ_ERR_SHAPE;
  s = check_rows(q, q_stride, q_heads, cache->head_dim, dtype);
  if (s != RQ_OK) return s;
  if (!aligned(out, 16) || !aligned(page_table, 4) || !aligned(length, 4) || !aligned(tree, 8))
    return RQ_ERR_SHAPE;
  if (batch == 0) return RQ_OK;
  const AttnCall call = {cache, dtype,     q,          q_stride,  out,    batch, new_tokens,
                         q_heads, page_table, max_pages, length, tree, scale};
  return launch_cache_attention(call, &ctx->attn, reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_ctx_attention_launches(const rq_ctx* ctx, int64_t* few_rows_host,
                                    int64_t* many_rows_host) {
  if (ctx == nullptr) return RQ_ERR_NULL;
  if (few_rows_host) *few_rows_host = ctx->attn.few_rows;
  if (many_rows_host) *many_rows_host = ctx->attn.many_rows;
  return RQ_OK;
}

// ---------------------------------------------- verification of drafts --

static rq_status check_verify(const int32_t* token, const float* p, const float* u,
                              const int32_t* accepted, const int32_t* next, int batch, int drafts,
                              int vocab) {
  if (p == nullptr || u == nullptr || accepted == nullptr || next == nullptr ||
      (drafts > 0 && token == nullptr))
    return RQ_ERR_NULL;
  // (drafts + 1 rows, counted in steps of a block's threads, in 32 bits)
  if (batch < 0 || batch > (1 << 27) || drafts < 0 || drafts > (1 << 30) || vocab < 1 ||
      vocab > (1 << 20) || !aligned(p, 4) || !aligned(u, 4) || !aligned(token, 4) ||
      !aligned(accepted, 4) || !aligned(next, 4))
    return RQ_ERR_SHAPE;
  return RQ_OK;
}

rq_status rq_verify_chain(const int32_t* token, const float* p, const float* q, const float* u,
                          int32_t* accepted, int32_t* next, int batch, int drafts, int vocab,
                          rq_stream_t stream) {
  const rq_status s = check_verify(token, p, u, accepted, next, batch, drafts, vocab);
  if (s != RQ_OK) return s;
  if (!aligned(q, 4)) return RQ_ERR_SHAPE;
  if (batch == 0) return RQ_OK;
  return launch_verify_chain(token, p, q, u, accepted, next, batch, drafts, vocab,
                             reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_verify_tree(const int32_t* token, const int32_t* parent, const float* p,
                         const float* u, int32_t* accepted, int32_t* next, int32_t* path,
                         int batch, int drafts, int vocab, rq_stream_t stream) {
  const rq_status s = check_verify(token, p, u, accepted, next, batch, drafts, vocab);
  if (s != RQ_OK) return s;
  if (drafts > 0 && (parent == nullptr || path == nullptr)) return RQ_ERR_NULL;
  if (drafts > 1024 || !aligned(parent, 4) || !aligned(path, 4)) return RQ_ERR_SHAPE;
  if (batch == 0) return RQ_OK;
  return launch_verify_tree(token, parent, p, u, accepted, next, path, batch, drafts, vocab,
                            reinterpret_cast<cudaStream_t>(stream));
}

// -------------------------------------------------- logits to tokens --

static rq_status check_sampling(const rq_sampling* f, int dtype, const void* logits,
                                int64_t stride, int rows, int vocab) {
  if (f == nullptr || (rows != 0 && logits == nullptr)) return RQ_ERR_NULL;
  const rq_status s = check_dtype(dtype);
  if (s != RQ_OK) return s;
  if (rows < 0 || rows > (1 << 27) || vocab < 1 || vocab > (1 << 20) || !stride_ok(stride, vocab) ||
      !aligned(logits, width_of(dtype)) || !aligned(f->temperature, 4) || !aligned(f->top_k, 4) ||
      !aligned(f->top_p, 4) || !aligned(f->min_p, 4))
    return RQ_ERR_SHAPE;
  return RQ_OK;
}

rq_status rq_sample(const rq_sampling* sampling, int dtype, const void* logits, int64_t stride,
                    const float* u, int32_t* token, int rows, int vocab, rq_stream_t stream) {
  if (rows != 0 && (u == nullptr || token == nullptr)) return RQ_ERR_NULL;
  const rq_status s = check_sampling(sampling, dtype, logits, stride, rows, vocab);
  if (s != RQ_OK) return s;
  if (!aligned(u, 4) || !aligned(token, 4)) return RQ_ERR_SHAPE;
  if (rows == 0) return RQ_OK;
  return launch_sample(*sampling, dtype, logits, stride, u, token, nullptr, rows, vocab,
                       reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_token_probs(const rq_sampling* sampling, int dtype, const void* logits,
                         int64_t stride, float* p, int rows, int vocab, rq_stream_t stream) {
  if (rows != 0 && p == nullptr) return RQ_ERR_NULL;
  const rq_status s = check_sampling(sampling, dtype, logits, stride, rows, vocab);
  if (s != RQ_OK) return s;
  if (rows == 0) return RQ_OK;
  if (!aligned(p, 4) || static_cast<const void*>(p) == logits) return RQ_ERR_SHAPE;
  return launch_sample(*sampling, dtype, logits, stride, nullptr, nullptr, p, rows, vocab,
                       reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_ctx_trace_begin(rq_ctx* ctx, int capacity) {
  if (ctx == nullptr) return RQ_ERR_NULL;
  if (capacity < 1) return RQ_ERR_SHAPE;
  while ((int)ctx->trace.size() < capacity) {
    TraceSlot t;
    if (cudaEventCreate(&t.start) != cudaSuccess) return RQ_ERR_ALLOC;
    if (cudaEventCreate(&t.stop) != cudaSuccess) {
      cudaEventDestroy(t.start);
      return RQ_ERR_ALLOC;
    }
    ctx->trace.push_back(t);
  }
  ctx->trace_cap = capacity;
  ctx->trace_used = 0;
  ctx->trace_on = true;
  return RQ_OK;
}

rq_status rq_ctx_trace_kinds(rq_ctx* ctx, unsigned int mask) {
  if (ctx == nullptr) return RQ_ERR_NULL;
  if (mask == 0u || (mask >> RQ_TRACE_KINDS) != 0u) return RQ_ERR_SHAPE;
  ctx->trace_mask = mask;
  return RQ_OK;
}

rq_status rq_ctx_trace_end(rq_ctx* ctx, int64_t* counts_host, double* ms_host) {
  if (ctx == nullptr) return RQ_ERR_NULL;
  int64_t counts[RQ_TRACE_KINDS] = {0};
  double ms[RQ_TRACE_KINDS] = {0.0};
  rq_status s = RQ_OK;
  for (int i = 0; i < ctx->trace_used; ++i) {
    const TraceSlot& t = ctx->trace[i];
    float e = 0.f;
    if (cudaEventSynchronize(t.stop) != cudaSuccess ||
        cudaEventElapsedTime(&e, t.start, t.stop) != cudaSuccess) {
      s = RQ_ERR_CUDA;
      continue;
    }
    counts[t.kind] += t.kernels;
    ms[t.kind] += e;
  }
  ctx->trace_on = false;
  ctx->trace_used = 0;
  for (int k = 0; k < RQ_TRACE_KINDS; ++k) {
    if (counts_host) counts_host[k] = counts[k];
    if (ms_host) ms_host[k] = ms[k];
  }
  return s;
}

rq_status rq_act_cache_invalidate(rq_ctx* ctx) {
  if (ctx == nullptr) return RQ_ERR_NULL;
  ++ctx->gen;
  return RQ_OK;
}

rq_status rq_get_device_status(rq_stream_t stream) {
  return read_and_clear_device_error(reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_debug_wait_timeout(int64_t limit_ns, rq_stream_t stream) {
  if (limit_ns < 1 || limit_ns > 10000000000LL) return RQ_ERR_SHAPE;
  return launch_debug_wait_timeout(limit_ns, reinterpret_cast<cudaStream_t>(stream));
}

rq_status rq_gemv_exact_outputs(rq_stream_t stream, int64_t* count_host) {
  if (count_host == nullptr) return RQ_ERR_NULL;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return RQ_ERR_CUDA;
  return read_and_clear_gemv_exact_outputs(count_host);
}

}  // extern "C"
