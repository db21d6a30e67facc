// token_logprobs.cu -- log probabilities of given tokens under the softmax of each row of logits,
// with the row's entropy and its most likely alternatives, and the gradient of both.
//
//   z = a l,  lse = log sum_j exp(z_j),  logprob = z_t - lse,  H = lse - sum_j p_j z_j,  p_j = exp(z_j - lse)
//   dl_j = a (dlp (1[j = t] - p_j) - dH p_j (log p_j + H))
//
// One pass: a thread keeps the running maximum m of its logits, s = sum exp(a (l - m)) and
// q = sum exp(a (l - m)) (l - m), all FP32; a larger maximum m' scales s by f = exp(a (m - m')) and
// makes q (q + s (m - m')) f. Partial triples join by the same rule, so threads, warps and the CTAs of
// a cluster that share a row combine in any fixed order: lse = a m + log s, H = log s - a q / s.
//
// Alternatives: logits are ordered by 64-bit keys (value, then the lower index), all different. The k-th
// largest of the threads' maxima is no larger than the row part's k-th largest logit, so only the k
// threads at or above it hold candidates, and only their logits are read again (from L2).
//
// Bound by the bytes of the logits. A row is split over a cluster of 1 to 8 CTAs that join through
// shared memory, so few rows still use many SMs and no workspace or second launch is needed.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "host_common.h"

namespace dtcp {

constexpr int kLogprobThreads = 512;
constexpr int kLogprobWarps = kLogprobThreads / 32;
constexpr int kLogprobMaxTop = 32;
constexpr float kLog2e = 1.4426950408889634f;

struct LogprobParams {
  const void* logits;
  const long long* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  float* top_logprobs;
  int* top_ids;
  long long ld;
  int rows, vocab, top, cluster;
  float scale;
};

struct LogprobBackwardParams {
  const void* logits;
  const long long* tokens;
  const float* lse;
  const float* entropy;
  const float* dlogprob;
  const float* dentropy;
  void* dlogits;
  long long ld, ldd;
  int rows, vocab, parts;
  float scale;
};

namespace {

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kMinusInf = -__builtin_huge_valf();

// One aligned 16-byte vector of logits.
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {  // BF16
  static constexpr int N = 8;
  static __device__ __forceinline__ float value(uint16_t e) { return __uint_as_float(static_cast<uint32_t>(e) << 16); }
  static __device__ __forceinline__ uint16_t minus_inf() { return 0xFF80u; }
  static __device__ __forceinline__ void unpack(uint4 p, float (&v)[8]) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2_rn(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ uint16_t element(float v) {
    return static_cast<uint16_t>(pack_bf16x2_rn(__float_as_uint(v), 0u) & 0xFFFFu);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float value(float e) { return e; }
  static __device__ __forceinline__ float minus_inf() { return kMinusInf; }
  static __device__ __forceinline__ void unpack(uint4 p, float (&v)[4]) {
    v[0] = __uint_as_float(p.x);
    v[1] = __uint_as_float(p.y);
    v[2] = __uint_as_float(p.z);
    v[3] = __uint_as_float(p.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  static __device__ __forceinline__ float element(float v) { return v; }
};

// A row as aligned vectors: vector v holds logits v N - phase .. v N - phase + N - 1; the first and
// the last may be partly outside the row.
template <typename T>
struct Row {
  const T* base;
  int vocab, phase, vectors;
  __device__ __forceinline__ Row(const T* row, int n) : base(row), vocab(n) {
    phase = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    vectors = static_cast<int>((static_cast<long long>(n) + phase + Vec<T>::N - 1) / Vec<T>::N);
  }
  __device__ __forceinline__ int first(int v) const { return v * Vec<T>::N - phase; }
  __device__ __forceinline__ bool whole(int v) const { return first(v) >= 0 && first(v) <= vocab - Vec<T>::N; }
  // Minus infinity outside the row.
  __device__ __forceinline__ void load(int v, float (&x)[Vec<T>::N]) const {
    const int c = first(v);
    if (whole(v)) {
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(base + c), x);
      return;
    }
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) x[j] = (c + j >= 0 && c + j < vocab) ? Vec<T>::value(base[c + j]) : kMinusInf;
  }
};

// Order of logits: larger value first (-0 as 0, NaN first of all), then the lower index. 0 is no logit.
__device__ __forceinline__ unsigned long long key_of(float l, int index) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  uint32_t hi = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  if (l != l) hi = 0xFFFFFFFFu;
  return static_cast<unsigned long long>(hi) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ int key_index(unsigned long long key) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}
__device__ __forceinline__ float key_value(unsigned long long key) {
  const uint32_t hi = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((hi & 0x80000000u) ? (hi == 0xFFFFFFFFu ? 0x7FFFFFFFu : hi & 0x7FFFFFFFu) : ~hi);
}

__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long key) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
  return static_cast<unsigned long long>(hi) << 32 | lo;
}

// Descending order over the lanes of a warp (bitonic).
__device__ __forceinline__ unsigned long long warp_sort(unsigned long long key) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int stride = size / 2; stride > 0; stride >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, stride);
      const bool keep_max = ((lane & stride) == 0) == ((lane & size) == 0);
      key = keep_max ? (key > other ? key : other) : (key < other ? key : other);
    }
  }
  return key;
}

struct Triple {
  float m, s, q;
};

__device__ __forceinline__ float clamp_low(float d) { return max_nan(d, -1.0e30f); }

// Joins two parts of a row; c = a log2(e). A part whose maximum is minus infinity holds no mass.
__device__ __forceinline__ Triple join(const Triple& a, const Triple& b, float c) {
  if (a.m == kMinusInf) return b;
  if (b.m == kMinusInf) return a;
  Triple r;
  r.m = max_nan(a.m, b.m);
  const float da = clamp_low(a.m - r.m), db = clamp_low(b.m - r.m);
  const float fa = ex2_approx(da * c), fb = ex2_approx(db * c);
  r.s = a.s * fa + b.s * fb;
  r.q = (a.q + a.s * da) * fa + (b.q + b.s * db) * fb;
  return r;
}

__device__ __forceinline__ Triple warp_join(Triple t, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Triple u;
    u.m = __shfl_xor_sync(0xffffffffu, t.m, o);
    u.s = __shfl_xor_sync(0xffffffffu, t.s, o);
    u.q = __shfl_xor_sync(0xffffffffu, t.q, o);
    t = join(t, u, c);
  }
  return t;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

struct LogprobShared {
  Triple parts[kLogprobWarps];
  Triple total;
  unsigned long long lists[kLogprobWarps][32];  // each warp's thread maxima in order; then candidates
  unsigned long long winners[kLogprobMaxTop];   // the CTA's k largest thread maxima
  unsigned long long top[kLogprobMaxTop];       // the CTA's k largest logits
  unsigned long long best[kLogprobWarps];
  unsigned long long joined[8 * kLogprobMaxTop];
  int candidates;
};

// The `top` largest logits of this CTA's vectors [v0, v1) into sh.top, in order (0 where there are fewer).
template <typename T>
__device__ void select_top(LogprobShared& sh, const Row<T>& row, int v0, int v1, int thread_vector, int top) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // this thread's largest logit, the lowest index first
  unsigned long long mine = 0;
  if (thread_vector < v1) {
    float x[N];
    row.load(thread_vector, x);
    const int c = row.first(thread_vector);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (c + j >= 0 && c + j < row.vocab) {
        const unsigned long long key = key_of(x[j], c + j);
        mine = key > mine ? key : mine;
      }
  }
  sh.lists[warp][lane] = warp_sort(mine);
  if (tid < kLogprobMaxTop) sh.top[tid] = 0;
  if (tid == 0) sh.candidates = 0;
  __syncthreads();
  if (warp == 0) {
    int at = 0;
    unsigned long long head = lane < kLogprobWarps ? sh.lists[lane][0] : 0ull;
    for (int j = 0; j < top; ++j) {
      const unsigned long long best = warp_max_key(head);
      if (lane == 0) sh.winners[j] = best;
      if (head == best && best != 0) {
        ++at;
        head = at < 32 ? sh.lists[lane][at] : 0ull;
      }
    }
  }
  __syncthreads();
  const unsigned long long threshold = sh.winners[top - 1];  // 0: fewer threads hold logits than are wanted
  unsigned long long* cand = &sh.lists[0][0];
  for (int j = warp; j < top; j += kLogprobWarps) {
    const unsigned long long key = sh.winners[j];
    if (key == 0) break;
    const int owner = ((key_index(key) + row.phase) / N - v0) % kLogprobThreads;
    for (int v = v0 + owner + lane * kLogprobThreads; v < v1; v += 32 * kLogprobThreads) {
      float x[N];
      row.load(v, x);
      const int c = row.first(v);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i >= 0 && c + i < row.vocab) {
          const unsigned long long k = key_of(x[i], c + i);
          if (k >= threshold) {
            const int n = atomicAdd(&sh.candidates, 1);
            if (n < kLogprobThreads) cand[n] = k;
          }
        }
    }
  }
  __syncthreads();
  const int n = sh.candidates;
  if (n <= kLogprobThreads) {
    // the order by counting: keys are all different, so the places do not depend on the order of arrival
    if (tid < n) {
      const unsigned long long key = cand[tid];
      int rank = 0;
      for (int i = 0; i < n; ++i) rank += cand[i] > key ? 1 : 0;
      if (rank < top) sh.top[rank] = key;
    }
    __syncthreads();
    return;
  }
  // more candidates than places for them (long runs of large logits in few threads): the largest one below the last, `top` times
  unsigned long long last = ~0ull;
  for (int j = 0; j < top; ++j) {
    unsigned long long best = 0;
    for (int w = warp; w < top; w += kLogprobWarps) {
      const unsigned long long key = sh.winners[w];
      if (key == 0) break;
      const int owner = ((key_index(key) + row.phase) / N - v0) % kLogprobThreads;
      for (int v = v0 + owner + lane * kLogprobThreads; v < v1; v += 32 * kLogprobThreads) {
        float x[N];
        row.load(v, x);
        const int c = row.first(v);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (c + i >= 0 && c + i < row.vocab) {
            const unsigned long long k = key_of(x[i], c + i);
            if (k < last && k > best) best = k;
          }
      }
    }
    best = warp_max_key(best);
    if (lane == 0) sh.best[warp] = best;
    __syncthreads();
    last = warp_max_key(lane < kLogprobWarps ? sh.best[lane] : 0ull);
    if (tid == 0) sh.top[j] = last;
    __syncthreads();
  }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kLogprobThreads) token_logprobs_kernel(const LogprobParams p) {
  constexpr int N = Vec<T>::N;
  __shared__ LogprobShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long long r = blockIdx.x / p.cluster;
  pdl_launch_dependents();
  pdl_wait();
  const Row<T> row(static_cast<const T*>(p.logits) + r * p.ld, p.vocab);
  const int v0 = static_cast<int>(static_cast<long long>(row.vectors) * rank / p.cluster);
  const int v1 = static_cast<int>(static_cast<long long>(row.vectors) * (rank + 1) / p.cluster);
  const float c = p.scale * kLog2e;

  Triple t{kMinusInf, 0.0f, 0.0f};
  float ref = 0.0f;  // t.m, or 0 while it is minus infinity
  int best_vector = v0 + tid;
  for (int v = v0 + tid; v < v1; v += kLogprobThreads) {
    float x[N];
    row.load(v, x);
    float top = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) top = max_nan(top, x[j]);
    if (!(top <= t.m)) {
      const float m = max_nan(t.m, top);
      if (t.m != kMinusInf) {
        const float d = clamp_low(t.m - m), f = ex2_approx(d * c);
        t.q = (t.q + t.s * d) * f;
        t.s *= f;
      }
      if (t.m == t.m) best_vector = v;  // (the first NaN stays the largest)
      t.m = ref = m;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float d = clamp_low(x[j] - ref), e = ex2_approx(d * c);
      t.s += e;
      t.q = fmaf(e, d, t.q);
    }
  }
  t = warp_join(t, c);
  if (lane == 0) sh.parts[warp] = t;
  __syncthreads();
  if (warp == 0) {
    t = lane < kLogprobWarps ? sh.parts[lane] : Triple{kMinusInf, 0.0f, 0.0f};
    t = warp_join(t, c);
    if (lane == 0) sh.total = t;
  }
  if constexpr (TOP) select_top(sh, row, v0, v1, best_vector, p.top);

  if (p.cluster > 1) cluster_sync_all();
  else __syncthreads();
  if (rank == 0) {
    const uint32_t total_addr = smem_u32(&sh.total);
    Triple all = sh.total;
    for (int k = 1; k < p.cluster; ++k) {
      const uint32_t a = mapa_shared(total_addr, k);
      all = join(all, Triple{__uint_as_float(ld_cluster_u32(a)), __uint_as_float(ld_cluster_u32(a + 4)),
                             __uint_as_float(ld_cluster_u32(a + 8))},
                 c);
    }
    const bool empty = all.m == kMinusInf;  // no logit has any mass
    const float log_s = logf(all.s);
    const float lse = empty ? kMinusInf : fmaf(p.scale, all.m, log_s);
    if (tid == 0) {
      p.lse[r] = lse;
      p.entropy[r] = empty ? 0.0f : log_s - p.scale * (all.q / all.s);
      if (p.logprob != nullptr) {
        const long long token = p.tokens[r];
        float lp = 0.0f;
        if (token >= p.vocab) lp = __uint_as_float(0x7FFFFFFFu);
        else if (token >= 0) lp = empty ? kMinusInf : p.scale * (Vec<T>::value(row.base[token]) - all.m) - log_s;
        p.logprob[r] = lp;
      }
    }
    if constexpr (TOP) {
      const int n = p.cluster * p.top;
      unsigned long long key = 0;
      if (tid < n) key = ld_cluster_u64(mapa_shared(smem_u32(&sh.top[tid % p.top]), tid / p.top));
      if (tid < n) sh.joined[tid] = key;
      __syncthreads();
      if (key != 0) {
        int place = 0;
        for (int i = 0; i < n; ++i) place += sh.joined[i] > key ? 1 : 0;
        if (place < p.top) {
          const long long at = r * p.top + place;
          p.top_ids[at] = key_index(key);
          p.top_logprobs[at] = empty ? kMinusInf : p.scale * (key_value(key) - all.m) - log_s;
        }
      }
    }
  }
  if (p.cluster > 1) cluster_sync_all();  // the others' shared memory is read until here
}

// ---------------------------------------------------------------- backward

constexpr int kLogprobBackThreads = 256;
constexpr int kLogprobBackVectors = 8;  // per thread

template <typename T>
__global__ void __launch_bounds__(kLogprobBackThreads) token_logprobs_backward_kernel(const LogprobBackwardParams p) {
  constexpr int N = Vec<T>::N;
  pdl_launch_dependents();
  pdl_wait();
  const long long r = blockIdx.x / p.parts;
  const int part = static_cast<int>(blockIdx.x % p.parts);
  const Row<T> row(static_cast<const T*>(p.logits) + r * p.ld, p.vocab);
  T* out = static_cast<T*>(p.dlogits) + r * p.ldd;
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.base)) & 15u) == 0;
  const long long token = p.tokens != nullptr ? p.tokens[r] : -1;
  const float lse = p.lse[r];
  const float dlp = token >= 0 ? p.dlogprob[r] : 0.0f;
  const float dh = p.dentropy != nullptr ? p.dentropy[r] : 0.0f;
  // dl_j = p_j (A + B log p_j), and a dlp more at the token
  const float bad = token >= p.vocab ? __uint_as_float(0x7FFFFFFFu) : 0.0f;
  const float A = -p.scale * (dlp + (dh != 0.0f ? dh * p.entropy[r] : 0.0f)) + bad, B = -p.scale * dh;
  const bool empty = lse == kMinusInf;
  const int v0 = part * (kLogprobBackThreads * kLogprobBackVectors) + static_cast<int>(threadIdx.x);
#pragma unroll 2
  for (int k = 0; k < kLogprobBackVectors; ++k) {
    const int v = v0 + k * kLogprobBackThreads;
    if (v >= row.vectors) break;
    float x[N];
    row.load(v, x);
    const int c = row.first(v);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float logp = clamp_low(fmaf(x[j], p.scale, -lse));
      x[j] = ex2_approx(logp * kLog2e) * fmaf(B, logp, A);
      if (empty) x[j] = 0.0f;
    }
    if (token >= c && token < c + N && !empty) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c + j == token) x[j] = fmaf(p.scale, dlp, x[j]);
    }
    if (same && row.whole(v)) {
      *reinterpret_cast<uint4*>(out + c) = Vec<T>::pack(x);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c + j >= 0 && c + j < row.vocab) out[c + j] = Vec<T>::element(x[j]);
    }
  }
}

// ---------------------------------------------------------------- host side

void launch_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], long long grid, int threads, int cluster,
                  cudaStream_t stream) {
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
}

template <typename T>
int run_token_logprobs(const LogprobParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  launch_config(cfg, attr, static_cast<long long>(p.rows) * p.cluster, kLogprobThreads, p.cluster, stream);
  const auto kernel = p.top > 0 ? token_logprobs_kernel<T, true> : token_logprobs_kernel<T, false>;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

template <typename T>
int run_token_logprobs_backward(LogprobBackwardParams p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  const long long vectors = (static_cast<long long>(p.vocab) + Vec<T>::N - 1) / Vec<T>::N + 1;
  const long long each = kLogprobBackThreads * kLogprobBackVectors;
  p.parts = static_cast<int>((vectors + each - 1) / each);
  if (static_cast<long long>(p.rows) * p.parts > 0x7FFFFFFFLL) return GEMM_ERR_UNSUPPORTED_SHAPE;
  launch_config(cfg, attr, static_cast<long long>(p.rows) * p.parts, kLogprobBackThreads, 1, stream);
  if (cudaLaunchKernelEx(&cfg, token_logprobs_backward_kernel<T>, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace
}  // namespace dtcp

using namespace dtcp;

extern "C" {

int gemm_token_logprobs(const void* logits, int type, const long long* tokens, float* logprob, float* entropy, float* lse,
                        int top, float* top_logprobs, int* top_ids, int rows, int vocab, long long ld, float scale,
                        void* stream) {
  if (rows < 0 || vocab < 0 || top < 0 || ld < 0 || (type != GEMM_LOGITS_BF16 && type != GEMM_LOGITS_F32))
    return GEMM_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || scale > 3.0e38f) return GEMM_ERR_INVALID_ARG;
  if (top > kLogprobMaxTop) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return GEMM_OK;
  if (vocab == 0 || top > vocab) return GEMM_ERR_INVALID_ARG;
  if (logits == nullptr || entropy == nullptr || lse == nullptr || (logprob != nullptr && tokens == nullptr) ||
      (top > 0 && (top_logprobs == nullptr || top_ids == nullptr)))
    return GEMM_ERR_INVALID_ARG;
  if (ld == 0) ld = vocab;
  if (ld < vocab) return GEMM_ERR_INVALID_ARG;
  if (vocab > (1 << 30) || rows > (1 << 27)) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (off(logits, type == GEMM_LOGITS_BF16 ? 2 : 4) || off(tokens, 8) || off(logprob, 4) || off(entropy, 4) ||
      off(lse, 4) || off(top_logprobs, 4) || off(top_ids, 4))
    return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  LogprobParams p;
  p.logits = logits;
  p.tokens = tokens;
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.top_logprobs = top_logprobs;
  p.top_ids = top_ids;
  p.ld = ld;
  p.rows = rows;
  p.vocab = vocab;
  p.top = top;
  p.scale = scale;
  // CTAs a row: while the rows alone leave SMs idle, and each CTA keeps at least a vector a thread
  const long long vectors = vocab / (type == GEMM_LOGITS_BF16 ? 8 : 4);
  p.cluster = 1;
  while (p.cluster < 8 && static_cast<long long>(rows) * p.cluster < 2LL * info->num_sms &&
         vectors > static_cast<long long>(p.cluster) * kLogprobThreads)
    p.cluster *= 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == GEMM_LOGITS_BF16 ? run_token_logprobs<uint16_t>(p, s) : run_token_logprobs<float>(p, s);
}

int gemm_token_logprobs_backward(const void* logits, int type, const long long* tokens, const float* lse,
                                 const float* entropy, const float* dlogprob, const float* dentropy, void* dlogits,
                                 int rows, int vocab, long long ld, long long ldd, float scale, void* stream) {
  if (rows < 0 || vocab < 0 || ld < 0 || ldd < 0 || (type != GEMM_LOGITS_BF16 && type != GEMM_LOGITS_F32))
    return GEMM_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || scale > 3.0e38f) return GEMM_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_OK;
  if (vocab == 0) return GEMM_ERR_INVALID_ARG;
  if (logits == nullptr || lse == nullptr || dlogits == nullptr || (dlogprob == nullptr) != (tokens == nullptr) ||
      (dentropy != nullptr && entropy == nullptr))
    return GEMM_ERR_INVALID_ARG;
  if (ld == 0) ld = vocab;
  if (ldd == 0) ldd = vocab;
  if (ld < vocab || ldd < vocab) return GEMM_ERR_INVALID_ARG;
  if (vocab > (1 << 30) || rows > (1 << 27)) return GEMM_ERR_UNSUPPORTED_SHAPE;
  const unsigned size = type == GEMM_LOGITS_BF16 ? 2 : 4;
  if (off(logits, size) || off(dlogits, size) || off(tokens, 8) || off(lse, 4) || off(entropy, 4) || off(dlogprob, 4) ||
      off(dentropy, 4))
    return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  if (current_device_info(&device, &err) == nullptr) return err;
  LogprobBackwardParams p;
  p.logits = logits;
  p.tokens = tokens;
  p.lse = lse;
  p.entropy = entropy;
  p.dlogprob = dlogprob;
  p.dentropy = dentropy;
  p.dlogits = dlogits;
  p.ld = ld;
  p.ldd = ldd;
  p.rows = rows;
  p.vocab = vocab;
  p.parts = 1;
  p.scale = scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == GEMM_LOGITS_BF16 ? run_token_logprobs_backward<uint16_t>(p, s) : run_token_logprobs_backward<float>(p, s);
}

}  // extern "C"
