// token_logprobs.cu -- log probabilities of given tokens under the softmax of each row of logits,
// with the row's entropy and its most likely alternatives, and the gradient of both.
//
//   z = a l,  lse = log sum_j exp(z_j),  logprob = z_t - lse,  H = lse - sum_j p_j z_j,  p_j = exp(z_j - lse)
//   dl_j = a (dlp (1[j = t] - p_j) - dH p_j (log p_j + H))
//
// One pass in powers of two: with c = a log2(e), a thread keeps the maximum m of its logits and, over t = c (l - m) of
// all of them but one that is m itself, s = sum 2^t and q = sum t 2^t, all FP32. When m grows by d / c, the old one
// joins the others: s becomes (s + 1) 2^-d and q (q - (s + 1) d) 2^-d. Partial results join by the same rule, so
// threads, warps and the CTAs of a cluster that share a row combine in a fixed order: lse = a m + log1p(s), H =
// log1p(s) - ln 2 q / (1 + s). The largest logit's own term is never rounded into s, and no two numbers of the results
// cancel, so a row that one logit dominates keeps its digits, a log probability is never above 0 and an entropy never
// below it. Where c m is beyond 2^60, logits that differ at all have no mass next to m: s counts the logits equal to
// m.
//
// Alternatives: a value that k threads' maxima reach is no larger than the k-th largest logit. At a row's end the CTA
// takes such a bound, and the threads whose maxima reach it have the logits read again (from L2) that may: each thread
// remembers its two largest chunk maxima and the chunk of the first, so that is one chunk's part of 8 vectors for most
// of them. The few logits that reach the bound are put in order by 64-bit keys (value, then the lower index), all
// different; the order in which they arrive (shared-memory atomics) does not matter. Logits of minus infinity take no
// part: where there are fewer others than are wanted, the lowest indices follow.
//
// Powers of two are ex2.approx (2^-22): the sums average that out, and the results' errors are those of FP32 (log
// probabilities 3e-8, entropy 5e-8 of their size). The gradient's p_j = exp(z_j - lse) takes lse as it was written,
// rounded to FP32: an error of p_j of up to |lse| 2^-24, the same for all of a row (7e-7 at an lse of 12).
//
// Bound by the bytes of the logits: measured on GB300, 4096 x 131072 BF16 160.5 us (6.7 TB/s), with 20 alternatives
// 214; 4096 x 65536 FP32 151 (7.1); their gradients 330 us (6.5 TB/s) and 319 (6.7). Following the maximum in every
// chunk costs 1% against a reference that may trail it (158.6 us). A row is split over a cluster of 1 to 8 CTAs that
// join through shared memory, so few rows still use many SMs and no workspace or second launch is needed.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "host_common.h"

namespace dtcp {

constexpr int kLogprobThreads = 256;
constexpr int kLogprobWarps = kLogprobThreads / 32;
constexpr int kLogprobMaxTop = 32;
// The row parts stream through a ring of chunks in shared memory: bulk copies keep chunks in flight without
// holding registers, also through the reductions at a row's end, when they are the next row's.
constexpr int kLogprobBatch = 8;  // vectors per thread and chunk
constexpr int kLogprobChunk = kLogprobBatch * kLogprobThreads;  // vectors
constexpr int kLogprobStages = 3;  // of the ring with two CTAs an SM; two with three CTAs
constexpr int kLogprobCtas = 3;    // per SM at most
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LogprobParams {
  const void* logits;
  const long long* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  float* top_logprobs;
  int* top_ids;
  long long ld;
  int rows, vocab, top, cluster, stages;
  float scale;
  unsigned* status;
  unsigned long long wait_limit_ns;
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
  static constexpr uint32_t kMinusInfWord = 0xFF80FF80u;
  static __device__ __forceinline__ uint16_t minus_inf() { return 0xFF80u; }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // Largest element (NaN if one is) of `n` vectors, and pair j of the elements in packed FP32.
  template <int M>
  static __device__ __forceinline__ float largest(const uint4 (&p)[M]) {
    uint32_t a[M];
#pragma unroll
    for (int u = 0; u < M; ++u) a[u] = max2(max2(p[u].x, p[u].y), max2(p[u].z, p[u].w));
#pragma unroll
    for (int u = 1; u < M; ++u) a[0] = max2(a[0], a[u]);
    return max_nan(__uint_as_float(a[0] << 16), __uint_as_float(a[0] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint64_t pair(uint4 p, int j) {
    const uint32_t w = j == 0 ? p.x : j == 1 ? p.y : j == 2 ? p.z : p.w;
    return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
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
  static constexpr uint32_t kMinusInfWord = 0xFF800000u;
  static __device__ __forceinline__ float minus_inf() { return kMinusInf; }
  template <int M>
  static __device__ __forceinline__ float largest(const uint4 (&p)[M]) {
    float a[M];
#pragma unroll
    for (int u = 0; u < M; ++u)
      a[u] = max_nan(max_nan(__uint_as_float(p[u].x), __uint_as_float(p[u].y)),
                     max_nan(__uint_as_float(p[u].z), __uint_as_float(p[u].w)));
#pragma unroll
    for (int u = 1; u < M; ++u) a[0] = max_nan(a[0], a[u]);
    return a[0];
  }
  static __device__ __forceinline__ uint64_t pair(uint4 p, int j) {
    return j == 0 ? f2_pack(__uint_as_float(p.x), __uint_as_float(p.y))
                  : f2_pack(__uint_as_float(p.z), __uint_as_float(p.w));
  }
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
  // First vector of part `k` of `parts`.
  __device__ __forceinline__ int begin(int k, int parts) const {
    return static_cast<int>(static_cast<long long>(vectors) * k / parts);
  }
  __device__ __forceinline__ int first(int v) const { return v * Vec<T>::N - phase; }
  __device__ __forceinline__ bool whole(int v) const { return first(v) >= 0 && first(v) <= vocab - Vec<T>::N; }
  __device__ __forceinline__ uint4 raw(int v) const { return *reinterpret_cast<const uint4*>(base + first(v)); }
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

// Part `k` of `parts` of a row: vectors [v0, v1), of which [n0, n1) are whole.
template <typename T>
struct Part {
  int v0, v1, n0, n1;
  __device__ __forceinline__ Part(const Row<T>& row, int k, int parts) {
    v0 = row.begin(k, parts);
    v1 = row.begin(k + 1, parts);
    n0 = v0;
    n1 = v1;
    if (v0 == v1) return;
    if (v0 == 0 && !row.whole(0)) n0 = 1;
    if (n1 == row.vectors && n1 > n0 && !row.whole(n1 - 1)) --n1;
  }
};

// Copies `bytes` (a multiple of 16) from global to this CTA's shared memory, both at 16-byte boundaries; completion is
// counted on the mbarrier `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// The chunks of this CTA's row parts in order, one row after another (one thread's state).
template <typename T>
struct Feed {
  const T* logits;
  long long ld, row, step;
  int rows, vocab, rank, cluster;
  int at, end;  // next vector and end of the current row part
  const T* base;
  int phase;

  __device__ __forceinline__ void start(long long r) {
    for (row = r; row < rows; row += step) {
      const Row<T> x(logits + row * ld, vocab);
      const Part<T> part(x, rank, cluster);
      if (part.n0 < part.n1) {
        base = x.base;
        phase = x.phase;
        at = part.n0;
        end = part.n1;
        return;
      }
    }
  }
  __device__ __forceinline__ void issue(uint32_t dst, uint32_t bar) {
    if (row >= rows) return;
    const int n = min(end - at, kLogprobChunk);
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n) * 16u);
    bulk_load(dst, base + (static_cast<long long>(at) * Vec<T>::N - phase), static_cast<uint32_t>(n) * 16u, bar);
    at += n;
    if (at == end) start(row + step);
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

// The order of logits as unsigned numbers: 0 for minus infinity (and for none).
__device__ __forceinline__ uint32_t order_of(float l) {
  return l == kMinusInf ? 0u : static_cast<uint32_t>(key_of(l, 0) >> 32);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return o == 0 ? kMinusInf : key_value(static_cast<unsigned long long>(o) << 32);
}

__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long key) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
  return static_cast<unsigned long long>(hi) << 32 | lo;
}

constexpr float kOrdinary = 1.152921504606847e18f;  // |m c| below 2^60

// Sums of a part of a row relative to its maximum, without one logit that is the maximum (see above); m minus infinity:
// no mass.
struct Sums {
  float m, s, q;
};

// c (from - to), with no mass (and no NaN) left where that has no finite value, nor where it multiplies a sum.
__device__ __forceinline__ float shift(float from, float to, float c) { return fmaxf((from - to) * c, -1.0e20f); }

// The sums of a warp's lanes as one, the same in every lane, relative to the largest of their maxima. The maximum left
// out is that of the first lane that has it.
__device__ __forceinline__ Sums warp_join(const Sums& a, float c) {
  const bool mass = a.m != kMinusInf;
  Sums r;
  r.m = order_value(__reduce_max_sync(0xffffffffu, order_of(a.m)));
  const bool has = mass && a.m == r.m;
  const uint32_t holders = __ballot_sync(0xffffffffu, has);  // (every lane takes part)
  const bool first = static_cast<int>(threadIdx.x & 31) == __ffs(static_cast<int>(holders)) - 1;
  const float d = has ? 0.0f : shift(a.m, r.m, c), f = ex2_approx(d);
  const float all = first ? a.s : a.s + 1.0f;
  r.s = mass ? all * f : 0.0f;
  r.q = mass ? fmaf(all, d, a.q) * f : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
    r.q += __shfl_xor_sync(0xffffffffu, r.q, o);
  }
  return r;
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

constexpr int kLogprobList = 768;  // candidates of a row part
constexpr int kLogprobDeep = 6;    // largest values of each warp that a bound is taken from

struct LogprobShared {
  Sums parts[kLogprobWarps];
  Sums total;
  uint32_t highest[2][kLogprobDeep][kLogprobWarps];  // each warp's largest values in order, for the two bounds of a row
  unsigned long long cand[kLogprobList];
  unsigned long long survivors[kLogprobThreads];
  unsigned long long top[kLogprobMaxTop];  // the CTA's k largest logits
  unsigned long long best[kLogprobWarps];
  unsigned long long full[kLogprobStages], empty[kLogprobStages];  // mbarriers of the ring
  uint32_t winner[kLogprobThreads];  // threads whose logits are read again, with the chunk
  int candidates, left, winners, scanners;
  uint32_t abort;
};

// An order that at least `top` of the threads' orders reach, or 0: if j of them in each of r warps reach one and
// j r >= top, top do; the largest such one over j is the r-th largest of the warps' j-th largest. One barrier.
__device__ __forceinline__ uint32_t cta_bound(uint32_t (&highest)[kLogprobDeep][kLogprobWarps], uint32_t mine,
                                              int top) {
  static_assert(kLogprobWarps == 8, "groups of 8 lanes take one value of each warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < kLogprobDeep; ++j) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, mine);
    if (lane == __ffs(static_cast<int>(__ballot_sync(0xffffffffu, mine == most))) - 1) {
      highest[j][warp] = most;
      mine = 0u;
    }
  }
  __syncthreads();
  uint32_t bound = 0u;
#pragma unroll
  for (int j0 = 0; j0 < kLogprobDeep; j0 += 4) {
    const int j = j0 + (lane >> 3), i = lane & 7;
    const uint32_t v = j < kLogprobDeep ? highest[j][i] : 0u;
    int larger = 0;
#pragma unroll
    for (int x = 1; x < 8; ++x) {
      const uint32_t other = __shfl_xor_sync(0xffffffffu, v, x);
      larger += other > v || (other == v && (i ^ x) < i) ? 1 : 0;
    }
    if (larger == (top + j) / (j + 1) - 1) bound = v > bound ? v : bound;
  }
  return __reduce_max_sync(0xffffffffu, bound);
}

__device__ __forceinline__ void list_candidate(LogprobShared& sh, unsigned long long key) {
  const int n = atomicAdd(&sh.candidates, 1);
  if (n < kLogprobList) sh.cand[n] = key;
}

// The largest logit of a thread's part of each chunk: the largest of them, its chunk, and the second largest (NaN:
// there may be any number of large ones).
struct Peaks {
  float first, second;
  int chunk;
  __device__ __forceinline__ void see(float most, int at) {
    const bool more = most > first || (most != most && first == first);
    float low;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(low) : "f"(most), "f"(first));
    second = max_nan(second, low);
    first = max_nan(first, most);
    chunk = more ? at : chunk;
  }
};

// The `top` largest keys into sh.top by taking the largest one below the last, `top` times. up_to(limit): the
// thread's largest key that is no larger than `limit` (all of them at first: a NaN at index 0 has the largest there
// is).
template <typename F>
__device__ __forceinline__ void extract_top(LogprobShared& sh, int top, F up_to) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long limit = ~0ull;
  for (int j = 0; j < top; ++j) {
    const unsigned long long best = warp_max_key(up_to(limit));
    if (lane == 0) sh.best[warp] = best;
    __syncthreads();
    const unsigned long long next = warp_max_key(lane < kLogprobWarps ? sh.best[lane] : 0ull);
    if (threadIdx.x == 0) sh.top[j] = next;
    limit = next == 0 ? 0 : next - 1;
    __syncthreads();
  }
}

// The `top` largest logits of this CTA's part of a row into sh.top, in order (0 where there are fewer). The logits of
// vectors that are not whole have been listed (before a barrier).
template <typename T>
__device__ void select_top(LogprobShared& sh, const Row<T>& row, const Part<T>& part, const Peaks& peaks, int top) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x;
  const float bound = order_value(cta_bound(sh.highest[0], order_of(peaks.first), top));
  auto reaches = [&](float l) { return !(l < bound) && l != kMinusInf; };  // (a NaN does)
  // the threads whose logits are read again: one chunk of them, or all
  if (reaches(peaks.first)) {
    if (reaches(peaks.second)) sh.winner[kLogprobThreads - 1 - atomicAdd(&sh.scanners, 1)] = static_cast<uint32_t>(tid);
    else sh.winner[atomicAdd(&sh.winners, 1)] = static_cast<uint32_t>(tid) | static_cast<uint32_t>(peaks.chunk) << 8;
  }
  __syncthreads();
  auto list = [&](int v) {
    if (v >= part.n1) return;
    const uint4 w[1] = {row.raw(v)};
    if (!reaches(Vec<T>::largest(w))) return;
    float x[N];
    Vec<T>::unpack(w[0], x);
    const int c = row.first(v);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (reaches(x[j])) list_candidate(sh, key_of(x[j], c + j));
  };
  for (int i = tid; i < sh.winners * kLogprobBatch; i += kLogprobThreads) {
    const uint32_t w = sh.winner[i / kLogprobBatch];
    list(part.n0 + static_cast<int>(w >> 8) * kLogprobChunk + (i % kLogprobBatch) * kLogprobThreads +
         static_cast<int>(w & 0xFFu));
  }
  const int steps = (part.n1 - part.n0 + kLogprobThreads - 1) / kLogprobThreads;
  for (int k = 0; k < sh.scanners; ++k)
    for (int i = tid; i < steps; i += kLogprobThreads)
      list(part.n0 + static_cast<int>(sh.winner[kLogprobThreads - 1 - k]) + i * kLogprobThreads);
  __syncthreads();
  const int n = sh.candidates;
  if (n > kLogprobList) {
    // more candidates than the list holds (very many equal ones): from the row itself
    extract_top(sh, top, [&](unsigned long long limit) {
      unsigned long long best = 0;
      for (int v = part.v0 + tid; v < part.v1; v += kLogprobThreads) {
        float x[N];
        row.load(v, x);
        const int c = row.first(v);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (x[i] != kMinusInf && c + i >= 0 && c + i < row.vocab) {
            const unsigned long long k = key_of(x[i], c + i);
            if (k <= limit && k > best) best = k;
          }
      }
      return best;
    });
    return;
  }
  const unsigned long long* keys = sh.cand;
  int left = n;
  if (n > kLogprobThreads) {
    // cut the list by a bound of its own
    uint32_t mine = 0;
    for (int i = tid; i < n; i += kLogprobThreads) mine = max(mine, static_cast<uint32_t>(sh.cand[i] >> 32));
    const uint32_t cut = cta_bound(sh.highest[1], mine, top);
    for (int i = tid; i < n; i += kLogprobThreads)
      if (static_cast<uint32_t>(sh.cand[i] >> 32) >= cut) {
        const int k = atomicAdd(&sh.left, 1);
        if (k < kLogprobThreads) sh.survivors[k] = sh.cand[i];
      }
    __syncthreads();
    keys = sh.survivors;
    left = sh.left;
  }
  if (left <= kLogprobThreads) {
    // the order by counting: keys are all different, so the places do not depend on the order of arrival
    if (tid < left) {
      const unsigned long long key = keys[tid];
      int place = 0;
#pragma unroll 8
      for (int i = 0; i < left; ++i) place += keys[i] > key ? 1 : 0;
      if (place < top) sh.top[place] = key;
    }
    __syncthreads();
    return;
  }
  extract_top(sh, top, [&](unsigned long long limit) {
    unsigned long long best = 0;
    for (int i = tid; i < n; i += kLogprobThreads)
      if (sh.cand[i] <= limit && sh.cand[i] > best) best = sh.cand[i];
    return best;
  });
}

// What a thread has seen of its row.
struct Running {
  float m, s, q;

  // (not NaN, not infinite)
  __device__ __forceinline__ bool ordinary(float c) const { return fabsf(m * c) < kOrdinary; }
  // Logits follow of which `top` is the largest: whether it is the new maximum (then one of them is left out of s).
  // Without a branch: some lane of a warp has a new maximum in almost every chunk.
  __device__ __forceinline__ bool see(float top, float c) {
    const float most = max_nan(m, top);
    const bool fresh = most != m;
    const float d = shift(m, most, c), f = ex2_approx(d);  // (0 and 1 where it stays)
    const float all = fresh && m != kMinusInf ? s + 1.0f : s;
    q = fmaf(all, d, q) * f;
    s = all * f;
    m = most;
    return fresh;
  }
  // The sums of a chunk or of a row's end, in two lanes of packed FP32, added to this. A new maximum's own term comes
  // out of the lane that has it (rounding could leave the sum of the others a little below 0 there).
  __device__ __forceinline__ void take(uint64_t s2, uint64_t q2, bool fresh) {
    float s0, s1, q0, q1;
    f2_unpack(s2, s0, s1);
    f2_unpack(q2, q0, q1);
    s += max_nan(max_nan(s0, s1) - (fresh ? 1.0f : 0.0f) + fminf(s0, s1), 0.0f);
    q += q0 + q1;
  }
};

// 2^t and t 2^t of two logits. CLAMP: they may be minus infinity, or so low that c l is (t 2^t is no number then).
template <bool CLAMP>
__device__ __forceinline__ uint64_t add_pair(uint64_t x2, uint64_t c2, uint64_t minus_m2, uint64_t& q2) {
  uint64_t t2 = f2_mul(f2_add(x2, minus_m2), c2);
  float t0, t1;
  f2_unpack(t2, t0, t1);
  if (CLAMP) {
    t0 = fmaxf(t0, -1.0e30f);
    t1 = fmaxf(t1, -1.0e30f);
    t2 = f2_pack(t0, t1);
  }
  const uint64_t e2 = f2_pack(ex2_approx(t0), ex2_approx(t1));
  q2 = f2_fma(e2, t2, q2);
  return e2;
}

// The same of a vector, its powers added among themselves first: next to the maximum's 1 fewer of them are rounded off.
template <typename T, bool CLAMP>
__device__ __forceinline__ void add_vector(uint4 raw, uint64_t c2, uint64_t minus_m2, uint64_t& s2, uint64_t& q2) {
  uint64_t e2 = f2_add(add_pair<CLAMP>(Vec<T>::pair(raw, 0), c2, minus_m2, q2),
                       add_pair<CLAMP>(Vec<T>::pair(raw, 1), c2, minus_m2, q2));
  if constexpr (Vec<T>::N == 8) {
    const uint64_t f2 = f2_add(add_pair<CLAMP>(Vec<T>::pair(raw, 2), c2, minus_m2, q2),
                               add_pair<CLAMP>(Vec<T>::pair(raw, 3), c2, minus_m2, q2));
    e2 = f2_add(e2, f2);
  }
  s2 = f2_add(s2, e2);
}

// Where the maximum is no ordinary number: 1 for a logit equal to it, NaN if it is infinite or NaN.
__device__ __forceinline__ float count_one(float x, float m) {
  if (m != m || m == -kMinusInf) return __uint_as_float(0x7FFFFFFFu);
  return x == m ? 1.0f : 0.0f;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kLogprobThreads, kLogprobCtas) token_logprobs_kernel(const LogprobParams p) {
  constexpr int N = Vec<T>::N;
  __shared__ LogprobShared sh;
  extern __shared__ __align__(128) uint8_t ring[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int clusters = gridDim.x / p.cluster;
  const long long r0 = blockIdx.x / p.cluster;
  const uint32_t full = smem_u32(sh.full), empty = smem_u32(sh.empty), ring_addr = smem_u32(ring);
  constexpr uint32_t STAGE = kLogprobChunk * 16;
  if (tid == 0) {
    for (int s = 0; s < kLogprobStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, kLogprobWarps);
    }
    sh.abort = 0u;
    fence_mbarrier_init_cluster();
  }
  __syncthreads();
  const WaitCtx wctx{&sh.abort, p.status, p.wait_limit_ns};
  pdl_launch_dependents();
  pdl_wait();
  Feed<T> feed;
  if (tid == 0) {
    feed.logits = static_cast<const T*>(p.logits);
    feed.ld = p.ld;
    feed.step = clusters;
    feed.rows = p.rows;
    feed.vocab = p.vocab;
    feed.rank = rank;
    feed.cluster = p.cluster;
    feed.start(r0);
    for (int s = 0; s < p.stages; ++s) feed.issue(ring_addr + s * STAGE, full + 8 * s);
  }
  const float c = p.scale * kLog2e;
  const uint64_t c2 = f2_pack(c, c);
  uint32_t stage = 0, parity = 0;  // of the next chunk
  uint32_t chunks = 0;
  bool ok = true;  // after a wait that gave up: no more waiting, the launch runs out (its results are void)
  for (long long r = r0; r < p.rows; r += clusters) {
    const Row<T> row(static_cast<const T*>(p.logits) + r * p.ld, p.vocab);
    const Part<T> part(row, rank, p.cluster);
    Running run{kMinusInf, 0.0f, 0.0f};
    bool masked = false;
    // the logits of vectors at the row's ends that are partly outside it, one per lane of the last warp: asked for
    // here, taken after the chunks
    T end_logit = Vec<T>::minus_inf();
    int end_index = -1;
    if (warp == kLogprobWarps - 1 && lane < 2 * N) {
      const bool tail = lane >= N;
      if (tail ? part.n1 < part.v1 : part.v0 < part.n0) end_index = row.first(tail ? part.n1 : part.v0) + lane % N;
      if (end_index >= row.vocab) end_index = -1;
      if (end_index >= 0) end_logit = row.base[end_index];
    }
    Peaks peaks{kMinusInf, kMinusInf, 0};
    if (TOP && tid == 0) sh.candidates = sh.left = sh.winners = sh.scanners = 0;
    if (TOP && tid < kLogprobMaxTop) sh.top[tid] = 0;
    if (TOP) __syncthreads();
    for (int v = part.n0; v < part.n1; v += kLogprobChunk) {
      if (tid == 0 && chunks > 0 && ok) {
        // the chunk before this one: refill its place once every warp has read it
        const uint32_t s = stage == 0 ? p.stages - 1 : stage - 1;
        const uint32_t ph = stage == 0 ? parity ^ 1u : parity;
        ok = wait_phase(empty + 8 * s, ph, wctx, status_code(kRoleProducer, s));
        if (ok) feed.issue(ring_addr + s * STAGE, full + 8 * s);
      }
      if (ok) ok = wait_phase(full + 8 * stage, parity, wctx, status_code(kRoleEpilogue, stage));
      const uint32_t src = ring_addr + stage * STAGE + static_cast<uint32_t>(tid) * 16u;
      const int left = part.n1 - v - tid;
      uint4 raw[kLogprobBatch];
      if (part.n1 - v >= kLogprobChunk) {
#pragma unroll
        for (int u = 0; u < kLogprobBatch; ++u)
          ld_shared_v4(src + u * (kLogprobThreads * 16), raw[u].x, raw[u].y, raw[u].z, raw[u].w);
      } else {
#pragma unroll
        for (int u = 0; u < kLogprobBatch; ++u) {
          constexpr uint32_t kNone = Vec<T>::kMinusInfWord;
          raw[u] = make_uint4(kNone, kNone, kNone, kNone);
          if (u * kLogprobThreads < left)
            ld_shared_v4(src + u * (kLogprobThreads * 16), raw[u].x, raw[u].y, raw[u].z, raw[u].w);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_local(empty + 8 * stage);
      ++chunks;
      stage = stage + 1 == static_cast<uint32_t>(p.stages) ? 0u : stage + 1;
      parity = stage == 0 ? parity ^ 1u : parity;
      if (left <= 0) continue;  // none of a row's last chunk (whole warps of a short one)
      const float most = Vec<T>::largest(raw);
      if (TOP) peaks.see(most, (v - part.n0) / kLogprobChunk);
      const bool fresh = run.see(most, c);
      uint64_t s2 = 0, q2 = 0;
      if (run.ordinary(c)) {
        const uint64_t minus_m2 = f2_pack(-run.m, -run.m);
        const bool full_chunk = part.n1 - v >= kLogprobChunk;  // (else some of `raw` is minus infinity)
        if (!masked && full_chunk) {
#pragma unroll
          for (int u = 0; u < kLogprobBatch; ++u) add_vector<T, false>(raw[u], c2, minus_m2, s2, q2);
          float q0, q1;
          f2_unpack(q2, q0, q1);
          if (q0 != q0 || q1 != q1) {  // logits without mass among them: from here on with a clamp
            masked = true;
            s2 = q2 = 0;
          }
        }
        if (masked || !full_chunk) {
#pragma unroll
          for (int u = 0; u < kLogprobBatch; ++u) {
            if (u * kLogprobThreads >= left) continue;
            add_vector<T, true>(raw[u], c2, minus_m2, s2, q2);
          }
        }
      } else if (run.m != kMinusInf) {
        float n = 0.0f;
#pragma unroll 1
        for (int u = 0; u < kLogprobBatch; ++u) {
          float x[N];
          uint4 w = raw[0];
#pragma unroll
          for (int i = 1; i < kLogprobBatch; ++i)
            if (u == i) w = raw[i];
          Vec<T>::unpack(w, x);
#pragma unroll
          for (int j = 0; j < N; ++j) n += count_one(x[j], run.m);
        }
        s2 = f2_pack(n, 0.0f);
      }
      run.take(s2, q2, fresh);
    }
    if (end_index >= 0) {
      const float x = Vec<T>::value(end_logit);
      if (TOP && x != kMinusInf) list_candidate(sh, key_of(x, end_index));
      const bool fresh = run.see(x, c);
      if (run.m != kMinusInf) {
        uint64_t e2, q2 = 0;
        if (run.ordinary(c)) e2 = add_pair<true>(f2_pack(x, kMinusInf), c2, f2_pack(-run.m, -run.m), q2);
        else e2 = f2_pack(count_one(x, run.m), 0.0f);
        run.take(e2, q2, fresh);
      }
    }
    Sums t = warp_join(Sums{run.m, run.s, run.q}, c);
    if (lane == 0) sh.parts[warp] = t;
    __syncthreads();
    if (warp == 0) {
      t = lane < kLogprobWarps ? sh.parts[lane] : Sums{kMinusInf, 0.0f, 0.0f};
      t = warp_join(t, c);
      if (lane == 0) sh.total = t;
    }
    if constexpr (TOP) select_top(sh, row, part, peaks, p.top);

    if (p.cluster > 1) cluster_sync_all();
    else __syncthreads();
    if (rank == 0) {
      Sums all{kMinusInf, 0.0f, 0.0f};
      if (lane < p.cluster) {
        const uint32_t at = mapa_shared(smem_u32(&sh.total), lane);
        all = Sums{__uint_as_float(ld_cluster_u32(at)), __uint_as_float(ld_cluster_u32(at + 4)),
                   __uint_as_float(ld_cluster_u32(at + 8))};
      }
      all = warp_join(all, c);
      const bool empty = all.m == kMinusInf;  // no logit has any mass
      const float log_s = log1pf(all.s);
      const float lse = empty ? kMinusInf : fmaf(p.scale, all.m, log_s);
      // log probability of a logit: no mass next to a maximum that is no ordinary number, unless it is that number
      const bool ordinary = fabsf(all.m * c) < kOrdinary;
      auto logp = [&](float l) {
        if (empty) return kMinusInf;
        if (ordinary || all.s != all.s) return p.scale * (l - all.m) - log_s;
        return l == all.m ? -log_s : kMinusInf;
      };
      if (tid == 0) {
        p.lse[r] = lse;
        p.entropy[r] = empty ? 0.0f : log_s - kLn2 * (all.q / (1.0f + all.s));
        if (p.logprob != nullptr) {
          // (Asked for at the row's start and carried to here, the token and its logit cost registers that the
          // alternatives need: 4096 x 131072 BF16 with 20 of them 230 us instead of 214, though 1500 x 50001 FP32 without
          // alternatives took 49.4 instead of 51.)
          const long long token = p.tokens[r];
          float lp = 0.0f;
          if (token >= p.vocab) lp = __uint_as_float(0x7FFFFFFFu);
          else if (token >= 0) lp = logp(Vec<T>::value(row.base[token]));
          p.logprob[r] = lp;
        }
      }
      if constexpr (TOP) {
        const int n = p.cluster * p.top;
        unsigned long long key = 0;
        if (tid < n) key = ld_cluster_u64(mapa_shared(smem_u32(&sh.top[tid % p.top]), tid / p.top));
        if (tid < n) sh.cand[tid] = key;
        const int listed = __syncthreads_count(key != 0);  // (n <= 256)
        auto write = [&](int place, int index, float l) {
          if (place >= p.top) return;
          p.top_ids[r * p.top + place] = index;
          p.top_logprobs[r * p.top + place] = logp(l);
        };
        if (key != 0) {
          int place = 0;
#pragma unroll 8
          for (int i = 0; i < n; ++i) place += sh.cand[i] > key ? 1 : 0;
          write(place, key_index(key), key_value(key));
        }
        if (listed < p.top && tid < 32) {
          // logits of minus infinity take the places left: the lowest indices, all among the first `top`
          const bool none = lane < p.top && Vec<T>::value(row.base[lane]) == kMinusInf;
          const uint32_t all_none = __ballot_sync(0xffffffffu, none);
          if (none) write(listed + __popc(all_none & ((1u << lane) - 1u)), lane, kMinusInf);
        }
      }
    }
    // the CTAs' shared memory is read until here
    if (p.cluster > 1) cluster_sync_all();
    else __syncthreads();
  }
  if (tid == 0 && !ok) settle_after_abort();
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
  const float row_lse = p.lse[r];
  const float dlp = token >= 0 ? p.dlogprob[r] : 0.0f;
  const float dh = p.dentropy != nullptr ? p.dentropy[r] : 0.0f;
  const float bad = token >= p.vocab ? __uint_as_float(0x7FFFFFFFu) : 0.0f;
  // dl_j = p_j (A + B log p_j), and a dlp more at the token. Where no logit has any mass every p_j is 0, against any
  // lse.
  const bool empty = row_lse == kMinusInf;
  const float lse = empty ? 0.0f : row_lse;
  const float A = empty ? bad : -p.scale * (dlp + (dh != 0.0f ? dh * p.entropy[r] : 0.0f)) + bad;
  const float B = empty ? 0.0f : -p.scale * dh;
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
      // (no mass is left far above -1e4, and B times it stays finite for any B below 3e34)
      const float logp = max_nan(fmaf(x[j], p.scale, -lse), -1.0e4f);
      x[j] = ex2_approx(logp * kLog2e) * fmaf(B, logp, A);
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
int run_token_logprobs(const LogprobParams& p, int ctas, int device, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  const auto kernel = p.top > 0 ? token_logprobs_kernel<T, true> : token_logprobs_kernel<T, false>;
  static std::atomic<unsigned long long> sized[2] = {};  // devices whose limit of shared memory is raised, by kernel
  const unsigned long long bit = 1ull << device;
  if ((sized[p.top > 0].load(std::memory_order_acquire) & bit) == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kLogprobStages * kLogprobChunk * 16) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
    sized[p.top > 0].fetch_or(bit, std::memory_order_release);
  }
  launch_config(cfg, attr, static_cast<long long>(std::min(p.rows, ctas / p.cluster)) * p.cluster, kLogprobThreads,
                p.cluster, stream);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.stages) * kLogprobChunk * 16;
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

int gemm_token_logprobs(const void* logits, int type, const long long* tokens, float* logprob, float* entropy,
                        float* lse, int top, float* top_logprobs, int* top_ids, int rows, int vocab, long long ld,
                        float scale, void* stream) {
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
  p.status = device_status_word(device);
  p.wait_limit_ns = RunOptions().wait_limit_ns;
  if (p.status == nullptr) return GEMM_ERR_NO_DEVICE;
  // Two or three CTAs an SM, each stepping over the rows (or its part of them), and 1 to 8 CTAs a row, by the time of
  // the launch: its rounds, each as long as a part at the CTA's share of the memory's rate (44 KB a microsecond and
  // SM) and about 2.5 us of reductions; each thread has a vector at least. Measured on GB300: 1500 x 50001 FP32
  // 51.1 us with two CTAs an SM and 53.9 with three, 4096 x 131072 BF16 166.8 and 159.2.
  const double row_bytes = static_cast<double>(vocab) * (type == GEMM_LOGITS_BF16 ? 2 : 4);
  double best = 0.0;
  int ctas = 0;
  for (int per_sm = kLogprobCtas; per_sm >= 2; --per_sm) {
    const int n = per_sm * info->num_sms / 8 * 8;
    for (int c = 1; c <= 8; c *= 2) {
      const double us = static_cast<double>((static_cast<long long>(rows) * c + n - 1) / n) *
                        (row_bytes * per_sm / (44e3 * c) + 2.5);
      if (ctas != 0 && (us >= best || row_bytes < c * 16.0 * kLogprobThreads)) continue;
      best = us;
      ctas = n;
      p.cluster = c;
      p.stages = per_sm == 2 ? 3 : 2;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == GEMM_LOGITS_BF16 ? run_token_logprobs<uint16_t>(p, ctas, device, s)
                                  : run_token_logprobs<float>(p, ctas, device, s);
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
  return type == GEMM_LOGITS_BF16 ? run_token_logprobs_backward<uint16_t>(p, s)
                                  : run_token_logprobs_backward<float>(p, s);
}

}  // extern "C"
