// embedding.cu -- rows of an embedding table for given token ids, scaled, and the gradient of the table.
//
//   y[i] = scale * table[token_i],   dtable[v] = base[v] + scale * sum over i with token_i = v of dy[i]
//
// Lookup: a copy with a product, bound by the bytes of the rows. A thread takes 16 bytes (8 columns of FP32: 32) at a time.
//
// Gradient: positions are sorted by token (stable, so a token's rows are added in the order of their positions and the
// same inputs give the same bits), then a CTA takes a run of sorted positions and 8 columns a thread, adds dy's rows in
// FP32 and writes a token's row once where the token begins and ends inside its run. What a run's first and last token
// share with other runs is left as FP32 partial rows, which a last kernel adds in order: a token that is a tenth of all
// positions costs no more than the others.
// The sort is a least-significant-digit radix sort of 9 bits a pass (two passes up to 262143 tokens) by one cluster of 8
// CTAs: a warp counts the digits of its part of the list, the CTAs exchange their totals through shared memory, and every
// warp then knows where its part's digits go. Lists lie in global memory (L2), so their length is not limited. The other
// CTAs of the same launch meanwhile write the rows that no token will touch, zeros or the base: that is most of the bytes
// of a dense gradient, and it hides the sort.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "host_common.h"

namespace dtcp {
namespace {

__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ void from_float(uint16_t& d, float v) {
  d = static_cast<uint16_t>(pack_bf16x2_rn(__float_as_uint(v), 0u) & 0xFFFFu);
}
__device__ __forceinline__ void from_float(float& d, float v) { d = v; }

struct Eight {
  float v[8];
};
__device__ __forceinline__ Eight load8(const uint16_t* p) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  Eight r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.v[2 * j] = __uint_as_float(w[j] << 16);
    r.v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
  return r;
}
__device__ __forceinline__ Eight load8(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(uint16_t* p, const Eight& e) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2_rn(__float_as_uint(e.v[2 * j]), __float_as_uint(e.v[2 * j + 1]));
  *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store8(float* p, const Eight& e) {
  *reinterpret_cast<float4*>(p) = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
}

// A thread's 8 columns: next to one another where rows start on 16-byte boundaries and have a multiple of 8 columns
// (VECTOR), else `step` apart, so that a warp reads and writes side by side.
template <bool VECTOR>
struct Columns {
  int first, step, cols;
  template <class T>
  __device__ __forceinline__ Eight load(const T* row) const {
    if constexpr (VECTOR) return load8(row + first);
    Eight r = {};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (first + j * step < cols) r.v[j] = to_float(row[first + j * step]);
    return r;
  }
  template <class T>
  __device__ __forceinline__ void store(T* row, const Eight& e) const {
    if constexpr (VECTOR) {
      store8(row + first, e);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (first + j * step < cols) from_float(row[first + j * step], e.v[j]);
    }
  }
};

// ---------------------------------------------------------------- lookup

struct LookupParams {
  const void* table;
  const long long* tokens;
  void* y;
  long long ldt, ldy;
  int rows, vocab, cols;
  int row_threads;  // a power of two: threads of a CTA that share a row
  float scale;
};

constexpr int kLookupThreads = 256;

// Each thread: UNITS times 8 columns of a row.
template <class T, bool VECTOR, int UNITS>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(const LookupParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int in_row = threadIdx.x & (p.row_threads - 1);
  const long long row = static_cast<long long>(blockIdx.x) * (kLookupThreads / p.row_threads) + threadIdx.x / p.row_threads;
  if (row >= p.rows) return;
  const long long token = p.tokens[row];
  const bool given = token >= 0 && token < p.vocab;
  const T* from = static_cast<const T*>(p.table) + (given ? token : 0) * p.ldt;
  T* to = static_cast<T*>(p.y) + row * p.ldy;
  const float other = token < 0 ? 0.0f : __int_as_float(0x7FC00000);
  Columns<VECTOR> at[UNITS];
  Eight e[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int unit = (static_cast<int>(blockIdx.y) * UNITS + u) * p.row_threads;
    at[u] = Columns<VECTOR>{VECTOR ? 8 * (unit + in_row) : 8 * unit + in_row, p.row_threads, p.cols};
    e[u] = Eight{{other, other, other, other, other, other, other, other}};
    if (given && at[u].first < p.cols) e[u] = at[u].load(from);
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    if (at[u].first >= p.cols) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) e[u].v[j] *= p.scale;
    at[u].store(to, e[u]);
  }
}

// ---------------------------------------------------------------- positions by token, and the rows of no token

constexpr int kSortCtas = 8, kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;

struct SortParams {
  const long long* tokens;
  int count, vocab, passes, digit_bits;
  int per_warp;      // positions of a warp, a multiple of 32
  uint32_t* key[2];  // lists of `count` tokens and positions; the last pass writes list 0
  uint32_t* pos[2];
  // rows that no token touches
  void* table;
  const void* base;  // or null: zeros
  long long bytes;   // 0: nothing to write
};

struct SortShared {
  uint32_t counts[kSortWarps][kDigits];  // of a warp's digits; then where the warp's next one goes, within the CTA's
  uint32_t totals[kDigits];              // of the CTA (read by the cluster)
  uint32_t first[kDigits];               // where the CTA's digits go
  uint32_t sums[kSortWarps];
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ void sort_positions(const SortParams& p, SortShared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = static_cast<int>(cluster_ctarank());
  const long long begin = static_cast<long long>(rank * kSortWarps + warp) * p.per_warp;
  const long long end = min(begin + p.per_warp, static_cast<long long>(p.count));
  const uint32_t mask = (1u << p.digit_bits) - 1u;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int from = (p.passes - pass) & 1, shift = pass * p.digit_bits;
    auto key_at = [&](long long i) -> uint32_t {
      if (pass > 0) return p.key[from][i];
      const long long t = p.tokens[i];
      // (no token: behind all others)
      return t >= 0 && t < p.vocab ? static_cast<uint32_t>(t) : static_cast<uint32_t>(p.vocab);
    };
    for (int d = threadIdx.x; d < kSortWarps * kDigits; d += kSortThreads) (&s.counts[0][0])[d] = 0u;
    __syncthreads();
    uint32_t* const mine = s.counts[warp];
#pragma unroll 4
    for (long long i = begin; i < end; i += 32) {
      const bool in = i + lane < end;
      const uint32_t digit = in ? (key_at(i + lane) >> shift) & mask : kDigits;  // (lanes past the end among themselves)
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (in && (same & ((1u << lane) - 1u)) == 0u) mine[digit] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x < kDigits) {
      uint32_t run = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = s.counts[w][threadIdx.x];
        s.counts[w][threadIdx.x] = run;
        run += c;
      }
      s.totals[threadIdx.x] = run;
    }
    cluster_sync_all();
    uint32_t all = 0, before = 0;
    if (threadIdx.x < kDigits) {
      const uint32_t at = smem_u32(&s.totals[threadIdx.x]);
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        const uint32_t c = ld_cluster_u32(mapa_shared(at, r));
        if (r < rank) before += c;
        all += c;
      }
    }
    uint32_t scan = all;  // over the digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) s.sums[warp] = scan;
    __syncthreads();
    if (threadIdx.x < kDigits) {
      uint32_t lower = 0;
      for (int w = 0; w < warp; ++w) lower += s.sums[w];
      s.first[threadIdx.x] = lower + scan - all + before;
    }
    __syncthreads();
#pragma unroll 4
    for (long long i = begin; i < end; i += 32) {
      const bool in = i + lane < end;
      const uint32_t key = in ? key_at(i + lane) : 0u;
      const uint32_t pos = !in ? 0u : pass > 0 ? p.pos[from][i + lane] : static_cast<uint32_t>(i + lane);
      const uint32_t digit = in ? (key >> shift) & mask : kDigits;
      const uint32_t same = __match_any_sync(0xffffffffu, digit), lower = same & ((1u << lane) - 1u);
      uint32_t to = 0;
      if (in) to = s.first[digit] + mine[digit] + __popc(lower);
      __syncwarp();
      if (in) {
        if (lower == 0u) mine[digit] += __popc(same);
        p.key[from ^ 1][to] = key;
        p.pos[from ^ 1][to] = pos;
      }
      __syncwarp();
    }
    cluster_sync_all();  // the list is written, and the totals are read
  }
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) sort_kernel(const SortParams p) {
  extern __shared__ uint4 sort_shared[];
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x < kSortCtas) {
    if (p.count > 0) sort_positions(p, *reinterpret_cast<SortShared*>(sort_shared));
    return;
  }
  const long long ctas = gridDim.x - kSortCtas, step = ctas * kSortThreads;
  const long long first = static_cast<long long>(blockIdx.x - kSortCtas) * kSortThreads + threadIdx.x;
  uint8_t* const to = static_cast<uint8_t*>(p.table);
  const uint8_t* const from = static_cast<const uint8_t*>(p.base);
  const long long vectors = p.bytes / 16;
  if (from == nullptr) {
    for (long long v = first; v < vectors; v += step) reinterpret_cast<uint4*>(to)[v] = make_uint4(0u, 0u, 0u, 0u);
  } else {
    long long v = first;
    for (; v + 3 * step < vectors; v += 4 * step) {
      uint4 r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = __ldcs(reinterpret_cast<const uint4*>(from) + v + j * step);
#pragma unroll
      for (int j = 0; j < 4; ++j) reinterpret_cast<uint4*>(to)[v + j * step] = r[j];
    }
    for (; v < vectors; v += step) reinterpret_cast<uint4*>(to)[v] = reinterpret_cast<const uint4*>(from)[v];
  }
  const long long at = vectors * 16 + 2 * first;  // (fewer than 16 bytes are left, a multiple of two)
  if (at < p.bytes)
    *reinterpret_cast<uint16_t*>(to + at) = from != nullptr ? *reinterpret_cast<const uint16_t*>(from + at) : uint16_t(0);
}

// ---------------------------------------------------------------- sums

struct SumParams {
  const void* dy;
  const uint32_t* key;  // sorted tokens and their positions
  const uint32_t* pos;
  const void* base;  // or null
  void* table;
  float* partial;  // [runs][2][cols]: what a run's first and last token share with others
  long long ldd;
  int count, vocab, cols, run;  // positions, tokens, columns, positions of a run
  float scale;
};

constexpr int kMaxRun = 256;
constexpr int kSumThreads = 128;

template <class TABLE, bool VECTOR>
__device__ __forceinline__ void write_row(const SumParams& p, const Columns<VECTOR>& at, uint32_t token, const Eight& sum) {
  const long long row = static_cast<long long>(token) * p.cols;
  Eight o = {};
  if (p.base != nullptr) o = at.load(static_cast<const TABLE*>(p.base) + row);
#pragma unroll
  for (int j = 0; j < 8; ++j) o.v[j] = fmaf(p.scale, sum.v[j], o.v[j]);
  at.store(static_cast<TABLE*>(p.table) + row, o);
}

template <bool VECTOR>
__device__ __forceinline__ Columns<VECTOR> sum_columns(int cols) {
  const int threads = static_cast<int>(blockDim.x), block = static_cast<int>(blockIdx.y) * threads;
  const int t = static_cast<int>(threadIdx.x);
  return Columns<VECTOR>{VECTOR ? 8 * (block + t) : 8 * block + t, threads, cols};
}

// A run of sorted positions, 8 columns a thread.
template <class DY, class TABLE, bool VECTOR>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const SumParams p) {
  __shared__ uint32_t key[kMaxRun + 2], pos[kMaxRun];  // the tokens before and behind the run as well
  pdl_launch_dependents();
  pdl_wait();
  const long long begin = static_cast<long long>(blockIdx.x) * p.run;
  const int length = static_cast<int>(min(static_cast<long long>(p.run), p.count - begin));
  for (int i = threadIdx.x; i < length + 2; i += blockDim.x) {
    const long long at = begin + i - 1;
    key[i] = at >= 0 && at < p.count ? p.key[at] : 0xFFFFFFFFu;
    if (i >= 1 && i <= length) pos[i - 1] = p.pos[at];
  }
  __syncthreads();
  const Columns<VECTOR> at = sum_columns<VECTOR>(p.cols);
  if (at.first >= p.cols) return;
  const Columns<VECTOR> part = at;
  float* const partial = p.partial + 2LL * blockIdx.x * p.cols;
  const DY* const dy = static_cast<const DY*>(p.dy);
  Eight sum = {};
  int start = 0;  // of the current token's part
  constexpr int AHEAD = 4;
  for (int i = 0; i < length; i += AHEAD) {
    Eight e[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
      if (i + a < length && key[i + a + 1] < static_cast<uint32_t>(p.vocab)) e[a] = at.load(dy + pos[i + a] * p.ldd);
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (i + a >= length) break;
      const uint32_t token = key[i + a + 1];
      if (token >= static_cast<uint32_t>(p.vocab)) return;  // (no token: the list's end)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum.v[j] += e[a].v[j];
      const bool last = i + a + 1 == length;
      if (!last && key[i + a + 2] == token) continue;
      // the token's part of this run is complete
      const bool before = start == 0 && key[0] == token, behind = last && key[length + 1] == token;
      if (before) part.store(partial, sum);
      else if (behind) part.store(partial + p.cols, sum);
      else write_row<TABLE>(p, at, token, sum);
      sum = Eight{};
      start = i + a + 1;
    }
  }
}

// The tokens that begin in one run and end in a later one: the first run's last part and the later ones' first parts, in
// order. The CTA's four groups of threads take every fourth run; their sums are added in order.
constexpr int kJoinGroups = 4;
template <class TABLE, bool VECTOR>
__global__ void __launch_bounds__(kJoinGroups* kSumThreads) join_rows_kernel(const SumParams p, int runs) {
  __shared__ float parts[kJoinGroups - 1][8][kSumThreads];
  pdl_launch_dependents();
  pdl_wait();
  const long long end = (static_cast<long long>(blockIdx.x) + 1) * p.run;
  if (end >= p.count) return;
  const uint32_t token = p.key[end - 1];
  if (token >= static_cast<uint32_t>(p.vocab) || p.key[end] != token) return;
  const long long begin = end - p.run;
  if (begin > 0 && p.key[begin] == token && p.key[begin - 1] == token) return;  // it begins in an earlier run
  // the runs that it reaches: a binary search for its end
  long long low = end, high = p.count;  // key[low] == token; key[high] is another one (or the list's end)
  while (high - low > 1) {
    const long long mid = (low + high) / 2;
    if (p.key[mid] == token) low = mid;
    else high = mid;
  }
  const int last = static_cast<int>(low / p.run);
  const Columns<VECTOR> at = sum_columns<VECTOR>(p.cols);
  const bool live = at.first < p.cols;
  Eight sum = {};
  if (live) {
#pragma unroll 4
    for (int r = static_cast<int>(blockIdx.x) + static_cast<int>(threadIdx.y); r <= last; r += kJoinGroups) {
      const bool first = r == static_cast<int>(blockIdx.x);
      const Eight e = at.load(p.partial + (2LL * r + (first ? 1 : 0)) * p.cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum.v[j] += e.v[j];
    }
    if (threadIdx.y > 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) parts[threadIdx.y - 1][j][threadIdx.x] = sum.v[j];
  }
  __syncthreads();
  if (threadIdx.y > 0 || !live) return;
#pragma unroll
  for (int g = 0; g < kJoinGroups - 1; ++g)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum.v[j] += parts[g][j][threadIdx.x];
  write_row<TABLE>(p, at, token, sum);
}

// ---------------------------------------------------------------- host side

int launch(const void* kernel, dim3 grid, dim3 threads, size_t smem, cudaStream_t stream, void** args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

constexpr int kMaxVocab = (1 << 27) - 1;  // three digits
constexpr int kMaxCols = 1 << 22;

bool known_type(int t) { return t == GEMM_TABLE_BF16 || t == GEMM_TABLE_F32; }
int type_bytes(int t) { return t == GEMM_TABLE_BF16 ? 2 : 4; }
bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
// Rows of 8 columns at a time: each starts on a 16-byte boundary.
bool rows_aligned(const void* p, int type, long long ld) { return aligned(p, 16) && ld * type_bytes(type) % 16 == 0; }

template <class T, bool VECTOR>
const void* lookup(int units) {
  return units == 1 ? reinterpret_cast<const void*>(lookup_kernel<T, VECTOR, 1>)
                    : reinterpret_cast<const void*>(lookup_kernel<T, VECTOR, 4>);
}

template <class DY, class TABLE>
const void* sum(bool vector) {
  return vector ? reinterpret_cast<const void*>(sum_kernel<DY, TABLE, true>)
                : reinterpret_cast<const void*>(sum_kernel<DY, TABLE, false>);
}
template <class TABLE>
const void* join_rows(bool vector) {
  return vector ? reinterpret_cast<const void*>(join_rows_kernel<TABLE, true>)
                : reinterpret_cast<const void*>(join_rows_kernel<TABLE, false>);
}

bool prepare_sort(int device) {
  static std::mutex mu;
  static bool done[64] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return false;
  if (!done[device]) {
    if (cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortShared)) !=
        cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    done[device] = true;
  }
  return true;
}

}  // namespace
}  // namespace dtcp

using namespace dtcp;

extern "C" {

int gemm_embedding(const void* table, int type, const long long* tokens, void* Y, int rows, int vocab, int cols,
                   long long ldt, long long ldy, float scale, void* stream) {
  if (rows < 0 || vocab < 0 || cols < 0 || !known_type(type) || !std::isfinite(scale)) return GEMM_ERR_INVALID_ARG;
  if (ldt == 0) ldt = cols;
  if (ldy == 0) ldy = cols;
  if (ldt < cols || ldy < cols) return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (cols > kMaxCols) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (tokens == nullptr || Y == nullptr || (vocab > 0 && table == nullptr)) return GEMM_ERR_INVALID_ARG;
  const unsigned bytes = type_bytes(type);
  if (!aligned(table, bytes) || !aligned(Y, bytes) || !aligned(tokens, 8)) return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  LookupParams p = {table, tokens, Y, ldt, ldy, rows, vocab, cols, 1, scale};
  const bool vector = cols % 8 == 0 && rows_aligned(table, type, ldt) && rows_aligned(Y, type, ldy);
  const int units = ceil_div(cols, 8);
  // four loads a thread in flight where there are rows enough for that, else as many threads as there are vectors
  const int each = 1LL * rows * units >= 4096LL * info->num_sms ? 4 : 1;
  while (p.row_threads < kLookupThreads && p.row_threads * each < units) p.row_threads *= 2;
  const int a_cta = kLookupThreads / p.row_threads;
  const dim3 grid(ceil_div(rows, a_cta), ceil_div(units, p.row_threads * each));
  void* args[] = {&p};
  const void* kernel = type == GEMM_TABLE_BF16 ? (vector ? lookup<uint16_t, true>(each) : lookup<uint16_t, false>(each))
                                               : (vector ? lookup<float, true>(each) : lookup<float, false>(each));
  return launch(kernel, grid, dim3(kLookupThreads), 0, static_cast<cudaStream_t>(stream), args);
}

int gemm_embedding_backward(const void* dY, int dy_type, const long long* tokens, const void* base, void* dtable,
                            int table_type, int rows, int vocab, int cols, long long ldd, float scale, void* stream) {
  if (rows < 0 || vocab < 0 || cols < 0 || !known_type(dy_type) || !known_type(table_type) || !std::isfinite(scale))
    return GEMM_ERR_INVALID_ARG;
  if (ldd == 0) ldd = cols;
  if (ldd < cols) return GEMM_ERR_INVALID_ARG;
  if (vocab == 0 || cols == 0) return GEMM_OK;
  if (dtable == nullptr || (rows > 0 && (dY == nullptr || tokens == nullptr))) return GEMM_ERR_INVALID_ARG;
  if (vocab > kMaxVocab || cols > kMaxCols) return GEMM_ERR_UNSUPPORTED_SHAPE;
  const bool in_place = base == dtable;
  if (!aligned(dY, type_bytes(dy_type)) || !aligned(tokens, 8) || !aligned(base, in_place ? type_bytes(table_type) : 16) ||
      !aligned(dtable, in_place ? type_bytes(table_type) : 16))
    return GEMM_ERR_MISALIGNED;
  if (rows == 0 && in_place) return GEMM_OK;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  if (!prepare_sort(device)) return GEMM_ERR_LAUNCH;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  // runs of at least 16 positions, and about 512 of them at most
  SumParams q = {};
  q.run = std::min(kMaxRun, std::max(16, ceil_div(ceil_div(std::max(rows, 1), 512), 8) * 8));
  const int runs = ceil_div(rows, q.run);
  const size_t list = (size_t(rows) * 4 + 255) / 256 * 256;
  uint8_t* ws = nullptr;
  if (rows > 0) {
    cudaMemPool_t pool = workspace_pool(device);
    void* got = nullptr;
    if (pool == nullptr || cudaMallocFromPoolAsync(&got, 4 * list + size_t(runs) * 2 * cols * 4, pool, s) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_OUT_OF_MEMORY;
    }
    ws = static_cast<uint8_t*>(got);
  }
  SortParams p = {};
  p.tokens = tokens;
  p.count = rows;
  p.vocab = vocab;
  int bits = 1;
  while ((vocab >> bits) != 0) ++bits;  // (the token after the last stands for none)
  p.passes = ceil_div(bits, kDigitBits);
  p.digit_bits = ceil_div(bits, p.passes);
  p.per_warp = ceil_div(ceil_div(rows, kSortCtas * kSortWarps), 32) * 32;
  for (int i = 0; i < 2; ++i) {
    p.key[i] = reinterpret_cast<uint32_t*>(ws + i * list);
    p.pos[i] = reinterpret_cast<uint32_t*>(ws + (2 + i) * list);
  }
  p.table = dtable;
  p.base = base;
  p.bytes = in_place ? 0 : static_cast<long long>(vocab) * cols * type_bytes(table_type);
  const long long fill = (p.bytes + 16LL * kSortThreads - 1) / (16LL * kSortThreads);
  const int fill_ctas = static_cast<int>(std::min<long long>((fill + kSortCtas - 1) / kSortCtas * kSortCtas,
                                                             info->num_sms * 2 / kSortCtas * kSortCtas));
  void* sort_args[] = {&p};
  int st = launch(reinterpret_cast<const void*>(sort_kernel), dim3(kSortCtas + fill_ctas), dim3(kSortThreads),
                  sizeof(SortShared), s, sort_args);
  if (rows == 0) return st;

  q.dy = dY;
  q.key = p.key[0];
  q.pos = p.pos[0];
  q.base = base;
  q.table = dtable;
  q.partial = reinterpret_cast<float*>(ws + 4 * list);
  q.ldd = ldd;
  q.count = rows;
  q.vocab = vocab;
  q.cols = cols;
  q.scale = scale;
  const bool vector = cols % 8 == 0 && rows_aligned(dY, dy_type, ldd) && rows_aligned(base, table_type, cols) &&
                      rows_aligned(dtable, table_type, cols);
  const int units = ceil_div(cols, 8), threads = std::min(kSumThreads, ceil_div(units, 32) * 32);
  const dim3 grid(runs, ceil_div(units, threads));
  const void* kernel = dy_type == GEMM_TABLE_BF16
                           ? (table_type == GEMM_TABLE_BF16 ? sum<uint16_t, uint16_t>(vector) : sum<uint16_t, float>(vector))
                           : (table_type == GEMM_TABLE_BF16 ? sum<float, uint16_t>(vector) : sum<float, float>(vector));
  void* sum_args[] = {&q};
  if (st == GEMM_OK) st = launch(kernel, grid, dim3(threads), 0, s, sum_args);
  if (st == GEMM_OK && runs > 1) {
    int n = runs;
    void* join_args[] = {&q, &n};
    st = launch(table_type == GEMM_TABLE_BF16 ? join_rows<uint16_t>(vector) : join_rows<float>(vector), grid,
                dim3(threads, kJoinGroups), 0, s, join_args);
  }
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == GEMM_OK) st = GEMM_ERR_LAUNCH;
  return st;
}

}  // extern "C"
