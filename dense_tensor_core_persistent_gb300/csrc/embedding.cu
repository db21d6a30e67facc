// embedding.cu -- rows of an embedding table for given token ids, scaled, and the gradient of the table.
//
//   y[i] = scale * table[token_i],   dtable[v] = base[v] + scale * sum over i with token_i = v of dy[i]
//
// Lookup: a copy with a product, bound by the bytes of the rows. A thread takes 16 bytes (8 columns of FP32: 32) at a time.
//
// Gradient: positions are sorted by token (stable, so a token's rows are added in the order of their positions and the
// same inputs give the same bits), then a CTA takes a run of sorted positions and 8 columns a thread, adds dy's rows in
// FP32 and writes each token's row once. Tokens of more than 16 positions are summed by run, into FP32 partial rows that a
// last kernel adds in order: a token that is a tenth of all positions costs no more than the others. (Up to 256 positions
// need no sort: direct_kernel.)
// The sort is a least-significant-digit radix sort of up to 10 bits a pass (two passes below 2^20 tokens) by one cluster of
// 8 or 16 CTAs: a warp counts the digits of its part of the list, the CTAs exchange their totals through shared memory, and every
// warp then knows where its part's digits go. The lists lie in global memory (L2), so their length is not limited. Beside
// the sort another kernel writes the whole table, zeros or the base: that is most of the bytes of a dense gradient, and it
// hides the sort.
//
// Both are bound by bytes. Measured on GB300: 16384 rows of 131072 x 4096 looked up in 30.5 us (8.8 TB/s, as frequent rows
// come from L2); their gradient 180 us in a table of zeros (6.7 TB/s: 138 the table, 42 the sums), 75 in place (sort 15,
// sums 47, parts of long tokens 8).
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
// (VECTOR), else STEP apart (the threads that share a row; 0: known at run time), so that a warp reads and writes side by
// side.
template <bool VECTOR, int STEP>
struct Columns {
  int first, cols, run_step;
  __device__ __forceinline__ int step() const { return STEP > 0 ? STEP : run_step; }
  template <class T>
  __device__ __forceinline__ Eight load(const T* row) const {
    if constexpr (VECTOR) return load8(row + first);
    Eight r = {};
    const T* const at = row + first;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (first + j * step() < cols) r.v[j] = to_float(at[j * step()]);
    return r;
  }
  template <class T>
  __device__ __forceinline__ void store(T* row, const Eight& e) const {
    if constexpr (VECTOR) {
      store8(row + first, e);
    } else {
      T* const at = row + first;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (first + j * step() < cols) from_float(at[j * step()], e.v[j]);
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
  Columns<VECTOR, 0> at[UNITS];
  Eight e[UNITS];
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int unit = (static_cast<int>(blockIdx.y) * UNITS + u) * p.row_threads;
    at[u] = Columns<VECTOR, 0>{VECTOR ? 8 * (unit + in_row) : 8 * unit + in_row, p.cols, p.row_threads};
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

// ---------------------------------------------------------------- positions by token

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMostDigitBits = 10, kMostDigits = 1 << kMostDigitBits;
constexpr int kSortAhead = 8;  // steps of 32 positions that a warp asks for together

// A position and its token, as they are sorted.
struct __align__(8) Entry {
  uint32_t token, pos;
};

struct SortParams {
  const long long* tokens;
  int count, vocab, passes, digit_bits;
  int per_warp;    // positions of a warp, a multiple of 32
  Entry* list[2];  // of `count`; the last pass writes list 0
  int* spans;      // two counts that the sums start from zero
};

struct SortShared {
  uint32_t totals[kMostDigits];  // of the CTA (read by the cluster)
  uint32_t first[kMostDigits];   // where the CTA's digits go
  uint32_t sums[kSortWarps];
  uint32_t counts[1];  // [kSortWarps][digits]: of a warp's digits; then where its next one goes, within the CTA's
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kSortThreads) sort_kernel(const SortParams p) {
  extern __shared__ uint4 sort_shared[];
  SortShared& s = *reinterpret_cast<SortShared*>(sort_shared);
  pdl_wait();
  pdl_launch_dependents();  // (only now: the rows' kernel starts beside this one, see there)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = static_cast<int>(cluster_ctarank());
  if (blockIdx.x == 0 && threadIdx.x < 2) p.spans[threadIdx.x] = 0;
  const long long begin = static_cast<long long>(rank * kSortWarps + warp) * p.per_warp;
  const long long end = min(begin + p.per_warp, static_cast<long long>(p.count));
  const uint32_t digits = 1u << p.digit_bits, mask = digits - 1u;
  uint32_t* const mine = s.counts + warp * digits;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int from = (p.passes - pass) & 1, shift = pass * p.digit_bits;
    auto entry_at = [&](long long i) -> Entry {
      if (pass > 0) return p.list[from][i];
      const long long t = p.tokens[i];
      // (no token: behind all others)
      return Entry{t >= 0 && t < p.vocab ? static_cast<uint32_t>(t) : static_cast<uint32_t>(p.vocab),
                   static_cast<uint32_t>(i)};
    };
    auto load = [&](Entry(&e)[kSortAhead], long long i) {
#pragma unroll
      for (int a = 0; a < kSortAhead; ++a)
        e[a] = i + 32 * a + lane < end ? entry_at(i + 32 * a + lane) : Entry{0u, 0u};
    };
    Entry e[kSortAhead];
    uint32_t among[kSortAhead];  // earlier entries of the warp with its digit
    for (uint32_t d = threadIdx.x; d < kSortWarps * digits; d += kSortThreads) s.counts[d] = 0u;
    __syncthreads();
    for (long long i = begin; i < end; i += 32 * kSortAhead) {
      load(e, i);
#pragma unroll
      for (int a = 0; a < kSortAhead; ++a) {
        if (i + 32 * a >= end) break;
        const bool in = i + 32 * a + lane < end;
        const uint32_t digit = in ? (e[a].token >> shift) & mask : digits;  // (lanes past the end among themselves)
        const uint32_t same = __match_any_sync(0xffffffffu, digit), lower = same & ((1u << lane) - 1u);
        const uint32_t seen = in ? mine[digit] : 0u;
        among[a] = seen + __popc(lower);
        __syncwarp();
        if (in && lower == 0u) mine[digit] = seen + __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();
    if (threadIdx.x < digits) {
      uint32_t run = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = s.counts[w * digits + threadIdx.x];
        s.counts[w * digits + threadIdx.x] = run;
        run += c;
      }
      s.totals[threadIdx.x] = run;
    }
    cluster_sync_all();
    uint32_t all = 0, before = 0;
    if (threadIdx.x < digits) {
      const uint32_t at = smem_u32(&s.totals[threadIdx.x]);
#pragma unroll
      for (int r = 0; r < CTAS; ++r) {
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
    if (threadIdx.x < digits) {
      uint32_t lower = 0;
      for (int w = 0; w < warp; ++w) lower += s.sums[w];
      s.first[threadIdx.x] = lower + scan - all + before;
    }
    __syncthreads();
    if (p.per_warp <= 32 * kSortAhead) {  // (the entries and their ranks still are here)
#pragma unroll
      for (int a = 0; a < kSortAhead; ++a) {
        if (begin + 32 * a + lane >= end) break;
        const uint32_t digit = (e[a].token >> shift) & mask;
        p.list[from ^ 1][s.first[digit] + mine[digit] + among[a]] = e[a];
      }
    } else {
      for (long long i = begin; i < end; i += 32 * kSortAhead) {
        load(e, i);
#pragma unroll
        for (int a = 0; a < kSortAhead; ++a) {
          if (i + 32 * a >= end) break;
          const bool in = i + 32 * a + lane < end;
          const uint32_t digit = in ? (e[a].token >> shift) & mask : digits;
          const uint32_t same = __match_any_sync(0xffffffffu, digit), lower = same & ((1u << lane) - 1u);
          uint32_t to = 0;
          if (in) to = s.first[digit] + mine[digit] + __popc(lower);
          __syncwarp();
          if (in) {
            if (lower == 0u) mine[digit] += __popc(same);
            p.list[from ^ 1][to] = e[a];
          }
          __syncwarp();
        }
      }
    }
    cluster_sync_all();  // the list is written, and the totals are read
  }
}

// ---------------------------------------------------------------- the rows of no token

struct RowsParams {
  void* table;
  const void* base;  // or null: zeros
  long long bytes;
  int beside;  // it runs beside the sort, which has waited for all work before it
};

constexpr int kRowsThreads = 512, kRowsVectors = 4;  // of 16 bytes a thread

// The whole table, zeros or the base (rows that tokens touch are written again by the sums). 32 KB a CTA, next to one
// another: CTAs that come and go write 1 GB at 7.7 TB/s, resident ones that step over it by the grid's size at 6.4.
// Beside the sort nothing here waits for it but the last CTA, so that the sums, which wait for this grid, find both done. What
// was done before the sort is done: the sort lets this grid start only behind its own wait for that. The base is read past L1
// all the same, as only a grid that waits is promised an L1 without lines from before.
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const RowsParams p) {
  if (!p.beside) pdl_wait();
  pdl_launch_dependents();
  uint8_t* const to = static_cast<uint8_t*>(p.table);
  const uint8_t* const from = static_cast<const uint8_t*>(p.base);
  const long long vectors = p.bytes / 16;
  const long long first = static_cast<long long>(blockIdx.x) * kRowsVectors * kRowsThreads + threadIdx.x;
  uint4 v[kRowsVectors];
#pragma unroll
  for (int j = 0; j < kRowsVectors; ++j) {
    const long long i = first + j * kRowsThreads;
    v[j] = make_uint4(0u, 0u, 0u, 0u);
    if (from != nullptr && i < vectors) v[j] = __ldcg(reinterpret_cast<const uint4*>(from) + i);
  }
#pragma unroll
  for (int j = 0; j < kRowsVectors; ++j) {
    const long long i = first + j * kRowsThreads;
    if (i < vectors) reinterpret_cast<uint4*>(to)[i] = v[j];
  }
  if (blockIdx.x + 1 == gridDim.x) {
    const long long at = vectors * 16 + 2 * threadIdx.x;  // (fewer than 16 bytes are left, a multiple of two)
    if (at < p.bytes)
      *reinterpret_cast<uint16_t*>(to + at) = from != nullptr ? __ldcg(reinterpret_cast<const uint16_t*>(from + at)) : uint16_t(0);
    if (p.beside) pdl_wait();
  }
}

// ---------------------------------------------------------------- sums

struct SumParams {
  const void* dy;
  const Entry* list;  // sorted
  const void* base;   // or null
  void* table;
  float* partial;  // [runs][2][cols]: a run's parts of a long token that began before it, and of one that goes on behind it
  int* spans;      // the long tokens of up to kJoinAlone runs and of more: two counts, then for either the runs in which they
                   // begin, with the tokens; room for one a run
  long long ldd;
  int count, vocab, cols, run;  // positions, tokens, columns, positions of a run
  float scale;
};

constexpr int kMaxRun = 256;
constexpr int kSumThreads = 128;
// A token of more positions is long. Whole gradient in place, us, with 32, 16 and 8: 16384 positions into 131072 x 4096 78.5,
// 75.5, 77.2; 5003 into 50001 x 1027 FP32 27.3, 25.8, 25.3 (the rows that one CTA adds are its longest path).
constexpr int kLong = 16;
constexpr int kBeside = 32;  // positions that a CTA sees before and behind its run
constexpr int kJoinAlone = 8;  // parts of a long token that one warp adds
template <bool VECTOR, bool BASE>
constexpr int kSumAhead = VECTOR && !BASE ? 8 : 4;  // rows of dy (and of the base) that a thread asks for together

// table[token] = base + scale * sum, at this thread's columns.
template <class TABLE, bool VECTOR, int STEP>
__device__ __forceinline__ void write_row(const SumParams& p, const Columns<VECTOR, STEP>& at, uint32_t token, const Eight& sum,
                                          Eight base) {
#pragma unroll
  for (int j = 0; j < 8; ++j) base.v[j] = fmaf(p.scale, sum.v[j], base.v[j]);
  at.store(static_cast<TABLE*>(p.table) + static_cast<long long>(token) * p.cols, base);
}
template <class TABLE, bool BASE, bool VECTOR, int STEP>
__device__ __forceinline__ Eight base_row(const SumParams& p, const Columns<VECTOR, STEP>& at, uint32_t token) {
  if constexpr (BASE) return at.load(static_cast<const TABLE*>(p.base) + static_cast<long long>(token) * p.cols);
  return Eight{};
}

// The columns of a thread of blockDim.x that share a row (STEP of them where columns are STEP apart).
template <bool VECTOR, int STEP>
__device__ __forceinline__ Columns<VECTOR, STEP> sum_columns(int cols) {
  const int threads = VECTOR ? static_cast<int>(blockDim.x) : STEP, block = static_cast<int>(blockIdx.y) * threads;
  const int t = static_cast<int>(threadIdx.x);
  return Columns<VECTOR, STEP>{VECTOR ? 8 * (block + t) : 8 * block + t, cols, STEP};
}

// How many lanes from the first one on say yes.
__device__ __forceinline__ int leading(bool yes) {
  const uint32_t no = ~__ballot_sync(0xffffffffu, yes);
  return no == 0u ? 32 : __ffs(no) - 1;
}

// The tokens that begin in a run of sorted positions, 8 columns a thread. Tokens of up to kLong positions are summed by the
// run in which they begin, even past its end; of longer ones every run sums its part, and join_rows_kernel adds those.
template <class DY, class TABLE, bool BASE, bool VECTOR>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const SumParams p) {
  constexpr int AHEAD = kSumAhead<VECTOR, BASE>;
  __shared__ uint32_t keys[kBeside + kMaxRun + kBeside], places[kMaxRun + kBeside];
  pdl_launch_dependents();
  pdl_wait();
  const long long begin = static_cast<long long>(blockIdx.x) * p.run;
  constexpr uint32_t NONE = 0xFFFFFFFFu;
  for (int i = threadIdx.x; i < p.run + 2 * kBeside; i += blockDim.x) {
    const long long at = begin + i - kBeside;
    const Entry e = at >= 0 && at < p.count ? p.list[at] : Entry{NONE, 0u};
    keys[i] = e.token < static_cast<uint32_t>(p.vocab) ? e.token : NONE;
    if (i >= kBeside) places[i - kBeside] = e.pos;
  }
  __syncthreads();
  const uint32_t* const key = keys + kBeside;  // of the run's positions; from -kBeside to run + kBeside - 1
  const int lane = threadIdx.x & 31;
  if (key[0] == NONE) return;  // (positions without a token are behind all others)
  // positions first .. end - 1 are this CTA's
  int first = 0, end = p.run;
  bool before = key[-1] == key[0], behind = false;  // its first token is a long one that began earlier; its last one goes on
  if (before) {
    const int back = leading(key[-1 - lane] == key[0]), on = leading(key[lane] == key[0]);
    if (back + on <= kLong) {  // a short one: the run in which it began has it
      first = on;
      before = false;
    }
  }
  if (key[p.run - 1] == NONE) {
    end = 0;
    for (int i = 0; i < p.run; i += 32) end += __popc(__ballot_sync(0xffffffffu, i + lane < p.run && key[i + lane] != NONE));
  } else if (key[p.run] == key[p.run - 1] && !(before && key[p.run - 1] == key[0]) && first < p.run) {
    const uint32_t last = key[p.run - 1];
    const int back = leading(p.run - 1 - lane >= 0 && key[p.run - 1 - lane] == last), on = leading(key[p.run + lane] == last);
    if (back + on <= kLong) end += on;
    else behind = true;
  }
  if (first >= end) return;
  if (behind && threadIdx.x == 0 && blockIdx.y == 0) {
    const long long past = begin + static_cast<long long>(kJoinAlone) * p.run;
    const bool more = past < p.count && p.list[past].token == key[p.run - 1];
    reinterpret_cast<int2*>(p.spans)[1 + (more ? gridDim.x : 0u) + atomicAdd(p.spans + more, 1)] =  // (in any order)
        make_int2(static_cast<int>(blockIdx.x), static_cast<int>(key[p.run - 1]));
  }
  const Columns<VECTOR, kSumThreads> at = sum_columns<VECTOR, kSumThreads>(p.cols);
  if (at.first >= p.cols) return;
  float* const partial = p.partial + 2LL * blockIdx.x * p.cols;
  const DY* const dy = static_cast<const DY*>(p.dy);
  Eight sum = {};
  for (int i = first; i < end; i += AHEAD) {
    Eight e[AHEAD], base[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) e[a] = at.load(dy + places[min(i + a, end - 1)] * p.ldd);
    if constexpr (BASE) {  // (asked for with dy's rows: the stores in between would keep them apart)
#pragma unroll
      for (int a = 0; a < AHEAD; ++a)
        if (i + a < end && (i + a + 1 == end || key[i + a + 1] != key[i + a]))
          base[a] = base_row<TABLE, true>(p, at, key[i + a]);
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (i + a >= end) break;
      const uint32_t token = key[i + a];
#pragma unroll
      for (int j = 0; j < 8; ++j) sum.v[j] += e[a].v[j];
      const bool last = i + a + 1 == end;
      if (!last && key[i + a + 1] == token) continue;
      // the token is complete, or the run's part of a long one
      if (before) at.store(partial, sum);
      else if (last && behind) at.store(partial + p.cols, sum);
      else write_row<TABLE>(p, at, token, sum, BASE ? base[a] : Eight{});
      sum = Eight{};
      before = false;
    }
  }
}

// Long tokens: the part of the run in which one begins and those of the runs that it reaches, 256 columns at a time. A warp
// adds up to kJoinAlone of them by itself; of more each of the CTA's warps takes every 16th, and their sums are added in
// order. Measured on GB300, whole gradient, with all tokens taken by a CTA and with those of few parts by a warp each: 65536
// uniform positions into 1000 x 1024 63.6 and 45.7 us, 16384 into 131072 x 4096 186.1 and 184.1.
constexpr int kJoinGroups = 16;
template <class TABLE, bool VECTOR>
__global__ void __launch_bounds__(kJoinGroups * 32) join_rows_kernel(const SumParams p, int runs) {
  __shared__ float parts[kJoinGroups][8][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = static_cast<int>(threadIdx.y), lane = static_cast<int>(threadIdx.x);
  const Columns<VECTOR, 32> at = sum_columns<VECTOR, 32>(p.cols);
  const bool live = at.first < p.cols;
  const int2* const spans = reinterpret_cast<const int2*>(p.spans) + 1;
  const int2 counts = *reinterpret_cast<const int2*>(p.spans);
  auto begins_with = [&](int r, uint32_t token) {
    return r < runs && p.list[static_cast<long long>(r) * p.run].token == token;
  };
  auto part = [&](int r, int from) { return at.load(p.partial + (2LL * r + (r == from ? 1 : 0)) * p.cols); };
  for (int n = blockIdx.x; n < counts.y; n += gridDim.x) {
    const int from = spans[runs + n].x;
    const uint32_t token = static_cast<uint32_t>(spans[runs + n].y);
    Eight base = {};
    if (p.base != nullptr && live && warp == 0) base = base_row<TABLE, true>(p, at, token);
    // the runs that begin with the token
    constexpr int THREADS = kJoinGroups * 32;
    int last = from;
    for (int more = THREADS; more == THREADS; last += more)
      more = __syncthreads_count(begins_with(last + 1 + warp * 32 + lane, token));
    Eight sum = {};
    if (live) {
#pragma unroll 4
      for (int r = from + warp; r <= last; r += kJoinGroups) {
        const Eight e = part(r, from);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] += e.v[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) parts[warp][j][lane] = sum.v[j];
    __syncthreads();
    if (warp == 0 && live) {
      const int groups = min(kJoinGroups, last - from + 1);
#pragma unroll 4
      for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] += parts[g][j][lane];
      write_row<TABLE>(p, at, token, sum, base);
    }
    __syncthreads();  // the warps' sums are read
  }
  // (from the last CTA on, as the others begin with the first one)
  const int step = static_cast<int>(gridDim.x) * kJoinGroups;
  for (int n = static_cast<int>(gridDim.x - 1 - blockIdx.x) * kJoinGroups + warp; n < counts.x; n += step) {
    const int from = spans[n].x;
    const uint32_t token = static_cast<uint32_t>(spans[n].y);
    const uint32_t ends = ~__ballot_sync(0xffffffffu, lane < kJoinAlone - 1 && begins_with(from + 1 + lane, token));
    const int count = __ffs(ends);  // with the run in which it begins
    if (!live) continue;
    Eight base = {}, sum = {};
    if (p.base != nullptr) base = base_row<TABLE, true>(p, at, token);
#pragma unroll
    for (int i = 0; i < kJoinAlone; i += 4) {
      Eight e[4] = {};
#pragma unroll
      for (int a = 0; a < 4; ++a)
        if (i + a < count) e[a] = part(from + i + a, from);
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] += e[a].v[j];
    }
    write_row<TABLE>(p, at, token, sum, base);
  }
}

// Few positions, without a sort: a CTA for each position looks whether its token stands before it; if not, it collects the
// token's positions in their order and adds their rows.
constexpr int kDirect = 256;
template <class DY, class TABLE, bool BASE, bool VECTOR>
__global__ void __launch_bounds__(kSumThreads) direct_kernel(const SumParams p, const long long* tokens) {
  constexpr int AHEAD = kSumAhead<VECTOR, BASE>;
  __shared__ uint32_t mask[kDirect / 32];
  __shared__ int places[kDirect];
  pdl_launch_dependents();
  pdl_wait();
  const int mine = blockIdx.x, lane = threadIdx.x & 31;
  const long long token = tokens[mine];
  if (token < 0 || token >= p.vocab) return;
  for (int i = threadIdx.x; i < kDirect; i += blockDim.x) {  // (blockDim is a multiple of 32)
    const uint32_t m = __ballot_sync(0xffffffffu, i < p.count && tokens[i] == token);
    if (lane == 0) mask[i / 32] = m;
  }
  __syncthreads();
  int count = 0;
  for (int w = 0; w < kDirect / 32; ++w) {
    const uint32_t m = mask[w];
    if (w * 32 <= mine && (m & (mine - w * 32 >= 32 ? 0xffffffffu : (1u << (mine - w * 32)) - 1u)) != 0u) return;  // it stands before
    if (threadIdx.x < 32 && (m >> lane & 1u) != 0u) places[count + __popc(m & ((1u << lane) - 1u))] = w * 32 + lane;
    count += __popc(m);
  }
  __syncthreads();
  const Columns<VECTOR, kSumThreads> at = sum_columns<VECTOR, kSumThreads>(p.cols);
  if (at.first >= p.cols) return;
  const DY* const dy = static_cast<const DY*>(p.dy);
  const Eight base = base_row<TABLE, BASE>(p, at, static_cast<uint32_t>(token));
  Eight sum = {};
  for (int i = 0; i < count; i += AHEAD) {
    Eight e[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
      if (i + a < count) e[a] = at.load(dy + places[i + a] * p.ldd);
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
      if (i + a < count)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] += e[a].v[j];
  }
  write_row<TABLE>(p, at, static_cast<uint32_t>(token), sum, base);
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

constexpr int kMaxVocab = (1 << 27) - 1;
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

template <class DY, class TABLE, bool BASE, bool VECTOR>
const void* sum(bool direct) {
  return direct ? reinterpret_cast<const void*>(direct_kernel<DY, TABLE, BASE, VECTOR>)
                : reinterpret_cast<const void*>(sum_kernel<DY, TABLE, BASE, VECTOR>);
}
template <class DY, class TABLE>
const void* sum(bool direct, bool base, bool vector) {
  return base ? (vector ? sum<DY, TABLE, true, true>(direct) : sum<DY, TABLE, true, false>(direct))
              : (vector ? sum<DY, TABLE, false, true>(direct) : sum<DY, TABLE, false, false>(direct));
}
const void* sum(int dy_type, int table_type, bool direct, bool base, bool vector) {
  return dy_type == GEMM_TABLE_BF16
             ? (table_type == GEMM_TABLE_BF16 ? sum<uint16_t, uint16_t>(direct, base, vector)
                                              : sum<uint16_t, float>(direct, base, vector))
             : (table_type == GEMM_TABLE_BF16 ? sum<float, uint16_t>(direct, base, vector)
                                              : sum<float, float>(direct, base, vector));
}
template <class TABLE>
const void* join_rows(bool vector) {
  return vector ? reinterpret_cast<const void*>(join_rows_kernel<TABLE, true>)
                : reinterpret_cast<const void*>(join_rows_kernel<TABLE, false>);
}

// The sort's cluster. Measured on GB300, whole gradient in place: 65536 positions into 131072 x 1024 90.4 us with 8 CTAs and
// 82.2 with 16, into 262144 x 64 49.6 and 44.9; 16384 into 131072 x 4096 80 and 79, 5003 into 50001 x 1027 28.2 and 28.7.
constexpr int kSortCtas = 8, kManySortCtas = 16, kManySorted = 16384;

int sort_bytes(int digit_bits) { return static_cast<int>(sizeof(SortShared)) + (kSortWarps << digit_bits) * 4; }

const void* sort_kernel_of(int ctas) {
  return ctas == kManySortCtas ? reinterpret_cast<const void*>(sort_kernel<kManySortCtas>)
                               : reinterpret_cast<const void*>(sort_kernel<kSortCtas>);
}

// CTAs of the sort's cluster; 0 on an error. Eight fit everywhere; a device whose SMs are shared out may not have room for
// more in one cluster.
int sort_ctas(int device, int rows) {
  static std::mutex mu;
  static int most[64] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  if (most[device] == 0) {
    for (int ctas : {kSortCtas, kManySortCtas})
      if (cudaFuncSetAttribute(sort_kernel_of(ctas), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               sort_bytes(kMostDigitBits)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
      }
    most[device] = kSortCtas;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(kManySortCtas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sort_bytes(kMostDigitBits);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kManySortCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const void* many = sort_kernel_of(kManySortCtas);
    if (cudaFuncSetAttribute(many, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, many, &cfg) == cudaSuccess && n > 0)
      most[device] = kManySortCtas;
    else
      cudaGetLastError();
  }
  return rows > kManySorted ? most[device] : kSortCtas;
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  const bool vector = cols % 8 == 0 && rows_aligned(dY, dy_type, ldd) && rows_aligned(base, table_type, cols) &&
                      rows_aligned(dtable, table_type, cols);
  RowsParams rest = {dtable, base, in_place ? 0 : static_cast<long long>(vocab) * cols * type_bytes(table_type),
                     rows > kDirect};
  constexpr long long FILL = 16LL * kRowsVectors * kRowsThreads;  // bytes of a CTA
  const long long fill_ctas = (rest.bytes + FILL - 1) / FILL;
  if (fill_ctas > 0x7FFFFFFF) return GEMM_ERR_UNSUPPORTED_SHAPE;
  void* rest_args[] = {&rest};
  auto write_rest = [&] {
    return rest.bytes == 0 ? GEMM_OK
                           : launch(reinterpret_cast<const void*>(rows_kernel), dim3(static_cast<unsigned>(fill_ctas)),
                                    dim3(kRowsThreads), 0, s, rest_args);
  };
  if (rows == 0) return write_rest();

  SumParams q = {};
  q.dy = dY;
  q.base = base;
  q.table = dtable;
  q.ldd = ldd;
  q.count = rows;
  q.vocab = vocab;
  q.cols = cols;
  q.scale = scale;
  const int units = ceil_div(cols, 8), threads = vector ? std::min(kSumThreads, ceil_div(units, 32) * 32) : kSumThreads;
  const void* kernel = sum(dy_type, table_type, rows <= kDirect, base != nullptr, vector);
  if (rows <= kDirect) {
    const int st = write_rest();
    if (st != GEMM_OK) return st;
    void* args[] = {&q, &tokens};
    return launch(kernel, dim3(rows, ceil_div(units, threads)), dim3(threads), 0, s, args);
  }

  // runs of as many positions as a thread asks for at a time, longer ones where there would be more than 2048 of them
  const int ctas = sort_ctas(device, rows);
  if (ctas == 0) return GEMM_ERR_LAUNCH;
  const int ahead = vector && base == nullptr ? kSumAhead<true, false> : kSumAhead<false, false>;
  q.run = std::min(kMaxRun, ceil_div(ceil_div(rows, 2048), ahead) * ahead);
  const int runs = ceil_div(rows, q.run);
  const size_t list = (size_t(rows) * sizeof(Entry) + 255) / 256 * 256, spans = (size_t(runs) * 16 + 8 + 255) / 256 * 256;
  cudaMemPool_t pool = workspace_pool(device);
  void* got = nullptr;
  if (pool == nullptr ||
      cudaMallocFromPoolAsync(&got, 2 * list + spans + size_t(runs) * 2 * cols * 4, pool, s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_OUT_OF_MEMORY;
  }
  uint8_t* const ws = static_cast<uint8_t*>(got);
  SortParams p = {};
  p.tokens = tokens;
  p.count = rows;
  p.vocab = vocab;
  int bits = 1;
  while ((vocab >> bits) != 0) ++bits;  // (the token after the last stands for none)
  p.passes = ceil_div(bits, kMostDigitBits);
  p.digit_bits = ceil_div(bits, p.passes);
  p.per_warp = ceil_div(ceil_div(rows, ctas * kSortWarps), 32) * 32;
  for (int i = 0; i < 2; ++i) p.list[i] = reinterpret_cast<Entry*>(ws + i * list);
  p.spans = reinterpret_cast<int*>(ws + 2 * list);
  void* sort_args[] = {&p};
  int st = launch(sort_kernel_of(ctas), dim3(ctas), dim3(kSortThreads), sort_bytes(p.digit_bits), s, sort_args);
  if (st == GEMM_OK) st = write_rest();

  q.list = p.list[0];
  q.spans = p.spans;
  q.partial = reinterpret_cast<float*>(ws + 2 * list + spans);
  const dim3 grid(runs, ceil_div(units, threads));
  void* sum_args[] = {&q};
  if (st == GEMM_OK) st = launch(kernel, grid, dim3(threads), 0, s, sum_args);
  if (st == GEMM_OK && runs > 1) {
    int n = runs;
    void* join_args[] = {&q, &n};
    const int blocks = ceil_div(units, 32);
    const dim3 join_grid(std::min(runs, std::max(1, 4 * info->num_sms / blocks)), blocks);
    st = launch(table_type == GEMM_TABLE_BF16 ? join_rows<uint16_t>(vector) : join_rows<float>(vector), join_grid,
                dim3(32, kJoinGroups), 0, s, join_args);
  }
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == GEMM_OK) st = GEMM_ERR_LAUNCH;
  return st;
}

}  // extern "C"
