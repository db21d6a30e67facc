// layer_norm.cu -- layer norm of the rows of a residual stream, with the residual's addition in front and the operand of
// the next product behind: BF16, E4M3 with one scale a row, or NVFP4 as gemm_nvfp4 reads it; and its gradient.
//
//   s = bf16(x + r),  mu = mean(s),  rstd = 1 / sqrt(mean((s - mu)^2) + eps),  y = (s - mu) rstd w + b
//   xh = (s - mu) rstd,  c1 = mean(dy w),  c2 = mean(dy w xh),  dx = rstd (dy w - c1 - xh c2) + ds,
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// The variance is of differences, never a difference of means of squares: a warp takes the mean of its own part of the
// row and the squares about that; the CTA's warps then exchange (mean, squares) across one barrier and every thread adds
// M2_w + n_w (mu_w - mu)^2 over them (Chan, Golub and LeVeque's update), so a row whose mean is far larger than its spread
// keeps its digits and the row costs one barrier, as in the RMS norm. All sums are FP32; every output is rounded once from FP32.
//
// Rows are held, fetched ahead and stored as rms_norm.cu's (norm_common.cuh): both directions are bound by the bytes they
// move (forward at most 8 per element, gradient 8). The weight's and the bias's gradients are summed in registers by the
// threads that own the columns, one partial row of each per CTA, which a second kernel adds in a fixed order.
// Measured on GB300: 8192 x 4096 with residual 42.8 us (6.3 TB/s), to E4M3 37.6, gradient 41.0 (6.5 TB/s), and 47.1 with
// weight and bias; 4000 x 8192 to E4M3 37.2 (6.2 TB/s).
#include "norm_common.cuh"

namespace dtcp {

struct LayerNormParams {
  const uint16_t* x;
  const uint16_t* r;  // or null
  const uint16_t* w;  // or null: all ones
  const uint16_t* b;  // or null: zeros
  uint16_t* s;        // or null
  void* y;
  void* scales;
  float* mean;  // or null
  float* rstd;  // or null
  long long ldx, ldr, lds, ldy;
  int rows, cols;
  float eps;
};

struct LayerNormBackwardParams {
  const uint16_t* dy;
  const uint16_t* s;
  const uint16_t* w;
  const float* mean;
  const float* rstd;
  const uint16_t* ds;  // or null
  uint16_t* dx;
  float* partial;  // [grid][2][cols]: dw, db; or null
  long long lddy, lds, ldds, lddx;
  int rows, cols;
};

namespace {

// The columns of a group that lie in the row.
template <int ACCESS>
__device__ __forceinline__ int group_size(int c, int cols) {
  if (ACCESS == kAligned) return c < cols ? 8 : 0;
  return max(0, min(c + 8, cols) - max(c, 0));
}

// Whether a group lies in the row as a whole (then f2), else f1 for its columns that do.
template <int ACCESS, class Whole, class Part>
__device__ __forceinline__ void by_group(int c, int cols, Whole whole_group, Part part) {
  if (ACCESS == kAligned ? c < cols : whole(c, cols)) {
    whole_group();
  } else if (ACCESS != kAligned && edge(c, cols)) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j >= 0 && c + j < cols) part(j);
  }
}

__device__ __forceinline__ float pair_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ float element(const P8& v, int j) {
  float lo, hi;
  f2_unpack(v.v[j >> 1], lo, hi);
  return j & 1 ? hi : lo;
}
__device__ __forceinline__ uint4 pack8_pairs(const P8& p) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi;
    f2_unpack(p.v[j], lo, hi);
    o[j] = pack2(lo, hi);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int VPT, int ACCESS>
__device__ __forceinline__ void load_bias(uint4 (&b)[VPT], const uint16_t* bias, const int (&col)[VPT], int cols) {
  if (bias != nullptr) {
    load_weight<VPT, ACCESS>(b, bias, col, cols);
  } else {
#pragma unroll
    for (int k = 0; k < VPT; ++k) b[k] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// The rows of a CTA (or a team) on their way, `step` apart: SLOTS of them in shared memory, the current one and those
// fetched ahead (1: the next one is fetched once the current one is read).
template <int SLOTS>
struct Ring {
  int slot = 0;
  // Before the first row: fetch(row, slot) for as many as go ahead.
  template <class Fetch>
  __device__ __forceinline__ void start(uint32_t row, uint32_t step, uint32_t rows, const Fetch& fetch) {
#pragma unroll
    for (int i = 0; i < (SLOTS > 1 ? SLOTS - 1 : 1); ++i) one(row + i * step, rows, i, fetch);
  }
  // Fetches the row that is SLOTS - 1 behind `row`, waits for `row` and gives its slot.
  template <class Fetch>
  __device__ __forceinline__ int next(uint32_t row, uint32_t step, uint32_t rows, const Fetch& fetch) {
    if (SLOTS > 1)
      one(row + (SLOTS - 1) * step, rows, SLOTS == 2 ? slot ^ 1 : (slot + SLOTS - 1) % SLOTS, fetch);
    asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
    const int now = slot;
    slot = SLOTS == 2 ? slot ^ 1 : (slot + 1) % SLOTS;
    return now;
  }
  template <class Fetch>
  __device__ __forceinline__ void one(uint32_t row, uint32_t rows, int to, const Fetch& fetch) {
    if (row < rows) fetch(row, to);
    else asm volatile("cp.async.commit_group;" ::: "memory");  // (groups are counted)
  }
};

// 1 / sqrt(v) to FP32's last place: the approximation and one Newton step (0 and infinity are past it).
__device__ __forceinline__ float inverse_sqrt(float v) {
  const float r = rsqrtf(v);
  const float better = fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
  return v > 0.0f && v < INFINITY ? better : r;
}

// The next kernel may start its CTAs beside those of one row each. CTAs that stay, as many as fill the SMs' shared memory,
// have to come together: placed in the gaps that the CTAs of the kernel before leave one by one, the next norm's find no
// room for the last of an SM, which then starts when another ends. 8192 x 4096 forward and gradient, without the weight's,
// in turn: 122 us a pair with this always on, 88 so.
__device__ __forceinline__ void launch_dependents(int rows) {
  if (rows <= static_cast<int>(gridDim.x)) pdl_launch_dependents();
}

// Rows off the 16-byte boundary whose tensors share it (kShared): the whole vectors between a row's first and last boundary
// are the groups of the CTA's threads, as on the boundary, and the up to 14 elements around them belong to the lanes of one
// more warp, the last. With the ends as masked groups of the first and last warp instead, which the others then waited for,
// 2001 x 5123 took 16.5 us forward (13.3 so) and its gradient 25.0 (22.3), 16000 x 1023 29.6 (25.4) and 39.7 (33.2), groups
// and registers as they were then: 13.4 and 19.8, 19.7 and 27.9 with those below.
template <int ACCESS>
struct RowPart {
  static constexpr int AS = ACCESS == kShared ? kAligned : ACCESS;  // how groups are read and written
  int threads, lead, end, phase;  // of the groups; columns before them; where they end; kElements: columns they start early
  __device__ __forceinline__ RowPart(const uint16_t* row, int cols) {
    const int off = ACCESS == kAligned ? 0 : row_phase(row);
    threads = static_cast<int>(blockDim.x) - (ACCESS == kShared ? 32 : 0);
    lead = ACCESS == kShared ? (8 - off) & 7 : 0;
    end = ACCESS == kShared ? lead + (cols - lead) / 8 * 8 : cols;
    phase = ACCESS == kElements ? off : 0;
  }
  __device__ __forceinline__ int column(int k) const {
    return lead + 8 * (static_cast<int>(threadIdx.x) + k * threads) - phase;
  }
  __device__ __forceinline__ bool at_edge() const { return ACCESS == kShared && static_cast<int>(threadIdx.x) >= threads; }
  // The column of a lane of the last warp, or -1.
  __device__ __forceinline__ int edge_column(int cols) const {
    const int lane = threadIdx.x & 31;
    if (lane < 8) return lane < lead ? lane : -1;
    return end + lane - 8 < cols ? end + lane - 8 : -1;
  }
};

__device__ __forceinline__ void cta_sync() { asm volatile("bar.sync 0;" ::: "memory"); }
__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return static_cast<uint16_t>(pack2(v, 0.0f) & 0xFFFFu); }

// ---------------------------------------------------------------- forward

// Mean and variance of the row from its warps' moments, behind the barrier.
// They are taken about the first warp's mean: its distance from the row's mean is at most sqrt(warps) spreads, so taking it
// out again costs five bits of the variance's at the worst, and both sums run side by side.
__device__ __forceinline__ void row_moments(const float2* moments, const float* counts, int warps, float inverse_cols,
                                            float& mean, float& var) {
  const int lane = threadIdx.x & 31;
  const float about = moments[0].x;
  float first = 0.0f, second = 0.0f;
  if (lane < warps) {
    const float2 part = moments[lane];
    const float off = part.x - about, n_off = counts[lane] * off;
    first = n_off;
    second = fmaf(n_off, off, part.y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    first += __shfl_xor_sync(0xffffffffu, first, o);
    second += __shfl_xor_sync(0xffffffffu, second, o);
  }
  const float shift = first * inverse_cols;
  mean = about + shift;
  var = fmaxf(fmaf(-first, shift, second), 0.0f) * inverse_cols + (second - second);  // (NaN and infinity make it NaN)
}

struct NormShared {
  float2 moments[2][32];  // a warp's mean and squares about it
  float counts[32];       // its columns
  uint32_t top[2][32];    // its largest result
};

// The elements around a row's vectors: a lane of the last warp each (column -1: none).
template <int FORMAT>
__device__ __forceinline__ void norm_edge(const LayerNormParams& p, NormShared& sh, int column, uint32_t rows, int warps,
                                          float inverse_count, float inverse_cols) {
  const bool on = column >= 0;
  const int lane = threadIdx.x & 31;
  const float w = on && p.w != nullptr ? bf16_value(p.w[column]) : 1.0f;
  const float b = on && p.b != nullptr ? bf16_value(p.b[column]) : 0.0f;
  auto load = [&](uint32_t row, uint16_t& x, uint16_t& r) {
    x = on ? p.x[row * p.ldx + column] : uint16_t(0);
    r = on && p.r != nullptr ? p.r[row * p.ldr + column] : uint16_t(0);
  };
  uint16_t x, r, x_next = 0, r_next = 0;
  load(blockIdx.x, x, r);
  int parity = 0;
  for (uint32_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
    if (row + gridDim.x < rows) load(row + gridDim.x, x_next, r_next);
    if (p.r != nullptr) x = bf16_bits(bf16_value(x) + bf16_value(r));
    if (on && p.s != nullptr) p.s[row * p.lds + column] = x;
    const float s = bf16_value(x);
    const float warp_mean = warp_sum(s) * inverse_count, d = on ? s - warp_mean : 0.0f;
    const float squares = warp_sum(d * d);
    if (lane == 0) sh.moments[parity][threadIdx.x >> 5] = make_float2(warp_mean, squares);
    cta_sync();
    float mean, var;
    row_moments(sh.moments[parity], sh.counts, warps, inverse_cols, mean, var);
    const float y = on ? fmaf((s - mean) * inverse_sqrt(var + p.eps), w, b) : 0.0f;
    if constexpr (FORMAT == GEMM_NORM_BF16) {
      if (on) static_cast<uint16_t*>(p.y)[row * p.ldy + column] = bf16_bits(y);
    } else {
      const E4m3Scale scale(block_max_bits(abs_bits(y), sh.top[parity], warps));
      if (on) static_cast<uint8_t*>(p.y)[row * p.ldy + column] = static_cast<uint8_t>(e4m3_code(y * scale.inverse));
    }
    x = x_next;
    r = r_next;
  }
}

template <int VPT, int SLOTS, int FORMAT, int ACCESS>
__global__ void __maxnreg__(norm_regs<VPT>(96, 128)) layer_norm_kernel(const LayerNormParams p) {
  constexpr int AS = RowPart<ACCESS>::AS;
  extern __shared__ uint4 fetched[];  // [SLOTS][2][VPT][threads], then (KEPT) weight and bias: [2][VPT][threads]
  __shared__ NormShared sh;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4* const mine = fetched + threadIdx.x;
  const uint32_t rows = static_cast<uint32_t>(p.rows);
  const int slot_size = 2 * VPT * static_cast<int>(blockDim.x);
  launch_dependents(p.rows);
  pdl_wait();
  const RowPart<ACCESS> part(p.x + blockIdx.x * p.ldx, p.cols);
  int col[VPT], size = 0;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    col[k] = part.column(k);
    size += group_size<AS>(col[k], part.end);
  }
  const int edge = part.at_edge() ? part.edge_column(p.cols) : -1;
  if (part.at_edge()) size = edge >= 0 ? 1 : 0;
  const float count = warp_sum(static_cast<float>(size)), inverse_count = count > 0.0f ? 1.0f / count : 0.0f;
  if (lane == 0) sh.counts[warp] = count;  // (read behind the first row's barrier)
  const float inverse_cols = 1.0f / static_cast<float>(p.cols);
  if (part.at_edge()) {
    if constexpr (ACCESS == kShared && FORMAT != GEMM_NORM_NVFP4)
      norm_edge<FORMAT>(p, sh, edge, rows, warps, inverse_count, inverse_cols);
    return;
  }
  auto fetch = [&](uint32_t row, int slot) {
    const uint16_t* const rows[2] = {p.x + row * p.ldx, p.r != nullptr ? p.r + row * p.ldr : nullptr};
    fetch_rows<2, VPT, AS>(mine + slot * slot_size, rows, col, part.end, row);
  };
  // (groups past the row's end stay zero)
  for (int i = 0; i < SLOTS * 2 * VPT; ++i) mine[i * static_cast<int>(blockDim.x)] = make_uint4(0u, 0u, 0u, 0u);
  Ring<SLOTS> ring;
  ring.start(blockIdx.x, gridDim.x, rows, fetch);
  // Weight and bias: in shared memory too, each thread's its own, so that registers do not bound the CTAs (with eight groups
  // there is no room).
  constexpr bool KEPT = VPT < 8;
  uint4* const affine = mine + SLOTS * slot_size;
  uint4 w[VPT], b[VPT];
  load_weight<VPT, ACCESS>(w, p.w, col, part.end);
  load_bias<VPT, ACCESS>(b, p.b, col, part.end);
  if constexpr (KEPT) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      affine[k * static_cast<int>(blockDim.x)] = w[k];
      affine[(VPT + k) * static_cast<int>(blockDim.x)] = b[k];
    }
  }
  int parity = 0;
  for (uint32_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {  // (no sum of them passes 32 bits)
    const uint4* const in = mine + ring.next(row, gridDim.x, rows, fetch) * slot_size;
    P8 s[VPT];  // the stream (zeros outside the row), then the results
    uint64_t sum = 0;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      uint4 v = in[k * static_cast<int>(blockDim.x)];
      if (p.r != nullptr) {
        P8 a = unpack8_pairs(v);
        const P8 e = unpack8_pairs(in[(VPT + k) * static_cast<int>(blockDim.x)]);
#pragma unroll
        for (int j = 0; j < 4; ++j) a.v[j] = f2_add(a.v[j], e.v[j]);
        v = pack8_pairs(a);
      }
      if (p.s != nullptr) store8<AS>(p.s + row * p.lds, col[k], part.end, v);
      s[k] = unpack8_pairs(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = f2_add(sum, s[k].v[j]);
    }
    if (SLOTS == 1 && row + gridDim.x < rows) fetch(row + gridDim.x, 0);
    const float warp_mean = warp_sum(pair_sum(sum)) * inverse_count;
    const uint64_t minus = f2_pack(-warp_mean, -warp_mean);
    uint64_t squares2 = 0;
    float squares = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      by_group<AS>(
          col[k], part.end,
          [&] {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t d = f2_add(s[k].v[j], minus);
              squares2 = f2_fma(d, d, squares2);
            }
          },
          [&](int j) {
            const float d = element(s[k], j) - warp_mean;
            squares = fmaf(d, d, squares);
          });
    squares = warp_sum(squares + pair_sum(squares2));
    float mean = warp_mean, var = squares * inverse_cols + (squares - squares);  // (infinite squares make the row NaN)
    if (warps > 1) {
      if (lane == 0) sh.moments[parity][warp] = make_float2(warp_mean, squares);
      cta_sync();
      row_moments(sh.moments[parity], sh.counts, warps, inverse_cols, mean, var);
    }
    const float rstd = inverse_sqrt(var + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean + (var - var);  // (of a row with an infinity NaN, as its other outputs)
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    const uint64_t mean2 = f2_pack(-mean, -mean), rstd2 = f2_pack(rstd, rstd);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const P8 g = unpack8_pairs(KEPT ? affine[k * static_cast<int>(blockDim.x)] : w[k]);
      const P8 h = unpack8_pairs(KEPT ? affine[(VPT + k) * static_cast<int>(blockDim.x)] : b[k]);
      P8 y = {};
      by_group<AS>(
          col[k], part.end,
          [&] {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              y.v[j] = f2_fma(f2_mul(f2_add(s[k].v[j], mean2), rstd2), g.v[j], h.v[j]);
          },
          [&](int j) {
            const float v = fmaf((element(s[k], j) - mean) * rstd, element(g, j), element(h, j));
            float lo, hi;
            f2_unpack(y.v[j >> 1], lo, hi);
            y.v[j >> 1] = j & 1 ? f2_pack(lo, v) : f2_pack(v, hi);
          });
      s[k] = y;
    }
    auto value = [&](int k) {
      F8 y;
#pragma unroll
      for (int j = 0; j < 4; ++j) f2_unpack(s[k].v[j], y.v[2 * j], y.v[2 * j + 1]);
      return y;
    };
    norm_output<VPT, FORMAT, AS>(value, p.y, p.ldy, p.scales, row, part.end, col, sh.top[parity], warps);
  }
}

// ---------------------------------------------------------------- backward

// Two sums over the CTA, the same bits in every thread (see block_sum).
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* slots, int warps) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (warps == 1) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = make_float2(a, b);
  cta_sync();
  const float2 v = (threadIdx.x & 31) < warps ? slots[threadIdx.x & 31] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// The elements around a row's vectors, as norm_edge.
__device__ __forceinline__ void norm_backward_edge(const LayerNormBackwardParams& p, float2 (&slots)[2][32], int column,
                                                   uint32_t rows, int warps, float inverse_cols) {
  const bool on = column >= 0;
  const float w = on && p.w != nullptr ? bf16_value(p.w[column]) : 1.0f;
  struct Element {
    uint16_t s, dy, ds;
    float mean, rstd;
  };
  auto load = [&](uint32_t row) {
    Element e = {0, 0, 0, p.mean[row], p.rstd[row]};
    if (on) {
      e.s = p.s[row * p.lds + column];
      e.dy = p.dy[row * p.lddy + column];
      if (p.ds != nullptr) e.ds = p.ds[row * p.ldds + column];
    }
    return e;
  };
  Element e = load(blockIdx.x), next = e;
  float dw = 0.0f, db = 0.0f;
  int parity = 0;
  for (uint32_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
    if (row + gridDim.x < rows) next = load(row + gridDim.x);
    const float off = bf16_value(e.s) - e.mean, xh = off * e.rstd, dy = bf16_value(e.dy), dyw = dy * w;
    if (on) {
      dw = fmaf(dy, xh, dw);
      db += dy;
    }
    const float2 c = block_sum2(on ? dyw : 0.0f, on ? dyw * xh : 0.0f, slots[parity], warps);
    const float c1 = c.x * inverse_cols * -e.rstd, c2 = c.y * inverse_cols * -(e.rstd * e.rstd);
    if (on)
      p.dx[row * p.lddx + column] = bf16_bits(fmaf(dyw, e.rstd, fmaf(off, c2, c1)) + bf16_value(e.ds));
    e = next;
  }
  if (p.partial != nullptr) {
    pdl_launch_dependents();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      cta_sync();
      cta_sync();
      if (on) p.partial[(2LL * blockIdx.x + t) * p.cols + column] = t == 0 ? dw : db;
    }
  }
}

// TEAMS: rows of a warp, kTeams of them in a CTA at a time, so that the gradients of weight and bias leave a CTA as one
// partial row instead of eight. Measured on GB300 with them: 65536 x 256 39 us in CTAs of a warp and 27, 8192 x 512 20 and
// 15. (Wider rows lose by it what they gain: with as many teams as an SM holds 8192 x 4096 58 and 61.)
constexpr int kTeams = 8;
// REGS: what holds a row, its weight and the sums of dw and db without spills, 128 with two groups a thread, even if a CTA
// is alone on its SM then: 8192 x 4096 46.9 us with 80 registers and two CTAs, 41.3 so; 4000 x 8192 42.4, with four groups
// (which spill) 52.3; 16000 x 1023 33.1 with 88, 28.0 so. One group with a row a warp: 64 and 80 the same 65536 x 255 in 48.7
// and 44.4. Off the boundary 96 where a second CTA of the warps with a row's ends fits an SM so, nine and ten of them (4000 x
// 4099 31.3 with 128, 27.1 so; 4000 x 4401 34.2 and 30.1), or the only one (seventeen).
// Three and four groups leave no registers for the weight: 4000 x 10000 82.9 us with four and the weight in registers, 78.2
// with three, 73.3 with three and it in shared memory; 4000 x 16384 105.0 and 96.4 with four.
__host__ __device__ constexpr bool weight_in_shared(int vpt) { return vpt == 3 || vpt == 4; }
constexpr int backward_regs(int vpt, int slots, bool teams) { return vpt > 1 ? 128 : slots == 4 && !teams ? 80 : 64; }
inline bool fewer_regs_pay(int threads) {
  const auto ctas = [&](int regs) { return 65536 / (regs * threads); };  // of an SM
  return ctas(128) < 2 && ctas(96) > ctas(128);
}
template <int VPT, int SLOTS, int ACCESS, bool TEAMS, int REGS = backward_regs(VPT, SLOTS, TEAMS)>
__global__ void __maxnreg__(REGS) layer_norm_backward_kernel(const LayerNormBackwardParams p) {
  constexpr int AS = RowPart<ACCESS>::AS;
  constexpr bool KEPT = weight_in_shared(VPT);
  extern __shared__ uint4 fetched[];  // [teams][SLOTS][3][VPT][threads], then (KEPT) the weight: [VPT][threads]
  __shared__ float2 slots[2][32];
  const int warps = blockDim.x >> 5;
  const int team = TEAMS ? static_cast<int>(threadIdx.y) : 0;
  const uint32_t first_row = blockIdx.x + (TEAMS ? gridDim.x * team : 0u), step = gridDim.x * (TEAMS ? kTeams : 1);
  const uint32_t rows = static_cast<uint32_t>(p.rows);
  const int slot_size = 3 * VPT * static_cast<int>(blockDim.x);
  uint4* const mine = fetched + team * SLOTS * slot_size + threadIdx.x;
  launch_dependents(p.rows);
  pdl_wait();
  const RowPart<ACCESS> part(p.s + blockIdx.x * p.lds, p.cols);
  const float inverse_cols = 1.0f / static_cast<float>(p.cols);
  if (part.at_edge()) {
    if constexpr (ACCESS == kShared) norm_backward_edge(p, slots, part.edge_column(p.cols), rows, warps, inverse_cols);
    return;
  }
  int col[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) col[k] = part.column(k);
  auto fetch = [&](uint32_t row, int slot) {
    const uint16_t* const rows[3] = {p.s + row * p.lds, p.dy + row * p.lddy,
                                     p.ds != nullptr ? p.ds + row * p.ldds : nullptr};
    fetch_rows<3, VPT, AS>(mine + slot * slot_size, rows, col, part.end, row);
  };
  // (groups past the row's end stay zero)
  for (int i = 0; i < SLOTS * 3 * VPT; ++i) mine[i * static_cast<int>(blockDim.x)] = make_uint4(0u, 0u, 0u, 0u);
  Ring<SLOTS> ring;
  ring.start(first_row, step, rows, fetch);
  uint4 w[VPT];
  P8 dw[VPT], db[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[k].v[j] = db[k].v[j] = 0;
  load_weight<VPT, ACCESS>(w, p.w, col, part.end);
  uint4* const kept = mine + SLOTS * slot_size;
  if constexpr (KEPT) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) kept[k * static_cast<int>(blockDim.x)] = w[k];
  }
  auto weight = [&](int k) { return unpack8_pairs(KEPT ? kept[k * static_cast<int>(blockDim.x)] : w[k]); };
  float rstd = 0.0f, mean = 0.0f, rstd_next = 0.0f, mean_next = 0.0f;
  if (!TEAMS || first_row < rows) {
    rstd = p.rstd[first_row];
    mean = p.mean[first_row];
  }
  int parity = 0;
  for (uint32_t row = first_row; row < rows; row += step, parity ^= 1) {  // (no sum of them passes 32 bits)
    const bool more = row + step < rows;
    if (more) {
      rstd_next = p.rstd[row + step];
      mean_next = p.mean[row + step];
    }
    const uint4* const in = mine + ring.next(row, step, rows, fetch) * slot_size;
    const uint64_t r2 = f2_pack(rstd, rstd), m2 = f2_pack(-mean, -mean);
    uint64_t sum1 = 0, sum2 = 0;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const uint4 v[2] = {in[k * static_cast<int>(blockDim.x)], in[(VPT + k) * static_cast<int>(blockDim.x)]};
      // (outside the row dy is 0, and so is what it adds)
      const P8 a = unpack8_pairs(v[0]), d = unpack8_pairs(v[1]), g = weight(k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t xh = f2_mul(f2_add(a.v[j], m2), r2), dyw = f2_mul(d.v[j], g.v[j]);
        dw[k].v[j] = f2_fma(d.v[j], xh, dw[k].v[j]);
        db[k].v[j] = f2_add(d.v[j], db[k].v[j]);
        sum1 = f2_add(dyw, sum1);
        sum2 = f2_fma(dyw, xh, sum2);
      }
    }
    const float2 c = block_sum2(pair_sum(sum1), pair_sum(sum2), slots[parity], warps);
    // rstd (dy w - c1 - xh c2) = rstd dy w + (s - mean) (-rstd^2 c2) - rstd c1
    const float c1 = c.x * inverse_cols * -rstd, c2 = c.y * inverse_cols * -(rstd * rstd);
    const uint64_t c1_2 = f2_pack(c1, c1), c2_2 = f2_pack(c2, c2);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const P8 a = unpack8_pairs(in[k * static_cast<int>(blockDim.x)]);
      const P8 d = unpack8_pairs(in[(VPT + k) * static_cast<int>(blockDim.x)]), g = weight(k);
      P8 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o.v[j] = f2_fma(f2_mul(d.v[j], g.v[j]), r2, f2_fma(f2_add(a.v[j], m2), c2_2, c1_2));
      if (p.ds != nullptr) {
        const P8 e = unpack8_pairs(in[(2 * VPT + k) * static_cast<int>(blockDim.x)]);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = f2_add(o.v[j], e.v[j]);
      }
      store8<AS>(p.dx + row * p.lddx, col[k], part.end, pack8_pairs(o));
    }
    if (SLOTS == 1 && more) fetch(row + step, 0);
    rstd = rstd_next;
    mean = mean_next;
  }
  if (p.partial != nullptr) {  // through shared memory: teams are added there, and a warp writes 32 columns side by side
    pdl_launch_dependents();  // (the next kernel is small and waits for this one's end: 0.3 us)
    const int team_floats = SLOTS * slot_size * 4, threads = part.threads * static_cast<int>(blockDim.y);
    const int from = part.lead - part.phase;  // the column of the first place
    float* const sums = reinterpret_cast<float*>(fetched);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      cta_sync();
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const P8& v = t == 0 ? dw[k] : db[k];
        ulonglong2* at = reinterpret_cast<ulonglong2*>(sums + team * team_floats + col[k] - from);
        at[0] = make_ulonglong2(v.v[0], v.v[1]);
        at[1] = make_ulonglong2(v.v[2], v.v[3]);
      }
      cta_sync();
      float* out = p.partial + (2LL * blockIdx.x + t) * p.cols;
      for (int c = part.lead + team * part.threads + static_cast<int>(threadIdx.x); c < part.end; c += threads) {
        float v = sums[c - from];
        if (TEAMS)
#pragma unroll
          for (int i = 1; i < kTeams; ++i) v += sums[i * team_floats + c - from];
        out[c] = v;
      }
    }
  }
}

// dw and db (either may be null) from the partial rows in a fixed order: 32 warps take every 32nd row of 32 columns,
// then a column each. blockIdx.y: 0 dw, 1 db.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps)
    layer_norm_sum_kernel(const float* partial, int rows, int cols, float* dw, float* db) {
  __shared__ float part[kSumWarps][33];
  pdl_launch_dependents();
  pdl_wait();
  float* const out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < cols)
#pragma unroll 16
    for (int r = warp; r < rows; r += kSumWarps) v += partial[(2LL * r + blockIdx.y) * cols + c];
  part[warp][lane] = v;
  __syncthreads();
  v = warp_sum(part[lane][warp]);  // one column a warp
  if (lane == 0 && blockIdx.x * 32 + warp < cols) out[blockIdx.x * 32 + warp] = v;
}

// ---------------------------------------------------------------- host side

// Threads, groups a thread and rows in shared memory. Measured on GB300, us:
//   up to 256 columns a warp a row, without a barrier; an SM holds 32 of those at most, so three rows go ahead:
//     65536 x 256 forward 26 with two groups a thread and one row ahead, 17 so; gradient 43 and 26;
//   forward on the 16-byte boundary four groups a thread, as what a row costs whatever its length (some 130 instructions a
//     warp, in reductions and addresses) is most of it: 4000 x 8192 to E4M3 40.3 with two and 37.3, 16000 x 1024 14.8 and
//     12.7; off the boundary two where two CTAs fit: 16000 x 1023 31.4 with four and 25.4, 4000 x 7001 38.5 and 45.2;
//   four streams that pass L2 (two in, two out), on the boundary: with all rows that fit on their way, memory turns between
//     reads and writes more than it need, so an SM has 8192 columns of rows at a time, two groups a thread and (from 4096
//     columns on) two rows ahead: 8192 x 4096 46.5 with four groups and four CTAs an SM and 42.7, 32000 x 1024 45.3 and
//     41.6, 4000 x 8192 44.5 and 41.5 (5000 x 4096, in L2 for the most part, 27.2 and 26.3);
//   gradient two up to 512 threads, then three, then four (see backward_regs); with two of them two rows ahead: one ahead
//     instead cost 8192 x 4096 50.9 instead of 47.0 (with 80 registers), three 42.4 instead of 41.3.
constexpr int kSmemOfSm = 228 * 1024;
struct LayerNormShape {
  NormShape at;
  int slots;
  int most = 0;  // CTAs of an SM (0: as many as fit)
  int smem(int tensors, int kept) const {
    // (a limit by shared memory that one more CTA does not find, as a smaller grid would not spread evenly over the SMs)
    return std::max((slots * tensors + kept) * at.vpt * at.threads * 16, most > 0 ? kSmemOfSm / (most + 1) : 0);
  }
};
LayerNormShape layer_norm_shape(int rows, int cols, int num_sms, NormAccess access, bool forward, bool four_streams) {
  if (access == kShared) {  // the whole groups, and a warp for the elements around them
    const int groups = cols / 8;
    if (groups <= 32 && rows > num_sms) return LayerNormShape{{64, 1}, 4};
    NormShape s{0, rows <= num_sms ? 1 : forward && groups > 704 ? 4 : 2};
    for (;; s.vpt *= 2) {
      s.threads = std::max(32, ceil_div(ceil_div(groups, s.vpt), 32) * 32);
      if (s.threads <= (s.vpt == 1 ? 992 : s.vpt == 2 ? 512 : 480)) break;
    }
    if (s.vpt == 4 && !forward && groups <= 3 * 480) s = NormShape{ceil_div(ceil_div(groups, 3), 32) * 32, 3};
    s.threads += 32;
    return LayerNormShape{s, s.vpt == 2 && !forward ? 3 : s.vpt == 3 ? 2 : norm_slots(s.vpt)};
  }
  const bool is_aligned = access == kAligned;
  const int groups = ceil_div(cols, 8) + (is_aligned ? 0 : 1);
  if (groups <= 32 && rows > num_sms) return LayerNormShape{{32, 1}, 4};
  if (four_streams && rows > num_sms && groups > 96 && groups <= 1024) {
    return LayerNormShape{{ceil_div(ceil_div(groups, 2), 32) * 32, 2}, groups < 512 ? 2 : 3, (1024 + groups / 2) / groups};
  }
  NormShape s = norm_shape(rows, cols, num_sms, is_aligned);
  if (s.vpt == 2 && is_aligned && forward && groups > 96) s = NormShape{ceil_div(ceil_div(groups, 4), 32) * 32, 4};
  if (s.vpt == 4 && !forward && groups <= 3 * 512) return LayerNormShape{{ceil_div(ceil_div(groups, 3), 32) * 32, 3}, 2};
  const bool three = s.vpt == 2 && is_aligned && !forward && s.threads > 32;
  return LayerNormShape{s, three ? 3 : norm_slots(s.vpt)};
}

template <int FORMAT, int ACCESS>
const void* forward_kernel(const LayerNormShape& s) {
  switch (s.at.vpt) {
    case 1:
      return s.slots == 1 ? reinterpret_cast<const void*>(layer_norm_kernel<1, 1, FORMAT, ACCESS>)
                          : reinterpret_cast<const void*>(layer_norm_kernel<1, 4, FORMAT, ACCESS>);
    case 2:
      if constexpr (FORMAT == GEMM_NORM_BF16 && ACCESS == kAligned)
        if (s.slots == 3) return reinterpret_cast<const void*>(layer_norm_kernel<2, 3, FORMAT, ACCESS>);
      return reinterpret_cast<const void*>(layer_norm_kernel<2, 2, FORMAT, ACCESS>);
    case 4: return reinterpret_cast<const void*>(layer_norm_kernel<4, 2, FORMAT, ACCESS>);
    default: return reinterpret_cast<const void*>(layer_norm_kernel<8, 1, FORMAT, ACCESS>);
  }
}
template <int FORMAT>
const void* forward_kernel(const LayerNormShape& s, NormAccess access) {
  return access == kAligned  ? forward_kernel<FORMAT, kAligned>(s)
         : access == kShared ? forward_kernel<FORMAT, kShared>(s)
                             : forward_kernel<FORMAT, kElements>(s);
}

template <int ACCESS>
const void* backward_kernel(const LayerNormShape& s, bool teams) {
  if constexpr (ACCESS != kShared) {
    if (teams && s.at.vpt == 1) return reinterpret_cast<const void*>(layer_norm_backward_kernel<1, 4, ACCESS, true>);
    if (teams) return reinterpret_cast<const void*>(layer_norm_backward_kernel<2, 2, ACCESS, true>);
  }
  switch (s.at.vpt) {
    case 1:
      return s.slots == 1 ? reinterpret_cast<const void*>(layer_norm_backward_kernel<1, 1, ACCESS, false>)
                          : reinterpret_cast<const void*>(layer_norm_backward_kernel<1, 4, ACCESS, false>);
    case 2:
      if constexpr (ACCESS == kShared) {
        if (fewer_regs_pay(s.at.threads))
          return reinterpret_cast<const void*>(layer_norm_backward_kernel<2, 3, ACCESS, false, 96>);
        return reinterpret_cast<const void*>(layer_norm_backward_kernel<2, 3, ACCESS, false>);
      } else {
        if constexpr (ACCESS == kAligned)
          if (s.slots == 3) return reinterpret_cast<const void*>(layer_norm_backward_kernel<2, 3, ACCESS, false>);
        return reinterpret_cast<const void*>(layer_norm_backward_kernel<2, 2, ACCESS, false>);
      }
    case 3: return reinterpret_cast<const void*>(layer_norm_backward_kernel<3, 2, ACCESS, false>);
    case 4: return reinterpret_cast<const void*>(layer_norm_backward_kernel<4, 2, ACCESS, false>);
    default: return reinterpret_cast<const void*>(layer_norm_backward_kernel<8, 1, ACCESS, false>);
  }
}

// How a call's rows lie: for kShared a row needs a whole vector between its boundaries, and no more of them than eight a
// thread of 15 warps.
NormAccess norm_access(bool aligned, bool shared, int cols) {
  return aligned ? kAligned : shared && cols >= 16 && cols <= 30720 ? kShared : kElements;
}

}  // namespace
}  // namespace dtcp

using namespace dtcp;

extern "C" {

int gemm_layer_norm(const void* X, const void* R, const void* W, const void* B, void* S, void* Y, void* scales,
                    float* mean, float* rstd, int rows, int cols, float eps, int format, void* stream,
                    const gemm_norm_strides_t* strides) {
  if (rows < 0 || cols < 0 || !(eps >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  if (format != GEMM_NORM_BF16 && format != GEMM_NORM_E4M3 && format != GEMM_NORM_NVFP4) return GEMM_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_OK;
  if (cols == 0) {  // rows without columns: what is one number a row is 0
    void* const numbers[] = {format == GEMM_NORM_E4M3 ? scales : nullptr, mean, rstd};
    if (numbers[0] == nullptr && mean == nullptr && rstd == nullptr) return GEMM_OK;
    for (void* n : numbers)
      if (misaligned(n, 4)) return GEMM_ERR_MISALIGNED;
    int device = 0, err = 0;
    if (current_device_info(&device, &err) == nullptr) return err;
    int st = GEMM_OK;
    for (void* n : numbers)
      if (st == GEMM_OK) st = zero_floats(n, rows, static_cast<cudaStream_t>(stream));
    return st;
  }
  if (X == nullptr || Y == nullptr || (format != GEMM_NORM_BF16 && scales == nullptr)) return GEMM_ERR_INVALID_ARG;
  if (R != nullptr && S == nullptr) return GEMM_ERR_INVALID_ARG;
  LayerNormParams p;
  p.ldx = p.ldr = p.lds = p.ldy = cols;
  if (strides != nullptr) {
    if (strides->x) p.ldx = strides->x;
    if (strides->residual) p.ldr = strides->residual;
    if (strides->sum) p.lds = strides->sum;
    if (strides->y) p.ldy = strides->y;
    if (p.ldx < cols || p.ldr < cols || p.lds < cols || p.ldy < cols) return GEMM_ERR_INVALID_ARG;
  }
  if (cols > kNormMaxCols || (format == GEMM_NORM_NVFP4 && (cols % 16 != 0 || p.ldy != cols)))
    return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (misaligned(X, 2) || misaligned(R, 2) || misaligned(W, 2) || misaligned(B, 2) || misaligned(S, 2) ||
      misaligned(mean, 4) || misaligned(rstd, 4) ||
      misaligned(Y, format == GEMM_NORM_BF16 ? 2 : format == GEMM_NORM_E4M3 ? 1 : 4) ||
      misaligned(scales, format == GEMM_NORM_E4M3 ? 4 : 1))
    return GEMM_ERR_MISALIGNED;
  p.x = static_cast<const uint16_t*>(X);
  p.r = static_cast<const uint16_t*>(R);
  p.w = static_cast<const uint16_t*>(W);
  p.b = static_cast<const uint16_t*>(B);
  p.s = static_cast<uint16_t*>(S);
  p.y = Y;
  p.scales = scales;
  p.mean = mean;
  p.rstd = rstd;
  p.rows = rows;
  p.cols = cols;
  p.eps = eps;
  const RowPlace place(X, p.ldx, 2);
  bool shared = (R == nullptr || RowPlace(R, p.ldr, 2) == place) && (S == nullptr || RowPlace(S, p.lds, 2) == place);
  if (format == GEMM_NORM_BF16) shared = shared && RowPlace(Y, p.ldy, 2) == place;
  if (format == GEMM_NORM_E4M3) shared = shared && RowPlace(Y, p.ldy, 1) == place;  // (8-byte vectors of codes)
  const bool aligned = shared && place.aligned() && cols % 8 == 0 && !misaligned(W, 16) && !misaligned(B, 16);
  if (format == GEMM_NORM_NVFP4 && !aligned) return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  const NormAccess access = norm_access(aligned, shared, cols);
  const bool four_streams =  // (some 1.5 times L2)
      access == kAligned && R != nullptr && format == GEMM_NORM_BF16 && 16LL * rows * cols > 3 * info->l2_bytes;
  const LayerNormShape shape = layer_norm_shape(rows, cols, info->num_sms, access, true, four_streams);
  const void* kernel = format == GEMM_NORM_NVFP4  ? forward_kernel<GEMM_NORM_NVFP4, kAligned>(shape)
                       : format == GEMM_NORM_E4M3 ? forward_kernel<GEMM_NORM_E4M3>(shape, access)
                                                  : forward_kernel<GEMM_NORM_BF16>(shape, access);
  void* args[] = {&p};
  const int smem = shape.smem(2, shape.at.vpt < 8 ? 2 : 0);
  const int grid = norm_grid(kernel, rows, shape.at.threads, smem, info->num_sms);
  if (grid == 0) return GEMM_ERR_LAUNCH;
  return norm_launch(kernel, dim3(grid), dim3(shape.at.threads), smem, static_cast<cudaStream_t>(stream), args);
}

int gemm_layer_norm_backward(const void* dY, const void* S, const void* W, const float* mean, const float* rstd,
                             const void* dS, void* dX, float* dW, float* dB, int rows, int cols, void* stream,
                             const gemm_norm_backward_strides_t* strides) {
  if (rows < 0 || cols < 0) return GEMM_ERR_INVALID_ARG;
  if (cols == 0) return GEMM_OK;
  if (rows > 0 && (dY == nullptr || S == nullptr || mean == nullptr || rstd == nullptr || dX == nullptr))
    return GEMM_ERR_INVALID_ARG;
  LayerNormBackwardParams p;
  p.lddy = p.lds = p.ldds = p.lddx = cols;
  if (strides != nullptr) {
    if (strides->dy) p.lddy = strides->dy;
    if (strides->sum) p.lds = strides->sum;
    if (strides->dsum) p.ldds = strides->dsum;
    if (strides->dx) p.lddx = strides->dx;
    if (p.lddy < cols || p.lds < cols || p.ldds < cols || p.lddx < cols) return GEMM_ERR_INVALID_ARG;
  }
  if (cols > kNormMaxCols) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (misaligned(dY, 2) || misaligned(S, 2) || misaligned(W, 2) || misaligned(mean, 4) || misaligned(rstd, 4) ||
      misaligned(dS, 2) || misaligned(dX, 2) || misaligned(dW, 4) || misaligned(dB, 4))
    return GEMM_ERR_MISALIGNED;
  const bool sums = dW != nullptr || dB != nullptr;
  if (rows == 0 && !sums) return GEMM_OK;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // the sums over no rows
    const int rc = zero_floats(dW, cols, st);
    return rc != GEMM_OK ? rc : zero_floats(dB, cols, st);
  }
  p.dy = static_cast<const uint16_t*>(dY);
  p.s = static_cast<const uint16_t*>(S);
  p.w = static_cast<const uint16_t*>(W);
  p.mean = mean;
  p.rstd = rstd;
  p.ds = static_cast<const uint16_t*>(dS);
  p.dx = static_cast<uint16_t*>(dX);
  p.partial = nullptr;
  p.rows = rows;
  p.cols = cols;
  const RowPlace place(S, p.lds, 2);
  const bool shared = RowPlace(dY, p.lddy, 2) == place && (dS == nullptr || RowPlace(dS, p.ldds, 2) == place) &&
                      RowPlace(dX, p.lddx, 2) == place;
  const bool aligned = shared && place.aligned() && cols % 8 == 0 && !misaligned(W, 16);
  const NormAccess access = norm_access(aligned, shared, cols);
  const LayerNormShape shape = layer_norm_shape(rows, cols, info->num_sms, access, false, false);
  // (a grid of a multiple of 8, or a row a team: rows of a CTA share the column at which their boundary lies)
  const bool teams = sums && shape.at.threads == 32 && rows > info->num_sms && info->num_sms % 8 == 0;
  const void* kernel = access == kAligned  ? backward_kernel<kAligned>(shape, teams)
                       : access == kShared ? backward_kernel<kShared>(shape, teams)
                                           : backward_kernel<kElements>(shape, teams);
  const dim3 threads(shape.at.threads, teams ? kTeams : 1);
  const int smem = shape.smem(3, weight_in_shared(shape.at.vpt) ? 1 : 0) * static_cast<int>(threads.y);
  const int grid = norm_grid(kernel, rows, static_cast<int>(threads.x * threads.y), smem, info->num_sms);
  if (grid == 0) return GEMM_ERR_LAUNCH;
  void* ws = nullptr;
  if (sums) {
    cudaMemPool_t pool = workspace_pool(device);
    if (pool == nullptr ||
        cudaMallocFromPoolAsync(&ws, static_cast<size_t>(grid) * 2 * cols * 4, pool, st) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_OUT_OF_MEMORY;
    }
    p.partial = static_cast<float*>(ws);
  }
  void* args[] = {&p};
  int rc = norm_launch(kernel, dim3(grid), threads, smem, st, args);
  if (ws != nullptr) {
    if (rc == GEMM_OK) {
      const float* partial = p.partial;
      int partial_rows = grid;
      void* sum_args[] = {&partial, &partial_rows, &cols, &dW, &dB};
      rc = norm_launch(reinterpret_cast<const void*>(layer_norm_sum_kernel), dim3(ceil_div(cols, 32), 2),
                       dim3(32 * kSumWarps), 0, st, sum_args);
    }
    if (cudaFreeAsync(ws, st) != cudaSuccess && rc == GEMM_OK) rc = GEMM_ERR_LAUNCH;
  }
  return rc;
}

}  // extern "C"
