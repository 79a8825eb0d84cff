// RMS norm in front of the layer, with the residual's addition and an output
// in MX blocks of 8 bits, and its backward.
//
//   forward   r = round(res + x), rstd = 1 / sqrt(mean r^2 + eps),
//             y = round(r rstd w), codes | scales = MX blocks of y
//   backward  n = r rstd, g = dy w, d_r = rstd (g - n mean(g n)) + d_res,
//             d_w = sum over the rows of dy n
//
// Both are bound by memory: a row is read once, its elements stay in
// registers between the sum and the outputs (a thread holds NV units of 8
// consecutive elements, 16 bytes of bf16 and 32 of fp32), and everything
// that goes out is written from there.  Short rows go to a wave or a part of one
// (no barrier between the sum and the outputs), others to a workgroup; rows
// longer than 16384 elements are read twice.  Workgroups stride over the
// rows; the weight is read again for every row, from the caches.
//
// Measured, bf16 (a copy of the same bytes streams at 5.2 TB/s): 16384 x 2048
// with y and MX blocks 58 us, 5.2 TB/s; 32749 x 7168 with an fp32 stream 511
// us, 5.5 TB/s; its backward on 16381 rows 360 us, 5.2 TB/s, 7 of them the
// second sum of d_w.  1 x 7168 forward 6.7 us a call, 3.6 of kernel, 512 x 256
// fp32 backward 6.0 and 4.5; a call of one wave takes 4.3 and 1.8.
#include "mok_internal.h"
#include "mok_lanes.h"
#include "mok_mx.h"
#include "mok_unit.h"

namespace mok {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 8;              // consecutive elements that a thread handles together

// Threads of a workgroup whose rows have L threads each.
template <int L>
constexpr int block_of() { return L <= 64 ? kThreads : L; }
// Waves that share a row.
template <int L>
constexpr int waves_of() { return L <= 64 ? 1 : L / 64; }

struct Unit {
  float v[kUnit];
};

template <typename T>
__device__ __forceinline__ Unit load_unit(const T* p) {
  Unit u;
  load8(p, u.v);
  return u;
}
template <typename T>
__device__ __forceinline__ void store_unit(T* p, const Unit& u) {
  store8(p, u.v);
}

// The values of a unit rounded to the type that stores them.
template <typename T>
__device__ __forceinline__ void round_unit(Unit& u) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) u.v[i] = bf16_to_f32(f32_to_bf16(u.v[i]));
  }
}

// Sum over the L threads that share a row, the same bits in every one of
// them: a butterfly in the wave, then the waves in order.  red: two sets of
// values taken in turn, so that one barrier per sum is enough (a wave writes a
// set again only behind the barrier of the sum in between).
template <int L>
__device__ __forceinline__ float row_sum(float x, float (&red)[2][waves_of<L>()], int& turn) {
  x = group_sum<(L < 64 ? L : 64)>(x);
  if constexpr (L > 64) {
    float(&r)[waves_of<L>()] = red[turn];
    turn ^= 1;
    if (lane_id() == 0) r[threadIdx.x >> 6] = x;
    __syncthreads();
    x = r[0];
#pragma unroll
    for (int w = 1; w < L / 64; ++w) x += r[w];
  }
  return x;
}

template <int L>
__device__ __forceinline__ double row_sum64(double x, double (&red)[waves_of<L>()]) {
#pragma unroll
  for (int off = (L < 64 ? L : 64) / 2; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  if constexpr (L > 64) {
    __syncthreads();
    if (lane_id() == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0];
    for (int w = 1; w < L / 64; ++w) x += red[w];
  }
  return x;
}

// The row's 1 / sqrt(mean + eps), rounded as fp32 operations.
__device__ __forceinline__ float rstd_of(float sum, int d, float eps) { return 1.0f / sqrtf(sum / (float)d + eps); }

// fp32 squares leave their range for elements beyond 1.8e19, and lose bits
// that count where eps is as small as they are: such rows are summed again in
// 64 bits.  (NaN and infinite rows stay what they are.)
__device__ __forceinline__ bool needs_64(float sum, float eps) {
  return sum > 1e37f || (sum < 1e-30f && eps < 1e-25f);
}
__device__ __forceinline__ float rstd_of64(double sum, int d, float eps) {
  return (float)(1.0 / sqrt(sum / (double)d + (double)eps));
}

// MX codes of a unit whose block (32 elements, four adjacent lanes) they
// share: the layer's codec (mok_mx.h), on the stored values of y.  A block
// with a value that is not finite becomes NaN as a whole.
__device__ __forceinline__ void store_mx(const Unit& y, uint8_t* codes, uint8_t* scales, size_t row, int d, int u) {
  int top = 0;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) top = max(top, (int)(__float_as_uint(y.v[i]) & 0x7FFFFFFFu));
  top = group_max<4>(top);
  const bool fine = top < 0x7F800000;
  const int sh = mx_shared_exp(__uint_as_float((uint32_t)top));
  uint2 w = make_uint2(e4m3_pack4(y.v[0], y.v[1], y.v[2], y.v[3], sh), e4m3_pack4(y.v[4], y.v[5], y.v[6], y.v[7], sh));
  if (!fine) w = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  *reinterpret_cast<uint2*>(codes + row * d + (size_t)u * kUnit) = w;
  if ((u & 3) == 0) scales[row * (size_t)(d / 32) + u / 4] = fine ? (uint8_t)(sh + 127) : 255;
}

struct NormArgs {
  const void* x;        // [T, d] or null
  const void* res;      // [T, d] or null (not both)
  const void* weight;   // [d]
  void* res_out;        // [T, d] or null
  void* y;              // [T, d] or null
  uint8_t* codes;       // [T, d] or null
  uint8_t* scales;
  float* rstd;          // [T] or null
  float eps;
  int T, d;
};

// r = round(res + x) of one unit.
template <typename TX, typename TR>
__device__ __forceinline__ Unit residual_unit(const NormArgs& a, size_t at) {
  Unit r;
  if (a.res) {
    r = load_unit(reinterpret_cast<const TR*>(a.res) + at);
    if (!a.x) return r;
    const Unit x = load_unit(reinterpret_cast<const TX*>(a.x) + at);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) r.v[i] += x.v[i];
  } else {
    r = load_unit(reinterpret_cast<const TX*>(a.x) + at);
  }
  round_unit<TR>(r);
  return r;
}

template <typename TX>
__device__ __forceinline__ void norm_out(const NormArgs& a, Unit y, const Unit& w, float rstd, size_t row, int u) {
#pragma unroll
  for (int i = 0; i < kUnit; ++i) y.v[i] = y.v[i] * rstd * w.v[i];
  round_unit<TX>(y);
  if (a.y) store_unit(reinterpret_cast<TX*>(a.y) + row * a.d + (size_t)u * kUnit, y);
  if (a.codes) store_mx(y, a.codes, a.scales, row, a.d, u);
}

// L threads per row, NV units per thread: d <= 8 L NV.
template <typename TX, typename TR, int L, int NV>
__global__ __launch_bounds__(block_of<L>()) void norm_fwd_kernel(NormArgs a) {
  __shared__ float red[2][waves_of<L>()];
  __shared__ double red64[waves_of<L>()];
  constexpr int RPW = block_of<L>() / L;     // rows of a workgroup at once
  const int me = threadIdx.x % L, units = a.d / kUnit;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / L; row < a.T; row += (int64_t)gridDim.x * RPW) {
    Unit r[NV];
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int u = me + q * L;
      if (u < units) r[q] = residual_unit<TX, TR>(a, (size_t)row * a.d + (size_t)u * kUnit);
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      if (me + q * L >= units) continue;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) s = __builtin_fmaf(r[q].v[i], r[q].v[i], s);
      sum += s;
    }
    sum = row_sum<L>(sum, red, turn);
    float rstd = rstd_of(sum, a.d, a.eps);
    if (needs_64(sum, a.eps)) {          // the same for all threads of a row
      double s64 = 0.0;
#pragma unroll
      for (int q = 0; q < NV; ++q)
        if (me + q * L < units)
          for (int i = 0; i < kUnit; ++i) s64 += (double)r[q].v[i] * (double)r[q].v[i];
      rstd = rstd_of64(row_sum64<L>(s64, red64), a.d, a.eps);
    }
    if (a.rstd && me == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int u = me + q * L;
      if (u >= units) continue;
      if (a.res_out) store_unit(reinterpret_cast<TR*>(a.res_out) + (size_t)row * a.d + (size_t)u * kUnit, r[q]);
      norm_out<TX>(a, r[q], load_unit(reinterpret_cast<const TX*>(a.weight) + (size_t)u * kUnit), rstd, (size_t)row, u);
    }
  }
}

// Rows of any length, read twice by a workgroup: the second time r comes from
// res_out, which may be res itself (a thread reads what it wrote).
template <typename TX, typename TR>
__global__ __launch_bounds__(kThreads) void norm_fwd_long_kernel(NormArgs a) {
  __shared__ double red64[kThreads / 64];
  const int units = a.d / kUnit;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    double sum = 0.0;
    for (int u = threadIdx.x; u < units; u += kThreads) {
      const size_t at = (size_t)row * a.d + (size_t)u * kUnit;
      const Unit r = residual_unit<TX, TR>(a, at);
      if (a.res_out) store_unit(reinterpret_cast<TR*>(a.res_out) + at, r);
      for (int i = 0; i < kUnit; ++i) sum += (double)r.v[i] * (double)r.v[i];
    }
    const float rstd = rstd_of64(row_sum64<kThreads>(sum, red64), a.d, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    for (int u = threadIdx.x; u < units; u += kThreads) {
      const size_t at = (size_t)row * a.d + (size_t)u * kUnit;
      const Unit r = a.res_out ? load_unit(reinterpret_cast<const TR*>(a.res_out) + at) : residual_unit<TX, TR>(a, at);
      norm_out<TX>(a, r, load_unit(reinterpret_cast<const TX*>(a.weight) + (size_t)u * kUnit), rstd, (size_t)row, u);
    }
  }
}

// ------------------------------------------------------------------ backward
struct NormBwdArgs {
  const void* dy;       // [T, d]
  const void* res;      // [T, d] the forward's r
  const void* weight;   // [d]
  const float* rstd;    // [T]
  const void* d_res;    // [T, d] or null
  void* d_r;            // [T, d] or null
  void* d_x;            // [T, d] or null (the same gradient in the layer's type)
  void* part;           // [workgroups, d] sums of dy n, fp32 or 64 bits, or null
  bool narrow;          // fp32: no workgroup has more rows than a thread adds in fp32
  float* dw;            // [d]
  int add;
  int T, d;
};

// Rows that a thread adds in fp32 before the sum joins the workgroup's 64-bit
// one: the error of d_w does not grow with the number of rows.
constexpr int kFlushRows = 64;

// Workgroups of the backward (a constant, so that d_w is the same on every
// device): two per compute unit hold the loads of two rows in flight.
constexpr int kBwdGroups = 512;

template <typename TX, typename TR>
__device__ __forceinline__ void norm_bwd_out(const NormBwdArgs& a, const Unit& g, const Unit& n, const Unit& up, float mean,
                                             float rstd, size_t at) {
  Unit o;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) o.v[i] = rstd * __builtin_fmaf(-n.v[i], mean, g.v[i]);
  if (a.d_res) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) o.v[i] += up.v[i];
  }
  if (a.d_r) store_unit(reinterpret_cast<TR*>(a.d_r) + at, o);
  if (a.d_x) store_unit(reinterpret_cast<TX*>(a.d_x) + at, o);
}

// The rows of workgroup `block` of `blocks`.  DW: with the workgroup's sums of
// dy n, in its row of a.part.
template <typename TX, typename TR, int L, int NV, bool DW>
__device__ __forceinline__ void norm_bwd_rows(const NormBwdArgs& a, int block, int blocks) {
  constexpr int BLOCK = block_of<L>(), RPW = BLOCK / L;
  __shared__ float red[2][waves_of<L>()];
  __shared__ float s_dw[L <= 64 && DW ? RPW * L * NV * kUnit : 1];
  const int me = threadIdx.x % L, units = a.d / kUnit;
  int turn = 0, held = 0;
  bool first = true;
  Unit acc[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q)
#pragma unroll
    for (int i = 0; i < kUnit; ++i) acc[q].v[i] = 0.0f;
  // the workgroup's rows: a part's turn may be past the last row while the
  // others still work, so every wave runs the same number of turns
  const int64_t step = (int64_t)blocks * RPW;
  const int64_t turns = (a.T - (int64_t)block * RPW + step - 1) / step;
  auto flush = [&]() {
    if (!a.part) return;
    double* part = reinterpret_cast<double*>(a.part) + (size_t)block * a.d;
    if constexpr (L <= 64) {
      const int mine = threadIdx.x / L;
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) s_dw[(mine * L * NV + q * L + me) * kUnit + i] = acc[q].v[i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.d; c += BLOCK) {
        double s = first ? 0.0 : part[c];
        for (int w = 0; w < RPW; ++w) s += (double)s_dw[w * L * NV * kUnit + c];
        part[c] = s;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int u = me + q * L;
        if (u >= units) continue;
        if (a.narrow) {
          store_unit(reinterpret_cast<float*>(a.part) + (size_t)block * a.d + (size_t)u * kUnit, acc[q]);
          continue;
        }
        double* p = part + (size_t)u * kUnit;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) p[i] = (first ? 0.0 : p[i]) + (double)acc[q].v[i];
      }
    }
    first = false;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) acc[q].v[i] = 0.0f;
  };
  for (int64_t it = 0; it < turns; ++it) {
    const int64_t row = (int64_t)block * RPW + threadIdx.x / L + it * step;
    const bool live = row < a.T;
    if (live) {
      const float rstd = a.rstd[row];
      Unit g[NV], n[NV], up[NV];
      float sum = 0.0f;
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int u = me + q * L;
        if (u >= units) continue;
        const size_t at = (size_t)row * a.d + (size_t)u * kUnit;
        g[q] = load_unit(reinterpret_cast<const TX*>(a.dy) + at);
        n[q] = load_unit(reinterpret_cast<const TR*>(a.res) + at);
        if (a.d_res) up[q] = load_unit(reinterpret_cast<const TR*>(a.d_res) + at);
      }
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int u = me + q * L;
        if (u >= units) continue;
        const Unit w = load_unit(reinterpret_cast<const TX*>(a.weight) + (size_t)u * kUnit);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          n[q].v[i] *= rstd;
          if constexpr (DW) acc[q].v[i] = __builtin_fmaf(g[q].v[i], n[q].v[i], acc[q].v[i]);
          g[q].v[i] *= w.v[i];
          s = __builtin_fmaf(g[q].v[i], n[q].v[i], s);
        }
        sum += s;
      }
      const float mean = row_sum<L>(sum, red, turn) / (float)a.d;
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int u = me + q * L;
        if (u < units) norm_bwd_out<TX, TR>(a, g[q], n[q], up[q], mean, rstd, (size_t)row * a.d + (size_t)u * kUnit);
      }
    }
    if constexpr (DW)
      if (++held == kFlushRows) {
        flush();
        held = 0;
      }
  }
  if constexpr (DW)
    if (held || first) flush();
}

template <typename TX, typename TR, int L, int NV>
__global__ __launch_bounds__(block_of<L>()) void norm_bwd_kernel(NormBwdArgs a) {
  norm_bwd_rows<TX, TR, L, NV, true>(a, blockIdx.x, gridDim.x);
}

// The columns of d_w that a workgroup of few_columns() takes, all rows: eight
// columns a thread, its rows (16 of them at most, for kFewRows) in fp32, then
// threads and waves in 64 bits in order.  64 rows are under way at once (1024 x
// 2048, bf16: 8.2 us with 32 columns of 256 threads, 12.1 with 64, 10.3 with 16;
// 1024 x 7168: 13.3 with 64 columns of 512 threads, 18.3 with 32).
constexpr int kFewRows = 1024;
constexpr int few_columns(int block) { return block / kUnit; }

template <typename TX, typename TR, int BLOCK>
__device__ __forceinline__ void norm_dw_columns(const NormBwdArgs& a, int tile) {
  constexpr int COLUMNS = few_columns(BLOCK), WIDE = COLUMNS / kUnit, STEP = BLOCK / WIDE;
  __shared__ double s[BLOCK / 64][COLUMNS];
  const int u = threadIdx.x % WIDE, c = tile * COLUMNS + u * kUnit;
  Unit acc;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) acc.v[i] = 0.0f;
#pragma unroll 4
  for (int row = threadIdx.x / WIDE; row < a.T; row += STEP) {
    const Unit g = load_unit(reinterpret_cast<const TX*>(a.dy) + (size_t)row * a.d + c);
    const Unit r = load_unit(reinterpret_cast<const TR*>(a.res) + (size_t)row * a.d + c);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) acc.v[i] = __builtin_fmaf(g.v[i], r.v[i] * rstd, acc.v[i]);
  }
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    double v = acc.v[i];
#pragma unroll
    for (int off = WIDE; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
    if (lane_id() < WIDE) s[threadIdx.x >> 6][u * kUnit + i] = v;
  }
  __syncthreads();
  if (threadIdx.x >= COLUMNS) return;
  double v = s[0][threadIdx.x];
  for (int w = 1; w < BLOCK / 64; ++w) v += s[w][threadIdx.x];
  float* dw = a.dw + tile * COLUMNS + threadIdx.x;
  *dw = (float)(a.add ? (double)*dw + v : v);
}

// Few rows: d_w needs no row's sum, so its columns are summed in the same
// launch by workgroups of their own, which read dy and r a second time (us a
// call, in two launches and in one: 512 x 256 8.6 and 6.0; 1024 x 1024 8.5 and
// 6.0; 1024 x 7168 19.5 and 13.3; 2000 x 2048 11 and 26).
template <typename TX, typename TR, int L, int NV>
__global__ __launch_bounds__(block_of<L>()) void norm_bwd_few_kernel(NormBwdArgs a) {
  const int tiles = a.dw ? a.d / few_columns(block_of<L>()) : 0;
  if ((int)blockIdx.x < tiles) norm_dw_columns<TX, TR, block_of<L>()>(a, blockIdx.x);
  else if (a.d_r || a.d_x) norm_bwd_rows<TX, TR, L, NV, false>(a, blockIdx.x - tiles, gridDim.x - tiles);
}

// Rows of any length: dy n goes to the workgroup's 64-bit sums row by row.
template <typename TX, typename TR>
__global__ __launch_bounds__(kThreads) void norm_bwd_long_kernel(NormBwdArgs a) {
  __shared__ double red64[kThreads / 64];
  const int units = a.d / kUnit;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float rstd = a.rstd[row];
    double sum = 0.0;
    auto fetch = [&](int u, Unit& g, Unit& n) {
      const size_t at = (size_t)row * a.d + (size_t)u * kUnit;
      g = load_unit(reinterpret_cast<const TX*>(a.dy) + at);
      n = load_unit(reinterpret_cast<const TR*>(a.res) + at);
      for (int i = 0; i < kUnit; ++i) n.v[i] *= rstd;
    };
    for (int u = threadIdx.x; u < units; u += kThreads) {
      Unit g, n;
      fetch(u, g, n);
      const Unit w = load_unit(reinterpret_cast<const TX*>(a.weight) + (size_t)u * kUnit);
      double* p = a.part ? reinterpret_cast<double*>(a.part) + (size_t)blockIdx.x * a.d + (size_t)u * kUnit : nullptr;
      for (int i = 0; i < kUnit; ++i) {
        if (p) p[i] = (first ? 0.0 : p[i]) + (double)g.v[i] * (double)n.v[i];
        sum += (double)(g.v[i] * w.v[i]) * (double)n.v[i];
      }
    }
    const float mean = (float)(row_sum64<kThreads>(sum, red64) / (double)a.d);
    for (int u = threadIdx.x; u < units; u += kThreads) {
      Unit g, n;
      fetch(u, g, n);
      const Unit w = load_unit(reinterpret_cast<const TX*>(a.weight) + (size_t)u * kUnit);
      for (int i = 0; i < kUnit; ++i) g.v[i] *= w.v[i];
      const size_t at = (size_t)row * a.d + (size_t)u * kUnit;
      Unit up;
      if (a.d_res) up = load_unit(reinterpret_cast<const TR*>(a.d_res) + at);
      norm_bwd_out<TX, TR>(a, g, n, up, mean, rstd, at);
    }
    first = false;
  }
}

// d_w: the workgroups' sums, kDwColumns columns per workgroup (a cache line of
// each sum), 64 threads a column, each with every 64th sum, joined in order.
constexpr int kDwThreads = 1024, kDwColumns = 16;

template <typename T>
__global__ __launch_bounds__(kDwThreads) void norm_dw_kernel(const T* part, int groups, float* dw, int d, int add) {
  __shared__ double s[kDwThreads / 64][kDwColumns];
  const int at = threadIdx.x % kDwColumns, c = blockIdx.x * kDwColumns + at;   // d % 64 == 0
  double v = 0.0;
#pragma unroll 8
  for (int g = threadIdx.x / kDwColumns; g < groups; g += kDwThreads / kDwColumns) v += (double)part[(size_t)g * d + c];
#pragma unroll
  for (int off = kDwColumns; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
  if (lane_id() < kDwColumns) s[threadIdx.x >> 6][at] = v;
  __syncthreads();
  if (threadIdx.x >= kDwColumns) return;
  for (int u = 1; u < kDwThreads / 64; ++u) v += s[u][at];
  dw[c] = (float)(add ? (double)dw[c] + v : v);
}

// Rows that a workgroup of the kernel for d works on at once.  Rows of up to
// 1024 elements take a wave or a part of one (65536 x 1024, bf16: backward 96
// us, with a workgroup a row 163; 16384 x 2048 forward 68 us with a wave a row,
// 59 with a workgroup), unless there are so few of them that a workgroup a row
// spreads over more of the chip.
int rows_at_once(int T, int d) {
  if (d <= 128) return kThreads / 16;
  if (d <= 256) return kThreads / 32;
  return d <= 512 || (d <= 1024 && T >= 1024) ? kThreads / 64 : 1;
}

// The kernel for rows of d elements: L threads a row with NV units each.
#define MOK_NORM_PICK(KERNEL, LONG, TX, TR)                                        \
  do {                                                                             \
    const int u = d / kUnit, rows = rows_at_once(T, d);                            \
    if (u <= 16) launch(KERNEL<TX, TR, 16, 1>, kThreads, rows);                    \
    else if (u <= 32) launch(KERNEL<TX, TR, 32, 1>, kThreads, rows);               \
    else if (u <= 64) launch(KERNEL<TX, TR, 64, 1>, kThreads, rows);               \
    else if (rows > 1) launch(KERNEL<TX, TR, 64, 2>, kThreads, rows);              \
    else if (u <= 256) launch(KERNEL<TX, TR, 256, 1>, 256, rows);                  \
    else if (u <= 1024) launch(KERNEL<TX, TR, 512, 2>, 512, rows);                 \
    else if (u <= 2048) launch(KERNEL<TX, TR, 512, 4>, 512, rows);                 \
    else launch(LONG<TX, TR>, kThreads, rows);                                     \
  } while (0)

int bwd_groups(int T, int d) {
  const int rows = rows_at_once(T, d);
  const int64_t need = ((int64_t)T + rows - 1) / rows;
  return (int)(need < kBwdGroups ? need : kBwdGroups);
}

// Up to kFewRows rows of a length that a thread holds in registers: one launch.
bool few_rows(int T, int d) { return T > 0 && T <= kFewRows && d <= 2048 * kUnit; }

}  // namespace

size_t norm_bwd_ws_bytes(int T, int d) { return (size_t)(T > 0 ? bwd_groups(T, d) : 1) * d * sizeof(double); }

mok_status launch_norm_fwd(int prec, int res_type, int T, int d, const void* x, const void* res, const void* weight,
                           float eps, void* res_out, void* y, uint8_t* codes, uint8_t* scales, float* rstd,
                           hipStream_t stream, mok_trace* tr) {
  if (T == 0) return MOK_OK;
  const NormArgs a = {x, res, weight, res_out, y, codes, scales, rstd, eps, T, d};
  auto launch = [&](void (*kernel)(NormArgs), int threads, int rows) {
    const int64_t need = ((int64_t)T + rows - 1) / rows;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(need < 4096 ? need : 4096)), dim3(threads), 0, stream, a);
  };
  if (prec == MOK_F32) MOK_NORM_PICK(norm_fwd_kernel, norm_fwd_long_kernel, float, float);
  else if (res_type == MOK_F32) MOK_NORM_PICK(norm_fwd_kernel, norm_fwd_long_kernel, bf16_t, float);
  else MOK_NORM_PICK(norm_fwd_kernel, norm_fwd_long_kernel, bf16_t, bf16_t);
  trace_mark(tr, "norm_fwd", stream);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

mok_status launch_norm_bwd(int prec, int res_type, int T, int d, const void* dy, const void* res, const void* weight,
                           const float* rstd, const void* d_res, void* d_r, void* d_x, float* dw, bool add, void* ws,
                           hipStream_t stream, mok_trace* tr) {
  const int groups = T > 0 ? bwd_groups(T, d) : 0;
  const bool narrow = rows_at_once(T, d) == 1 && d <= 2048 * kUnit && T <= (int64_t)groups * kFlushRows;
  const NormBwdArgs a = {dy, res, weight, rstd, d_res, d_r, d_x, dw ? ws : nullptr, narrow, dw, add ? 1 : 0, T, d};
  if (few_rows(T, d)) {
    auto launch = [&](void (*kernel)(NormBwdArgs), int threads, int rows) {
      const int64_t more = (dw ? d / few_columns(threads) : 0) + (d_r || d_x ? ((int64_t)T + rows - 1) / rows : 0);
      hipLaunchKernelGGL(kernel, dim3((unsigned)more), dim3(threads), 0, stream, a);
    };
    if (prec == MOK_F32) MOK_NORM_PICK(norm_bwd_few_kernel, norm_bwd_long_kernel, float, float);
    else if (res_type == MOK_F32) MOK_NORM_PICK(norm_bwd_few_kernel, norm_bwd_long_kernel, bf16_t, float);
    else MOK_NORM_PICK(norm_bwd_few_kernel, norm_bwd_long_kernel, bf16_t, bf16_t);
    trace_mark(tr, "norm_bwd", stream);
    return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
  }
  if (T > 0) {
    auto launch = [&](void (*kernel)(NormBwdArgs), int threads, int) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(threads), 0, stream, a);
    };
    if (prec == MOK_F32) MOK_NORM_PICK(norm_bwd_kernel, norm_bwd_long_kernel, float, float);
    else if (res_type == MOK_F32) MOK_NORM_PICK(norm_bwd_kernel, norm_bwd_long_kernel, bf16_t, float);
    else MOK_NORM_PICK(norm_bwd_kernel, norm_bwd_long_kernel, bf16_t, bf16_t);
    trace_mark(tr, "norm_bwd", stream);
  }
  if (dw && (T > 0 || !add)) {
    const dim3 grid((unsigned)(d / kDwColumns));
    if (a.narrow) hipLaunchKernelGGL(norm_dw_kernel<float>, grid, dim3(kDwThreads), 0, stream, (const float*)ws, groups, dw, d, a.add);
    else hipLaunchKernelGGL(norm_dw_kernel<double>, grid, dim3(kDwThreads), 0, stream, (const double*)ws, groups, dw, d, a.add);
    trace_mark(tr, "norm_dw", stream);
  }
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

}  // namespace mok
