// Balance loss, z-loss and per-expert counts of the router, and the gradient
// with respect to its logits.
//
// Mathematics (per group g of N_g counted rows, p = softmax(z), c = counts):
//   L_balance = alpha / G+ sum_g E / (k N_g^2) sum_e c_ge (sum_t p_te)
//   L_z       = beta / N sum_t lse_t^2
//   dz_te     = p_te ((w_ge - sum_i p_ti w_gi) + 2 beta d1 lse_t / N),
//               w_ge = alpha d0 E / (k N_g^2 G+) (c_ge - k N_g / E).
// A constant subtracted from all w of a group drops out of the gradient
// (p sums to one); with the mean count taken off, nearly balanced counts do
// not leave a small difference of large numbers.
//
// Forward: a workgroup takes a chunk of consecutive rows, whatever groups they
// belong to, so ragged groups load the chip evenly (a fixed number of slices
// per group took 60 us where chunks took 35 on 131072 x 256 in 32 random groups).  A
// row is held by LPR lanes (NV logits each, 16-byte loads where E and the
// alignment allow), so a wave takes 64 / LPR rows at a time, U times over,
// with the next rows' loads issued before this step's arithmetic, and each
// lane keeps the column sums of its own NV experts over the rows of a group;
// counts are integer LDS atomics (their order cannot change the result).
// For every group that a chunk meets, the column sums, counts, row count and
// sum of lse^2 go to a slot of the workspace: chunk + group, which no two
// (chunk, group) pairs that meet share, because both only ascend.  A second
// kernel adds each group's slots in order in 64 bits, and its last workgroup
// the groups.  A call of one group and chunk ends in the first kernel.
// Backward: the same chunks and row layout, one pass, the row's softmax
// formed again from registers.
//
// Bound by HBM when large: 131072 x 256, k = 8 in 32 groups, forward 30 us
// (138 MB of logits and ids, 4.6 TB/s: the counts' LDS atomics and the row
// reductions are not hidden entirely), finishing kernel 7, backward 46 (134 MB
// read and as much written, 5.8 TB/s; part of the logits comes from the
// memory-side cache); in one group the finishing kernel has E / 64 workgroups
// for all chunks and takes 12.  Bound by latency when small: 16384 x 64 takes
// 8 + 7 + 7 us, 512 x 8 6 + 4.
#include "mok_internal.h"
#include "mok_lanes.h"

namespace mok {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / 64;
constexpr int kBalWgs = 1024;   // chunks at most: four workgroups per CU
constexpr int kMaxE = 512;
constexpr int kFold = 16;       // steps of a lane's fp32 sums
constexpr int kFinCols = 64;    // experts per workgroup of the finishing kernel
constexpr int kFinThreads = 512;

struct BalArgs {
  const float* z;
  const int32_t* topk;
  const uint8_t* mask;
  const int32_t* off;    // [G+1] or null: one group of T rows
  int T, E, k, G;
  int chunks, rows;      // chunks of `rows` rows
  int32_t* status;
  // workspace of the forward; slots = chunks + G
  float* part;           // [slots][E] column sums
  int32_t* cnt;          // [slots][E]
  double* zz;            // [slots]
  int32_t* nrow;         // [slots]
  int32_t* ticket;       // [0] workgroups of the finishing kernel that are done, [1] the offsets are good
  double* lossp;         // [G * ceil(E / kFinCols)]
  double* zzp;           // [G]
  // outputs and the backward's inputs
  int32_t* counts;
  float* prob;
  int32_t* n_tok;
  float* loss;
  const float* d_loss;
  float* dz;
  int stream;            // gradients past the caches
  float alpha, beta;
};

// Sum of every thread's x over the workgroup, in a fixed order; every thread
// gets it.
template <class T, int THREADS>
__device__ __forceinline__ T block_sum(T x) {
  __shared__ T s_w[THREADS / 64];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) x += s_w[i];
  return x;
}
// Sum of value(i) for i in [0, n).
template <class T, int THREADS, class F>
__device__ __forceinline__ T block_sum(int n, F value) {
  T x = 0;
  for (int i = threadIdx.x; i < n; i += THREADS) x += value(i);
  return block_sum<T, THREADS>(x);
}

__device__ __forceinline__ int group_begin(const BalArgs& a, int g) { return a.off ? a.off[g] : g == 0 ? 0 : a.T; }

// The first group that ends behind `row`, or -1 (MOK_EGROUP latched) if the
// offsets do not ascend within [0, T].  Every wave reads them all, so every
// one comes to the same answer without a barrier.
__device__ __forceinline__ int first_group(const BalArgs& a, int row) {
  if (!a.off) return 0;
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    const int g = g0 + lane;
    const bool in = g < a.G;
    const int b = in ? a.off[g] : 0, e = in ? a.off[g + 1] : 0;
    if (__any(in && (b < 0 || e < b || e > a.T))) {
      if (lane == 0) latch(a.status, MOK_EGROUP);
      return -1;
    }
    before += (int)__popcll(__ballot(in && e <= row));
  }
  return before;
}

// The row layout: lane l of LPR holds experts 4 (l + LPR u) + 0..3 (VEC) or
// l + LPR i.  expert(i) is the expert of value i of this lane.
template <int LPR, int NV, bool VEC>
struct RowLayout {
  static constexpr int kRows = 64 / LPR;  // rows of a wave at a time
  __device__ __forceinline__ static int expert(int l, int i) {
    return VEC ? 4 * (l + LPR * (i >> 2)) + (i & 3) : l + LPR * i;
  }
  // logits of U rows; -inf past E
  template <int U>
  __device__ __forceinline__ static void load(const float* const (&row)[U], int l, int E, float (&v)[U][NV]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[u][i] = -__builtin_inff();
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < NV / 4; ++i) {
        const int e = 4 * (l + LPR * i);
        if (e < E) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float4 q = *reinterpret_cast<const float4*>(row[u] + e);
            v[u][4 * i] = q.x, v[u][4 * i + 1] = q.y, v[u][4 * i + 2] = q.z, v[u][4 * i + 3] = q.w;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = l + LPR * i;
        if (e < E) {
#pragma unroll
          for (int u = 0; u < U; ++u) v[u][i] = row[u][e];
        }
      }
    }
  }
  template <bool STREAM>
  __device__ __forceinline__ static void store(float* row, int l, int E, const float (&v)[NV]) {
    if constexpr (VEC) {
#pragma unroll
      for (int u = 0; u < NV / 4; ++u) {
        const int e = 4 * (l + LPR * u);
        const f32x4_t q = {v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]};
        if (e >= E) continue;
        if constexpr (STREAM) __builtin_nontemporal_store(q, reinterpret_cast<f32x4_t*>(row + e));
        else *reinterpret_cast<f32x4_t*>(row + e) = q;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = l + LPR * i;
        if (e < E) row[e] = v[i];
      }
    }
  }
};

// Rows of a lane at once, so their loads are in flight together.
constexpr int kRowsAtOnce = 2;
// Chosen slots of a row per lane (k <= 16 and k <= E).
template <int LPR, bool VEC>
constexpr int slots_per_lane() {
  return !VEC || LPR >= 16 ? 1 : LPR == 8 ? 2 : 4;
}

// U rows of a wave on their way: logits, mask bytes and whether each row is
// one of the slice (a row past its end reads the last row instead).
template <int LPR, int NV, bool VEC>
struct Rows {
  static constexpr int U = kRowsAtOnce;
  float v[U][NV];
  uint32_t mask[U];
  bool in[U];
  __device__ __forceinline__ void load(const BalArgs& a, int r0, int hi, int l, int sub) {
    const float* row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * (64 / LPR) + sub;
      in[u] = r < hi;
      row[u] = a.z + (size_t)min(r, hi - 1) * a.E;
      mask[u] = 1;
    }
    RowLayout<LPR, NV, VEC>::load(row, l, a.E, v);
    if (a.mask) {
#pragma unroll
      for (int u = 0; u < U; ++u) mask[u] = a.mask[min(r0 + u * (64 / LPR) + sub, hi - 1)];
    }
  }
};

// Softmax of U rows in place (v becomes p) and their log-sum-exp.  live: the
// row counts (in the slice, not masked, not all -inf); v and lse are zero
// where not.  A NaN among the logits of a live row reaches p and lse.
// p = 2^(z log2 e - c) / sum with c = max log2 e: c's rounding is the same
// factor in every term and in lse = (c + log2 sum) ln 2, so only the product
// with z rounds (one fused operation); exponential, logarithm and reciprocal
// are the hardware's (1 ulp).  Rows that do not count are rare enough to be
// dealt with in a branch, and so are rows whose c is so large (all logits at a
// mask's -1e9, or at the type's lowest value) that its rounding, or c itself,
// would leave the exponent's range: those subtract the maximum first.
// Returns whether there was one in the wave.
template <int LPR, int NV, int U>
__device__ __forceinline__ bool softmax_rows(float (&v)[U][NV], const uint32_t (&mask)[U], const bool (&in)[U],
                                             int lane, bool (&live)[U], float (&lse)[U]) {
  constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kLarge = 0x1p24f;
  float m[U], c[U], off[U];
  bool rare = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    int mx = float_order(v[u][0]);
#pragma unroll
    for (int i = 1; i < NV; ++i) mx = max(mx, float_order(v[u][i]));
    m[u] = order_float(group_max<LPR>(mx));
    c[u] = m[u] * kLog2e;
    off[u] = 0.0f;
    live[u] = true;
    rare = rare || !in[u] || mask[u] == 0 || !(__builtin_fabsf(c[u]) < kLarge);
  }
  rare = __any(rare);
  if (rare) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // all -inf, or -inf and negative NaN only: look for one
      bool some = m[u] != -__builtin_inff();
#pragma unroll
      for (int i = 0; i < NV; ++i) some = some || __builtin_isnan(v[u][i]);
      const uint64_t vote = __ballot(some);
      const uint64_t grp = LPR == 64 ? ~0ull : ((1ull << (LPR & 63)) - 1) << (lane & ~(LPR - 1));
      live[u] = in[u] && mask[u] != 0 && (vote & grp) != 0;
      if (!live[u]) {
        c[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) v[u][i] = -__builtin_inff();
      } else if (__builtin_fabsf(c[u]) >= kLarge && __builtin_fabsf(m[u]) < __builtin_inff()) {
        c[u] = 0.0f;
        off[u] = m[u];
#pragma unroll
        for (int i = 0; i < NV; ++i) v[u][i] -= m[u];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[u][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[u][i], kLog2e, -c[u]));
      sum += v[u][i];
    }
    sum = group_sum<LPR>(sum);
    const float inv = live[u] ? __builtin_amdgcn_rcpf(sum) : 0.0f;
    lse[u] = live[u] ? __builtin_fmaf(c[u] + __builtin_amdgcn_logf(sum), kLn2, off[u]) : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[u][i] *= inv;
  }
  return rare;
}

// n_tok[G], n_tok[G+1] and the losses from the groups' terms.
__device__ __forceinline__ void write_totals(const BalArgs& a, int N, int groups, double bal, double zz) {
  a.n_tok[a.G] = N;
  a.n_tok[a.G + 1] = groups;
  a.loss[0] = groups > 0 ? (float)(a.alpha * bal / groups) : 0.0f;
  a.loss[1] = N > 0 && a.beta != 0.0f ? (float)(a.beta * zz / N) : 0.0f;   // lse^2 may be infinite
}
__device__ __forceinline__ double group_term(const BalArgs& a, int n, double cp) {
  return n > 0 ? cp * a.E / ((double)a.k * n * n) : 0.0;
}

template <int LPR, int NV, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_fwd_kernel(BalArgs a) {
  typedef RowLayout<LPR, NV, VEC> RL;
  constexpr int U = kRowsAtOnce, KJ = slots_per_lane<LPR, VEC>();
  __shared__ float s_sum[kBalWaves][kMaxE];
  __shared__ int s_cnt[kMaxE];
  __shared__ double s_zz[kBalWaves];
  __shared__ double s_fold[NV][kBalThreads];
  __shared__ int s_n[kBalWaves];
  const int chunk = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane & (LPR - 1), sub = lane / LPR;
  const int c_lo = chunk * a.rows, c_hi = min(a.T, c_lo + a.rows);
  const int step = kBalWaves * RL::kRows * U;
  const int g0 = first_group(a, c_lo);
  if (chunk == 0 && tid == 0) {  // for the kernel that follows
    a.ticket[0] = 0;
    a.ticket[1] = g0 >= 0;
  }
  bool bad = false;
  auto load = [&](int r0, int hi, Rows<LPR, NV, VEC>& rows, int (&ids)[U][KJ]) {
#pragma unroll
    for (int q = 0; q < KJ; ++q) {
      const int j = l + LPR * q;
#pragma unroll
      for (int u = 0; u < U; ++u) ids[u][q] = 0;
      if (j < a.k) {
#pragma unroll
        for (int u = 0; u < U; ++u) ids[u][q] = a.topk[(size_t)min(r0 + u * RL::kRows + sub, hi - 1) * a.k + j];
      }
    }
    rows.load(a, r0, hi, l, sub);
  };
  // (a lone chunk and group also writes its zeros when nothing counts)
  const bool lone = gridDim.x == 1 && a.G == 1;
  for (int g = lone ? 0 : g0; g < a.G && (g0 >= 0 || lone); ++g) {
    const int g_lo = g0 < 0 ? 0 : group_begin(a, g), g_hi = g0 < 0 ? 0 : group_begin(a, g + 1);
    if (g_lo >= c_hi && !lone) break;
    const int lo = max(g_lo, c_lo), hi = min(g_hi, c_hi);
    if (lo >= hi && !lone) continue;
    for (int e = tid; e < a.E; e += kBalThreads) s_cnt[e] = 0;
    __syncthreads();
    // a lane adds kFold steps' probabilities in fp32, and those sums in 64
    // bits, so that the error does not grow with the chunk (in LDS: as
    // registers they cost 8 % of 131072 x 256, where no chunk is that long);
    // squares of lse would overflow in fp32 where their mean does not
    float acc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
    double zz = 0.0;
    int n = 0, steps = 0;
    Rows<LPR, NV, VEC> now, next;
    int id[U][KJ], id_next[U][KJ];
    int r0 = lo + wave * RL::kRows * U;
    if (r0 < hi) load(r0, hi, now, id);
    while (r0 < hi) {
      // the next rows' loads go out before this step's arithmetic
      const bool more = hi - r0 > step;
      if (more) load(r0 + step, hi, next, id_next);
      bool live[U];
      float lse[U];
      softmax_rows<LPR, NV, U>(now.v, now.mask, now.in, lane, live, lse);
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += now.v[u][i];
        zz = __builtin_fma((double)lse[u], (double)lse[u], zz);   // every lane of the row: lane 0's is used
        n += live[u];
      }
#pragma unroll
      for (int q = 0; q < KJ; ++q)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool slot = live[u] && l + LPR * q < a.k;
          const bool known = (uint32_t)id[u][q] < (uint32_t)a.E;
          if (slot && known) atomicAdd(&s_cnt[id[u][q]], 1);
          bad = bad || (slot && !known);
        }
      if (!more) break;
      if (++steps % kFold == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          s_fold[i][tid] = (steps > kFold ? s_fold[i][tid] : 0.0) + (double)acc[i];
          acc[i] = 0.0f;
        }
      }
      r0 += step;
      now = next;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < KJ; ++q) id[u][q] = id_next[u][q];
    }
    // the wave's row groups, then the four waves
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (steps >= kFold) acc[i] = (float)(s_fold[i][tid] + (double)acc[i]);
#pragma unroll
      for (int o = LPR; o < 64; o <<= 1) acc[i] += __shfl_xor(acc[i], o, 64);
      const int e = RL::expert(l, i);
      if (sub == 0 && e < a.E) s_sum[wave][e] = acc[i];
    }
#pragma unroll
    for (int o = LPR; o < 64; o <<= 1) {
      zz += __shfl_xor(zz, o, 64);
      n += __shfl_xor(n, o, 64);
    }
    if (lane == 0) {
      s_zz[wave] = zz;
      s_n[wave] = n;
    }
    __syncthreads();
    const int rows = s_n[0] + s_n[1] + s_n[2] + s_n[3];
    const double zsum = (s_zz[0] + s_zz[1]) + (s_zz[2] + s_zz[3]);
    auto column = [&](int e) { return (s_sum[0][e] + s_sum[1][e]) + (s_sum[2][e] + s_sum[3][e]); };
    if (lone) {  // nothing is left to add up
      const double cp = block_sum<double, kBalThreads>(a.E, [&](int e) {
        const double p = column(e);
        a.counts[e] = s_cnt[e];
        a.prob[e] = rows > 0 ? (float)(p / rows) : 0.0f;
        return p * s_cnt[e];
      });
      if (tid == 0) {
        a.n_tok[0] = rows;
        write_totals(a, rows, rows > 0, group_term(a, rows, cp), zsum);
      }
      break;
    }
    const size_t slot = (size_t)chunk + g;
    for (int e = tid; e < a.E; e += kBalThreads) {
      a.part[slot * a.E + e] = column(e);
      a.cnt[slot * a.E + e] = s_cnt[e];
    }
    if (tid == 0) {
      a.zz[slot] = zsum;
      a.nrow[slot] = rows;
    }
    __syncthreads();   // the sums are read before the next group's begin
  }
  if (bad) latch(a.status, MOK_EROUTE);
}

// Slots of one group, kFinCols experts: thread (c, q) adds slots q, q + Q,
// ... of experts 4 c .. 4 c + 3; the Q partial sums meet in LDS in order.
// The workgroup that finishes last (a ticket per workgroup) adds the groups.
// What it reads of the others -- terms and row counts -- is written and read
// with device-scope atomics, which pass by the XCDs' separate L2s, and every
// write has completed (vmcnt 0) before its workgroup takes a ticket; a fence
// would write back the whole L2 once per workgroup (17 us against 6 us for
// 512 workgroups).
__global__ __launch_bounds__(kFinThreads) void balance_finish_kernel(BalArgs a) {
  constexpr int C = kFinCols / 4, Q = kFinThreads / C, W = kFinThreads / 64;
  static_assert(kFinCols == 64, "an expert per lane of wave 0");
  __shared__ double s_p[Q][kFinCols + 1];
  __shared__ int s_c[Q][kFinCols + 1];
  __shared__ double s_a[W], s_b[W];
  __shared__ int s_n[W], s_m[W];
  __shared__ int s_last;
  const int g = blockIdx.x, c = threadIdx.x % C, q = threadIdx.x / C;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = blockIdx.y * kFinCols;
  // the chunks that meet the group; none if it is empty or the offsets are bad
  const int g_lo = group_begin(a, g), g_hi = group_begin(a, g + 1);
  const bool some = a.ticket[1] && g_hi > g_lo;
  const int first = some ? g_lo / a.rows : 0, slots = some ? (g_hi - 1) / a.rows - first + 1 : 0;
  const size_t s0 = (size_t)first + g;
  double p[4] = {0.0, 0.0, 0.0, 0.0}, zz = 0.0;
  int cn[4] = {0, 0, 0, 0}, n = 0;
  for (int i = threadIdx.x; i < slots; i += kFinThreads) {
    n += a.nrow[s0 + i];
    zz += a.zz[s0 + i];
  }
  const int ec = e0 + 4 * c;
  if (a.E % 4 == 0) {
#pragma unroll 4
    for (int s = ec < a.E ? q : slots; s < slots; s += Q) {
      const size_t i = (s0 + s) * a.E + ec;
      const float4 x = *reinterpret_cast<const float4*>(a.part + i);
      const int4 y = *reinterpret_cast<const int4*>(a.cnt + i);
      p[0] += (double)x.x, p[1] += (double)x.y, p[2] += (double)x.z, p[3] += (double)x.w;
      cn[0] += y.x, cn[1] += y.y, cn[2] += y.z, cn[3] += y.w;
    }
  } else {
    for (int s = q; s < slots; s += Q) {
      const size_t i = (s0 + s) * a.E + ec;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (ec + j >= a.E) break;
        p[j] += (double)a.part[i + j];
        cn[j] += a.cnt[i + j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s_p[q][4 * c + j] = p[j];
    s_c[q][4 * c + j] = cn[j];
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    n += __shfl_xor(n, o, 64);
    zz += __shfl_xor(zz, o, 64);
  }
  if (lane == 0) s_n[wave] = n, s_a[wave] = zz;
  __syncthreads();
  if (wave == 0) {
    const int e = e0 + lane;
    double ps = 0.0;
    int cs = 0;
#pragma unroll 8
    for (int i = 0; i < Q; ++i) ps += s_p[i][lane], cs += s_c[i][lane];
    n = 0, zz = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) n += s_n[i], zz += s_a[i];
    if (e < a.E) {
      a.counts[(size_t)g * a.E + e] = cs;
      a.prob[(size_t)g * a.E + e] = n > 0 ? (float)(ps / n) : 0.0f;
    }
    double term = e < a.E ? ps * cs : 0.0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) term += __shfl_xor(term, o, 64);
    if (lane == 0) {
      __hip_atomic_store(&a.lossp[(size_t)g * gridDim.y + blockIdx.y], group_term(a, n, term), __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
      if (blockIdx.y == 0) {
        __hip_atomic_store(&a.n_tok[g], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&a.zzp[g], zz, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      s_last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               (int)(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  int N = 0, groups = 0;
  double bal = 0.0;
  zz = 0.0;
  for (int i = threadIdx.x; i < a.G; i += kFinThreads) {
    const int r = __hip_atomic_load(&a.n_tok[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    N += r;
    groups += r > 0;
    zz += __hip_atomic_load(&a.zzp[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  for (int i = threadIdx.x; i < a.G * (int)gridDim.y; i += kFinThreads)
    bal += __hip_atomic_load(&a.lossp[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    N += __shfl_xor(N, o, 64);
    groups += __shfl_xor(groups, o, 64);
    zz += __shfl_xor(zz, o, 64);
    bal += __shfl_xor(bal, o, 64);
  }
  if (lane == 0) s_n[wave] = N, s_m[wave] = groups, s_a[wave] = zz, s_b[wave] = bal;
  __syncthreads();
  if (threadIdx.x == 0) {
    N = groups = 0, zz = bal = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) N += s_n[i], groups += s_m[i], zz += s_a[i], bal += s_b[i];
    write_totals(a, N, groups, bal, zz);
  }
}

// STREAM: nontemporal stores (a template parameter: as a branch the compiler
// merges both stores into one plain one).
template <int LPR, int NV, bool VEC, bool STREAM>
__global__ __launch_bounds__(kBalThreads) void balance_bwd_kernel(BalArgs a) {
  typedef RowLayout<LPR, NV, VEC> RL;
  constexpr int U = kRowsAtOnce;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & (LPR - 1), sub = lane / LPR;
  const int c_lo = blockIdx.x * a.rows, c_hi = min(a.T, c_lo + a.rows);
  const int step = kBalWaves * RL::kRows * U;
  const int g0 = first_group(a, c_lo);
  if (g0 < 0) return;
  const int N = a.n_tok[a.G], groups = a.n_tok[a.G + 1];
  const double d0 = a.d_loss ? a.d_loss[0] : 1.0, d1 = a.d_loss ? a.d_loss[1] : 1.0;
  const float cz = N > 0 ? (float)(2.0 * a.beta * d1 / N) : 0.0f;
  for (int g = g0; g < a.G; ++g) {
    const int g_lo = group_begin(a, g), g_hi = group_begin(a, g + 1);
    if (g_lo >= c_hi) break;
    const int lo = max(g_lo, c_lo), hi = min(g_hi, c_hi);
    if (lo >= hi) continue;
    Rows<LPR, NV, VEC> now, next;
    // last rows first: the forward read them last, so they are likeliest to be
    // in a cache still
    const int first = lo + wave * RL::kRows * U;
    int r0 = first < hi ? first + (hi - 1 - first) / step * step : first;
    if (r0 < hi) now.load(a, r0, hi, l, sub);
    const int n = a.n_tok[g];
    const float cw = n > 0 && groups > 0 ? (float)(a.alpha * d0 * a.E / ((double)a.k * n * n * groups)) : 0.0f;
    const double mean = (double)a.k * n / a.E;
    float w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = RL::expert(l, i);
      w[i] = e < a.E ? cw * (float)(a.counts[(size_t)g * a.E + e] - mean) : 0.0f;
    }
    while (r0 < hi) {
      const bool more = r0 > first;
      if (more) next.load(a, r0 - step, hi, l, sub);
      bool live[U];
      float lse[U], dot[U];
      const bool rare = softmax_rows<LPR, NV, U>(now.v, now.mask, now.in, lane, live, lse);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        dot[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) dot[u] = __builtin_fmaf(now.v[u][i], w[i], dot[u]);
        dot[u] = group_sum<LPR>(dot[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float c = __builtin_fmaf(cz, lse[u], -dot[u]);
#pragma unroll
        for (int i = 0; i < NV; ++i) now.v[u][i] *= w[i] + c;
      }
      if (rare) {  // exact zeros where nothing counts, whatever d_loss holds
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < NV; ++i) now.v[u][i] = live[u] ? now.v[u][i] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!now.in[u]) continue;
        RL::template store<STREAM>(a.dz + (size_t)(r0 + u * RL::kRows + sub) * a.E, l, a.E, now.v[u]);
      }
      if (!more) break;
      r0 -= step;
      now = next;
    }
  }
}

struct Shape {
  int lpr, nv;
  bool vec;
};

// Lanes per row and values per lane: 16-byte units where rows start aligned,
// at most 64 lanes, the fewest that hold the row with one unit (value) each.
// Rows of 33 to 64 units take 32 lanes when there are many: two rows of a
// wave then share the steps of the row reductions (131072 x 256: 87 us against
// 91, in one group 90 against 94; 65536 x 256: 54.7 against 55.3), while fewer
// rows are over sooner with twice the waves (16384 x 256: 27.4 against 28.9;
// at 50000 the 32 lanes would take 44.3 against 45.3).
Shape row_shape(int T, int E, uintptr_t align) {
  Shape s;
  s.vec = E % 4 == 0 && align % 16 == 0;
  const int units = s.vec ? E / 4 : E;
  const int most = s.vec && units <= 64 && T >= 1 << 16 ? 32 : 64;
  s.lpr = 1;
  while (s.lpr < most && s.lpr < units) s.lpr <<= 1;
  int per = 1;
  while (per * s.lpr < units) per <<= 1;
  s.nv = s.vec ? 4 * per : per;
  return s;
}

// Rows per chunk: whole steps of a workgroup, at most kBalWgs chunks; one
// group of up to four steps is one chunk, whose workgroup needs no second
// kernel to finish (512 x 8, forward and backward: 13.6 us against 17.4).
int chunk_rows(int T, int E, int G) {
  const Shape s = row_shape(T, E, 0);
  const int64_t step = (int64_t)kBalWaves * (64 / s.lpr) * kRowsAtOnce;
  if (G == 1 && T <= 4 * step) return (int)(4 * step);
  const int64_t n = (T + kBalWgs * step - 1) / (kBalWgs * step);
  return (int)(step * (n < 1 ? 1 : n));
}
int chunk_count(int T, int E, int G) {
  const int rows = chunk_rows(T, E, G);
  return T > rows ? (T + rows - 1) / rows : 1;
}

int fin_blocks(int E) { return (E + kFinCols - 1) / kFinCols; }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <bool BWD, int LPR, int NV, bool VEC>
void launch_rows(const BalArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.chunks), blk(kBalThreads);
  if constexpr (BWD) {
    if constexpr (VEC) {
      if (a.stream) {
        hipLaunchKernelGGL((balance_bwd_kernel<LPR, NV, true, true>), grid, blk, 0, st, a);
        return;
      }
    }
    hipLaunchKernelGGL((balance_bwd_kernel<LPR, NV, VEC, false>), grid, blk, 0, st, a);
  } else
    hipLaunchKernelGGL((balance_fwd_kernel<LPR, NV, VEC>), grid, blk, 0, st, a);
}

template <bool BWD>
void launch_shape(const Shape& s, const BalArgs& a, hipStream_t st) {
#define MOK_BAL(L, N, V) \
  if (s.lpr == L && s.nv == N && s.vec == V) return launch_rows<BWD, L, N, V>(a, st)
  MOK_BAL(1, 4, true);
  MOK_BAL(2, 4, true);
  MOK_BAL(4, 4, true);
  MOK_BAL(8, 4, true);
  MOK_BAL(16, 4, true);
  MOK_BAL(32, 4, true);
  MOK_BAL(32, 8, true);
  MOK_BAL(64, 4, true);
  MOK_BAL(64, 8, true);
  MOK_BAL(1, 1, false);
  MOK_BAL(2, 1, false);
  MOK_BAL(4, 1, false);
  MOK_BAL(8, 1, false);
  MOK_BAL(16, 1, false);
  MOK_BAL(32, 1, false);
  MOK_BAL(64, 1, false);
  MOK_BAL(64, 2, false);
  MOK_BAL(64, 4, false);
  MOK_BAL(64, 8, false);
#undef MOK_BAL
}

}  // namespace

size_t balance_ws_bytes(int T, int E, int G) {
  const size_t slots = (size_t)G + chunk_count(T, E, G);
  return 2 * align256(slots * E * 4) + align256(slots * 8) + align256(slots * 4) + align256((size_t)G * fin_blocks(E) * 8) +
         align256((size_t)G * 8) + 256;
}

mok_status launch_balance_fwd(int T, int E, int k, int G, const mok_balance& b, const float* logits,
                              const int32_t* topk, int32_t* counts, float* prob, int32_t* n_tok,
                              float* loss, void* ws, int32_t* status, hipStream_t stream,
                              mok_trace* tr) {
  BalArgs a = {};
  a.z = logits;
  a.topk = topk;
  a.mask = b.token_mask;
  a.off = b.G > 0 ? b.group_offsets : nullptr;
  a.T = T, a.E = E, a.k = k, a.G = G;
  a.rows = chunk_rows(T, E, G);
  a.chunks = chunk_count(T, E, G);
  a.status = status;
  const size_t slots = (size_t)G + a.chunks;
  char* p = (char*)ws;
  auto take = [&](size_t bytes) {
    char* q = p;
    p += align256(bytes);
    return q;
  };
  a.part = (float*)take(slots * E * 4);
  a.cnt = (int32_t*)take(slots * E * 4);
  a.zz = (double*)take(slots * 8);
  a.nrow = (int32_t*)take(slots * 4);
  a.lossp = (double*)take((size_t)G * fin_blocks(E) * 8);
  a.zzp = (double*)take((size_t)G * 8);
  a.ticket = (int32_t*)p;
  a.counts = counts, a.prob = prob, a.n_tok = n_tok, a.loss = loss;
  a.alpha = b.alpha, a.beta = b.beta;
  launch_shape<false>(row_shape(T, E, (uintptr_t)logits), a, stream);
  trace_mark(tr, "balance_fwd", stream);
  if (a.chunks > 1 || G > 1) {
    hipLaunchKernelGGL(balance_finish_kernel, dim3(G, fin_blocks(E)), dim3(kFinThreads), 0, stream, a);
    trace_mark(tr, "balance_finish", stream);
  }
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

mok_status launch_balance_bwd(int T, int E, int k, int G, const mok_balance& b, const float* logits,
                              const int32_t* counts, const int32_t* n_tok, const float* d_loss,
                              float* d_logits, int32_t* status, hipStream_t stream, mok_trace* tr) {
  BalArgs a = {};
  a.z = logits;
  a.mask = b.token_mask;
  a.off = b.G > 0 ? b.group_offsets : nullptr;
  a.T = T, a.E = E, a.k = k, a.G = G;
  a.rows = chunk_rows(T, E, G);
  a.chunks = chunk_count(T, E, G);
  a.status = status;
  a.counts = const_cast<int32_t*>(counts);
  a.n_tok = const_cast<int32_t*>(n_tok);
  a.d_loss = d_loss;
  a.dz = d_logits;
  // Logits and gradients that the 256 MiB memory-side cache cannot hold
  // together: left in it, the gradients are written back under whatever runs
  // next, and push out the logits (131072 x 256, forward and backward: 100
  // us, 87 us with streaming stores; smaller ones are read again from the
  // cache by the router's backward).
  a.stream = (int64_t)T * E * 8 >= (int64_t)256 << 20;
  a.alpha = b.alpha, a.beta = b.beta;
  launch_shape<true>(row_shape(T, E, (uintptr_t)logits | (uintptr_t)d_logits), a, stream);
  trace_mark(tr, "balance_bwd", stream);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

}  // namespace mok
