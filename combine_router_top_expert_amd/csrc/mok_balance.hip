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
// Forward: a workgroup takes a slice of one group's rows.  A row is held by
// LPR lanes (NV logits each, 16-byte loads where E and the alignment allow),
// so a wave takes 64 / LPR rows at a time, U times over (all loads of these
// rows before the first use: one row at a time left the kernel waiting for
// memory, 144 us against 37 us on 131072 x 256), and each lane keeps the
// column sums of its own NV experts over all its rows; counts are integer
// LDS atomics (their order cannot change the result).  Per slice the column
// sums, counts, row count and sum of lse^2 go to the workspace; a second
// kernel adds the slices in order in 64 bits, and its last workgroup the
// groups.  A call whose rows fit one slice ends in the first kernel.
// Backward: the same slices and row layout, one pass, the row's softmax
// formed again from registers.
#include "mok_internal.h"
#include "mok_lanes.h"

namespace mok {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / 64;
constexpr int kBalWgs = 1024;   // slices aimed at: four workgroups per CU
constexpr int kMaxE = 512;
constexpr int kFinCols = 16;    // experts per workgroup of the finishing kernel

struct BalArgs {
  const float* z;
  const int32_t* topk;
  const uint8_t* mask;
  const int32_t* off;    // [G+1] or null: one group of T rows
  int T, E, k, G, splits;
  int32_t* status;
  // workspace of the forward
  float* part;           // [G * splits][E] column sums
  int32_t* cnt;          // [G * splits][E]
  float* zz;             // [G * splits]
  int32_t* rows;         // [G * splits]
  int32_t* ticket;       // workgroups of the finishing kernel that are done
  double* lossp;         // [G * ceil(E / kFinCols)]
  // outputs and the backward's inputs
  int32_t* counts;
  float* prob;
  int32_t* n_tok;
  float* loss;
  const float* d_loss;
  float* dz;
  float alpha, beta;
};

// Rows [lo, hi) of slice s of group g; false (and MOK_EGROUP latched) if the
// group's offsets do not ascend within [0, T].
__device__ __forceinline__ bool slice_rows(const BalArgs& a, int g, int s, int* lo, int* hi) {
  int b = 0, e = a.T;
  if (a.off) {
    b = a.off[g];
    e = a.off[g + 1];
    if (b < 0 || e < b || e > a.T) {
      if (threadIdx.x == 0) latch(a.status, MOK_EGROUP);
      return false;
    }
  }
  const int64_t n = e - b;
  *lo = b + (int)(n * s / a.splits);
  *hi = b + (int)(n * (s + 1) / a.splits);
  return true;
}

// The row layout: lane l of LPR holds experts 4 (l + LPR u) + 0..3 (VEC) or
// l + LPR i.  expert(i) is the expert of value i of this lane.
template <int LPR, int NV, bool VEC>
struct RowLayout {
  static constexpr int kRows = 64 / LPR;  // rows of a wave at a time
  __device__ __forceinline__ static int expert(int l, int i) {
    return VEC ? 4 * (l + LPR * (i >> 2)) + (i & 3) : l + LPR * i;
  }
  // logits of a row; -inf past E (and for a row that is not there)
  __device__ __forceinline__ static void load(const float* row, bool there, int l, int E, float (&v)[NV]) {
    if constexpr (VEC) {
#pragma unroll
      for (int u = 0; u < NV / 4; ++u) {
        const int e = 4 * (l + LPR * u);
        float4 q = make_float4(-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff());
        if (there && e < E) q = *reinterpret_cast<const float4*>(row + e);
        v[4 * u] = q.x, v[4 * u + 1] = q.y, v[4 * u + 2] = q.z, v[4 * u + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = l + LPR * i;
        v[i] = there && e < E ? row[e] : -__builtin_inff();
      }
    }
  }
  __device__ __forceinline__ static void store(float* row, int l, int E, const float (&v)[NV]) {
    if constexpr (VEC) {
#pragma unroll
      for (int u = 0; u < NV / 4; ++u) {
        const int e = 4 * (l + LPR * u);
        if (e < E) *reinterpret_cast<float4*>(row + e) = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
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

// Values of a lane in U rows at once, so their loads are in flight together.
template <int NV>
constexpr int rows_at_once() {
  return NV >= 8 ? 2 : 4;
}
// Chosen slots of a row per lane (k <= 16 and k <= E).
template <int LPR, bool VEC>
constexpr int slots_per_lane() {
  return !VEC || LPR >= 16 ? 1 : LPR == 8 ? 2 : 4;
}

// Softmax of a row in place (v becomes p) and its log-sum-exp; false if the
// row does not count (masked, absent or all -inf): v is then zero.  A NaN
// among the logits reaches p and lse.  exp and log are the hardware's base-2
// ones (1 ulp) on z - max, reciprocal of the sum likewise.
template <int LPR, int NV>
__device__ __forceinline__ bool row_softmax(float (&v)[NV], bool there, int lane, float* lse) {
  float mx = v[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) mx = __builtin_fmaxf(mx, v[i]);
  mx = group_reduce<LPR, OpMax>(mx);
  bool live = there;
  if (__any(mx == -__builtin_inff())) {  // fmax passes over NaN: look for one
    bool some = mx != -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NV; ++i) some = some || __builtin_isnan(v[i]);
    const uint64_t vote = __ballot(some);
    const uint64_t grp = LPR == 64 ? ~0ull : ((1ull << (LPR & 63)) - 1) << (lane & ~(LPR - 1));
    live = there && (vote & grp) != 0;
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = __builtin_amdgcn_exp2f((v[i] - mx) * 1.4426950408889634f);
    sum += v[i];
  }
  sum = group_reduce<LPR, OpAdd>(sum);
  const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = live ? v[i] * inv : 0.0f;
  *lse = live ? __builtin_fmaf(__builtin_amdgcn_logf(sum), 0.6931471805599453f, mx) : 0.0f;
  return live;
}

// Sums of n values v[i] (i < n) over the workgroup; every thread gets it.
template <class T, class F>
__device__ __forceinline__ T block_sum(int n, F value) {
  __shared__ T s_w[kBalWaves];
  T x = 0;
  for (int i = threadIdx.x; i < n; i += kBalThreads) x += value(i);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = x;
  __syncthreads();
  return (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
}

// n_tok[G], n_tok[G+1] and the losses from the groups' terms.
__device__ __forceinline__ void write_totals(const BalArgs& a, int N, int groups, double bal, double zz) {
  a.n_tok[a.G] = N;
  a.n_tok[a.G + 1] = groups;
  a.loss[0] = groups > 0 ? (float)(a.alpha * bal / groups) : 0.0f;
  a.loss[1] = N > 0 ? (float)(a.beta * zz / N) : 0.0f;
}
__device__ __forceinline__ double group_term(const BalArgs& a, int n, double cp) {
  return n > 0 ? cp * a.E / ((double)a.k * n * n) : 0.0;
}

template <int LPR, int NV, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_fwd_kernel(BalArgs a) {
  typedef RowLayout<LPR, NV, VEC> RL;
  constexpr int U = rows_at_once<NV>(), KJ = slots_per_lane<LPR, VEC>();
  __shared__ float s_sum[kBalWaves][kMaxE];
  __shared__ int s_cnt[kMaxE];
  __shared__ float s_zz[kBalWaves];
  __shared__ int s_n[kBalWaves];
  const int wg = blockIdx.x, g = wg / a.splits, s = wg % a.splits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane & (LPR - 1), sub = lane / LPR;
  for (int e = tid; e < a.E; e += kBalThreads) s_cnt[e] = 0;
  __syncthreads();
  int lo = 0, hi = 0;
  if (!slice_rows(a, g, s, &lo, &hi)) lo = hi = 0;
  float acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
  float zz = 0.0f;
  int n = 0;
  for (int64_t r0 = lo + wave * RL::kRows * U; r0 < hi; r0 += kBalWaves * RL::kRows * U) {
    float v[U][NV];
    int id[U][KJ];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * RL::kRows + sub;
      there[u] = r < hi;
      RL::load(a.z + (size_t)r * a.E, there[u], l, a.E, v[u]);
#pragma unroll
      for (int q = 0; q < KJ; ++q) {
        const int j = l + LPR * q;
        id[u][q] = there[u] && j < a.k ? a.topk[(size_t)r * a.k + j] : 0;
      }
      if (a.mask) there[u] = there[u] && a.mask[r];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float lse;
      const bool live = row_softmax<LPR, NV>(v[u], there[u], lane, &lse);
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += v[u][i];
      zz = __builtin_fmaf(lse, lse, zz);   // every lane of the row: lane 0's is used
      n += live;
#pragma unroll
      for (int q = 0; q < KJ; ++q) {
        if (!live || l + LPR * q >= a.k) continue;
        if (id[u][q] >= 0 && id[u][q] < a.E) atomicAdd(&s_cnt[id[u][q]], 1);
        else latch(a.status, MOK_EROUTE);
      }
    }
  }
  // the wave's row groups, then the four waves
#pragma unroll
  for (int i = 0; i < NV; ++i) {
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
  const float zsum = (s_zz[0] + s_zz[1]) + (s_zz[2] + s_zz[3]);
  auto column = [&](int e) { return (s_sum[0][e] + s_sum[1][e]) + (s_sum[2][e] + s_sum[3][e]); };
  if (gridDim.x == 1) {  // the only slice: nothing is left to add up
    const double cp = block_sum<double>(a.E, [&](int e) {
      const double p = column(e);
      a.counts[e] = s_cnt[e];
      a.prob[e] = rows > 0 ? (float)(p / rows) : 0.0f;
      return p * s_cnt[e];
    });
    if (tid == 0) {
      a.n_tok[0] = rows;
      write_totals(a, rows, rows > 0, group_term(a, rows, cp), zsum);
    }
    return;
  }
  for (int e = tid; e < a.E; e += kBalThreads) {
    a.part[(size_t)wg * a.E + e] = column(e);
    a.cnt[(size_t)wg * a.E + e] = s_cnt[e];
  }
  if (tid == 0) {
    a.zz[wg] = zsum;
    a.rows[wg] = rows;
    if (wg == 0) *a.ticket = 0;   // for the kernel that follows
  }
}

// Slices of one group, kFinCols experts: thread (c, q) adds slices q, q + 16,
// ... of expert c; the 16 partial sums meet in LDS in order.  The workgroup
// that finishes last (a ticket per workgroup; what the others wrote is made
// visible by their release and its acquire fence) adds the groups.
__global__ __launch_bounds__(kBalThreads) void balance_finish_kernel(BalArgs a) {
  constexpr int Q = kBalThreads / kFinCols;
  __shared__ double s_p[Q][kFinCols];
  __shared__ int s_c[Q][kFinCols];
  __shared__ int s_last;
  const int g = blockIdx.x, c = threadIdx.x % kFinCols, q = threadIdx.x / kFinCols;
  const int e = blockIdx.y * kFinCols + c;
  double p = 0.0;
  int cn = 0;
  if (e < a.E) {
    for (int s = q; s < a.splits; s += Q) {
      const size_t i = ((size_t)g * a.splits + s) * a.E + e;
      p += (double)a.part[i];
      cn += a.cnt[i];
    }
  }
  s_p[q][c] = p;
  s_c[q][c] = cn;
  const int n = block_sum<int>(a.splits, [&](int i) { return a.rows[(size_t)g * a.splits + i]; });
  if (threadIdx.x < 64) {  // wave 0; its first kFinCols lanes hold an expert each
    double term = 0.0;
    if (q == 0) {
      p = 0.0, cn = 0;
      for (int i = 0; i < Q; ++i) p += s_p[i][c], cn += s_c[i][c];
      if (e < a.E) {
        a.counts[(size_t)g * a.E + e] = cn;
        a.prob[(size_t)g * a.E + e] = n > 0 ? (float)(p / n) : 0.0f;
        term = p * cn;
      }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) term += __shfl_xor(term, o, 64);
    if (threadIdx.x == 0) {
      a.lossp[(size_t)g * gridDim.y + blockIdx.y] = group_term(a, n, term);
      if (blockIdx.y == 0) a.n_tok[g] = n;
      __threadfence();
      s_last = atomicAdd(a.ticket, 1) == (int)(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const int N = block_sum<int>(a.G, [&](int i) { return a.n_tok[i]; });
  const int groups = block_sum<int>(a.G, [&](int i) { return a.n_tok[i] > 0 ? 1 : 0; });
  const double bal = block_sum<double>(a.G * (int)gridDim.y, [&](int i) { return a.lossp[i]; });
  const double zz = block_sum<double>(a.G * a.splits, [&](int i) { return (double)a.zz[i]; });
  if (threadIdx.x == 0) write_totals(a, N, groups, bal, zz);
}

template <int LPR, int NV, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_bwd_kernel(BalArgs a) {
  typedef RowLayout<LPR, NV, VEC> RL;
  constexpr int U = rows_at_once<NV>();
  const int wg = blockIdx.x, g = wg / a.splits, s = wg % a.splits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & (LPR - 1), sub = lane / LPR;
  int lo, hi;
  if (!slice_rows(a, g, s, &lo, &hi)) return;
  const int n = a.n_tok[g], N = a.n_tok[a.G], groups = a.n_tok[a.G + 1];
  const double d0 = a.d_loss ? a.d_loss[0] : 1.0, d1 = a.d_loss ? a.d_loss[1] : 1.0;
  const float cw = n > 0 && groups > 0 ? (float)(a.alpha * d0 * a.E / ((double)a.k * n * n * groups)) : 0.0f;
  const float cz = N > 0 ? (float)(2.0 * a.beta * d1 / N) : 0.0f;
  const double mean = (double)a.k * n / a.E;
  float w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = RL::expert(l, i);
    w[i] = e < a.E ? cw * (float)(a.counts[(size_t)g * a.E + e] - mean) : 0.0f;
  }
  for (int64_t r0 = lo + wave * RL::kRows * U; r0 < hi; r0 += kBalWaves * RL::kRows * U) {
    float v[U][NV];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * RL::kRows + sub;
      there[u] = r < hi;
      RL::load(a.z + (size_t)r * a.E, there[u], l, a.E, v[u]);
      if (a.mask) there[u] = there[u] && a.mask[r];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float lse;
      const bool live = row_softmax<LPR, NV>(v[u], there[u], lane, &lse);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) dot = __builtin_fmaf(v[u][i], w[i], dot);
      dot = group_reduce<LPR, OpAdd>(dot);
      const float c = __builtin_fmaf(cz, lse, -dot);
#pragma unroll
      for (int i = 0; i < NV; ++i) v[u][i] = live ? v[u][i] * (w[i] + c) : 0.0f;
      const int64_t r = r0 + u * RL::kRows + sub;
      if (r < hi) RL::store(a.dz + (size_t)r * a.E, l, a.E, v[u]);
    }
  }
}

struct Shape {
  int lpr, nv;
  bool vec;
};

// Lanes per row and values per lane: 16-byte units where rows start aligned,
// at most 64 lanes, the fewest that hold the row with one unit (value) each.
Shape row_shape(int E, uintptr_t align) {
  Shape s;
  s.vec = E % 4 == 0 && align % 16 == 0;
  const int units = s.vec ? E / 4 : E;
  s.lpr = 1;
  while (s.lpr < 64 && s.lpr < units) s.lpr <<= 1;
  int per = 1;
  while (per * s.lpr < units) per <<= 1;
  s.nv = s.vec ? 4 * per : per;
  return s;
}

// Slices per group: about kBalWgs workgroups in all, no slice shorter than
// one step of a workgroup on average.
int split_count(int T, int E, int G) {
  const Shape s = row_shape(E, 0);
  const int64_t step = (int64_t)kBalWaves * (64 / s.lpr) * (s.nv >= 8 ? rows_at_once<8>() : rows_at_once<4>());
  int64_t n = kBalWgs / G;
  const int64_t most = (T + step * G - 1) / (step * G);
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

int fin_blocks(int E) { return (E + kFinCols - 1) / kFinCols; }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <bool BWD, int LPR, int NV, bool VEC>
void launch_rows(const BalArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.G * a.splits)), blk(kBalThreads);
  if constexpr (BWD)
    hipLaunchKernelGGL((balance_bwd_kernel<LPR, NV, VEC>), grid, blk, 0, st, a);
  else
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
  const size_t wgs = (size_t)G * split_count(T, E, G);
  return 2 * align256(wgs * E * 4) + 2 * align256(wgs * 4) + align256((size_t)G * fin_blocks(E) * 8) + 256;
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
  a.splits = split_count(T, E, G);
  a.status = status;
  const size_t wgs = (size_t)G * a.splits;
  char* p = (char*)ws;
  a.part = (float*)p;
  p += align256(wgs * E * 4);
  a.cnt = (int32_t*)p;
  p += align256(wgs * E * 4);
  a.zz = (float*)p;
  p += align256(wgs * 4);
  a.rows = (int32_t*)p;
  p += align256(wgs * 4);
  a.lossp = (double*)p;
  p += align256((size_t)G * fin_blocks(E) * 8);
  a.ticket = (int32_t*)p;
  a.counts = counts, a.prob = prob, a.n_tok = n_tok, a.loss = loss;
  a.alpha = b.alpha, a.beta = b.beta;
  launch_shape<false>(row_shape(E, (uintptr_t)logits), a, stream);
  trace_mark(tr, "balance_fwd", stream);
  if (wgs > 1) {
    hipLaunchKernelGGL(balance_finish_kernel, dim3(G, fin_blocks(E)), dim3(kBalThreads), 0, stream, a);
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
  a.splits = split_count(T, E, G);
  a.status = status;
  a.counts = const_cast<int32_t*>(counts);
  a.n_tok = const_cast<int32_t*>(n_tok);
  a.d_loss = d_loss;
  a.dz = d_logits;
  a.alpha = b.alpha, a.beta = b.beta;
  launch_shape<true>(row_shape(E, (uintptr_t)logits | (uintptr_t)d_logits), a, stream);
  trace_mark(tr, "balance_bwd", stream);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

}  // namespace mok
