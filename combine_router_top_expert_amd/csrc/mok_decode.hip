// The experts of a few tokens, with weights in 4 bits: for every token t
//   out_t = sum over its slots j of gate_tj W_down (silu(W_gate x_t) * W_up x_t)
// with the matrices of the slot's expert, E2M1 codes with one E8M0 scale per
// 32 along the contraction (MXFP4).  Two products and a sum:
//   gate_up   h_n = silu(a) b of every item n = (t, j), rounded to bf16;
//   down      y_n = W_down h_n, fp32;
//   combine   out_t, fp32 sums over j in order, rounded once.
// h is the second product's operand, which the matrix cores take in bf16 beside
// weights that need bf16's range, and is what the layer rounds to as well; as
// two bf16 parts it would take twice the instructions and LDS.  It makes the
// output's error 1.4 times that of one rounding at the end (2.3e-3 against
// 1.7e-3 of the norm).
//
// Bound by the weights' bytes.  A workgroup takes some columns of an expert's
// matrices and all of that expert's items, so a matrix is read once however
// many tokens (up to 32, or 64) chose it.  The matrix cores multiply 16 weight rows by
// 16 items at a time; with few items most columns are idle, which costs nothing
// that the loads do not hide.  In a chunk of 128 elements of the contraction,
// lane (r = lane % 16, g = lane / 16) holds block g of weight row r: 32 codes
// in one 16-byte load, and their scale; four operands of 8 values, converted by
// one instruction for two.  The order of the contraction within a chunk is
// free, so the items' operands follow: operand i of lane group g is elements
// 32 g + 8 i .. + 7.
//
// Two ways.  About 20 local items or fewer (one token's, or some more of a
// share of the experts): 16 columns a workgroup, whose waves share the
// contraction, everything asked for before the first product, and the second
// product with the sum over the slots in one launch; latency bounds it.  More:
// a wave takes columns of its own, weights four chunks ahead, and the sum is a
// launch of its own.
//
// Which items belong to an expert: with few of them every wave finds out by
// itself; up to kLongListItems the first product's workgroups look through all
// items while their first weights are on their way, and leave what they found
// to the second; beyond, one launch places the items of every expert, and from
// kPlanItems on the library's expert-contiguous layout.
//
// Measured, us (floor: the bytes at 6.27 TB/s): 1 token, d 2048, I 1408, 64
// experts, top-6: 12.2 (4.4), two launches of 6.6 and 5.8; 61 tokens: 61 (47),
// 37 + 20 + 5 in its launches, of which the weights' stream alone takes 36 + 18;
// 512 tokens at 8 of 256 experts, d 7168, I 2048, top-8: 55 (32), 33 + 16 + 6, the
// stream alone 31 + 13.
#include <string.h>

#include <type_traits>

#include "mok_internal.h"
#include "mok_mx.h"
#include "mok_unit.h"

namespace mok {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChunk = 128;           // contraction elements of a step: 4 blocks
// Items that a workgroup looks through itself: room for them costs registers
// and LDS whatever their number, a launch for the search (beyond the limit) 3 to
// 5 us.  First product of 61 tokens with room for 1024 38 us, for 4096 40.  Whole
// calls, d 7168, 8 of 256 experts, top-8, with a limit of 1024, 2048, 4096 and
// 8192: 256 tokens 43.2, 40.4, 40.5, 41.1 us; 512 tokens 49.9, 50.0, 46.1, 46.7; 513
// 51.3, 51.2, 51.3, 48.1; 1000 77, 77, 77, 68; d 2048, 64 experts, top-6: 300
// tokens 94.0, 88.9, 89.7, 91.0; 682 141, 141, 137, 140; 1000 176, 176, 176, 179.
// 4096 loses at most 0.8 us below it to a smaller limit; 8192 loses up to 3.
constexpr int kListItems = 1024, kLongListItems = 4096;

struct DecodeArgs {
  const void* x;            // [T, d] bf16, or E4M3 codes with x_scale
  const uint8_t* x_scale;   // [T, d/32] or null
  const int32_t* topk;      // [N]
  const int32_t* e2l;       // [E]
  const uint8_t *wg, *wu, *sg, *su;   // of [E_local, I, d/2], [E_local, I, d/32], tiled
  const uint8_t *wd, *sd;             // of [E_local, d, I/2], [E_local, d, I/32], tiled
  int32_t* heads;           // [slots][64]: what kHeads says of every slot
  int32_t* rows;            // [N] items in the order of their slots
  bf16_t* h;                // [N, I]
  float* y;                 // [N, d]
  int32_t* status;
  int N, k, d, I, E, E_local;
  int splits;               // workgroups that share the items of a slot, 32 at a time in turn
};

// The local expert of item i, -1 for none; -2 for an id outside [0, E) or a
// malformed entry of the table.
__device__ __forceinline__ int local_of(const DecodeArgs& a, int64_t i) {
  const int e = a.topk[i];
  if ((unsigned)e >= (unsigned)a.E) return -2;
  const int le = a.e2l[e];
  return le >= a.E_local ? -2 : le < 0 ? -1 : le;
}

// The items of slot `slot`: how many there are, their numbers in ascending
// order and their expert; the same for every thread of the workgroup.  With at
// most E_local items, slot s stands for item s and works if no earlier item
// has the same expert; else slot s is local expert s.
//   kWave    a lane per item, every wave for itself; lane m keeps number m
//   kSearch, kSearchLong   the waves look through the items together; numbers in LDS
//   kHeads   the first kHeadItems numbers in one load of a lane each, with the
//            lanes behind them for what else there is to know
enum { kWave, kSearch, kSearchLong, kHeads };
constexpr int kHeadItems = 32, kHeadN = 32, kHeadBase = 33, kHeadExpert = 34;

struct Items {
  const uint16_t* list;   // kSearch, kSearchLong
  const int32_t* rows;    // kHeads
  int mine;               // kWave, kHeads
  int n, expert;
};

template <int FIND>
__device__ __forceinline__ int item_number(const Items& it, int m) {
  if constexpr (FIND == kWave) {
    const int v = __shfl(it.mine, m & 63, 64);
    return m < it.n ? v : -1;
  } else if constexpr (FIND != kHeads) {
    return m < it.n ? it.list[m] : -1;
  } else {
    int v = __shfl(it.mine, m & 63, 64);
    if (m >= kHeadItems && m < it.n) v = it.rows[m];
    return m < it.n ? v : -1;
  }
}

// The local expert of item `lane` (-1 for none, -2 malformed).  The table of up
// to 256 experts is read beside the ids instead of behind them.
__device__ __forceinline__ int wave_local_of(const DecodeArgs& a) {
  const int lane = lane_id();
  if (a.E > 256) return lane < a.N ? local_of(a, lane) : -1;
  int tab[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) tab[q] = q * 64 + lane < a.E ? a.e2l[q * 64 + lane] : -1;
  const int e = lane < a.N ? a.topk[lane] : 0;
  int le = -1;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int v = __shfl(tab[q], e & 63, 64);
    if (e >> 6 == q) le = v;
  }
  if ((unsigned)e >= (unsigned)a.E || le >= a.E_local) le = -2;
  return lane < a.N ? (le == -2 ? -2 : le < 0 ? -1 : le) : -1;
}

// kWave.
__device__ __forceinline__ Items wave_items(const DecodeArgs& a, int slot) {
  Items it = {nullptr, nullptr, -1, 0, -1};
  const bool by_item = a.N <= a.E_local;
  const int lane = lane_id(), le = wave_local_of(a);
  if (__any(le == -2) && blockIdx.x == 0 && threadIdx.x == 0) latch(a.status, MOK_EROUTE);
  it.expert = by_item ? __builtin_amdgcn_readlane(le, slot) : slot;
  const uint64_t mask = it.expert >= 0 ? __ballot(le == it.expert) : 0;
  if (by_item && (mask & ((1ull << slot) - 1)) != 0) return it;   // an earlier slot has this expert
  it.n = __popcll(mask);
  // lane i of the mask sends its number to the lane of its rank; the others
  // send theirs behind them
  const uint64_t below = (1ull << lane) - 1;
  const int rank = (mask >> lane) & 1 ? __popcll(mask & below) : it.n + __popcll(~mask & below);
  it.mine = __builtin_amdgcn_ds_permute(rank * 4, lane);
  return it;
}

// kSearch, in two halves, so that other loads can be asked for between them:
// first the ids of a run of items per wave, 64 at a time, and the table.
constexpr int kMaxExperts = 512;

template <int WAVES, int ITEMS>
struct Search {
  static constexpr int ROUNDS = ITEMS / (64 * WAVES), TABS = (kMaxExperts + 64 * WAVES - 1) / (64 * WAVES);
  struct Lds {
    int16_t local[kMaxExperts];
    int count[WAVES], below[WAVES];
    uint16_t list[ITEMS];
  };
  int ids[ROUNDS], tab[TABS], rounds, mine;

  __device__ __forceinline__ void ask(const DecodeArgs& a, int slot) {
    const int wave = threadIdx.x >> 6;
    rounds = (a.N + 64 * WAVES - 1) / (64 * WAVES);
#pragma unroll
    for (int t = 0; t < TABS; ++t) tab[t] = a.e2l[min(t * 64 * WAVES + (int)threadIdx.x, a.E - 1)];
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q)
      if (q < rounds) ids[q] = a.topk[min((wave * rounds + q) * 64 + lane_id(), a.N - 1)];
    mine = a.topk[min(slot, a.N - 1)];
  }

  __device__ __forceinline__ Items answer(const DecodeArgs& a, int slot, bool first_of_slot, Lds& s) {
    Items it = {s.list, nullptr, -1, 0, slot};
    const bool by_item = a.N <= a.E_local;
    const int wave = threadIdx.x >> 6, lane = lane_id();
#pragma unroll
    for (int t = 0; t < TABS; ++t) {
      const int e = t * 64 * WAVES + threadIdx.x;
      if (e < kMaxExperts) s.local[e] = tab[t] >= a.E_local ? -2 : tab[t] < 0 ? -1 : tab[t];
    }
    __syncthreads();
    auto local = [&](int e) -> int { return (unsigned)e < (unsigned)a.E ? s.local[e] : -2; };
    if (by_item) it.expert = __builtin_amdgcn_readfirstlane(local(mine));
    uint64_t is[ROUNDS];
    int count = 0, below = 0;
    bool bad = false;
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
      is[q] = 0;
      if (q >= rounds) continue;
      const int le = (wave * rounds + q) * 64 + lane < a.N ? local(ids[q]) : -1;
      bad |= le == -2;
      is[q] = __ballot(le == it.expert && le >= 0);
      count += __popcll(is[q]);
      below += __popcll(__ballot(le < it.expert && le >= 0));
    }
    if (bad && blockIdx.x == 0) latch(a.status, MOK_EROUTE);
    if (lane == 0) s.count[wave] = count, s.below[wave] = below;
    __syncthreads();
    int at = 0, base = 0;
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) at += s.count[w];
      it.n += s.count[w];
      base += s.below[w];
    }
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
      if ((is[q] >> lane) & 1u)
        s.list[at + __popcll(is[q] & ((1ull << lane) - 1))] = (uint16_t)((wave * rounds + q) * 64 + lane);
      at += __popcll(is[q]);
    }
    __syncthreads();
    if (by_item && it.n > 0 && s.list[0] != slot) it.n = 0;
    if (first_of_slot) {                // for the second product
      if (wave == 0) {
        const int v = lane < kHeadItems ? (lane < it.n ? s.list[lane] : 0) : lane == kHeadN ? it.n : lane == kHeadBase ? base : it.expert;
        a.heads[(size_t)slot * 64 + lane] = v;
      }
      for (int m = kHeadItems + threadIdx.x; m < it.n; m += 64 * WAVES) a.rows[base + m] = s.list[m];
    }
    return it;
  }
};

// Eight values of weight codes (a dword) times 2^(byte - 127), as bf16: exact
// where bf16 holds them.
__device__ __forceinline__ bf16x8_t w4_operand(uint32_t codes, float scale) {
  const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8_t{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// Eight E4M3 codes times their block's factor, as bf16 (exact).
__device__ __forceinline__ bf16x8_t x8_operand(uint32_t lo, uint32_t hi, float f) {
  const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false);
  const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true);
  const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false);
  const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true);
  return bf16x8_t{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// An item's operand row: its token's x, or its h.
template <bool DOWN, bool X8>
__device__ __forceinline__ const void* item_row(const DecodeArgs& a, int item) {
  if constexpr (DOWN) return a.h + (size_t)item * a.I;
  const size_t at = (size_t)(item / a.k) * a.d;
  if constexpr (X8) return reinterpret_cast<const uint8_t*>(a.x) + at;
  return reinterpret_cast<const bf16_t*>(a.x) + at;
}

// h = silu(va) vb of an item, four columns from `at`.
__device__ __forceinline__ void store_h(const DecodeArgs& a, int item, int at, f32x4_t va, f32x4_t vb) {
  float hv[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) hv[e] = silu_f(va[e]) * vb[e];
  *reinterpret_cast<uint2*>(a.h + (size_t)item * a.I + at) = make_uint2(pack2_bf16(hv[0], hv[1]), pack2_bf16(hv[2], hv[3]));
}

// The four operands of chunk c of an item's row: operand i is elements
// 128 c + 32 g + 8 i .. + 7.  X8: E4M3 codes with their block's scale, decoded
// (exact in bf16).
template <bool X8>
__device__ __forceinline__ void item_operands(const void* row, const uint8_t* scale, int c, int g, bf16x8_t (&o)[4]) {
  const int at = c * kChunk + 32 * g;
  if constexpr (X8) {
    const uint4 lo = ld16(reinterpret_cast<const uint8_t*>(row) + at), hi = ld16(reinterpret_cast<const uint8_t*>(row) + at + 16);
    const float f = __uint_as_float((uint32_t)scale[c * 4 + g] << 23);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = x8_operand(w[2 * i], w[2 * i + 1], f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(bf16x8_t, ld16(reinterpret_cast<const bf16_t*>(row) + at + 8 * i));
  }
}

// NM matrices of one expert from a column tile on.  The weights are laid out in
// the order in which a wave reads them: per tile of 16 rows and chunk, 64 lanes
// of 16 bytes, lane (r, g) with block g of row r; per tile and four chunks, 64
// lanes of 4 scales, lane (r, g) with block g of row r in each of the four.  A
// load is one run of memory (the stream alone, four chunks ahead with a wait
// for all of them: 4.7 TB/s, row by row, in 16 runs of 64 bytes, 4.3; the loop as
// it is reaches 5.4 with the products).
template <int NM>
struct Weights {
  const uint8_t* codes[NM];
  const uint8_t* scales[NM];
  int chunks;               // of the whole contraction
};

// Tile j = NM p + m: column tile p of matrix m.
template <int NM>
__device__ __forceinline__ uint4 tile_codes(const Weights<NM>& w, int j, int c) {
  return ld16(w.codes[j % NM] + ((size_t)(j / NM) * w.chunks + c) * 1024 + 16 * lane_id());
}

// The scales of chunks c .. c + 3, c a multiple of 4.
template <int NM>
__device__ __forceinline__ uint32_t tile_scales(const Weights<NM>& w, int j, int c) {
  return *reinterpret_cast<const uint32_t*>(w.scales[j % NM] + ((size_t)(j / NM) * ((w.chunks + 3) / 4) + c / 4) * 256 + 4 * lane_id());
}

__device__ __forceinline__ float scale_of(uint32_t four, int p) {
  return __uint_as_float(((four >> (8 * p)) & 0xFFu) << 23);
}

// Columns n0 .. of an expert's matrices.
template <bool DOWN>
__device__ __forceinline__ auto expert_weights(const DecodeArgs& a, int local, int n0) {
  const int out = DOWN ? a.d : a.I, K = DOWN ? a.I : a.d;
  const size_t tile = ((size_t)__builtin_amdgcn_readfirstlane(local) * out + n0) / 16;
  Weights<DOWN ? 1 : 2> w;
  w.chunks = K / kChunk;
  const size_t codes = tile * w.chunks * 1024, scales = tile * ((w.chunks + 3) / 4) * 256;
  w.codes[0] = (DOWN ? a.wd : a.wg) + codes;
  w.scales[0] = (DOWN ? a.sd : a.sg) + scales;
  if constexpr (!DOWN) {
    w.codes[1] = a.wu + codes;
    w.scales[1] = a.su + scales;
  }
  return w;
}

// 16 rows of NM matrices times 16 items over chunks [lo, hi), lo a multiple of
// 4: everything that four chunks need is asked for before the first of them is
// multiplied (the last chunk again behind the end, so that no load depends on a
// condition).
constexpr int kGroup = 4;

template <int NM, bool X8>
__device__ __forceinline__ void product(const Weights<NM>& w, const void* row, const uint8_t* xs, int lo, int hi,
                                        f32x4_t (&acc)[NM]) {
  const int g = lane_id() >> 4;
  for (int c0 = lo; c0 < hi; c0 += kGroup) {
    uint32_t sc[NM];
    uint4 q[kGroup][NM];
    bf16x8_t xo[kGroup][4];
#pragma unroll
    for (int m = 0; m < NM; ++m) sc[m] = tile_scales(w, m, c0);
#pragma unroll
    for (int p = 0; p < kGroup; ++p) {
      const int c = min(c0 + p, hi - 1);
#pragma unroll
      for (int m = 0; m < NM; ++m) q[p][m] = tile_codes(w, m, c);
      item_operands<X8>(row, xs, c, g, xo[p]);
    }
    // (the compiler would put loads behind products to save registers)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < kGroup; ++p) {
      if (c0 + p >= hi) break;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const uint32_t word[4] = {q[p][m].x, q[p][m].y, q[p][m].z, q[p][m].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w4_operand(word[i], scale_of(sc[m], p)), xo[p][i], acc[m], 0, 0, 0);
      }
    }
  }
}

// Where the share of the contraction that part w of n takes begins: whole
// groups of four chunks, and w = n behind the last chunk.
__device__ __forceinline__ int chunk_cut(int chunks, int w, int n) { return min(chunks, (chunks + 3) / 4 * w / n * 4); }

// 16 columns of h for the items of a slot, when there are few items: the four
// waves share the contraction, so that few experts' matrices are under way on
// many compute units, and their sums are added in order.
template <bool X8>
__global__ __launch_bounds__(kThreads) void decode_up_few_kernel(DecodeArgs a) {
  __shared__ f32x4_t red[kWaves][2][64];
  const int tiles = a.I / 16, K = a.d;
  const int slot = blockIdx.x / tiles, n0 = blockIdx.x % tiles * 16;
  const Items it = wave_items(a, slot);
  if (it.n == 0) return;
  const int lane = lane_id(), wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int lo = chunk_cut(K / kChunk, wave, kWaves), hi = chunk_cut(K / kChunk, wave + 1, kWaves);
  const Weights<2> w = expert_weights<false>(a, it.expert, n0);
  for (int m0 = 0; m0 < it.n; m0 += 16) {
    // (columns without an item hold the last item again and are not stored)
    const int item = item_number<kWave>(it, m0 + r), shown = item_number<kWave>(it, min(m0 + r, it.n - 1));
    const void* row = item_row<false, X8>(a, shown);
    const uint8_t* xs = nullptr;
    if constexpr (X8) xs = a.x_scale + (size_t)(shown / a.k) * (K / 32);
    f32x4_t acc[2] = {};
    product<2, X8>(w, row, xs, lo, hi, acc);
    __syncthreads();
    red[wave][0][lane] = acc[0];
    red[wave][1][lane] = acc[1];
    __syncthreads();
    if (wave != 0 || item < 0) continue;
    f32x4_t va = red[0][0][lane], vb = red[0][1][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) {
      va += red[v][0][lane];
      vb += red[v][1][lane];
    }
    store_h(a, item, n0 + 4 * g, va, vb);
  }
}

// 64 NC columns of h (DOWN false) or of y (true) for the items of a slot, 16 MT
// at a time: a wave takes NC tiles of 16 columns over the whole contraction (of
// both matrices for h).  The items' elements go through LDS in slabs, four chunks
// of 16 items, two of 32 or one of 64, one barrier a slab (two buffers taken in
// turn), fetched four chunks ahead (two with 64); the weights come straight to registers, four chunks ahead,
// which keeps the loads of the chip in flight whatever the barriers do.  KG
// groups of four waves share the contraction when there are too few workgroups
// otherwise; their sums are added in order.  LDS rows are 16 bytes longer than
// a slab, so the 16 rows that a quarter of the wave reads lie in 64 different
// banks.  Columns without an item hold the last item again and are not stored.
constexpr int kAhead = 4;                      // chunks
// LDS of `sets` sets of 16 items: four chunks of 16, two of 32, one of 64 (each
// more than the one before).
constexpr int slab_bytes(int sets) { return 16 * sets * (4 / sets * kChunk * 2 + 16); }

template <bool DOWN, int FIND, int NC, int KG, bool X8, int MT>
__global__ __launch_bounds__(kThreads * KG, KG == 1 && NC < 4 && MT < 4 ? 3 : 2) void decode_kernel(DecodeArgs a) {
  constexpr int NM = DOWN ? 1 : 2, NT = NM * NC, kSlabBytes = slab_bytes(MT);
  constexpr int ESIZE = X8 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) char s_all[KG][2][kSlabBytes];
  static_assert(sizeof(s_all) >= (KG - 1) * kWaves * NT * MT * 64 * sizeof(f32x4_t), "the groups' sums fit");
  const int out = DOWN ? a.d : a.I, K = DOWN ? a.I : a.d;
  const int tiles = out / (64 * NC);             // d and I are multiples of 128
  const int slot = blockIdx.x / tiles / a.splits, split = blockIdx.x / tiles % a.splits;
  const int lane = lane_id(), r = lane & 15, g = lane >> 4, tid = threadIdx.x & (kThreads - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), kg = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  const int n0 = blockIdx.x % tiles * (64 * NC) + wave * 16 * NC;
  // this group's chunks, and the most that a group has (the barriers are common)
  const int first = KG == 1 ? 0 : chunk_cut(K / kChunk, kg, KG);
  const int chunks = KG == 1 ? K / kChunk : chunk_cut(K / kChunk, kg + 1, KG) - first;
  const int most = KG == 1 ? chunks : ((K / kChunk + 3) / 4 + KG - 1) / KG * 4;
  char(&s_x)[2][kSlabBytes] = s_all[kg];
  const uint8_t* const base = reinterpret_cast<const uint8_t*>(DOWN ? a.h : a.x);

  uint4 q[kAhead][NT];
  uint32_t sc[NT];
  Weights<NM> w;
  // Chunk c of this group's and the scales of c .. c + 3.  Behind the last
  // chunk every lane takes the same bytes, which costs nothing: a load that may
  // not happen would have the compiler wait for all loads at once.
  auto load = [&](int c, uint4 (&to)[NT]) {
    const uint32_t on = c < chunks ? ~0u : 0u;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      to[j] = ld16(w.codes[j % NM] + (on & (uint32_t)((j / NM * w.chunks + first + c) * 1024 + 16 * lane)));
  };
  auto load_scales = [&](int c) {
    const uint32_t on = c < chunks ? ~0u : 0u;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      sc[j] = *reinterpret_cast<const uint32_t*>(
          w.scales[j % NM] + (on & (uint32_t)((j / NM * ((w.chunks + 3) / 4) + (first + c) / 4) * 256 + 4 * lane)));
  };
  auto begin = [&]() {          // the first chunks of the weights
    load_scales(0);
#pragma unroll
    for (int p = 0; p < kAhead; ++p) load(p, q[p]);
  };
  // where a slot is an expert, its weights are on their way while its items are found
  const bool early = a.N > a.E_local;
  auto ahead = [&]() {
    if (!early) return;
    w = expert_weights<DOWN>(a, slot, n0);
    begin();
  };
  Items it = {};
  if constexpr (FIND != kHeads) {
    using Find = Search<kWaves * KG, FIND == kSearch ? kListItems : kLongListItems>;
    __shared__ typename Find::Lds s_find;
    Find find;
    find.ask(a, slot);
    ahead();
    it = find.answer(a, slot, blockIdx.x % (tiles * a.splits) == 0, s_find);
  } else {
    it.mine = a.heads[(size_t)slot * 64 + lane];
    ahead();
    it.n = __builtin_amdgcn_readlane(it.mine, kHeadN);
    it.rows = a.rows + __builtin_amdgcn_readlane(it.mine, kHeadBase);
    it.expert = __builtin_amdgcn_readlane(it.mine, kHeadExpert);
  }
  if (16 * MT * split >= it.n) return;
  if (!early) {
    w = expert_weights<DOWN>(a, it.expert, n0);
    begin();
  }

  // SETS sets of 16 items, beginning with number m0
  auto pass = [&](auto sets, int m0) {
    constexpr int SETS = decltype(sets)::value, SLAB = 4 / SETS, ROW = SLAB * kChunk * 2 + 16;
    // the units of 8 elements that this thread fetches of a slab: the same
    // columns of every `per`-th row (rows past the last item fetch that item again)
    static_assert(16 * SETS * ROW <= kSlabBytes, "a slab fits its buffer");
    constexpr int WIDE = SLAB * kChunk / 8, PER = kThreads / WIDE, FETCH = 16 * SETS / PER;
    const int col = (tid % WIDE) * 8;
    int src[FETCH];
#pragma unroll
    for (int i = 0; i < FETCH; ++i) {
      const int item = item_number<FIND>(it, min(m0 + tid / WIDE + PER * i, it.n - 1));
      src[i] = DOWN ? item : item / a.k;
    }
    // fetched four chunks ahead (one slab of four chunks, or two of two) or two
    constexpr int HELD = SLAB == 4 ? 1 : 2, XAHEAD = HELD * SLAB;
    uint4 held[HELD][FETCH];
    uint32_t held_scale[HELD][FETCH];
    // the slab that begins with chunk c; what lies behind the last chunk is not used
    auto fetch = [&](int c, uint4 (&xv)[FETCH], uint32_t (&xf)[FETCH]) {
      const int at = min(first * kChunk + min(c * kChunk + col, max(chunks * kChunk - 8, 0)), K - 8);
#pragma unroll
      for (int i = 0; i < FETCH; ++i) {
        const int64_t from = (int64_t)src[i] * K + at;
        if constexpr (X8) {
          const uint2 v = *reinterpret_cast<const uint2*>(base + from);
          xv[i].x = v.x;
          xv[i].y = v.y;
          xf[i] = a.x_scale[from >> 5];
        } else {
          xv[i] = ld16(base + from * ESIZE);
        }
      }
    };
    auto stash = [&](int buf, const uint4 (&xv)[FETCH], const uint32_t (&xf)[FETCH]) {
#pragma unroll
      for (int i = 0; i < FETCH; ++i) {
        uint4 v = xv[i];
        if constexpr (X8) v = __builtin_bit_cast(uint4, x8_operand(xv[i].x, xv[i].y, __uint_as_float(xf[i] << 23)));
        *reinterpret_cast<uint4*>(s_x[buf] + (tid / WIDE + PER * i) * ROW + col * 2) = v;
      }
    };
    fetch(0, held[0], held_scale[0]);
    if (HELD == 2) fetch(SLAB, held[HELD - 1], held_scale[HELD - 1]);
    stash(0, held[0], held_scale[0]);
    __syncthreads();
    f32x4_t acc[NT][SETS];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int s = 0; s < SETS; ++s) acc[j][s] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c0 = 0; c0 < most; c0 += kAhead) {
      float f[kAhead][NT];
#pragma unroll
      for (int p = 0; p < kAhead; ++p)
#pragma unroll
        for (int j = 0; j < NT; ++j) f[p][j] = scale_of(sc[j], p);
      load_scales(c0 + kAhead);
#pragma unroll
      for (int p = 0; p < kAhead; ++p) {
        const int c = c0 + p;
        if (p % SLAB == 0) fetch(c + XAHEAD, held[p / SLAB % HELD], held_scale[p / SLAB % HELD]);
        if (c < chunks) {
          const char* xrow = s_x[(SLAB == 4 ? c0 / 4 : p / SLAB) & 1] + r * ROW + (p % SLAB) * (kChunk * 2) + g * 64;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bf16x8_t xo[SETS];
#pragma unroll
            for (int s = 0; s < SETS; ++s) xo[s] = *reinterpret_cast<const bf16x8_t*>(xrow + s * 16 * ROW + i * 16);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const uint4 v = q[p][j];
              const bf16x8_t wo = w4_operand(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w, f[p][j]);
#pragma unroll
              for (int s = 0; s < SETS; ++s) acc[j][s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wo, xo[s], acc[j][s], 0, 0, 0);
            }
          }
        }
        load(c + kAhead, q[p]);
        if (p % SLAB == SLAB - 1) {
          const int next = (p / SLAB + 1) % HELD;
          stash((SLAB == 4 ? c0 / 4 + 1 : p / SLAB + 1) & 1, held[next], held_scale[next]);
          __syncthreads();
        }
      }
    }
    if (m0 + 16 * MT * a.splits < it.n) begin();
    if constexpr (KG > 1) {
      f32x4_t* red = reinterpret_cast<f32x4_t*>(s_all);
      if (kg > 0)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int s = 0; s < SETS; ++s) red[((((kg - 1) * kWaves + wave) * NT + j) * MT + s) * 64 + lane] = acc[j][s];
      __syncthreads();
      if (kg == 0)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int o = 0; o < KG - 1; ++o) acc[j][s] += red[(((o * kWaves + wave) * NT + j) * MT + s) * 64 + lane];
      __syncthreads();
      if (kg > 0) return;
    }
    // lane (r, g): output rows 4 g .. + 3 of a tile, item r of a set
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
      const int item = item_number<FIND>(it, m0 + 16 * s + r);
      if (item < 0) continue;
#pragma unroll
      for (int p = 0; p < NC; ++p) {
        const int at = n0 + 16 * p + 4 * g;
        if constexpr (DOWN) *reinterpret_cast<f32x4_t*>(a.y + (size_t)item * a.d + at) = acc[p][s];
        else store_h(a, item, at, acc[2 * p][s], acc[2 * p + 1][s]);
      }
    }
  };
  int m0 = 16 * MT * split;
  if constexpr (MT == 4)
    for (; it.n - m0 > 32; m0 += 64 * a.splits) pass(std::integral_constant<int, 4>{}, m0);
  for (; it.n - m0 > 16; m0 += 16 * MT * a.splits) pass(std::integral_constant<int, 2>{}, m0);
  if (m0 < it.n) pass(std::integral_constant<int, 1>{}, m0);
}

// The second product and the sum over the slots in one launch, for up to 16
// tokens and 64 items: 16 columns of out per workgroup, tokens as the columns
// of the matrix cores.  The waves share the (expert, chunk) pairs; a pair's
// product is weighed by each token's gate as it is added; a token that did not
// choose the expert multiplies another's h and adds nothing.
template <int THREADS>
__global__ __launch_bounds__(THREADS, 4) void decode_down_few_kernel(DecodeArgs a, const float* gate, bf16_t* out) {
  constexpr int kFewWaves = THREADS / 64;
  __shared__ f32x4_t red[kFewWaves][64];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, K = a.I, chunks = K / kChunk;
  const int le = wave_local_of(a);
  const float my_gate = lane < a.N ? gate[lane] : 0.0f;
  const bool token = r * a.k < a.N;
  // the experts, by their first items: lane i keeps expert number i's
  int lead = 0, experts = 0;
  for (uint64_t left = __ballot(le >= 0); left != 0; ++experts) {
    const int f = __ffsll((unsigned long long)left) - 1;
    if (lane == experts) lead = f;
    left &= ~__ballot(le == __builtin_amdgcn_readlane(le, f));
  }
  const int pairs = experts * chunks;
  f32x4_t total = {0.0f, 0.0f, 0.0f, 0.0f};
  // this wave's pairs are wave, wave + kFewWaves, ..: four at a time, all of
  // their loads first
  for (int u0 = wave; u0 < pairs; u0 += kGroup * kFewWaves) {
    uint4 q[kGroup];
    bf16x8_t ho[kGroup][4];
    uint32_t sc[kGroup];
    float weigh[kGroup];
    bool chose[kGroup];
#pragma unroll
    for (int p = 0; p < kGroup; ++p) {
      const int u = min(u0 + p * kFewWaves, pairs - 1);
      const int n = u / chunks, c = u % chunks;
      const int first = __builtin_amdgcn_readlane(lead, n), e = __builtin_amdgcn_readlane(le, first);
      const uint64_t mask = __ballot(le == e);
      const Weights<1> m = expert_weights<true>(a, e, n0);
      q[p] = tile_codes(m, 0, c);
      sc[p] = tile_scales(m, 0, c & ~3) >> (8 * (c & 3));
      // this lane's token: its items with this expert (more than one if the
      // expert is listed twice)
      const uint32_t mine = token ? (uint32_t)(mask >> (r * a.k)) & ((1u << a.k) - 1) : 0;
      const int at = mine ? (r * a.k + __ffs(mine) - 1) & 63 : first;
      item_operands<false>(a.h + (size_t)at * K, nullptr, c, g, ho[p]);
      const float one = __shfl(my_gate, at, 64);
      weigh[p] = one;
      chose[p] = mine != 0;
      if (__any(mine & (mine - 1))) {
        for (int j = 0; j < a.k; ++j) {
          const float more = __shfl(my_gate, (r * a.k + j) & 63, 64);
          if ((mine >> j) & 1u && ((r * a.k + j) & 63) != at) weigh[p] += more;
        }
      }
    }
#pragma unroll
    for (int p = 0; p < kGroup; ++p) {
      if (u0 + p * kFewWaves >= pairs) break;
      f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
      const uint32_t word[4] = {q[p].x, q[p].y, q[p].z, q[p].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w4_operand(word[i], scale_of(sc[p], 0)), ho[p][i], acc, 0, 0, 0);
      if (chose[p])
#pragma unroll
        for (int v = 0; v < 4; ++v) total[v] = __builtin_fmaf(weigh[p], acc[v], total[v]);
    }
  }
  red[wave][lane] = total;
  __syncthreads();
  if (wave != 0 || !token) return;
  f32x4_t v = red[0][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) v += red[w][lane];
  *reinterpret_cast<uint2*>(out + (size_t)r * a.d + n0 + 4 * g) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
}

// out[t] = sum over j in order of gate_tj y_tj, over the slots with a local
// expert: 8 columns per thread, a workgroup within one token, so that what it
// needs to know of the slots is the same for all of it.
__global__ __launch_bounds__(kThreads) void decode_combine_kernel(DecodeArgs a, const float* gate, bf16_t* out, int pieces) {
  const int64_t t = blockIdx.x / pieces;
  const int c = (blockIdx.x % pieces * kThreads + threadIdx.x) * 8;
  // the token's slots with a local expert, as bits
  uint32_t left = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < a.k && local_of(a, t * a.k + j) >= 0) left |= 1u << j;
  if (c >= a.d) return;
  float acc[8] = {};
  while (left != 0) {                    // the rows of four slots at a time
    float v[4][8], q[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (left == 0) break;
      const int64_t n = t * a.k + __ffs(left) - 1;
      left &= left - 1;
      q[s] = gate[n];
      load8(a.y + n * a.d + c, v[s]);
      if (s < 3 && left != 0) continue;
#pragma unroll
      for (int u = 0; u <= s; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(q[u], v[u][i], acc[i]);
      break;
    }
  }
  store8(out + t * a.d + c, acc);
}

// The layout of more items than a workgroup looks through, in one launch: one
// workgroup per local expert counts the items of the experts before it and its
// own and places its own, each thread a run of consecutive items (ascending
// order).  All workgroups read all items, so up to kPlanItems.
constexpr int kPlanItems = 32768;
constexpr int kPlanThreads = 1024;

__global__ __launch_bounds__(kPlanThreads) void decode_plan_kernel(DecodeArgs a) {
  __shared__ int s_below[kPlanThreads / 64], s_mine[kPlanThreads / 64];
  const int me = blockIdx.x, lane = lane_id(), wave = threadIdx.x >> 6;
  const int run = (a.N + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(a.N, (int)threadIdx.x * run), hi = min(a.N, lo + run);
  int below = 0, mine = 0;
  bool bad = false;
  for (int i = lo; i < hi; ++i) {
    const int le = local_of(a, i);
    bad |= le == -2;
    below += le >= 0 && le < me;
    mine += le == me;
  }
  if (bad && me == 0) latch(a.status, MOK_EROUTE);
  int before = mine;                    // items of this expert in the wave's lanes up to this one
  int all = below;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(before, off, 64);
    if (lane >= off) before += v;
    all += __shfl_xor(all, off, 64);
  }
  if (lane == 63) s_mine[wave] = before;
  if (lane == 0) s_below[wave] = all;
  __syncthreads();
  int base = 0, at = before - mine, total = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    base += s_below[w];
    total += s_mine[w];
    if (w < wave) at += s_mine[w];
  }
  int32_t* head = a.heads + (size_t)me * 64;
  if (threadIdx.x == 0) head[kHeadN] = total, head[kHeadBase] = base, head[kHeadExpert] = me;
  for (int i = lo; i < hi; ++i)
    if (local_of(a, i) == me) {
      if (at < kHeadItems) head[at] = i;
      a.rows[base + at++] = i;
    }
}

// The same from the library's expert-contiguous layout, whose rows are a.rows.
__global__ __launch_bounds__(64) void decode_heads_kernel(DecodeArgs a, const int32_t* offsets) {
  const int me = blockIdx.x, lane = lane_id(), lo = min(offsets[me], a.N), n = min(offsets[me + 1], a.N) - lo;
  a.heads[(size_t)me * 64 + lane] =
      lane < kHeadItems ? (lane < n ? a.rows[lo + lane] : 0) : lane == kHeadN ? n : lane == kHeadBase ? lo : me;
}

// ------------------------------------------------------------------ MXFP4 codes
// Rows of values -> E2M1 codes (element 2i in the low half of byte i) and E8M0
// scales per 32: shared exponent floor(log2 amax) - 2, nearest code, ties to
// even, saturating at +-6 (OCP Microscaling v1.0).  Weights, off the timed
// path.  A block with a value that is not finite gets scale 255 (NaN).
__device__ __forceinline__ uint32_t e2m1_code(float v, int sh) {
  const float y = __builtin_amdgcn_ldexpf(fabsf(v), -sh);
  const uint32_t m = (y > 0.25f) + (y >= 0.75f) + (y > 1.25f) + (y >= 1.75f) + (y > 2.5f) + (y >= 3.5f) + (y > 5.0f);
  return m | (__float_as_uint(v) >> 31 << 3);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void mxfp4_quantize_kernel(const T* src, uint8_t* codes, uint8_t* scales, int64_t units) {
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += (int64_t)gridDim.x * kThreads) {
    float v[8];
    load8(src + u * 8, v);
    int top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, (int)(__float_as_uint(v[i]) & 0x7FFFFFFFu));
    top = max(top, __shfl_xor(top, 1, 64));
    top = max(top, __shfl_xor(top, 2, 64));
    const bool fine = top < 0x7F800000;
    int sh = -127;
    if (fine && top > 0) sh = max(ilog2f(__uint_as_float((uint32_t)top)) - 2, -127);
    uint32_t w = 0;
    if (fine)
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= e2m1_code(v[i], sh) << (4 * i);
    *reinterpret_cast<uint32_t*>(codes + u * 4) = w;
    if ((u & 3) == 0) scales[u >> 2] = fine ? (uint8_t)(sh + 127) : 255;
  }
}

// Rows of codes and scales -> the order of mok_w4: a thread per 16 bytes of
// codes, and one per 4 scales.
__global__ __launch_bounds__(kThreads) void mxfp4_tile_kernel(const uint8_t* codes, const uint8_t* scales, uint8_t* codes_out,
                                                              uint8_t* scales_out, int64_t tiles, int64_t chunks) {
  const int64_t units = tiles * chunks * 64, groups = (chunks + 3) / 4, dwords = tiles * groups * 64;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < units; u += step) {
    const int lane = (int)(u % 64), r = lane & 15, g = lane >> 4;
    const int64_t c = u / 64 % chunks, tile = u / 64 / chunks;
    st16(codes_out + u * 16, ld16(codes + ((tile * 16 + r) * chunks + c) * 64 + 16 * g));
  }
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < dwords; u += step) {
    const int lane = (int)(u % 64), r = lane & 15, g = lane >> 4;
    const int64_t q = u / 64 % groups, tile = u / 64 / groups;
    uint32_t v = 0;
    for (int p = 0; p < 4; ++p)
      if (4 * q + p < chunks) v |= (uint32_t)scales[((tile * 16 + r) * chunks + 4 * q + p) * 4 + g] << (8 * p);
    *reinterpret_cast<uint32_t*>(scales_out + u * 4) = v;
  }
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct DecodeWs {
  size_t h, y, heads, rows, counts, offsets, dest_row, layout, total;
};
DecodeWs decode_ws(int64_t N, int d, int I, int E_local) {
  DecodeWs w;
  size_t at = 0;
  w.h = at;
  at += align256((size_t)N * I * 2);
  w.y = at;
  at += align256((size_t)N * d * 4);
  w.heads = at;
  at += align256((size_t)(N < E_local ? N : E_local) * 256);
  w.rows = at;
  at += align256((size_t)N * 4);
  const bool lay = N > kPlanItems;
  w.counts = at;
  if (lay) at += align256((size_t)E_local * 4);
  w.offsets = at;
  if (lay) at += align256((size_t)(E_local + 1) * 4);
  w.dest_row = at;
  if (lay) at += align256((size_t)N * 4);
  w.layout = at;
  if (lay) at += align256(layout_ws_bytes(N, E_local));
  w.total = at > 0 ? at : 256;
  return w;
}

}  // namespace

size_t decode_ws_bytes(int64_t N, int d, int I, int E_local) { return decode_ws(N, d, I, E_local).total; }

mok_status launch_decode(const DecodePlan& p, hipStream_t stream) {
  const int64_t N = (int64_t)p.T * p.k;
  if (N == 0) return MOK_OK;
  const DecodeWs ws = decode_ws(N, p.d, p.I, p.E_local);
  char* wsb = (char*)p.ws;
  DecodeArgs a;
  memset(&a, 0, sizeof(a));
  a.x = p.x, a.x_scale = p.x_scale, a.topk = p.topk, a.e2l = p.e2l;
  a.wg = p.w->w_gate, a.wu = p.w->w_up, a.wd = p.w->w_down;
  a.sg = p.w->s_gate, a.su = p.w->s_up, a.sd = p.w->s_down;
  a.h = (bf16_t*)(wsb + ws.h);
  a.y = (float*)(wsb + ws.y);
  a.heads = (int32_t*)(wsb + ws.heads);
  a.rows = (int32_t*)(wsb + ws.rows);
  a.status = p.status;
  a.N = (int)N, a.k = p.k, a.d = p.d, a.I = p.I, a.E = p.E, a.E_local = p.E_local;
  const int64_t slots = N < p.E_local ? N : p.E_local;
  const int cus = device_cus() > 0 ? device_cus() : 256;
  auto done = [&](const char* name) { trace_mark(p.tr, name, stream); };
  // few items, about 20 of them local: one token's, or some more of a share of
  // the experts (us, this path and the other, d 2048, 64 experts, top-6: 1 token
  // 12.4 and 17.9, 2 tokens 18.5 and 25.2, 3 tokens 24 and 27, 4 tokens 30.3 and
  // 28.7; d 7168, 256 experts, 8 tokens, top-8: 16 local 37 and 47, 64 local 78 and
  // 79, 100 local 108 and 99)
  if (N <= 64 && p.T <= 16 && N * p.E_local <= 20 * (int64_t)p.E) {
    const dim3 grid((unsigned)(slots * (p.I / 16)));
    if (p.x_scale) hipLaunchKernelGGL(decode_up_few_kernel<true>, grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL(decode_up_few_kernel<false>, grid, dim3(kThreads), 0, stream, a);
    done("decode_up_few");
    // one workgroup of 16 waves for each compute unit, or two of eight (8 tokens at
    // 32 of 256 experts, d 7168: 24.5 us, with 16 waves 27.8)
    if (p.d / 16 > cus) hipLaunchKernelGGL(decode_down_few_kernel<512>, dim3((unsigned)(p.d / 16)), dim3(512), 0, stream, a, p.gate, (bf16_t*)p.out);
    else hipLaunchKernelGGL(decode_down_few_kernel<1024>, dim3((unsigned)(p.d / 16)), dim3(1024), 0, stream, a, p.gate, (bf16_t*)p.out);
    done("decode_down_few");
    return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
  }
  if (N > kPlanItems) {
    int32_t* offsets = (int32_t*)(wsb + ws.offsets);
    const mok_status rc = launch_layout(N, p.E, p.E_local, (int)N, p.topk, p.e2l, (int32_t*)(wsb + ws.counts), offsets, a.rows,
                                        (int32_t*)(wsb + ws.dest_row), wsb + ws.layout, p.status, stream, p.tr);
    if (rc != MOK_OK) return rc;
    hipLaunchKernelGGL(decode_heads_kernel, dim3((unsigned)p.E_local), dim3(64), 0, stream, a, offsets);
    done("decode_heads");
  } else if (N > kLongListItems) {
    hipLaunchKernelGGL(decode_plan_kernel, dim3((unsigned)p.E_local), dim3(kPlanThreads), 0, stream, a);
    done("decode_plan");
  }
  // two groups of waves share the contraction where a workgroup per tile
  // leaves compute units with one or none
  const int64_t up = slots * (p.I / 64), down = slots * (p.d / 128);
  // and 256 columns of y a workgroup where that leaves two for each (61 tokens at
  // 64 experts: 21.7 us with 128 columns, 20.6)
  const int64_t items = N / p.E;         // of an expert, about
  const bool wide = p.d % 256 == 0 && down / 2 >= 2 * cus && items <= 32;
  auto launch = [&](auto one, auto two, auto more, int64_t tiles, const char* name) {
    // few columns and many items an expert: workgroups share the items too, as
    // long as that fills the chip and not more (each reads the weights; 200 tokens,
    // top-8 of 8 experts of 1024 x 512: 22.7 us, without 63).  64 items at a time,
    // with two workgroups for each compute unit, where that fills it (512 tokens at
    // 64 experts: 111 us, with 32 128; 512 at 2 of them 38 and 31; 512, top-8 at 8
    // experts of 7168 x 2048: 397 us, 909 TFLOP/s, with 32 461)
    const int64_t sets = (items + 31) / 32, sets64 = (items + 63) / 64;
    const bool many = items > 32 && tiles * sets64 >= 2 * cus;
    const int64_t most = many ? sets64 : sets, room = (many ? 2 : 3) * cus / tiles;
    a.splits = (int)(most < room ? most : room);
    if (a.splits < 1) a.splits = 1;
    tiles *= a.splits;
    if (many) hipLaunchKernelGGL(more, dim3((unsigned)tiles), dim3(kThreads), 0, stream, a);
    else if (2 * tiles < 3 * cus) hipLaunchKernelGGL(two, dim3((unsigned)tiles), dim3(2 * kThreads), 0, stream, a);
    else hipLaunchKernelGGL(one, dim3((unsigned)tiles), dim3(kThreads), 0, stream, a);
    done(name);
  };
#define MOK_DECODE_UP(FIND, MANY, X8)                                                                        \
  launch(decode_kernel<false, FIND, 1, 1, X8, 2>, decode_kernel<false, FIND, 1, 2, X8, 2>,                   \
         decode_kernel<false, MANY, 1, 1, X8, 4>, up, "decode_gate_up")
  if (N <= kListItems && p.x_scale) MOK_DECODE_UP(kSearch, kSearchLong, true);
  else if (N <= kListItems) MOK_DECODE_UP(kSearch, kSearchLong, false);
  else if (N <= kLongListItems && p.x_scale) MOK_DECODE_UP(kSearchLong, kSearchLong, true);
  else if (N <= kLongListItems) MOK_DECODE_UP(kSearchLong, kSearchLong, false);
  else if (p.x_scale) MOK_DECODE_UP(kHeads, kHeads, true);
  else MOK_DECODE_UP(kHeads, kHeads, false);
#undef MOK_DECODE_UP
  const auto four = decode_kernel<true, kHeads, 4, 1, false, 2>;
  if (wide) launch(four, four, four, down / 2, "decode_down");
  else launch(decode_kernel<true, kHeads, 2, 1, false, 2>, decode_kernel<true, kHeads, 2, 2, false, 2>,
              decode_kernel<true, kHeads, 2, 1, false, 4>, down, "decode_down");
  const int pieces = (p.d / 8 + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(decode_combine_kernel, dim3((unsigned)((int64_t)p.T * pieces)), dim3(kThreads), 0, stream, a, p.gate,
                     (bf16_t*)p.out, pieces);
  trace_mark(p.tr, "decode_combine", stream);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

mok_status launch_mxfp4_quantize(int64_t rows, int64_t K, int type, const void* src, uint8_t* codes, uint8_t* scales,
                                 hipStream_t stream) {
  const int64_t units = rows * (K / 8), need = (units + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(need < 8192 ? need : 8192));
  if (type == MOK_F32)
    hipLaunchKernelGGL(mxfp4_quantize_kernel<float>, grid, dim3(kThreads), 0, stream, (const float*)src, codes, scales, units);
  else
    hipLaunchKernelGGL(mxfp4_quantize_kernel<bf16_t>, grid, dim3(kThreads), 0, stream, (const bf16_t*)src, codes, scales, units);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

mok_status launch_mxfp4_tile(int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales, uint8_t* codes_out,
                             uint8_t* scales_out, hipStream_t stream) {
  const int64_t need = (rows / 16 * (K / kChunk) * 64 + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(mxfp4_tile_kernel, dim3((unsigned)(need < 8192 ? need : 8192)), dim3(kThreads), 0, stream, codes,
                     scales, codes_out, scales_out, rows / 16, K / kChunk);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

}  // namespace mok
