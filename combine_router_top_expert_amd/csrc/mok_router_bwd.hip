// Backward of the router projection z = x W^T + bias for a dense gradient dz
// of the logits:
//   dx[t][n] = sum_e dz[t][e] W[e][n]      (contraction over the experts)
//   dW[e][n] = sum_t dz[t][e] x[t][n]      (contraction over the tokens)
//   db[e]    = sum_t dz[t][e]
//
// fp32 layers: both products on the fp32 matrix cores
// (v_mfma_f32_32x32x2_f32), whose operands hold one k per lane, so operands
// that are strided along k need no transpose.
//
// bf16 layers: x and W are bf16, dz is fp32.  A fp32 value is the sum of
// three bf16 parts (hi = bf16(v), mid = bf16(v - hi), lo = bf16(v - hi -
// mid): 8 bits each, exact in between), so the products run on the bf16
// matrix cores, eight times the fp32 rate, once per part: dz is exact in both
// products, whose sums are fp32.  (Two parts are not enough for dx either,
// though it is rounded to bf16: rows of dz that sum to about zero cancel what
// the rows of W have in common, and the third part is what is left.)
//   1. router_split_kernel writes the parts of dz once (and sums db);
//   2. dx: a wave keeps the parts of its 32 token rows in registers for up to
//      128 experts (256 above 256) and walks column steps of 64, W coming
//      through LDS; above 128 experts two waves share the rows, half of the
//      experts each, and exchange halves of their sums;
//   3. dW: 64 x 64 of dW per wave, both operands through an LDS ring filled by
//      direct loads, split over the tokens; beside dx in one launch;
//   4. router_reduce_kernel adds the token chunks in order.
//
// What bounds it.  16384 x 2048 x 64: HBM (x read, d_x written, 67 MB each):
// split 6 us, both products 33, reduction 5.  4096 x 7168 x 256, added: the
// matrix cores, 90 GFLOP in six parts: split 6 us, both products 95 (0.95
// PFLOP/s; a large library product reaches 1.23), reduction 9.  fp32, 512 x
// 256 x 8: launch latency, 7 + 3 us; 4096 x 7168 x 256: 306 us call after
// call, 98 TFLOP/s of the 154 that a library product reaches (vector work for
// addresses and LDS stores beside the matrix cores, which are 68 % busy).
#include <math.h>

#include <algorithm>

#include "mok_gemm2.h"
#include "mok_internal.h"

namespace mok {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;   // fp32: tile side
constexpr int kKB = 16;     // and contraction steps staged through LDS at a time (32: up to 12 % slower, with half the waves)
constexpr int kPitch = kTile + 4;
constexpr int kDxWaves = 4;
constexpr int kDwWaves = 4;         // dW: two workgroups per CU (one of eight waves took a tenth longer in a launch of its own)
constexpr int kBf16Threads = 64 * kDwWaves;
constexpr int kBK = 16;             // token rows per LDS stage of dW

struct RArgs {
  const float* dz;
  const void* w;
  SrcTable x;
  DstTable d_x;
  float* dw;
  float* db;
  float* part;     // [chunks][E][d] partial dW, or null: one chunk, straight into dw
  double* dbp;     // [chunks][E]
  int T, T_src, d, E, own_lo, chunks;
  int64_t chunk_rows;
  int add;
  // bf16: the parts of dz in 1 KiB blocks of 32 tokens x 16 experts,
  // [T / 32][3 parts][E / 16] of [expert / 8 % 2][token % 32][expert % 8]: a
  // block is one MFMA operand of dx as it lies, and half of its tokens are
  // four 256-byte pieces of a dW stage; padded with zeros to whole blocks
  // and expert tiles
  bf16_t* parts;
  int ew, etiles;      // experts per tile (64, 128 or 256) and tiles
  int eblocks;         // blocks of 16 experts in the parts
  int64_t split_rows;  // token rows per workgroup of the split
  int db_parts;        // partial sums of db per expert
  int n_chunks;        // column chunks of dx, each a workgroup per row block
};

// row of accumulator register r in a 32 x 32 block (its column is lane % 32)
__device__ __forceinline__ int acc_row(int r, int lane) { return (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3); }

// ------------------------------------------------------------------ fp32
// Both products as C[m][n] = sum_k A(k, m) B(k, n) on 64 x 64 tiles, four
// waves of 32 x 32 (128 x 128 measured no faster).  kKB steps of k at a time
// go through LDS as [k][m] and [k][n]; the next block's global loads are in
// registers while this one is multiplied.  dx: m = token, k = expert (dz
// read along k); dW: m = expert, k = token.
template <bool DX>
__device__ __forceinline__ void f32_tile(const RArgs& a, int m0, int n0, int k_lo, int k_hi, int chunk, float* smem) {
  constexpr int NU = kTile * kKB / 4 / kThreads;   // 16-byte units per thread and operand
  constexpr int BUF = 2 * kKB * kPitch;            // two LDS buffers, one barrier a block
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const bool wide = a.E % 4 == 0 && ((uintptr_t)a.dz & 15) == 0;
  const float* w = reinterpret_cast<const float*>(a.w);
  float4 ra[NU], rb[NU];
  auto dz4 = [&](int t, int e) {  // four experts of a token, zeros past E
    const float* p = a.dz + (size_t)t * a.E + e;
    if (wide) return e < a.E ? *reinterpret_cast<const float4*>(p) : make_float4(0, 0, 0, 0);
    return make_float4(e < a.E ? p[0] : 0.0f, e + 1 < a.E ? p[1] : 0.0f, e + 2 < a.E ? p[2] : 0.0f,
                       e + 3 < a.E ? p[3] : 0.0f);
  };
  auto fetch = [&](int k0) {
    // the block's tokens usually come from one source: one division for all
    const int src = DX ? 0 : k0 / a.T_src, row = DX ? 0 : k0 % a.T_src;
    const float* xb = nullptr;
    if (!DX && a.dw && row + kKB <= a.T_src)
      xb = reinterpret_cast<const float*>(a.x.p[a.own_lo + src]) + (size_t)row * a.d + n0;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = tid + i * kThreads;
      const int kr = u / (kTile / 4), c = u % (kTile / 4) * 4;   // k-row and column of an operand with k rows
      const bool there = k0 + kr < k_hi;
      ra[i] = rb[i] = make_float4(0, 0, 0, 0);
      if constexpr (DX) {
        const int t = m0 + u / (kKB / 4), e = k0 + u % (kKB / 4) * 4;
        if (t < a.T) ra[i] = dz4(t, e);
        if (there) rb[i] = *reinterpret_cast<const float4*>(w + (size_t)(k0 + kr) * a.d + n0 + c);
      } else if (there) {
        const int t = k0 + kr;
        ra[i] = dz4(t, m0 + c);
        if (xb) rb[i] = *reinterpret_cast<const float4*>(xb + (size_t)kr * a.d + c);
        else if (a.dw)
          rb[i] = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.x.p[a.own_lo + t / a.T_src]) +
                                                   (size_t)(t % a.T_src) * a.d + n0 + c);
      }
    }
  };
  auto deposit = [&](float* sA, float* sB) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = tid + i * kThreads;
      const int kr = u / (kTile / 4), c = u % (kTile / 4) * 4;
      if constexpr (DX) {
        const int m = u / (kKB / 4), k = u % (kKB / 4) * 4;
        sA[k * kPitch + m] = ra[i].x;
        sA[(k + 1) * kPitch + m] = ra[i].y;
        sA[(k + 2) * kPitch + m] = ra[i].z;
        sA[(k + 3) * kPitch + m] = ra[i].w;
      } else {
        *reinterpret_cast<float4*>(sA + kr * kPitch + c) = ra[i];
      }
      *reinterpret_cast<float4*>(sB + kr * kPitch + c) = rb[i];
    }
  };
  const bool bias = !DX && a.db && n0 == 0 && tid < kTile;
  double bsum = 0.0;
  f32x16_t acc = {};
  const int c = lane & 31, h = lane >> 5;
  if (k_lo < k_hi) fetch(k_lo);
  for (int k0 = k_lo, buf = 0; k0 < k_hi; k0 += kKB, buf ^= 1) {
    // a buffer's readers of two blocks ago have passed the last barrier
    float* sA = smem + buf * BUF;
    float* sB = sA + kKB * kPitch;
    deposit(sA, sB);
    __syncthreads();
    if (k_hi - k0 > kKB) fetch(k0 + kKB);
#pragma unroll
    for (int k = 0; k < kKB; k += 2)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sA[(k + h) * kPitch + wm + c], sB[(k + h) * kPitch + wn + c], acc, 0, 0, 0);
    if (bias)
      for (int k = 0; k < kKB; ++k) bsum += (double)sA[k * kPitch + tid];
  }
  const int n = n0 + wn + c;   // d is a multiple of the tile
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int m = m0 + wm + acc_row(r, lane);
    if (m >= (DX ? a.T : a.E)) continue;
    float* row = nullptr;
    if constexpr (DX) row = reinterpret_cast<float*>(a.d_x.p[a.own_lo + m / a.T_src]) + (size_t)(m % a.T_src) * a.d;
    else if (a.part) row = a.part + ((size_t)chunk * a.E + m) * a.d;
    else if (a.dw) row = a.dw + (size_t)m * a.d;
    if (row) row[n] = a.add && (DX || !a.part) ? row[n] + acc[r] : acc[r];
  }
  if (bias && m0 + tid < a.E) {
    const int e = m0 + tid;
    if (a.dbp) a.dbp[(size_t)chunk * a.E + e] = bsum;
    else a.db[e] = (float)(a.add ? a.db[e] + bsum : bsum);
  }
}

// The tiles of both products in one launch: the first dw_tiles workgroups dW
// (chunk by chunk of tokens: the longer ones), the others dx.
__global__ __launch_bounds__(kThreads) void router_f32_kernel(RArgs a, int64_t dw_tiles) {
  __shared__ __attribute__((aligned(16))) float smem[4 * kKB * kPitch];
  const int nt = a.d / kTile;
  int64_t b = blockIdx.x;
  if (b >= dw_tiles) {
    b -= dw_tiles;
    f32_tile<true>(a, (int)(b / nt) * kTile, (int)(b % nt) * kTile, 0, a.E, 0, smem);
    return;
  }
  const int n = a.dw ? nt : 1, me = (a.E + kTile - 1) / kTile, tile = (int)(b % (n * me)), chunk = (int)(b / (n * me));
  const int64_t lo = (int64_t)chunk * a.chunk_rows;
  f32_tile<false>(a, tile / n * kTile, tile % n * kTile, (int)min(lo, (int64_t)a.T),
                  (int)min(lo + a.chunk_rows, (int64_t)a.T), chunk, smem);
}

// ------------------------------------------------------------------ bf16: split
// Workgroup: split_rows token rows (whole blocks of 32) of four expert
// blocks, one a wave; lane l token l % 32 and 8 experts of half l / 32, so a
// wave reads 64 bytes of 32 rows and writes whole blocks.  The column sums of
// db stay in registers (64 bits) over the rows, then over the 32 lanes.
__global__ __launch_bounds__(kThreads) void router_split_kernel(RArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tl = lane & 31, half = lane >> 5;
  const bool wide = a.E % 4 == 0 && ((uintptr_t)a.dz & 15) == 0;
  const int64_t lo = (int64_t)blockIdx.x * a.split_rows;
  const int64_t hi = lo + a.split_rows < a.T ? lo + a.split_rows : a.T;
  const int eb = blockIdx.y * (kThreads / 64) + wave;   // eblocks is a multiple of 4
  {
    const int e0 = eb * 16 + half * 8;
    double db[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) db[j] = 0.0;
#pragma unroll 2
    for (int64_t t0 = lo; t0 < hi; t0 += 32) {
      const int64_t t = t0 + tl;
      float v[8];
      const float* row = a.dz + (size_t)t * a.E + e0;
      if (wide) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float4 u = make_float4(0, 0, 0, 0);
          if (t < hi && e0 + 4 * h < a.E) u = *reinterpret_cast<const float4*>(row + 4 * h);
          v[4 * h] = u.x, v[4 * h + 1] = u.y, v[4 * h + 2] = u.z, v[4 * h + 3] = u.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = t < hi && e0 + j < a.E ? row[j] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) db[j] += (double)v[j];
      if (a.parts) {
        bf16_t* o = a.parts + ((size_t)(t0 / 32) * 3 * a.eblocks + eb) * 512 + lane * 8;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] = pack2_bf16(v[2 * j], v[2 * j + 1]);
            v[2 * j] -= __uint_as_float(w[j] << 16);
            v[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
          }
          st16(o + (size_t)p * a.eblocks * 512, make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
    }
    if (!a.db) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) db[j] += __shfl_xor(db[j], o, 64);
      if (tl != 0 || e0 + j >= a.E) continue;
      if (a.dbp) a.dbp[(size_t)blockIdx.x * a.E + e0 + j] = db[j];
      else a.db[e0 + j] = (float)(a.add ? a.db[e0 + j] + db[j] : db[j]);   // the only partial sum
    }
  }
}

// s_barrier for every wave's own LDS work and direct loads: no LDS access
// moves across it.
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// This wave's LDS work, and with LOADS its direct loads, are done; no access
// moves across it.
template <bool LOADS>
__device__ __forceinline__ void complete() {
  if constexpr (LOADS) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// ------------------------------------------------------------------ bf16: dx
// Fragment of 32 columns from n (k = 16 s ..) of an LDS tile of 64 columns
// (128-byte k-rows) read with ds_read_b64_tr_b16: in a 16-lane group lane a
// points at (k + a/4, n + 4 (a%4)) and lane i receives k..k+3 of column n + i.
// Chunk c (16 bytes) of k-row r sits at c ^ 4 ((r / 2) & 1): four consecutive
// k-rows of one column range then cover all banks.
__device__ __forceinline__ bf16x8_t frag64(const char* lds, int n0, int s) {
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const int n = n0 + 16 * (g & 1) + 4 * (li & 3), kb = 16 * s + 8 * (g >> 1) + (li >> 2);
  g2::v4s h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int kr = kb + 4 * i, c = (n >> 3) ^ (4 * ((kr >> 1) & 1));
    h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((g2::lds_v4s*)(lds + kr * 128 + c * 16 + (n & 7) * 2));
  }
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// NK: 16-expert steps (E <= 16 NK); KS: waves that share 32 token rows, each
// with NK / KS of the steps (three parts of 16 steps are all the registers of
// a wave where two workgroups share a CU).  Four waves, two workgroups per CU
// up to NK = 16 (one computes while the other stores).  STREAM: nontemporal
// stores of d_x.
template <int NK>
constexpr int dx_split() { return NK >= 16 ? 2 : 1; }
template <int NK>
constexpr int dx_rows() { return 32 * kDxWaves / dx_split<NK>(); }
template <int NK>
constexpr int dx_lds() { return 2 * NK * 16 * 128 + dx_rows<NK>() / 32 * 4096; }

template <int NK, bool STREAM>
__device__ __forceinline__ void dx_bf16(const RArgs& a, int b, char* smem) {
  constexpr int KS = dx_split<NK>(), NKW = NK / KS, ROWS = dx_rows<NK>();
  constexpr int STAGE = NK * 16 * 128;               // bytes of W per column step
  constexpr int LOADS = STAGE / 1024 / kDxWaves;     // direct loads per wave and step
  static_assert(KS == 1 || STAGE >= kDxWaves * 4096, "the exchange takes a stage of W");
  const int lane = threadIdx.x & 63;
  const int wave = (int)g2::wave_id();
  const int rg = wave / KS, kh = wave % KS;          // row group, part of the experts
  // workgroups of one row block on one XCD (b % 8), so its parts meet in an L2
  const int rb_n = (a.T + ROWS - 1) / ROWS;
  int rb, ch;
  const int full = rb_n / 8 * 8 * a.n_chunks;
  if (b < full) {
    rb = b % 8 + 8 * (b / 8 / a.n_chunks);
    ch = b / 8 % a.n_chunks;
  } else {
    b -= full;
    rb = rb_n / 8 * 8 + b / a.n_chunks;
    ch = b % a.n_chunks;
  }
  const int steps = a.d / 64;
  const int s0 = (int)((int64_t)steps * ch / a.n_chunks), s1 = (int)((int64_t)steps * (ch + 1) / a.n_chunks);
  const bf16_t* w = reinterpret_cast<const bf16_t*>(a.w);
  const unsigned lds0 = g2::lds_addr_of(smem);
  // this wave's direct loads: source of column 0, or the zero page past E
  const char* wp[LOADS];
  int adv[LOADS];
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int row = (wave * LOADS + j) * 8 + lane / 8;
    const int c = (lane % 8) ^ (4 * ((row >> 1) & 1));
    const bool there = row < a.E;
    wp[j] = there ? reinterpret_cast<const char*>(w + (size_t)row * a.d + c * 8)
                  : reinterpret_cast<const char*>(g2::g_zero);
    adv[j] = there ? 128 : 0;
  }
  auto issue = [&](int s, int slot) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      g2::load_lds16(wp[j] + (size_t)s * adv[j], lds0 + slot * STAGE + (wave * LOADS + j) * 1024);
  };
  if (s0 < s1) issue(s0, 0);
  // the wave's rows: all parts of its experts, in registers
  const int t0 = rb * ROWS + rg * 32;
  bf16x8_t part[3][NKW];
  {
    const bool there = t0 < a.T;
    const bf16_t* p = a.parts + ((size_t)(t0 / 32) * 3 * a.eblocks + kh * NKW) * 512 + lane * 8;
#pragma unroll
    for (int k = 0; k < NKW; ++k)
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (there) u = ld16(p + ((size_t)q * a.eblocks + k) * 512);
        part[q][k] = __builtin_bit_cast(bf16x8_t, u);
      }
  }
  // the rows this lane stores: 8 lanes per row, 4 / KS rows from row 32 / KS
  // kh of the row group; chunk c of a staged row (128 bytes) sits at c ^ (row
  // & 7), so this lane's chunk of row 8 i + lane / 8 is LDS position 64 i +
  // lane for the column chunk below
  const int col = ((lane % 8) ^ (lane / 8)) * 8;
  bf16_t* out[4 / KS];
#pragma unroll
  for (int i = 0; i < 4 / KS; ++i) {
    const int t = t0 + 32 / KS * kh + 8 * i + lane / 8;
    out[i] = t < a.T ? reinterpret_cast<bf16_t*>(a.d_x.p[a.own_lo + t / a.T_src]) + (size_t)(t % a.T_src) * a.d + col
                     : nullptr;
  }
  char* stg = smem + 2 * STAGE + rg * 4096;                      // the row group's tile
  const int stg_own = 4096 / KS * kh;                            // the rows that this wave stores
  const unsigned stg_lds = lds0 + 2 * STAGE + rg * 4096 + stg_own;
  auto store = [&](int s) {  // the staged tile of column step s
    uint4 u[4 / KS];
#pragma unroll
    for (int i = 0; i < 4 / KS; ++i) u[i] = *reinterpret_cast<const uint4*>(stg + stg_own + i * 1024 + lane * 16);
#pragma unroll
    for (int i = 0; i < 4 / KS; ++i)
      if (out[i]) {
        if constexpr (STREAM)
          __builtin_nontemporal_store(__builtin_bit_cast(i32x4_t, u[i]), reinterpret_cast<i32x4_t*>(out[i] + (size_t)s * 64));
        else
          st16(out[i] + (size_t)s * 64, u[i]);
      }
  };
  for (int s = s0; s < s1; ++s) {
    // this wave's loads of step s (and its stores of the step before last)
    // are done, everyone's are after the barrier; everyone has also left the
    // buffer that step s + 1 will fill
    g2::wait_vmcnt_lgkm0<0>();
    barrier();
    const int slot = (s - s0) & 1;
    if (s + 1 < s1) issue(s + 1, slot ^ 1);
    if (s > s0) store(s - 1);
    if (a.add) {
      // what d_x holds goes straight into the staging rows, which store()
      // has read into registers by now
      g2::wave_lds_fence();
#pragma unroll
      for (int i = 0; i < 4 / KS; ++i)
        g2::load_lds16(out[i] ? (const void*)(out[i] + (size_t)s * 64) : (const void*)g2::g_zero, stg_lds + i * 1024);
    }
    const char* W = smem + slot * STAGE + kh * NKW * 16 * 128;
    f32x16_t acc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][r] = 0.0f;
    // fragments are read kAhead k16 steps before their use; acc[0] holds
    // columns 32 kh.., acc[1] the other 32
    constexpr int kAhead = 2;
    bf16x8_t f[kAhead + 1][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) f[k][j] = frag64(W, 32 * (j ^ kh), k);
    __builtin_amdgcn_sched_group_barrier(0x100, 4 * kAhead, 0);
#pragma unroll
    for (int k = 0; k < NKW; ++k) {
      if (k + kAhead < NKW) {
#pragma unroll
        for (int j = 0; j < 2; ++j) f[(k + kAhead) % (kAhead + 1)][j] = frag64(W, 32 * (j ^ kh), k + kAhead);
      }
#pragma unroll
      for (int q = 2; q >= 0; --q)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[k % (kAhead + 1)][j], part[q][k], acc[j], 0, 0, 0);
      if (k + kAhead < NKW) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 6, 0);
    }
    if constexpr (KS == 2) {
      // This step's W is read by all behind the first barrier, so its buffer
      // takes the exchange: a wave gives acc[1] to the one with the other
      // experts of its rows and adds what that one gives.  Behind the second
      // barrier the pair's base rows are in place too.
      complete<false>();
      barrier();
      f32x4_t* ex = reinterpret_cast<f32x4_t*>(smem + slot * STAGE);
#pragma unroll
      for (int g = 0; g < 4; ++g)
        ex[(wave * 4 + g) * 64 + lane] = f32x4_t{acc[1][4 * g], acc[1][4 * g + 1], acc[1][4 * g + 2], acc[1][4 * g + 3]};
      if (a.add) complete<true>();
      else complete<false>();
      barrier();
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t o = ex[((wave ^ 1) * 4 + g) * 64 + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[0][4 * g + i] += o[i];
      }
    } else {
      if (a.add) g2::wait_vmcnt_lgkm0<0>();
      asm volatile("" ::: "memory");
    }
    // lane holds row lane % 32, columns 32 (j ^ kh) + 8 g + 4 (lane / 32) + 0..3
    const int r = lane & 31;
#pragma unroll
    for (int j = 0; j < 2 / KS; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = 32 * (j ^ kh) + 8 * g + 4 * (lane >> 5);
        uint2* p = reinterpret_cast<uint2*>(stg + r * 128 + ((c >> 3) ^ (r & 7)) * 16 + (c & 7) * 2);
        float v[4] = {acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
        if (a.add) {
          const uint2 u = *p;
          v[0] += __uint_as_float(u.x << 16), v[1] += __uint_as_float(u.x & 0xFFFF0000u);
          v[2] += __uint_as_float(u.y << 16), v[3] += __uint_as_float(u.y & 0xFFFF0000u);
        }
        *p = g2::pack4_bf16(v[0], v[1], v[2], v[3]);
      }
    if constexpr (KS == 2) complete<false>();
    else g2::wave_lds_fence();
  }
  if (KS == 2) barrier();   // the other wave's half of the staged rows
  if (s0 < s1) store(s1 - 1);
}

// ------------------------------------------------------------------ bf16: dW
// Tile EW experts x EN columns, four waves of 64 x 64; LDS ring of NS stages
// of 16 token rows, each [3 parts][EW / 16 expert blocks of 512 bytes | 16
// rows of EN columns of x].  Both operands are read with ds_read_b64_tr_b16:
// in a 16-lane group lane a points at 8 bytes of token k + a/4, columns n + 4
// (a%4)..+3, and lane i receives tokens k..k+3 of column n + i.  Placement so
// that a half wave covers all banks: 16-byte chunk c of x row r at c ^ 4 (r &
// 3); chunk (half h, token t) of expert block b at 16 h + (t + 4 h + 8 b) %
// 16.
template <int EW>
struct DwCfg {
  static constexpr int WE = EW / 64, WN = kDwWaves / WE;
  static constexpr int EN = 64 * WN;
  static constexpr int RB = 2 * EN;                    // bytes of a row of x
  static constexpr int A_BYTES = 3 * EW / 16 * 512, STAGE = A_BYTES + kBK * RB;
  static constexpr int LDS = 160 * 1024 * kDwWaves / 8 - 1024;     // eight waves per CU
  static constexpr int NS = LDS / STAGE > 6 ? 6 : LDS / STAGE;
  static constexpr int UNITS = STAGE / 1024;           // 1 KiB direct loads per stage
  static constexpr int Q = UNITS / kDwWaves, X = UNITS % kDwWaves;   // per wave; waves below X issue one more
  static_assert(STAGE % 1024 == 0 && A_BYTES % 1024 == 0 && NS >= 3, "ring");
};

__device__ __forceinline__ bf16x8_t frag_x(const char* lds, int rb, int n0) {
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const int n = n0 + 16 * (g & 1) + 4 * (li & 3), kb = 8 * (g >> 1) + (li >> 2);
  g2::v4s h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int kr = kb + 4 * i, c = (n >> 3) ^ (4 * (kr & 3));
    h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((g2::lds_v4s*)(lds + kr * rb + c * 16 + (n & 7) * 2));
  }
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}
// 32 experts from block eb (even) of a part
__device__ __forceinline__ bf16x8_t frag_parts(const char* lds, int eb) {
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const int b = g & 1, half = (li & 3) >> 1, t = 8 * (g >> 1) + (li >> 2);
  const char* base = lds + (eb + b) * 512 + half * 256 + (li & 1) * 8;
  g2::v4s h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((g2::lds_v4s*)(base + ((t + 4 * i + 4 * half + 8 * b) & 15) * 16));
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// One direct load (lane i's 16 bytes land at LDS byte lds + 16 i) from a
// uniform base and a lane offset; lds is wave-uniform.
__device__ __forceinline__ void load_lds16_at(const char* base, unsigned off, unsigned lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}

template <int EW>
constexpr int dw_lds() { return DwCfg<EW>::NS * DwCfg<EW>::STAGE + MOK_MAX_SOURCES * 8; }

template <int EW>
__device__ __forceinline__ void dw_bf16(const RArgs& a, int b, char* smem) {
  typedef DwCfg<EW> C;
  const bf16_t** s_x = reinterpret_cast<const bf16_t**>(smem + C::NS * C::STAGE);
  const int lane = threadIdx.x & 63;
  const int wave = (int)g2::wave_id();
  // a token chunk's tiles on one XCD (b % 8) while the chunks fill whole
  // rounds of eight: its parts are then read from one L2
  const int ntn = (a.d + C::EN - 1) / C::EN, per = ntn * a.etiles;
  int chunk, tile;
  const int full = a.chunks / 8 * 8 * per;
  if (b < full) {
    chunk = b % 8 + 8 * (b / 8 / per);
    tile = b / 8 % per;
  } else {
    b -= full;
    const int left = a.chunks - a.chunks / 8 * 8;
    chunk = a.chunks / 8 * 8 + b % left;
    tile = b / left;
  }
  const int et = tile / ntn, n0 = tile % ntn * C::EN;
  for (int i = threadIdx.x; i < MOK_MAX_SOURCES; i += kBf16Threads) s_x[i] = reinterpret_cast<const bf16_t*>(a.x.p[i]);
  __syncthreads();
  const int64_t lo64 = (int64_t)chunk * a.chunk_rows;
  const int lo = (int)min(lo64, (int64_t)a.T), hi = (int)min(lo64 + a.chunk_rows, (int64_t)a.T);
  const int KT = (hi - lo + kBK - 1) / kBK;
  const unsigned lds0 = g2::lds_addr_of(smem);
  // This wave's units w, w + 8, ... of a stage: unit u is LDS bytes
  // [1024 u, 1024 u + 1024), 16-byte positions 64 u + lane.  voff: the lane's
  // byte offset from the stage's first block of parts (or row of x).
  constexpr int QM = C::Q + (C::X ? 1 : 0);
  const int nq = C::Q + (wave < C::X ? 1 : 0);
  unsigned voff[QM];
  int krow[QM];   // x units: the row of the stage
#pragma unroll
  for (int j = 0; j < QM; ++j) {
    const int u = wave + kDwWaves * j;
    if (u * 1024 < C::A_BYTES) {
      const int p = u / (EW / 32), eb = 2 * (u % (EW / 32)) + lane / 32, q = lane % 32;
      const int h = q / 16, t = (q - 4 * h - 8 * (eb & 1)) & 15;
      krow[j] = 0;
      voff[j] = (unsigned)(p * a.eblocks + et * (EW / 16) + eb) * 1024 + h * 512 + t * 16;
    } else {
      const int pos = (u * 1024 - C::A_BYTES) / 16 + lane;
      krow[j] = pos / (C::RB / 16);
      int c = ((pos % (C::RB / 16)) ^ (4 * (krow[j] & 3))) * 8;
      if (n0 + c >= a.d) c = 0;   // past d any column will do: its sums are not stored
      voff[j] = (unsigned)(krow[j] * a.d + c) * 2;
    }
  }
  // The next stage to fill, all uniform: its first token, its block of parts,
  // its first row of x (source xs, row xt), its slot.  Kept as running
  // values: recomputed per stage they stood between the barrier and the
  // matrix work, with a scalar load among them.
  auto x_at = [&](int src, int row) {
    return reinterpret_cast<const char*>(reinterpret_cast<const bf16_t*>(a.x.p[a.own_lo + src]) + (size_t)row * a.d + n0);
  };
  const size_t block = (size_t)3 * a.eblocks * 1024, x_step = (size_t)kBK * a.d * 2;
  int t0 = lo, xs = lo / a.T_src, xt = lo % a.T_src, left = KT;
  const char* pa = reinterpret_cast<const char*>(a.parts) + (size_t)(t0 / 32) * block + t0 / 16 % 2 * 256;
  const char* px = KT > 0 ? x_at(xs, xt) : nullptr;
  unsigned slot = lds0;
  auto issue = [&]() {
    if (t0 + kBK <= hi && xt + kBK <= a.T_src) {
      // sixteen rows of one source: uniform bases, no address arithmetic
#pragma unroll
      for (int j = 0; j < QM; ++j) {
        if (j >= nq) continue;                          // wave-uniform
        const unsigned u = (wave + kDwWaves * j) * 1024;
        load_lds16_at(u < C::A_BYTES ? pa : px, voff[j], slot + u);
      }
    } else {
      // the last rows, or rows of several sources: row by row, zeros past hi
#pragma unroll
      for (int j = 0; j < QM; ++j) {
        if (j >= nq) continue;
        const unsigned u = (wave + kDwWaves * j) * 1024;
        if (u < C::A_BYTES) {
          load_lds16_at(pa, voff[j], slot + u);
          continue;
        }
        const int t = t0 + krow[j];
        const char* src = reinterpret_cast<const char*>(g2::g_zero);
        if (t < hi)
          src = reinterpret_cast<const char*>(s_x[a.own_lo + t / a.T_src] + (size_t)(t % a.T_src) * a.d + n0) +
                (voff[j] - (unsigned)krow[j] * a.d * 2);
        g2::load_lds16(src, slot + u);
      }
    }
    slot = slot + C::STAGE == lds0 + C::NS * C::STAGE ? lds0 : slot + C::STAGE;
    // past the last stage its tokens are loaded again into slots that nothing
    // reads, so that every stage counts as many loads
    if (--left > 0) {
      t0 += kBK;
      pa += t0 & 16 ? 256 : block - 256;
      xt += kBK;
      px += x_step;
      if (xt >= a.T_src) {
        xs += xt / a.T_src;
        xt %= a.T_src;
        px = x_at(xs, xt);
      }
    }
  };
  f32x16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int we = wave / C::WN * 64, wn = wave % C::WN * 64;
  struct Frags {
    bf16x8_t a[3][2], b[2];
  };
  auto read = [&](int kt, Frags& f) {
    const char* A = smem + kt % C::NS * C::STAGE;
    const char* B = A + C::A_BYTES;
#pragma unroll
    for (int j = 0; j < 2; ++j) f.b[j] = frag_x(B, C::RB, wn + 32 * j);
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
      for (int i = 0; i < 2; ++i) f.a[p][i] = frag_parts(A + p * (EW / 16) * 512, we / 16 + 2 * i);
  };
  auto stage = [&](int kt, const Frags& f, Frags& next) {
    // this wave's loads of stage kt + 1 have landed (NS - 2 later stages stay
    // in flight) and its fragments of stage kt are in registers; after the
    // barrier that holds for everyone, so stage kt's slot can be filled again
    // and the next fragments are read under this stage's matrix work
    if (wave < C::X) g2::wait_vmcnt_lgkm0<(C::NS - 2) * (C::Q + 1)>();
    else g2::wait_vmcnt_lgkm0<(C::NS - 2) * C::Q>();
    barrier();
    read(kt + 1, next);
    auto mma = [&](int p) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[p][i], f.b[j], acc[i][j], 0, 0, 0);
    };
    mma(2);
    g2::interleave_reads<4, 16, 0, 4>();
    issue();
    mma(1);
    mma(0);
  };
  if (KT > 0) {
    for (int s = 0; s < C::NS; ++s) issue();
    if (wave < C::X) g2::wait_vmcnt_lgkm0<(C::NS - 1) * (C::Q + 1)>();
    else g2::wait_vmcnt_lgkm0<(C::NS - 1) * C::Q>();
    barrier();
    Frags f0, f1;
    read(0, f0);
    int kt = 0;
    for (; kt + 1 < KT; kt += 2) {
      stage(kt, f0, f1);
      stage(kt + 1, f1, f0);
    }
    if (kt < KT) stage(kt, f0, f1);
  }
  g2::wait_vmcnt_lgkm0<0>();   // no load of this workgroup outlives it
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int e = et * EW + we + 32 * i + acc_row(r, lane), n = n0 + wn + 32 * j + (lane & 31);
        if (e >= a.E || n >= a.d) continue;
        const size_t k = (size_t)e * a.d + n;
        if (a.part) a.part[(size_t)chunk * a.E * a.d + k] = acc[i][j][r];
        else a.dw[k] = a.add ? a.dw[k] + acc[i][j][r] : acc[i][j][r];
      }
}

template <int NK, bool STREAM>
__global__ __launch_bounds__(kThreads, NK <= 16 ? 2 : 1) void router_dx_bf16_kernel(RArgs a) {
  __shared__ __attribute__((aligned(16))) char smem[dx_lds<NK>()];
  dx_bf16<NK, STREAM>(a, (int)blockIdx.x, smem);
}
template <int EW>
__global__ __launch_bounds__(kBf16Threads, 2) void router_dw_bf16_kernel(RArgs a) {
  __shared__ __attribute__((aligned(16))) char smem[dw_lds<EW>()];
  dw_bf16<EW>(a, (int)blockIdx.x, smem);
}
// Both products in one launch, dW's workgroups first: they are the longer
// ones, and the dx workgroups that fill the CUs beside and after them store
// under their loads (16384 x 2048 x 64: 51 us in all against 58 one after the
// other; 4096 x 7168 x 128: 65 against 69; x 256, which the matrix cores
// bound: 114 against 116).
template <int NK, int EW, bool STREAM>
__global__ __launch_bounds__(kThreads, 2) void router_both_bf16_kernel(RArgs a, int dw_wgs) {
  __shared__ __attribute__((aligned(16))) char smem[std::max(dx_lds<NK>(), dw_lds<EW>())];
  const int b = (int)blockIdx.x;
  if (b < dw_wgs) dw_bf16<EW>(a, b, smem);
  else dx_bf16<NK, STREAM>(a, b - dw_wgs, smem);
}

// dW from the chunks' partial sums (the first dw_blocks workgroups: 64
// 16-byte columns, four threads each adding every fourth chunk), and db:
// eight experts per workgroup, 32 threads an expert, each adding every 32nd
// partial sum.
__global__ __launch_bounds__(kThreads) void router_reduce_kernel(RArgs a, int dw_blocks) {
  __shared__ double s_db[32][8];
  if ((int)blockIdx.x < dw_blocks) {
    __shared__ float4 s_dw[4][64];
    const int c = threadIdx.x % 64, q = threadIdx.x / 64;
    const size_t n = (size_t)a.E * a.d, i = ((size_t)blockIdx.x * 64 + c) * 4;
    float4 s = make_float4(0, 0, 0, 0);
    const float4* part = reinterpret_cast<const float4*>(a.part + i);
#pragma unroll 4
    for (int k = i < n ? q : a.chunks; k < a.chunks; k += 4) {
      const float4 p = part[k * (n / 4)];
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    s_dw[q][c] = s;
    __syncthreads();
    if (q != 0 || i >= n) return;
    if (a.add) {
      const float4 p = *reinterpret_cast<const float4*>(a.dw + i);
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
#pragma unroll
    for (int j = 1; j < 4; ++j) {
      const float4 p = s_dw[j][c];
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    *reinterpret_cast<float4*>(a.dw + i) = s;
    return;
  }
  const int c = threadIdx.x % 8, q = threadIdx.x / 8, e = ((int)blockIdx.x - dw_blocks) * 8 + c;
  double s = 0.0;
  if (e < a.E) {
#pragma unroll 8
    for (int i = q; i < a.db_parts; i += 32) s += a.dbp[(size_t)i * a.E + e];
  }
  s_db[q][c] = s;
  __syncthreads();
  if (q == 0 && e < a.E) {
    s = a.add ? a.db[e] : 0.0;
    for (int i = 0; i < 32; ++i) s += s_db[i][c];
    a.db[e] = (float)s;
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Experts of a dW tile (128, or 64 where fewer experts are padded: 4096 x 7168
// x 128 takes 65 us in all against 84, x 256 114 against 116), and experts of the parts
// of dz: a power of two from 64 on, so that dx has whole operands.
int expert_tile(int E) { return (E + 63) / 64 % 2 ? 64 : 128; }
int padded_experts(int E) { return E <= 64 ? 64 : E <= 128 ? 128 : E <= 256 ? 256 : 512; }

// Token chunks of the dW product, at least 64 tokens each, and the workspace
// that follows from them.  fp32: workgroups for two per CU or a little more
// (for four: 4 to 15 % slower but at 448 tiles, where this rule takes two
// chunks as well).
struct Plan {
  int chunks = 1, ew = 0, etiles = 0, db_parts = 0;
  int64_t chunk_rows = 0, split_rows = 0;
  size_t parts = 0, dbp = 0, part = 0, total = 0;
};

Plan make_plan(int prec, int64_t T, int d, int E) {
  Plan p;
  const bool f32 = prec == MOK_F32;
  p.ew = expert_tile(E);
  p.etiles = (E + p.ew - 1) / p.ew;
  const int en = 64 * kDwWaves * 64 / p.ew;
  const int64_t tiles = f32 ? (int64_t)(d / kTile) * ((E + kTile - 1) / kTile) : (int64_t)((d + en - 1) / en) * p.etiles;
  const int64_t unit = f32 ? kKB : kBK;
  int64_t c;
  if (f32) {
    c = (512 + tiles - 1) / tiles;
  } else {
    // a chunk costs E d 8 bytes (written and read) at about 5 TB/s, 16 tokens
    // of a workgroup 0.25 us while there are fewer workgroups than CUs hold:
    // least in all at the root below.  From one workgroup per CU on, whole
    // rounds of the CUs, at most two (16384 x 2048 x 64: 32 chunks 51 us in
    // all, 64 chunks 60)
    c = (int64_t)(sqrt(9766.0 * (double)T / ((double)E * d)) + 0.5);
    const int64_t rounds = (c * tiles + 128) / 256;
    if (rounds > 0) c = 256 * (rounds < 2 ? rounds : 2) / tiles;
  }
  if (c > (T + 63) / 64) c = (T + 63) / 64;
  if (c < 1) c = 1;
  p.chunk_rows = ((T + c - 1) / c + unit - 1) / unit * unit;
  p.chunks = p.chunk_rows > 0 ? (int)((T + p.chunk_rows - 1) / p.chunk_rows) : 1;
  if (f32) {
    p.db_parts = p.chunks;
  } else {
    // blocks of 32 tokens, at most 512 workgroups a side; few tokens in one,
    // which then writes db itself (and with one chunk nothing is left to add)
    p.split_rows = (T + 512 * 32 - 1) / (512 * 32) * 32;
    if (T <= 128) p.split_rows = 128;
    p.db_parts = T > 0 ? (int)((T + p.split_rows - 1) / p.split_rows) : 0;
    p.parts = align256((size_t)((T + 31) / 32) * 3 * padded_experts(E) * 64);
  }
  p.dbp = align256((size_t)p.db_parts * E * 8);
  p.part = p.chunks > 1 ? align256((size_t)p.chunks * E * d * 4) : 0;
  p.total = p.parts + p.dbp + p.part + 256;
  return p;
}

// Workgroups of dx: for every CU as often as they fit, as far as there are
// column steps.
template <int NK>
int64_t plan_dx(RArgs& a, int per_cu) {
  const int64_t rb = ((int64_t)a.T + dx_rows<NK>() - 1) / dx_rows<NK>();
  int64_t n = (256 * per_cu + rb - 1) / rb;
  if (n > a.d / 64) n = a.d / 64;
  a.n_chunks = (int)n;
  return rb * n;
}
template <int EW>
unsigned dw_workgroups(const RArgs& a) {
  return (unsigned)((a.d + DwCfg<EW>::EN - 1) / DwCfg<EW>::EN) * a.etiles * a.chunks;
}
// d_x beyond the 32 MiB of the L2s is stored past them: kept, it is written
// back under the dW product's loads (16384 x 2048 x 64: 53 us in all against
// 51; 4096 x 7168 x 128: 68 against 65).
bool stream_dx(const RArgs& a) { return (int64_t)a.T * a.d * 2 > (int64_t)32 << 20; }

template <int NK>
void launch_dx(RArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)plan_dx<NK>(a, NK <= 4 ? 4 : NK <= 16 ? 2 : 1));
  if (stream_dx(a)) hipLaunchKernelGGL((router_dx_bf16_kernel<NK, true>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((router_dx_bf16_kernel<NK, false>), grid, dim3(kThreads), 0, stream, a);
}

template <int EW>
void launch_dw(const RArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(router_dw_bf16_kernel<EW>, dim3(dw_workgroups<EW>(a)), dim3(kBf16Threads), 0, stream, a);
}

template <int NK, int EW>
void launch_both(RArgs& a, hipStream_t stream) {
  const unsigned dw = dw_workgroups<EW>(a);
  const dim3 grid(dw + (unsigned)plan_dx<NK>(a, 2));
  if (stream_dx(a)) hipLaunchKernelGGL((router_both_bf16_kernel<NK, EW, true>), grid, dim3(kThreads), 0, stream, a, (int)dw);
  else hipLaunchKernelGGL((router_both_bf16_kernel<NK, EW, false>), grid, dim3(kThreads), 0, stream, a, (int)dw);
}

}  // namespace

size_t router_bwd_ws_bytes(int prec, int64_t T, int d, int E) {
  return make_plan(prec == MOK_F32 ? MOK_F32 : MOK_BF16, T, d, E).total;
}

mok_status launch_router_bwd(const RouterBwdPlan& p, hipStream_t stream) {
  const Plan pl = make_plan(p.prec, p.T, p.d, p.E);
  RArgs a = {};
  a.dz = p.dz;
  a.w = p.w;
  a.x = p.x;
  a.d_x = p.d_x;
  a.dw = p.dw;
  a.db = p.db;
  a.T = p.T, a.T_src = p.T_src > 0 ? p.T_src : 1, a.d = p.d, a.E = p.E, a.own_lo = p.own_lo;
  a.add = p.add;
  a.chunks = pl.chunks, a.chunk_rows = pl.chunk_rows;
  a.ew = pl.ew, a.etiles = pl.etiles, a.eblocks = padded_experts(p.E) / 16, a.split_rows = pl.split_rows, a.db_parts = pl.db_parts;
  char* ws = (char*)p.ws;
  a.part = pl.chunks > 1 ? (float*)(ws + pl.parts + pl.dbp) : nullptr;
  const dim3 blk(kThreads);
  const bool f32 = p.prec == MOK_F32;
  if (f32) {
    a.dbp = pl.chunks > 1 ? (double*)ws : nullptr;
    const int64_t nt = p.d / kTile;
    const int64_t dx = p.want_dx ? nt * (((int64_t)p.T + kTile - 1) / kTile) : 0;
    const int64_t dw = p.dw || p.db ? (p.dw ? nt : 1) * ((p.E + kTile - 1) / kTile) * a.chunks : 0;
    if (dx + dw > 0) {
      hipLaunchKernelGGL(router_f32_kernel, dim3((unsigned)(dx + dw)), blk, 0, stream, a, dw);
      trace_mark(p.tr, "router_f32", stream);
    }
  } else {
    if (p.T > 0) {
      a.parts = p.want_dx || p.dw ? (bf16_t*)ws : nullptr;
      a.dbp = pl.db_parts > 1 ? (double*)(ws + pl.parts) : nullptr;
      hipLaunchKernelGGL(router_split_kernel, dim3((unsigned)pl.db_parts, a.eblocks / 4), blk, 0, stream, a);
      trace_mark(p.tr, "router_split", stream);
    }
    const bool dx = p.want_dx && p.T > 0;
    if (dx && p.dw && p.E <= 256) {
      if (p.E <= 64) launch_both<4, 64>(a, stream);
      else if (p.E <= 128) launch_both<8, 128>(a, stream);
      else if (a.ew == 64) launch_both<16, 64>(a, stream);
      else launch_both<16, 128>(a, stream);
      trace_mark(p.tr, "router_dx_dw", stream);
    } else {
      // one product alone; above 256 experts a dx workgroup fills a CU
      if (dx) {
        if (p.E <= 64) launch_dx<4>(a, stream);
        else if (p.E <= 128) launch_dx<8>(a, stream);
        else if (p.E <= 256) launch_dx<16>(a, stream);
        else launch_dx<32>(a, stream);
        trace_mark(p.tr, "router_dx", stream);
      }
      if (p.dw) {
        if (a.ew == 64) launch_dw<64>(a, stream);
        else launch_dw<128>(a, stream);
        trace_mark(p.tr, "router_dw", stream);
      }
    }
  }
  // what is left to add up: dW over chunks, db over its partial sums
  const bool dw_left = p.dw && a.part, db_left = p.db && (a.dbp || (!f32 && p.T == 0));
  if (dw_left || db_left) {
    const unsigned dwb = dw_left ? (unsigned)(((size_t)p.E * p.d + 255) / 256) : 0;
    const unsigned dbb = db_left ? (unsigned)(p.E + 7) / 8 : 0;
    hipLaunchKernelGGL(router_reduce_kernel, dim3(dwb + dbb), blk, 0, stream, a, (int)dwb);
    trace_mark(p.tr, "router_reduce", stream);
  }
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

}  // namespace mok
