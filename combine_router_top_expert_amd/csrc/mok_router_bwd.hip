// Backward of the router projection z = x W^T + bias for a dense gradient dz
// of the logits:
//   dx[t][n] = sum_e dz[t][e] W[e][n]      (contraction over the experts)
//   dW[e][n] = sum_t dz[t][e] x[t][n]      (contraction over the tokens)
//   db[e]    = sum_t dz[t][e]
// dz stays fp32: both products run on the fp32 matrix cores
// (v_mfma_f32_32x32x2_f32), whose operands hold one k per lane, so operands
// that are strided along k need no transpose.
#include "mok_internal.h"

namespace mok {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;   // output tile 64 x 64, four waves of 32 x 32
constexpr int kKB = 32;     // contraction steps staged through LDS at a time
constexpr int kPitch = kTile + 4;

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
};

template <typename T>
__device__ __forceinline__ const T* x_row(const RArgs& a, int t) {
  return reinterpret_cast<const T*>(a.x.p[a.own_lo + t / a.T_src]) + (size_t)(t % a.T_src) * a.d;
}

// acc += A B over one staged block: sA [kKB][kPitch] (k, m), sB (k, n)
__device__ __forceinline__ void mma_block(const float* sA, const float* sB, int m0, int n0, f32x16_t& acc) {
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
#pragma unroll
  for (int k = 0; k < kKB; k += 2)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sA[(k + h) * kPitch + m0 + c], sB[(k + h) * kPitch + n0 + c], acc, 0, 0, 0);
}

// row of accumulator register r in a 32 x 32 block (its column is lane % 32)
__device__ __forceinline__ int acc_row(int r, int lane) { return (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3); }

template <typename T>
__global__ __launch_bounds__(kThreads) void router_dx_kernel(RArgs a) {
  __shared__ float sA[kKB * kPitch], sB[kKB * kPitch];
  const int nt = a.d / kTile;
  const int n0 = (int)(blockIdx.x % nt) * kTile, t0 = (int)(blockIdx.x / nt) * kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const T* w = reinterpret_cast<const T*>(a.w);
  f32x16_t acc = {};
  for (int e0 = 0; e0 < a.E; e0 += kKB) {
    for (int i = tid; i < kTile * kKB; i += kThreads) {
      const int t = i / kKB, e = i % kKB;
      sA[e * kPitch + t] = t0 + t < a.T && e0 + e < a.E ? a.dz[(size_t)(t0 + t) * a.E + e0 + e] : 0.0f;
      const int k = i / kTile, n = i % kTile;
      sB[k * kPitch + n] = e0 + k < a.E ? to_f32<T>(w[(size_t)(e0 + k) * a.d + n0 + n]) : 0.0f;
    }
    __syncthreads();
    mma_block(sA, sB, wm, wn, acc);
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int t = t0 + wm + acc_row(r, lane);
    if (t >= a.T) continue;
    T* o = reinterpret_cast<T*>(a.d_x.p[a.own_lo + t / a.T_src]) + (size_t)(t % a.T_src) * a.d + n0 + wn + (lane & 31);
    *o = from_f32<T>(a.add ? to_f32<T>(*o) + acc[r] : acc[r]);
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void router_dw_kernel(RArgs a) {
  __shared__ float sA[kKB * kPitch], sB[kKB * kPitch];
  const int n0 = blockIdx.x * kTile, e0 = blockIdx.y * kTile, chunk = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int64_t lo64 = (int64_t)chunk * a.chunk_rows;
  const int lo = (int)min(lo64, (int64_t)a.T), hi = (int)min(lo64 + a.chunk_rows, (int64_t)a.T);
  const bool bias = a.db && blockIdx.x == 0 && tid < kTile;
  double bsum = 0.0;
  f32x16_t acc = {};
  for (int t0 = lo; t0 < hi; t0 += kKB) {
    for (int i = tid; i < kTile * kKB; i += kThreads) {
      const int k = i / kTile, c = i % kTile;
      const bool there = t0 + k < hi;
      sA[k * kPitch + c] = there && e0 + c < a.E ? a.dz[(size_t)(t0 + k) * a.E + e0 + c] : 0.0f;
      sB[k * kPitch + c] = there && a.dw ? to_f32<T>(x_row<T>(a, t0 + k)[n0 + c]) : 0.0f;
    }
    __syncthreads();
    mma_block(sA, sB, wm, wn, acc);
    if (bias)
      for (int k = 0; k < kKB; ++k) bsum += (double)sA[k * kPitch + tid];
    __syncthreads();
  }
  if (a.dw) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int e = e0 + wm + acc_row(r, lane);
      if (e >= a.E) continue;
      const size_t i = (size_t)e * a.d + n0 + wn + (lane & 31);
      if (a.part) a.part[(size_t)chunk * a.E * a.d + i] = acc[r];
      else a.dw[i] = a.add ? a.dw[i] + acc[r] : acc[r];
    }
  }
  if (bias && e0 + tid < a.E) {
    const int e = e0 + tid;
    if (a.dbp) a.dbp[(size_t)chunk * a.E + e] = bsum;
    else a.db[e] = (float)(a.add ? a.db[e] + bsum : bsum);
  }
}

// dW and db from the chunks' partial sums, in chunk order
__global__ __launch_bounds__(kThreads) void router_reduce_kernel(RArgs a) {
  const size_t n = (size_t)a.E * a.d, i = ((size_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  if (a.dw && i < n) {
    float4 s = a.add ? *reinterpret_cast<const float4*>(a.dw + i) : make_float4(0, 0, 0, 0);
    for (int c = 0; c < a.chunks; ++c) {
      const float4 p = *reinterpret_cast<const float4*>(a.part + c * n + i);
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    *reinterpret_cast<float4*>(a.dw + i) = s;
  }
  const int e = blockIdx.x * kThreads + threadIdx.x;
  if (a.db && e < a.E) {
    double s = a.add ? a.db[e] : 0.0;
    for (int c = 0; c < a.chunks; ++c) s += a.dbp[(size_t)c * a.E + e];
    a.db[e] = (float)s;
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Token chunks of the dW product: enough workgroups for four per CU, at
// least 256 tokens each.
void dw_chunks(int64_t T, int d, int E, int* chunks, int64_t* rows) {
  const int64_t tiles = (int64_t)(d / kTile) * ((E + kTile - 1) / kTile);
  int64_t c = 1024 / tiles;
  if (c > (T + 255) / 256) c = (T + 255) / 256;
  if (c < 1) c = 1;
  const int64_t r = ((T + c - 1) / c + kKB - 1) / kKB * kKB;
  *rows = r;
  *chunks = r > 0 ? (int)((T + r - 1) / r) : 1;
}

}  // namespace

size_t router_bwd_ws_bytes(int prec, int64_t T, int d, int E) {
  (void)prec;
  int chunks;
  int64_t rows;
  dw_chunks(T, d, E, &chunks, &rows);
  return chunks > 1 ? align256((size_t)chunks * E * d * 4) + align256((size_t)chunks * E * 8) : 256;
}

mok_status launch_router_bwd(const RouterBwdPlan& p, hipStream_t stream) {
  RArgs a = {};
  a.dz = p.dz;
  a.w = p.w;
  a.x = p.x;
  a.d_x = p.d_x;
  a.dw = p.dw;
  a.db = p.db;
  a.T = p.T, a.T_src = p.T_src > 0 ? p.T_src : 1, a.d = p.d, a.E = p.E, a.own_lo = p.own_lo;
  a.add = p.add;
  dw_chunks(p.T, p.d, p.E, &a.chunks, &a.chunk_rows);
  if (a.chunks > 1) {
    a.part = (float*)p.ws;
    a.dbp = (double*)((char*)p.ws + align256((size_t)a.chunks * p.E * p.d * 4));
  }
  const dim3 blk(kThreads);
  const bool f32 = p.prec == MOK_F32;
  if (p.want_dx && p.T > 0) {
    const dim3 grid((unsigned)((int64_t)(p.d / kTile) * (((int64_t)p.T + kTile - 1) / kTile)));
    if (f32) hipLaunchKernelGGL(router_dx_kernel<float>, grid, blk, 0, stream, a);
    else hipLaunchKernelGGL(router_dx_kernel<bf16_t>, grid, blk, 0, stream, a);
    trace_mark(p.tr, "router_dx", stream);
  }
  if (p.dw || p.db) {
    const dim3 grid(p.dw ? p.d / kTile : 1, (p.E + kTile - 1) / kTile, a.chunks);
    if (f32) hipLaunchKernelGGL(router_dw_kernel<float>, grid, blk, 0, stream, a);
    else hipLaunchKernelGGL(router_dw_kernel<bf16_t>, grid, blk, 0, stream, a);
    trace_mark(p.tr, "router_dw", stream);
    if (a.chunks > 1) {
      const size_t n = (size_t)p.E * p.d / 4;
      hipLaunchKernelGGL(router_reduce_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), blk, 0, stream, a);
      trace_mark(p.tr, "router_reduce", stream);
    }
  }
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

}  // namespace mok
