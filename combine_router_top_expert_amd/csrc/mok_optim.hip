// Optimizer step over many tensors: global gradient norm with the clip
// factor, and AdamW with moments in 32 or 8 bits.
//
// Tensors come as descriptors in the kernel arguments (as many as fit their
// 4 KiB per launch; no device table to keep), cut into pieces of kPiece
// elements; a workgroup finds its tensor by a search over the pieces' prefix
// sums.  A lane takes 8 consecutive elements at a time (32 bytes of fp32, 16
// of bf16, 8 of codes); four lanes hold a 32-element block of an 8-bit
// moment, so its largest magnitude is two quad exchanges away.
//
// Both are bound by HBM.  Norm: 554 million fp32 gradients in 356 us (6.2
// TB/s; the streaming read probe reaches 6.3).  Step: the same tensors with
// fp32 gradient, master and moments and a bf16 copy, 30 bytes an element,
// 3.16 ms (5.2 TB/s, the copy probe's rate); 352 million elements with 8-bit
// moments, 18 bytes an element, 1.19 ms (5.3 TB/s).  120 bf16 tensors of 44
// million elements in all with 8-bit moments, 10 bytes an element, take 116 us
// in three launches (47 + 47 + 25): each start and end of a launch costs some
// 7 us, and the arithmetic of two encodings nearly as much as the bytes.  (With
// the step number on the device every thread forms the two corrections by
// itself, two powers in 64 bits; the figures are of host steps.)
#include "mok_internal.h"
#include "mok_lanes.h"

namespace mok {

namespace {

constexpr int kThreads = 256;
constexpr int kLane = 8;                       // elements per lane at a time
constexpr int kStep = kThreads * kLane;        // elements per workgroup step
constexpr int kPiece = 4 * kStep;              // elements per workgroup: of the norm and of fp32 moments,
constexpr int kPiece8 = 2 * kStep;             // of 8-bit ones (3 % faster over many tensors; fp32 1 % slower)
constexpr int kBatch = 50;                     // tensors per launch of the step
constexpr int kNormBatch = 192;                // and of the norm
constexpr int kNormWgs = 2048;                 // workgroups of the norm per launch at most

struct Desc {
  void* p;
  const void* g;
  float* master;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
  float wd;
  uint32_t tag;   // flags below, and from bit 4 on the place in the caller's array
};
enum : uint32_t { kPBf16 = 1, kGBf16 = 2, kEight = 4, kWide = 8 };

struct Batch {
  Desc d[kBatch];
  uint32_t first[kBatch + 1];   // pieces before tensor i
  int count;
};

struct AdamArgs {
  float lr, b1, c1, b2, c2, eps;   // c = 1 - b
  double beta1, beta2;
  float inv_bc1, inv_sqrt_bc2;     // of the host's step
  float grad_scale;
  int64_t step;
  uint64_t seed;
  const float* dev_scale;
  const double* dev_lr;
  const int64_t* dev_step;
  int random_params;
};

struct NormDesc {
  const void* g;
  int64_t n;        // elements, times 4, plus kNormBf16 and kNormWide
};
enum : int64_t { kNormBf16 = 1, kNormWide = 2 };
struct NormBatch {
  NormDesc d[kNormBatch];
  uint32_t first[kNormBatch + 1];
  int count;
};
static_assert(sizeof(Batch) + sizeof(AdamArgs) <= 4096 && sizeof(NormBatch) + 64 <= 4096, "kernel arguments");

template <class B>
__device__ __forceinline__ int find_tensor(const B& b, uint32_t piece) {
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= piece) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// 8 elements from element i of an fp32 or bf16 tensor; elements past n are 0.
__device__ __forceinline__ void load8_f32(const float* p, int64_t i, int64_t n, bool wide, float (&v)[8]) {
  if (wide && i <= n - 8) {
    const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < n ? p[i + j] : 0.0f;
  }
}
__device__ __forceinline__ void load8_bf16(const bf16_t* p, int64_t i, int64_t n, bool wide, float (&v)[8]) {
  if (wide && i <= n - 8) {
    const uint4 u = ld16(p + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < n ? bf16_to_f32(p[i + j]) : 0.0f;
  }
}
__device__ __forceinline__ void store8_f32(float* p, int64_t i, int64_t n, bool wide, const float (&v)[8]) {
  if (wide && i <= n - 8) {
    *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = v[j];
  }
}
__device__ __forceinline__ void store8_u16(bf16_t* p, int64_t i, int64_t n, bool wide, const uint32_t (&w)[4]) {
  if (wide && i <= n - 8) {
    st16(p + i, make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = (bf16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ void load8_u8(const uint8_t* p, int64_t i, int64_t n, bool wide, uint32_t (&w)[2]) {
  if (wide && i <= n - 8) {
    const uint2 u = *reinterpret_cast<const uint2*>(p + i);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = w[1] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) w[j >> 2] |= (uint32_t)p[i + j] << (8 * (j & 3));
  }
}
__device__ __forceinline__ void store8_u8(uint8_t* p, int64_t i, int64_t n, bool wide, const uint32_t (&w)[2]) {
  if (wide && i <= n - 8) {
    *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) p[i + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
}

// ------------------------------------------------------------------ norm
// Squares summed in 64 bits (fp32 squares would overflow from 1.8e19 on and
// vanish below 1e-23; conversion and fused multiply-add run under the loads):
// per lane over the workgroup's pieces, then wave and workgroup in a fixed
// order, one partial sum per workgroup.
__global__ __launch_bounds__(kThreads) void norm_kernel(NormBatch b, uint32_t pieces, double* part) {
  __shared__ double s_w[kThreads / 64];
  constexpr int S = kPiece / kStep;
  double s = 0.0;
  auto add = [&](const float (&g)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __builtin_fma((double)g[j], (double)g[j], s);
  };
  for (uint32_t pc = blockIdx.x; pc < pieces; pc += gridDim.x) {
    const int ti = find_tensor(b, pc);
    const void* p = b.d[ti].g;
    const int64_t tag = b.d[ti].n, n = tag >> 2;
    const bool bf = tag & kNormBf16, wide = tag & kNormWide;
    const int64_t base = (int64_t)(pc - b.first[ti]) * kPiece + threadIdx.x * kLane;
    float g[S][8];
    if (wide && base - threadIdx.x * kLane + kPiece <= n) {   // whole pieces: every load first
      if (bf) {
#pragma unroll
        for (int i = 0; i < S; ++i) load8_bf16((const bf16_t*)p, base + i * kStep, INT64_MAX, true, g[i]);
      } else {
#pragma unroll
        for (int i = 0; i < S; ++i) load8_f32((const float*)p, base + i * kStep, INT64_MAX, true, g[i]);
      }
#pragma unroll
      for (int i = 0; i < S; ++i) add(g[i]);
      continue;
    }
    for (int i = 0; i < S; ++i) {
      if (base + i * kStep >= n) break;
      if (bf) load8_bf16((const bf16_t*)p, base + i * kStep, n, wide, g[0]);
      else load8_f32((const float*)p, base + i * kStep, n, wide, g[0]);
      add(g[0]);
    }
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = (s_w[0] + s_w[1]) + (s_w[2] + s_w[3]);
}

__global__ __launch_bounds__(1024) void norm_total_kernel(const double* part, int64_t n, float max_norm, float* out) {
  __shared__ double s_w[16];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += part[i];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < 16; ++i) s += s_w[i];
    const double norm = sqrt(s);
    const float f = (float)norm;
    out[0] = f;
    const double c = max_norm > 0.0f ? max_norm / (norm + 1e-6) : 1.0;
    out[1] = __builtin_isfinite(f) ? (float)(c < 1.0 ? c : 1.0) : __builtin_nanf("");
  }
}

// ------------------------------------------------------------------ AdamW
// The 64-bit finaliser of SplitMix64 (Steele, Lea and Flood, OOPSLA 2014).
constexpr uint64_t kGold = 0x9E3779B97F4A7C15ull;
__device__ __forceinline__ uint64_t mix64(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// Smallest s with amax <= 448 2^s (448 = 1.75 2^8), from the bits: adding
// what is missing from 1.75 to 2 in the mantissa carries into the exponent
// exactly where the mantissa is above 1.75.  Clamped to E8M0's range.
__device__ __forceinline__ int block_scale(float amax) {
  const int s = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 127 - 8;
  return s < -127 ? -127 : (s > 127 ? 127 : s);
}

// fp32 bits of |x| 2^(-s-120) with random bits added below bit 20: bits 20..26
// are the E4M3 code of |x| 2^-s rounded up or down.  |x| 2^(-s-120) has the
// code's exponent field (bias 127 - 120 = 7), so its bits from 20 on are the
// code rounded down, subnormals included, and what is added below carries.
// The scale keeps finite |x| 2^-s at 448 or less, so nothing passes 0x7E.
// (Below the 2^-6 of the smallest full code the product is rounded to fp32's
// own subnormals, 2^-20 of the distance of two codes: 16 times finer than the
// random number.)
__device__ __forceinline__ uint32_t random_code(float x, int s, uint32_t rnd) {
  return __float_as_uint(__builtin_amdgcn_ldexpf(__builtin_fabsf(x), -s - 120)) + rnd;
}

// Largest of the quad's four values (as unsigned bits).
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true));
  return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true));
}

// Codes of eight values and the block's scale.  Magnitudes compare as
// integers (NaN above infinity above every number), so one comparison finds
// out whether a lane of the wave holds something that is not finite; only
// then the block's maximum is taken again over finite values.  ROOT: the
// values are square roots: no sign, above zero stays above zero, and what is
// not finite saturates (E4M3's NaN would be a divisor too).
template <bool ROOT>
__device__ __forceinline__ int encode8(const float (&x)[8], const uint32_t (&rnd)[8], uint32_t (&out)[2]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  constexpr uint32_t kInf = 0x7F800000u;
  const bool odd = __any(top >= kInf);
  if (odd) {
    top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = __float_as_uint(x[j]) & 0x7FFFFFFFu;
      top = max(top, m < kInf ? m : 0u);
    }
  }
  const int s = block_scale(__uint_as_float(quad_max(top)));
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = random_code(x[j], s, rnd[j]) << 4;     // the code in bits 24..30
    if constexpr (ROOT) c[j] = max(c[j], min(__float_as_uint(x[j]), 1u) << 24);
  }
  if (odd) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!__builtin_isfinite(x[j])) c[j] = ROOT ? 0x7E000000u : 0x7F000000u;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if constexpr (!ROOT) c[j] = (c[j] & 0x7FFFFFFFu) | (__float_as_uint(x[j]) & 0x80000000u);
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // the top bytes of four words
    const uint32_t lo = __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h], 0x0C0C0703u);
    const uint32_t up = __builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2], 0x07030C0Cu);
    out[h] = lo | up;
  }
  return s;
}

// The square root of v, rounded to nearest but for rare last bits, where v is
// zero or at least kRootMin: the hardware's reciprocal root (1 ulp) and one
// step of Newton's for the root, whose residual v - r r is exact there (a
// multiple of 2^-46 of r's power of two squared, which fp32 still holds).
// Below, the residual and from 2^-126 on the reciprocal root go wrong, so a
// wave with such a v takes the library's root (all waves: 6 us more on 43
// million elements of 8-bit moments).
constexpr float kRootMin = 0x1p-102f;
__device__ __forceinline__ float root(float v) {
  const float h = __builtin_amdgcn_rsqf(__builtin_fmaxf(v, kRootMin));
  const float r = v * h;
  const float e = __builtin_fmaf(-r, r, v);
  return v < __builtin_inff() ? __builtin_fmaf(e, 0.5f * h, r) : v;
}
__device__ __forceinline__ void roots8(const float (&v)[8], float (&r)[8]) {
  uint32_t least = ~0u;   // of the bits less one: zero comes last
#pragma unroll
  for (int j = 0; j < 8; ++j) least = min(least, __float_as_uint(v[j]) - 1);
  if (__any(least < __float_as_uint(kRootMin) - 1)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = sqrtf(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = root(v[j]);
  }
}

// The moments are formed as the formula says, each product and sum rounded by
// itself, and so is the root: a fused or 1-ulp form moves one stored code in
// about 2^21 to its neighbour, and where two gradients' histories are alike
// their codes should not depend on how a build contracts.  The reciprocal of
// the update is the hardware's (1 ulp): an error of 2^-23 of the update.
template <bool EIGHT>
__device__ __forceinline__ void adam_step(const Desc& d, const AdamArgs& a, int64_t i, float scale, float lr,
                                          float inv_bc1, float inv_sbc2, uint64_t key) {
  const bool wide = d.tag & kWide, pb = d.tag & kPBf16;
  float g[8], p[8], m[8], v[8];
  const int64_t n = d.n;
  if (d.tag & kGBf16) load8_bf16((const bf16_t*)d.g, i, n, wide, g);
  else load8_f32((const float*)d.g, i, n, wide, g);
  if (d.master) load8_f32(d.master, i, n, wide, p);
  else if (pb) load8_bf16((const bf16_t*)d.p, i, n, wide, p);
  else load8_f32((const float*)d.p, i, n, wide, p);
  if constexpr (EIGHT) {
    uint32_t mc[2], vc[2];
    load8_u8((const uint8_t*)d.m, i, n, wide, mc);
    load8_u8((const uint8_t*)d.v, i, n, wide, vc);
    const bool there = i < n;
    const int sm = there ? (int)d.ms[i >> 5] - 127 : 0, sv = there ? (int)d.vs[i >> 5] - 127 : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto m0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[h], false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[h], true);
      const auto v0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[h], false), v1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[h], true);
      m[4 * h] = m0[0], m[4 * h + 1] = m0[1], m[4 * h + 2] = m1[0], m[4 * h + 3] = m1[1];
      v[4 * h] = v0[0], v[4 * h + 1] = v0[1], v[4 * h + 2] = v1[0], v[4 * h + 3] = v1[1];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = __builtin_amdgcn_ldexpf(m[j], sm);
      v[j] = __builtin_amdgcn_ldexpf(v[j], sv);
      v[j] *= v[j];
    }
  } else {
    load8_f32((const float*)d.m, i, n, wide, m);
    load8_f32((const float*)d.v, i, n, wide, v);
  }
  const float decay = 1.0f - lr * d.wd, rate = -lr * inv_bc1;
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma clang fp contract(off)
    const float gj = g[j] * scale;
    m[j] = a.b1 * m[j] + a.c1 * gj;
    v[j] = a.b2 * v[j] + a.c2 * (gj * gj);
  }
  roots8(v, r);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u = m[j] * __builtin_amdgcn_rcpf(__builtin_fmaf(r[j], inv_sbc2, a.eps));
    p[j] = __builtin_fmaf(rate, u, p[j] * decay);
  }
  uint32_t w0 = 0, w1 = 0;
  if (EIGHT || a.random_params) {
    const uint64_t z = mix64(key + ((uint64_t)(i >> 3) + 1) * kGold);
    w0 = (uint32_t)z, w1 = (uint32_t)(z >> 32);
  }
  if constexpr (EIGHT) {
    uint32_t rm[8], rv[8], w = w0, mc[2], vc[2];
#pragma unroll
    for (int j = 0; j < 8; ++j, w += w1) {
      rm[j] = (w & 0xFFFFu) << 4;
      rv[j] = (w >> 16) << 4;
    }
    const int sm = encode8<false>(m, rm, mc), sr = encode8<true>(r, rv, vc);
    store8_u8((uint8_t*)d.m, i, n, wide, mc);
    store8_u8((uint8_t*)d.v, i, n, wide, vc);
    if ((threadIdx.x & 3) == 0 && i < n) {
      d.ms[i >> 5] = (uint8_t)(sm + 127);
      d.vs[i >> 5] = (uint8_t)(sr + 127);
    }
  } else {
    store8_f32((float*)d.m, i, n, wide, m);
    store8_f32((float*)d.v, i, n, wide, v);
  }
  if (d.master) store8_f32(d.master, i, n, wide, p);
  if (pb) {
    uint32_t o[4];
    if (a.random_params && !d.master) {
      uint32_t w = w1, b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j, w += w0) b[j] = __float_as_uint(p[j]) + (w >> 16);
      // infinity and NaN take no random bits: they would turn into others
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!__builtin_isfinite(p[j])) b[j] = __float_as_uint(p[j]) | (__builtin_isnan(p[j]) ? 0x400000u : 0u);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_perm(b[2 * j + 1], b[2 * j], 0x07060302u);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = pack2_bf16(p[2 * j], p[2 * j + 1]);
    }
    store8_u16((bf16_t*)d.p, i, n, wide, o);
  } else {
    store8_f32((float*)d.p, i, n, wide, p);
  }
}

__global__ __launch_bounds__(kThreads) void adamw_kernel(Batch b, AdamArgs a) {
  float scale = a.grad_scale;
  if (a.dev_scale) {
    const float s = *a.dev_scale;
    if (__builtin_isnan(s)) return;   // the whole step is left out
    scale *= s;
  }
  float lr = a.lr, inv_bc1 = a.inv_bc1, inv_sbc2 = a.inv_sqrt_bc2;
  int64_t step = a.step;
  if (a.dev_lr) lr = (float)*a.dev_lr;
  if (a.dev_step) {
    step = *a.dev_step;
    inv_bc1 = (float)(1.0 / (1.0 - pow(a.beta1, (double)step)));
    inv_sbc2 = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)step)));
  }
  const int ti = find_tensor(b, blockIdx.x);
  const Desc& d = b.d[ti];
  const uint64_t key = mix64(mix64(a.seed + (d.tag >> 4)) + (uint64_t)step * kGold);
  const int64_t place = blockIdx.x - b.first[ti];
  if (d.tag & kEight) {
    for (int it = 0; it < kPiece8 / kStep; ++it) {
      const int64_t at = place * kPiece8 + (int64_t)it * kStep;
      if (at >= d.n) break;
      adam_step<true>(d, a, at + threadIdx.x * kLane, scale, lr, inv_bc1, inv_sbc2, key);
    }
  } else {
    for (int it = 0; it < kPiece / kStep; ++it) {
      const int64_t at = place * kPiece + (int64_t)it * kStep;
      if (at >= d.n) break;
      adam_step<false>(d, a, at + threadIdx.x * kLane, scale, lr, inv_bc1, inv_sbc2, key);
    }
  }
}

uint32_t norm_grid(uint32_t pieces) { return pieces < kNormWgs ? pieces : kNormWgs; }
// Fills batches of at most N non-empty tensors and at most 2^30 pieces (a
// tensor never splits over batches) and calls run(batch, pieces) for each;
// put(descriptor, tensor, place) writes one; piece(tensor) is its elements
// per workgroup.
template <class B, int N, class Piece, class Put, class Run>
bool each_batch(int n_params, const mok_param* params, Piece piece, Put put, Run run) {
  B b = {};
  uint64_t pieces = 0;
  for (int t = 0; t < n_params; ++t) {
    if (params[t].n == 0) continue;
    const int per = piece(params[t]);
    const uint64_t k = (uint64_t)(params[t].n + per - 1) / per;
    if (b.count == N || (b.count && pieces + k > (1u << 30))) {
      if (!run(b, (uint32_t)pieces)) return false;
      b.count = 0;
      pieces = 0;
    }
    put(b.d[b.count], params[t], t);
    b.first[b.count] = (uint32_t)pieces;
    pieces += k;
    b.first[++b.count] = (uint32_t)pieces;
  }
  return b.count == 0 || run(b, (uint32_t)pieces);
}

}  // namespace

size_t grad_norm_ws_bytes(int n_params, const mok_param* params) {
  size_t parts = 1;
  each_batch<NormBatch, kNormBatch>(n_params, params, [](const mok_param&) { return kPiece; }, [](NormDesc&, const mok_param&, int) {},
                                    [&](const NormBatch&, uint32_t pieces) {
                                      parts += norm_grid(pieces);
                                      return true;
                                    });
  return parts * sizeof(double);
}

mok_status launch_grad_norm(int n_params, const mok_param* params, float max_norm, float* out, void* ws,
                            hipStream_t stream) {
  double* part = (double*)ws;
  int64_t done = 0;
  auto put = [](NormDesc& d, const mok_param& q, int) {
    d.g = q.g;
    d.n = q.n * 4 + (q.g_type == MOK_BF16 ? kNormBf16 : 0) + ((uintptr_t)q.g % 16 == 0 ? kNormWide : 0);
  };
  auto run = [&](const NormBatch& b, uint32_t pieces) {
    const uint32_t grid = norm_grid(pieces);
    hipLaunchKernelGGL(norm_kernel, dim3(grid), dim3(kThreads), 0, stream, b, pieces, part + done);
    done += grid;
    return hipGetLastError() == hipSuccess;
  };
  if (!each_batch<NormBatch, kNormBatch>(n_params, params, [](const mok_param&) { return kPiece; }, put, run)) return MOK_EDEVICE;
  hipLaunchKernelGGL(norm_total_kernel, dim3(1), dim3(1024), 0, stream, part, done, max_norm, out);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EDEVICE;
}

mok_status launch_adamw(int n_params, const mok_param* params, const mok_adamw_args& h, hipStream_t stream) {
  AdamArgs a = {};
  a.lr = (float)h.lr;
  a.b1 = (float)h.beta1, a.c1 = (float)(1.0 - h.beta1);
  a.b2 = (float)h.beta2, a.c2 = (float)(1.0 - h.beta2);
  a.eps = (float)h.eps;
  a.beta1 = h.beta1, a.beta2 = h.beta2;
  a.inv_bc1 = (float)(1.0 / (1.0 - pow(h.beta1, (double)h.step)));
  a.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
  a.grad_scale = h.grad_scale;
  a.step = h.step;
  a.seed = h.seed;
  a.dev_scale = h.dev_scale, a.dev_lr = h.dev_lr, a.dev_step = h.dev_step;
  a.random_params = h.random_params;
  auto put = [](Desc& d, const mok_param& q, int t) {
    d.p = q.p, d.g = q.g, d.master = q.master, d.m = q.m, d.v = q.v, d.ms = q.m_scale, d.vs = q.v_scale;
    d.n = q.n;
    d.wd = q.weight_decay;
    const uintptr_t all = (uintptr_t)q.p | (uintptr_t)q.g | (uintptr_t)q.master | (uintptr_t)q.m | (uintptr_t)q.v;
    d.tag = (uint32_t)t << 4 | (q.p_type == MOK_BF16 ? kPBf16 : 0) | (q.g_type == MOK_BF16 ? kGBf16 : 0) |
            (q.state_bits == 8 ? kEight : 0) | (all % 16 == 0 ? kWide : 0);
  };
  auto piece = [](const mok_param& q) { return q.state_bits == 8 ? kPiece8 : kPiece; };
  auto run = [&](const Batch& b, uint32_t pieces) {
    hipLaunchKernelGGL(adamw_kernel, dim3(pieces), dim3(kThreads), 0, stream, b, a);
    return hipGetLastError() == hipSuccess;
  };
  return each_batch<Batch, kBatch>(n_params, params, piece, put, run) ? MOK_OK : MOK_EDEVICE;
}

}  // namespace mok
