// Row-wise operators that write 8-bit-float activations, and the weight
// encoder:
//   quantize  q = e4m3(x / s), one scale s per row and 128 columns
//   swiglu    the same of silu(gate) * up
//   rmsnorm   t = x + residual;  h = t / sqrt(mean(t^2) + eps) * weight;
//             the same of h, and / or h as bf16
//   encode    q = e4m3(w / s), one scale per 128 x 128 block
// All are bound by HBM: each element is read once and written once, the
// block maximum and the row's sum of squares are taken from registers. (The
// forms for long or unaligned rows of the norm, and for unaligned rows of the
// encoder, read them twice.)
//
// Scales are powers of two, so the division is exact and a byte depends only
// on the value that is rounded: one rounding, to nearest even, to 4
// significand bits. Values of h and silu(g) * u are formed in fp32 (within 16
// 2^-24, far below that rounding); where such an error could move a block to
// the next scale the block is formed again in 64 bits (fp8_scale_unsure).
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>
#include <mutex>
#include <new>
#include <vector>

#include "hxq_fp8.cuh"

namespace hxq {
namespace {

// (Inputs are read with plain loads, not through the read-only path: the
// kernels may start while the one that writes their inputs still runs.)
constexpr int kVec = 8;                        // elements per thread and block of 128: 16 lanes share a block
constexpr int kLanesPerBlock = kFp8Block / kVec;

// Pieces of kVec columns in a row of any length below 2^31.
__host__ __device__ inline int pieces_of(int cols) { return cols / kVec + (cols % kVec != 0); }

// 8 elements from p (fp32 or bf16) as floats; VEC: p is 16-byte aligned and
// all 8 exist, else element by element with zeros past n.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t at, int n, float (&v)[8]) {
  if (VEC) {
    if (n <= 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    } else if (BF16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(u[j] << 16);
        v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
      const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.f;
      if (j < n)
        v[j] = BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(base)[at + j] << 16)
                    : static_cast<const float*>(base)[at + j];
    }
  }
}

// 8 floats to p as fp32 or bf16 (round to nearest even), as load8.
template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, const float (&v)[8]) {
  if (VEC) {
    if (n <= 0) return;
    if (BF16) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      float* p = static_cast<float*>(base) + at;
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        if (BF16)
          static_cast<__nv_bfloat16*>(base)[at + j] = __float2bfloat16_rn(v[j]);
        else
          static_cast<float*>(base)[at + j] = v[j];
      }
  }
}

__device__ __forceinline__ float round_bf16(float f) { return __bfloat162float(__float2bfloat16_rn(f)); }

// e4m3 bytes of 4 values already divided by their scale (NaN gives NaN; an
// infinity would give 448: see no_infinities).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Infinities become NaN (e4m3 has none) in a block whose maximum is infinite:
// 0 * v adds NaN to them and nothing to the others.
template <int N>
__device__ __forceinline__ void no_infinities(float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = fmaf(v[j], 0.f, v[j]);
}

__device__ __forceinline__ float absmax8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));  // (fmaxf skips NaN)
  return m;
}
// Over the 16 lanes that share a block of 128.
__device__ __forceinline__ float block_max(float m) {
#pragma unroll
  for (int o = kLanesPerBlock / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
__device__ __forceinline__ double block_max(double m) {
#pragma unroll
  for (int o = kLanesPerBlock / 2; o; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The 8 bytes of one lane (8 values of its block). `c` is the lane's first
// column: bytes are written up to the row's padded length.
__device__ __forceinline__ void put8(uint8_t* row, int64_t ld, int c, const float (&v)[8], float inv) {
  if (c >= ld) return;
  const uint2 w = make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                             e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  *reinterpret_cast<uint2*>(row + c) = w;
}

// silu(g) * u of two elements. e^-g = 2^p (1 + r ln 2) with p = -g log2(e)
// rounded and r what the rounding left (exact by FMA, plus the constant's own
// tail): 2^p is the hardware's (2 ulp), the reciprocal too (1 ulp), and four
// more roundings follow. For kGateMin <= g <= kGateMax: below, e^-g nears the end
// of fp32, which an up near that end makes large again; above, p leaves fp32. A
// block with such a gate is formed in 64 bits. g u comes first: what it loses
// below fp32's normal numbers is far below any block's maximum that is not
// formed in 64 bits, and beyond fp32's end it makes that maximum infinite.
constexpr float kGateMin = -87.f, kGateMax = 1e38f;
__device__ __forceinline__ float2 swiglu2(float2 g, float2 u) {
  constexpr float kLog2e = 1.44269504f;                                    // log2(e) to fp32,
  constexpr float kLog2eTail = (float)(1.4426950408889634 - 1.44269504f);  // and the rest
  const float2 k = make_float2(-kLog2e, -kLog2e), k2 = make_float2(-kLog2eTail, -kLog2eTail);
  const float2 p = __fmul2_rn(g, k);
  const float2 r = __ffma2_rn(g, k2, __ffma2_rn(g, k, make_float2(-p.x, -p.y)));
  float2 e, inv;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(p.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(p.y));
  e = __ffma2_rn(__fmul2_rn(e, r), make_float2(0.693147181f, 0.693147181f), e);
  const float2 d = __fadd2_rn(e, make_float2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.y) : "f"(d.y));
  return __fmul2_rn(__fmul2_rn(g, u), inv);
}
// (Blocks of zeros have no maximum to tell them by and come here too: 2048 x 14336
// bf16 into the same outputs takes 27 us, with every other row zeros 166, all zeros 294.)
// One thread's part of a block (8 columns from c0 + 8 lanes k on for each of
// its `pieces`, `lanes` threads a block) formed in 64 bits, for blocks whose scale
// fp32 cannot settle or with a gate outside swiglu2's range (a call: its registers
// are not the fast path's). at: the gate of column c0; n: columns from c0 on.
template <bool BF16, bool VEC>
__device__ __noinline__ void swiglu64(const void* x, int64_t at, int cols, int n, uint8_t* row, int64_t ld, int c0,
                                      int pieces, int lanes, float* scale) {
  double m = 0.0;
  float inv = 1.f, s = 1.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int k = 0; k < pieces; ++k) {
      float g[8], v[8];
      load8<BF16, VEC>(x, at + 8 * lanes * k, n - 8 * lanes * k, g);
      load8<BF16, VEC>(x, at + cols + 8 * lanes * k, n - 8 * lanes * k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = (double)g[j] / (1.0 + exp(-(double)g[j])) * (double)v[j];
        m = fmax(m, fabs(d));
        v[j] = (float)d;
      }
      if (pass == 1) {
        if (isinf((float)m)) no_infinities(v);
        if (row) put8(row, ld, c0 + 8 * lanes * k, v, inv);
      }
    }
    if (pass == 0) {
      for (int o = 1; o < lanes; o <<= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
      s = fp8_scale(m, &inv);
    }
  }
  if (scale) *scale = s;
}

// n / d for n < 2^31: with l = ceil(log2 d), m = floor(2^(31 + l) / d) + 1 the
// quotient is n m >> (31 + l) (Granlund and Montgomery's round-up method).
struct FastDiv {
  uint32_t m, s, d;
};
FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  return {(uint32_t)((((uint64_t)1 << (31 + l)) / d) + 1), l, d};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return f.s ? __umulhi(n, f.m) >> (f.s - 1) : n;
}

// A thread's 8 elements as they lie in memory.
template <bool BF16>
struct Raw8 {
  uint4 w[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_raw(const void* base, int64_t at, bool live) {
  Raw8<BF16> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + at * (BF16 ? 2 : 4));
#pragma unroll
  for (int k = 0; k < (BF16 ? 1 : 2); ++k) r.w[k] = live ? p[k] : make_uint4(0, 0, 0, 0);
  return r;
}
template <bool BF16>
__device__ __forceinline__ void unpack(const Raw8<BF16>& r, float (&v)[8]) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(r.w);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = __uint_as_float(!BF16 ? u[j] : j & 1 ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16);
}

// L = 16 / P threads per block of 128, blocks numbered row-major; thread l of
// them has the P pieces of 8 columns (L k + l) 8 .., all loaded before the
// first is worked on. GATED: x is gate|up of 2 * cols columns. Rows of whole
// 16-byte pieces. More pieces pay less often for what is done once per block
// and thread (shuffles, scale, addresses), and hold more registers: plain
// 2048 x 14336 bf16 takes 14.1 us with four (6.3 TB/s) and 17.6 with one,
// gated 31.2 with two (bound by issue slots; fp32 41, 6.4 TB/s) and 37 with
// four or one.
template <bool BF16, bool GATED>
__global__ void __launch_bounds__(256) quantize_kernel(const void* x, uint32_t n_all, int cols, FastDiv kb,
                                                      int64_t ld, uint8_t* q,
                                                      float* scales) {
  constexpr int P = GATED ? 2 : 4, L = kLanesPerBlock / P, kStep = L * kVec;  // pieces, threads of a block
  pdl_launch_dependents();
  pdl_wait();
  // whole warps take part in the shuffles: a block past the end has no columns
  const uint32_t i = blockIdx.x * (256 / L) + threadIdx.x / L;
  const bool live = i < n_all;
  const uint32_t row = div_by(i, kb);
  const int c0 = (int)(i - row * kb.d) * kFp8Block + threadIdx.x % L * kVec;
  const int n = live ? cols - c0 : 0;
  const int64_t at = (int64_t)row * cols * (GATED ? 2 : 1) + c0;
  Raw8<BF16> ra[P], rb[GATED ? P : 1];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    ra[k] = load_raw<BF16>(x, at + kStep * k, kStep * k < n);
    if (GATED) rb[k] = load_raw<BF16>(x, at + cols + kStep * k, kStep * k < n);
  }
  float v[P][8], amax = 0.f, gmin = 0.f, gmax = 0.f;
#pragma unroll
  for (int k = 0; k < P; ++k) {
    unpack<BF16>(ra[k], v[k]);
    if (GATED) {
      float u[8];
      unpack<BF16>(rb[k], u);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        gmin = fminf(gmin, fminf(v[k][j], v[k][j + 1]));
        gmax = fmaxf(gmax, fmaxf(v[k][j], v[k][j + 1]));
        const float2 h = swiglu2(make_float2(v[k][j], v[k][j + 1]), make_float2(u[j], u[j + 1]));
        v[k][j] = h.x;
        v[k][j + 1] = h.y;
      }
    }
    amax = fmaxf(amax, absmax8(v[k]));
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  uint8_t* out = live ? q + row * ld : nullptr;
  float* to = live && threadIdx.x % L == 0 ? scales + i : nullptr;
  if (GATED && __any_sync(0xffffffffu, live && (gmin < kGateMin || gmax > kGateMax || fp8_scale_unsure(amax)))) {
    swiglu64<BF16, true>(x, at, cols, n, out, ld, c0, P, L, to);
    return;
  }
  float inv;
  const float s = fp8_scale(amax, &inv);
  const bool inf = !GATED && __any_sync(0xffffffffu, isinf(amax));
  if (!live) return;
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if (inf) no_infinities(v[k]);
    put8(out, ld, c0 + kStep * k, v[k], inv);
  }
  if (to) *to = s;
}

// The same for any other rows: a half-warp per block, element by element. 2048 x
// 14335 bf16: 20.5 us against 13 for 14336; gated 1024 x 14335: 22 us.
template <bool BF16, bool GATED>
__global__ void __launch_bounds__(256) quantize_any_kernel(const void* x, uint32_t n_all, int cols,
                                                          FastDiv kb, int64_t ld, uint8_t* q,
                                                          float* scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x & (kLanesPerBlock - 1);
  const uint32_t i = blockIdx.x * 16 + threadIdx.x / kLanesPerBlock;
  const bool live = i < n_all;
  const uint32_t row = div_by(i, kb);
  const int c = (int)(i - row * kb.d) * kFp8Block + sub * kVec;
  const int n = live ? cols - c : 0;
  const int64_t at = (int64_t)row * cols * (GATED ? 2 : 1) + c;
  float v[8], gmin = 0.f, gmax = 0.f;
  load8<BF16, false>(x, at, n, v);
  if (GATED) {
    float u[8];
    load8<BF16, false>(x, at + cols, n, u);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      gmin = fminf(gmin, fminf(v[j], v[j + 1]));
      gmax = fmaxf(gmax, fmaxf(v[j], v[j + 1]));
      const float2 h = swiglu2(make_float2(v[j], v[j + 1]), make_float2(u[j], u[j + 1]));
      v[j] = h.x;
      v[j + 1] = h.y;
    }
  }
  const float amax = block_max(absmax8(v));
  uint8_t* out = live ? q + row * ld : nullptr;
  float* to = live && sub == 0 ? scales + i : nullptr;
  if (GATED && __any_sync(0xffffffffu, live && (gmin < kGateMin || gmax > kGateMax || fp8_scale_unsure(amax)))) {
    swiglu64<BF16, false>(x, at, cols, n, out, ld, c, 1, kLanesPerBlock, to);
    return;
  }
  float inv;
  const float s = fp8_scale(amax, &inv);
  if (!GATED && __any_sync(0xffffffffu, isinf(amax))) no_infinities(v);
  if (out) put8(out, ld, c, v, inv);
  if (to) *to = s;
}

// A thread's 8 elements as they lie in shared memory (bf16: 16 bytes, fp32: 32).
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint8_t* p, float (&v)[8]) {
  uint32_t u[BF16 ? 4 : 8];
#pragma unroll
  for (int k = 0; k < (BF16 ? 1 : 2); ++k) {
    const uint4 w = reinterpret_cast<const uint4*>(p)[k];
    u[4 * k] = w.x; u[4 * k + 1] = w.y; u[4 * k + 2] = w.z; u[4 * k + 3] = w.w;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = __uint_as_float(!BF16 ? u[j] : j & 1 ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16);
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// With eps 0 and a root mean square below 2.9e-39 (a row of subnormal numbers)
// 1 / root leaves fp32: root() is infinite. Such a row's t are taken times kLift
// (exact) and its factor divided by it. A row of zeros keeps 0 / 0. And where
// the factor is not finite (a NaN in the row, 0 / 0), 0 times it is no padding.
// Neither can happen with an eps and rows of whole 16 bytes: the forms of the
// kernels for those (CAREFUL false) have none of the checks, which cost fp32 rows
// 3 to 9 % (8192 x 2048 with both outputs 42.6 us without, 46.5 with).
constexpr double kLift = 0x1p64;
__device__ __forceinline__ float lifted_root(double mean) { return (float)(1.0 / (sqrt(mean) * kLift)); }

// What the norm kernels do with a thread's 8 values t of one chunk (columns
// c .., lifted if the row is), their weights and the row's statistics: h = t
// rstd g as bf16 and / or 8 bits. mean64(): the mean of squares (plus eps) in 64 bits, asked for by a
// whole warp and only where it decides a scale.
template <bool VEC, bool CAREFUL, typename Mean64>
__device__ __forceinline__ void norm_out(const NormArgs& a, int64_t row, int64_t ld, int kb, int c,
                                         const float (&t)[8], const float (&g)[8], float rstd, Mean64 mean64) {
  const int n = a.cols - c;
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = t[j] * rstd * g[j];
  if (a.y) store8<true, VEC>(a.y, row * a.cols + c, n, h);  // (the same whether 8 bits are asked for or not)
  if (a.q) {
    float inv;
    const float amax = block_max(absmax8(h));
    float s = fp8_scale(amax, &inv);
    bool unsure = c - (int)(threadIdx.x & (kLanesPerBlock - 1)) * kVec < a.cols && fp8_scale_unsure(amax);
    if (__any_sync(0xffffffffu, unsure)) {
      if (amax < 1e-30f) {  // a block of zeros is sure
        float any = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) any = fmaxf(any, t[j] != 0.f && g[j] != 0.f ? 1.f : 0.f);
        unsure = unsure && any != 0.f;
      }
      if (__any_sync(0xffffffffu, unsure)) {
        double r = 1.0 / sqrt(mean64());
        if (CAREFUL && isinf((float)r)) r /= kLift;
        double m = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double e = (double)t[j] * r * (double)g[j];
          m = fmax(m, fabs(e));
          h[j] = (float)e;
        }
        m = block_max(m);
        s = fp8_scale(m, &inv);
        if (isinf((float)m)) no_infinities(h);
      }
    }
    if (isinf(amax)) no_infinities(h);
    if (CAREFUL) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = j < n ? h[j] : 0.f;
    }
    put8(a.q + row * ld, ld, c, h, inv);
    const int b = c / kFp8Block;
    if ((threadIdx.x & (kLanesPerBlock - 1)) == 0 && b < kb) a.scales[row * kb + b] = s;
  }
}
// 1 / sqrt of a mean of squares, which may lie beyond the range of fp32: the
// hardware's root (2 ulp, the same for a whole row, and enough to turn some
// bytes) with one Newton step, its residual in 64 bits.
__device__ __forceinline__ float root(double mean) {
  if (!(mean < 1e37 && mean > 1e-37)) return (float)(1.0 / sqrt(mean));
  const float r = rsqrtf((float)mean);
  return fmaf(0.5f * r, (float)fma(-mean * r, (double)r, 1.0), r);
}

// Rows blockIdx.x, + gridDim.x, ... one after another; thread t has the columns
// 8 (i T + t) .. + 7 for i < NCH, and their weights in registers. It copies its
// own pieces of the next rows into shared memory (cp.async, D slots): a slot
// is filled again after the next row's barrier, when no warp can still want
// the row for its mean in 64 bits.
// Sums are fp32 in a warp (10 roundings deep at most, of positive terms, and
// the root halves their error) and 64 bits across warps; other 64 bits come on
// demand. 8192 x 2048 fp32 rows with both outputs: 43 us, 5.9 TB/s; 8192 x 3584 with
// 8 bits out: 86 us, 4.4 TB/s (its 64 registers spill).
template <bool XBF16, bool RBF16, int NCH, int D, bool CAREFUL>
__global__ void __launch_bounds__(NCH == 1 ? 256 : 1024) rmsnorm_kernel(NormArgs a, int64_t rows) {
  constexpr int XB = XBF16 ? 16 : 32, RB = RBF16 ? 16 : 32;  // bytes of 8 elements
  const int T = blockDim.x, tid = threadIdx.x, cols = a.cols;
  const int64_t ld = fp8_ld(cols), step = gridDim.x;
  const int kb = fp8_blocks(cols);
  extern __shared__ __align__(16) uint8_t ring[];  // [D][NCH][T] pieces of x, then of the residual
  __shared__ float part[2][32];
  pdl_launch_dependents();
  auto col = [&](int i) { return (i * T + tid) * kVec; };
  auto xslot = [&](int d, int i, int t) { return ring + ((d * NCH + i) * T + t) * XB; };
  auto rslot = [&](int d, int i, int t) { return ring + D * NCH * T * XB + ((d * NCH + i) * T + t) * RB; };
  const uint8_t* px = static_cast<const uint8_t*>(a.x) + ((int64_t)blockIdx.x * cols + tid * kVec) * (XB / 8);
  const uint8_t* pr = static_cast<const uint8_t*>(a.res) + ((int64_t)blockIdx.x * cols + tid * kVec) * (RB / 8);
  const int64_t xstep = step * cols * (XB / 8), rstep = step * cols * (RB / 8);
  int64_t fetched = blockIdx.x;
  auto fetch = [&](int d) {  // the next row into slot d
    if (fetched < rows) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (col(i) < cols) {
          cp_async16(xslot(d, i, tid), px + i * T * XB);
          if (!XBF16) cp_async16(xslot(d, i, tid) + 16, px + i * T * XB + 16);
          if (a.res) {
            cp_async16(rslot(d, i, tid), pr + i * T * RB);
            if (!RBF16) cp_async16(rslot(d, i, tid) + 16, pr + i * T * RB + 16);
          }
        }
    }
    fetched += step;
    px += xstep;
    pr += rstep;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // t = x + res, rounded to the residual's type: what the next layer's
  // residual holds and what the norm of the unfused sequence would read; the
  // 16 bytes of a bf16 t come along as they are stored
  auto load_t = [&](int d, int i, int t, float (&v)[8], uint4& w) {
    unpack8<XBF16>(xslot(d, i, t), v);
    if (a.res) {
      float r[8];
      unpack8<RBF16>(rslot(d, i, t), r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
      if (RBF16) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          u[j] = *reinterpret_cast<const uint32_t*>(&p);
          v[2 * j] = __uint_as_float(u[j] << 16);
          v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
        w = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  };
  pdl_wait();
#pragma unroll
  for (int d = 0; d < (D > 1 ? D - 1 : 1); ++d) fetch(d);
  float g[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if (a.weight) {
      load8<false, true>(a.weight, col(i), cols - col(i), g[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = 1.f;
    }
  }
  const double inv_cols = 1.0 / cols;
  int flip = 0, d = 0;
  for (int64_t row = blockIdx.x; row < rows; row += step, flip ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(D > 1 ? D - 2 : 0) : "memory");  // the oldest row
    float t[NCH][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (col(i) < cols) {
        uint4 w;
        load_t(d, i, tid, t[i], w);
        if (a.sum) {
          if (RBF16)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.sum) + row * cols + col(i)) = w;
          else
            store8<false, true>(a.sum, row * cols + col(i), 8, t[i]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i][j] = 0.f;
      }
      float q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = fmaf(t[i][j + 4], t[i][j + 4], t[i][j] * t[i][j]);
      ss += (q[0] + q[1]) + (q[2] + q[3]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((tid & 31) == 0) part[flip][tid >> 5] = ss;
    __syncthreads();  // (the other half of `part` is written before the next barrier)
    if (D > 1) fetch(d == 0 ? D - 1 : d - 1);  // the last row's slot
    double sd = (tid & 31) < T / 32 ? (double)part[flip][tid & 31] : 0.0;
#pragma unroll
    for (int o = 16; o; o >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
    // the row's mean of squares in 64 bits, by one warp from shared memory
    auto mean64 = [&]() {
      double s64 = 0.0;
      for (int k = tid & 31; k < pieces_of(cols); k += 32) {
        float v[8];
        uint4 w;
        load_t(d, k / T, k % T, v, w);
        for (int j = 0; j < 8; ++j) s64 = fma((double)v[j], (double)v[j], s64);
      }
      for (int o = 16; o; o >>= 1) s64 += __shfl_xor_sync(0xffffffffu, s64, o);
      return s64 / cols + (double)a.eps;
    };
    const double mean = fma(sd, inv_cols, (double)a.eps);
    float rstd = root(mean);
    if (!(mean < 1e37 && mean > 1e-30)) {  // squares beyond the range of fp32
      const double m = mean64();
      rstd = root(m);
      if (CAREFUL && isinf(rstd)) {
        rstd = lifted_root(m);
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) t[i][j] *= (float)kLift;
      }
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) norm_out<true, CAREFUL>(a, row, ld, kb, col(i), t[i], g[i], rstd, mean64);
    if (D == 1) {
      __syncthreads();  // every warp is done with the slot
      fetch(0);
    }
    d = d + 1 == D ? 0 : d + 1;
  }
}

// Rows longer than that, or not of whole 16-byte pieces: one CTA per row, the
// row read twice, the sum in 64 bits. 1024 x 32768 bf16 with a residual: 75 us,
// 3.1 TB/s; 8192 x 3583, element by element: 168 us, 1.2 TB/s.
template <bool XBF16, bool RBF16, bool VEC, bool CAREFUL>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(NormArgs a) {
  const int64_t row = blockIdx.x;
  const int T = blockDim.x, tid = threadIdx.x, cols = a.cols;
  const int iters = (pieces_of(cols) + T - 1) / T;
  __shared__ double part[32];
  pdl_launch_dependents();
  pdl_wait();
  auto load_t = [&](int i, float (&v)[8]) {
    const int c = (i * T + tid) * kVec;
    load8<XBF16, VEC>(a.x, row * cols + c, cols - c, v);
    if (a.res) {
      float r[8];
      load8<RBF16, VEC>(a.res, row * cols + c, cols - c, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = RBF16 ? round_bf16(v[j] + r[j]) : v[j] + r[j];
    }
  };
  double ss = 0.0;
  float t[8];
  for (int i = 0; i < iters; ++i) {
    load_t(i, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fma((double)t[j], (double)t[j], ss);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((tid & 31) == 0) part[tid >> 5] = ss;
  __syncthreads();
  ss = 0.0;
  for (int w = 0; w < T / 32; ++w) ss += part[w];
  const double mean = ss / cols + (double)a.eps;
  float rstd = root(mean);
  const bool lift = CAREFUL && isinf(rstd);
  if (lift) rstd = lifted_root(mean);
  for (int i = 0; i < iters; ++i) {
    const int c = (i * T + tid) * kVec;
    load_t(i, t);
    if (a.sum) store8<RBF16, VEC>(a.sum, row * cols + c, cols - c, t);
    if (lift) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] *= (float)kLift;
    }
    float g[8];
    if (a.weight) {
      load8<false, VEC>(a.weight, c, cols - c, g);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 1.f;
    }
    norm_out<VEC, CAREFUL>(a, row, fp8_ld(cols), fp8_blocks(cols), c, t, g, rstd, [&]() { return mean; });
  }
}

// 8 values t of a bf16 row in shared memory: t = x + res, rounded to bf16:
// what the next layer's residual holds and what the norm of the unfused
// sequence would read; their 16 bytes come along as they are stored.
__device__ __forceinline__ void load_sum(const uint8_t* xs, const uint8_t* rs, bool res, float (&v)[8], uint4& w) {
  unpack8<true>(xs, v);
  if (res) {
    float r[8];
    unpack8<true>(rs, r);
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j] + r[2 * j], v[2 * j + 1] + r[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&p);
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// bf16 rows of up to 16384 columns: rows blockIdx.x, + gridDim.x, ... one after
// another. Four threads share a block of 128 columns: thread l of them has the
// four pieces of 8 columns (4 k + l) 8 .., and their weights in registers. Each thread copies its own
// pieces of the next rows into shared memory (cp.async, D slots); a slot is
// filled again after the next row's barrier, when no warp can still want the
// row for its mean in 64 bits.
// The kernel is bound by issue slots: with one piece of a block per thread,
// what is done once per block and thread (shuffles, scale, checks, addresses)
// made 48 instructions an element, and 8192 x 3584 took 50 us, 40 with four.
// (fp32 rows are better off in rmsnorm_kernel, 86 us for 8192 x 3584 against
// some 95 here: they are twice as long in shared memory, and fewer fit.)
constexpr int kPieces = 4, kBf16Slots = 3;
template <bool CAREFUL>
__global__ void __launch_bounds__(512) rmsnorm_bf16_kernel(NormArgs a, int64_t rows) {
  constexpr int D = kBf16Slots, P = kPieces, L = kLanesPerBlock / P, kStep = L * kVec;  // threads of a block, columns from piece to piece
  const int T = blockDim.x, tid = threadIdx.x, cols = a.cols;
  const int64_t ld = fp8_ld(cols), step = gridDim.x;
  const int kb = fp8_blocks(cols), half = T * 16;
  extern __shared__ __align__(16) uint8_t ring[];  // [D][piece][T] of x, then of the residual
  __shared__ float part[2][32];
  pdl_launch_dependents();
  const int blk = tid / L, c0 = blk * kFp8Block + tid % L * kVec;  // piece k starts at column c0 + kStep k
  uint8_t* const xring = ring + tid * 16;
  uint8_t* const rring = xring + (size_t)D * P * half;
  auto xslot = [&](int d, int k) { return xring + (d * P + k) * half; };
  auto rslot = [&](int d, int k) { return rring + (d * P + k) * half; };
  const uint8_t* px = static_cast<const uint8_t*>(a.x) + ((int64_t)blockIdx.x * cols + c0) * 2;
  const uint8_t* pr = static_cast<const uint8_t*>(a.res) + ((int64_t)blockIdx.x * cols + c0) * 2;
  const int64_t xstep = step * cols * 2, rstep = step * cols * 2;
  int64_t fetched = blockIdx.x;
  auto fetch = [&](int d) {  // the next row into slot d
    if (fetched < rows) {
#pragma unroll
      for (int k = 0; k < P; ++k)
        if (c0 + kStep * k < cols) {
          cp_async16(xslot(d, k), px + k * kStep * 2);
          if (a.res) cp_async16(rslot(d, k), pr + k * kStep * 2);
        }
    }
    fetched += step;
    px += xstep;
    pr += rstep;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  pdl_wait();
#pragma unroll
  for (int d = 0; d < D - 1; ++d) fetch(d);
  float g[P][8];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if (a.weight) {
      load8<false, true>(a.weight, c0 + kStep * k, cols - c0 - kStep * k, g[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[k][j] = 1.f;
    }
  }
  const double inv_cols = 1.0 / cols;
  int flip = 0, d = 0;
  for (int64_t row = blockIdx.x; row < rows; row += step, flip ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");  // the oldest row
    float t[P][8];
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if (c0 + kStep * k < cols) {
        uint4 w;
        load_sum(xslot(d, k), rslot(d, k), a.res, t[k], w);
        if (a.sum) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.sum) + row * cols + c0 + kStep * k) = w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[k][j] = 0.f;
      }
      // (two chains of 16 terms and 6 steps across lanes: 22 roundings deep at
      // most, of positive terms; the root halves their error, and its own rounding
      // and two products make 14 2^-24 in all)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 v = make_float2(t[k][j], t[k][j + 1]);
        sq = __ffma2_rn(v, v, sq);
      }
    }
    float ss = sq.x + sq.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if ((tid & 31) == 0) part[flip][tid >> 5] = ss;
    __syncthreads();  // (the other half of `part` is written before the next barrier)
    fetch(d == 0 ? D - 1 : d - 1);  // the last row's slot
    double sd = (tid & 15) < T / 32 ? (double)part[flip][tid & 15] : 0.0;
#pragma unroll
    for (int o = 8; o; o >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
    // the mean of squares (plus eps) in 64 bits, by one warp from shared memory
    auto mean64 = [&]() {
      double s = 0.0;
#pragma unroll 1
      for (int i = (tid & 31) - tid; i < T - tid; i += 32)  // thread tid + i's pieces
#pragma unroll 1
        for (int k = 0; k < P; ++k)
          if ((tid + i) / L * kFp8Block + (tid + i) % L * kVec + kStep * k < cols) {
            float v[8];
            uint4 w;
            load_sum(xslot(d, k) + i * 16, rslot(d, k) + i * 16, a.res, v, w);
            for (int j = 0; j < 8; ++j) s = fma((double)v[j], (double)v[j], s);
          }
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      return s / cols + (double)a.eps;
    };
    const double mean = fma(sd, inv_cols, (double)a.eps);
    float rstd = root(mean);
    if (!(mean < 1e37 && mean > 1e-30)) {  // squares beyond the range of fp32
      const double m = mean64();
      rstd = root(m);
      if (CAREFUL && isinf(rstd)) {
        rstd = lifted_root(m);
#pragma unroll
        for (int k = 0; k < P; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) t[k][j] *= (float)kLift;
      }
    }

    // p = t g, its maximum over the block gives the scale; h = p rstd
    float pm = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[k][j] *= g[k][j];
        pm = fmaxf(pm, fabsf(t[k][j]));
      }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, o));
    const float amax = fmaxf(pm * rstd, 0.f);  // (a row of NaN has no maximum)
    bool far = blk < kb && fp8_far(pm), in64 = false;  // (y is the same whether 8 bits are asked for or not)
    bool unsure = far || (a.q && blk < kb && fp8_scale_unsure(amax));
    if (__any_sync(0xffffffffu, unsure)) {
      // a block of zeros is sure; the others of this warp are formed again in
      // 64 bits, from shared memory
      if (pm == 0.f) {
        float any = 0.f;
#pragma unroll 1
        for (int k = 0; k < P; ++k)
          if (c0 + kStep * k < cols) {
            float v[8];
            uint4 w;
            load_sum(xslot(d, k), rslot(d, k), a.res, v, w);
            for (int j = 0; j < 8; ++j)
              if (v[j] != 0.f && (!a.weight || a.weight[c0 + kStep * k + j] != 0.f)) any = 1.f;
          }
        // (a block's threads are here together; each looks at its own pieces)
        const uint32_t peers = ((1u << L) - 1) << (tid & 31 & ~(L - 1));
        for (int o = 1; o < L; o <<= 1) any = fmaxf(any, __shfl_xor_sync(peers, any, o));
        if (any == 0.f) far = unsure = false;
      }
      if (__any_sync(0xffffffffu, unsure)) {
        const double r = 1.0 / sqrt(mean64());
        double m = 0.0;
        float inv = 1.f, s = 1.f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
          for (int k = 0; k < P; ++k) {
            const int c = c0 + kStep * k;
            float v[8];
            uint4 w;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.f;
            if (c < cols) load_sum(xslot(d, k), rslot(d, k), a.res, v, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const double e = (double)v[j] * r * (a.weight && c < cols ? (double)a.weight[c + j] : 1.0);
              m = fmax(m, fabs(e));
              v[j] = (float)e;
            }
            if (pass == 0) continue;
            if (a.y && far) store8<true, true>(a.y, row * cols + c, cols - c, v);
            if (isinf((float)m)) no_infinities(v);
            if (CAREFUL && c >= cols) {
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = 0.f;
            }
            if (a.q) put8(a.q + row * ld, ld, c, v, inv);
          }
          if (pass == 0) {
#pragma unroll
            for (int o = 1; o < L; o <<= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
            s = fp8_scale(m, &inv);
          }
        }
        if (a.q && tid % L == 0 && blk < kb) a.scales[row * kb + blk] = s;
        in64 = true;
      }
    }
    if (a.y && !(in64 && far)) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        float h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = t[k][j] * rstd;
        store8<true, true>(a.y, row * cols + c0 + kStep * k, cols - c0 - kStep * k, h);
      }
    }
    if (a.q && !in64) {
      float inv;
      const float s = fp8_scale(amax, &inv);
      uint8_t* q = a.q + row * ld;
#pragma unroll
      for (int k = 0; k < P; ++k)
        put8(q, ld, c0 + kStep * k, t[k], !CAREFUL || c0 + kStep * k < cols ? rstd * inv : 0.f);
      if (tid % L == 0 && blk < kb) a.scales[row * kb + blk] = s;
    }
    d = d + 1 == D ? 0 : d + 1;
  }
}

// Blocks of 128 x 128, blockIdx.x, + gridDim.x, ... one after another, the next
// ones on their way into shared memory (cp.async: each thread copies and reads
// its own pieces, no barrier). Of T threads, thread t has the pieces of 16
// bytes t, t + T, ... of the block's rows. Rows of whole pieces. 14336 x 3584
// fp32 takes 48 us (5.3 TB/s), 55 with 512 threads; held in registers from
// load to store, with two CTAs of 256 threads per SM taking turns, 52.
// 11008 x 2048 bf16: 16 us against 26.
template <bool BF16>
struct Enc {
  static constexpr int kThreads = BF16 ? 512 : 1024;
  static constexpr int kPer = BF16 ? 8 : 4;                     // elements of a piece
  static constexpr int kRow = kFp8Block / kPer;                 // pieces of a row
  static constexpr int kPieces = kFp8Block * kRow / kThreads;   // of a thread
  static constexpr int kSlots = BF16 ? 4 : 3;
  static constexpr int kSlot = kFp8Block * kFp8Block * (BF16 ? 2 : 4);
};
template <bool BF16>
__global__ void __launch_bounds__(Enc<BF16>::kThreads, 1) encode_kernel(const void* w, int N, int K, int nb, int kb,
                                                    int64_t n_all, uint8_t* q,
                                                    float* scales) {
  using E = Enc<BF16>;
  constexpr int S = E::kSlots, P = E::kPieces, T = E::kThreads, R = T / E::kRow;  // rows between a thread's pieces
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float part[2][32];
  const int tid = threadIdx.x, c_in = tid % E::kRow * E::kPer, r_in = tid / E::kRow;
  pdl_launch_dependents();
  pdl_wait();
  // (expert, row block, column block) of block i: its first row and column
  auto place = [&](int64_t i, int64_t& row, int& rows, int& c) {
    const int64_t en = i / kb;
    c = (int)(i - en * kb) * kFp8Block + c_in;
    const int64_t e = en / nb;
    const int rb = (int)(en - e * nb);
    row = e * N + rb * kFp8Block;
    rows = min(kFp8Block, N - rb * kFp8Block);
  };
  auto fetch = [&](int64_t i, int slot) {
    if (i < n_all) {
      int64_t row;
      int rows, c;
      place(i, row, rows, c);
      const uint8_t* src = static_cast<const uint8_t*>(w) + ((row + r_in) * K + c) * (BF16 ? 2 : 4);
#pragma unroll
      for (int k = 0; k < P; ++k)
        if (c < K && r_in + k * R < rows)
          cp_async16(ring + slot * E::kSlot + (k * T + tid) * 16, src + (int64_t)k * R * K * (BF16 ? 2 : 4));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < S; ++d) fetch(blockIdx.x + (int64_t)d * gridDim.x, d);
  int slot = 0, flip = 0;
  for (int64_t i = blockIdx.x; i < n_all; i += gridDim.x, flip ^= 1) {
    int64_t row;
    int rows, c;
    place(i, row, rows, c);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    float v[P][E::kPer], m = 0.f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const bool live = c < K && r_in + k * R < rows;
      const uint4 u = live ? *reinterpret_cast<const uint4*>(ring + slot * E::kSlot + (k * T + tid) * 16)
                           : make_uint4(0, 0, 0, 0);
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < E::kPer; ++j) {
        v[k][j] = __uint_as_float(!BF16 ? x[j % 4] : j & 1 ? x[j / 2] & 0xFFFF0000u : x[j / 2] << 16);
        m = fmaxf(m, fabsf(v[k][j]));
      }
    }
    fetch(i + (int64_t)S * gridDim.x, slot);
    if (++slot == S) slot = 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) part[flip][tid >> 5] = m;
    __syncthreads();  // (the other half of `part` is written before the next barrier)
    m = part[flip][tid & (T / 32 - 1)];
#pragma unroll
    for (int o = T / 64; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    const float s = fp8_scale(m, &inv);
    if (tid == 0) scales[i] = s;
    const bool inf = isinf(m);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if (inf) no_infinities(v[k]);
      if (c >= K || r_in + k * R >= rows) continue;
      uint8_t* p = q + (row + r_in + k * R) * K + c;
      uint32_t b[E::kPer / 4];
#pragma unroll
      for (int j = 0; j < E::kPer; j += 4)
        b[j / 4] = e4m3x4(v[k][j] * inv, v[k][j + 1] * inv, v[k][j + 2] * inv, v[k][j + 3] * inv);
      if (BF16)
        *reinterpret_cast<uint2*>(p) = make_uint2(b[0], b[E::kPer / 4 - 1]);
      else
        *reinterpret_cast<uint32_t*>(p) = b[0];
    }
  }
}

// The same for any other rows, one CTA per block, element by element: warp w
// holds rows w, w + 8, ..., lane l the columns l, l + 32, ... Bound by its chain of
// single loads: 14336 x 3583 fp32 takes 121 us, 11008 x 2049 bf16 48.
template <bool BF16>
__global__ void __launch_bounds__(256) encode_any_kernel(const void* w, int N, int K, int nb, int kb,
                                                        uint8_t* q, float* scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t blk = blockIdx.x, en = blk / kb, e = en / nb;
  const int c0 = (int)(blk - en * kb) * kFp8Block, rb = (int)(en - e * nb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nc = min(kFp8Block, K - c0);  // (c0 + 128 may be 2^31)
  auto each = [&](auto f) {
    for (int r = warp; r < min(kFp8Block, N - rb * kFp8Block); r += 8)
      for (int c = lane; c < nc; c += 32) {
        const int64_t at = (e * N + rb * kFp8Block + r) * (int64_t)K + c0 + c;
        f(at, BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(w)[at] << 16)
                   : static_cast<const float*>(w)[at]);
      }
  };
  float m = 0.f;
  each([&](int64_t, float v) { m = fmaxf(m, fabsf(v)); });
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  __shared__ float part[8];
  if (lane == 0) part[warp] = m;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, part[j]);
  float inv;
  const float s = fp8_scale(m, &inv);
  if (threadIdx.x == 0) scales[blk] = s;
  each([&](int64_t at, float v) {
    if (isinf(v)) v = fmaf(v, 0.f, v);
    q[at] = (uint8_t)e4m3x4(v * inv, 0.f, 0.f, 0.f);
  });
}

// Weights [N][K] of one expert into the tiles of the handle; one thread per
// 16 bytes of the destination.
__global__ void __launch_bounds__(256) retile_kernel(const uint8_t* __restrict__ src, uint8_t* __restrict__ dst, int N,
                                                    int K, int kb, int64_t n16) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (i >= n16) return;
  const int64_t tile = i / (kFp8TileBytes / 16);
  const int in = (int)(i % (kFp8TileBytes / 16));
  const int64_t r = tile / kb * kFp8Block + in / 8;
  const int c = (int)(tile % kb) * kFp8Block + in % 8 * 16;
  uint32_t u[4] = {0, 0, 0, 0};
  if (r < N) {
    if ((K & 15) == 0 && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
      if (c < K) {
        const uint4 t = *reinterpret_cast<const uint4*>(src + r * K + c);
        u[0] = t.x; u[1] = t.y; u[2] = t.z; u[3] = t.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c + j < K) u[j >> 2] |= (uint32_t)src[r * K + c + j] << (8 * (j & 3));
    }
  }
  reinterpret_cast<uint4*>(dst)[i] = make_uint4(u[0], u[1], u[2], u[3]);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <bool GATED>
cudaError_t launch_quant(const void* x, int bf16, int64_t rows, int cols, uint8_t* q, float* scales, cudaStream_t s) {
  const uint32_t n = (uint32_t)(rows * fp8_blocks(cols));  // < 2^31, checked by the caller
  const FastDiv kb = fast_div((uint32_t)fp8_blocks(cols));
  constexpr uint32_t kPer = 16 * (GATED ? 2 : 4);  // blocks per CTA
  auto go = [&](auto kern, uint32_t per) {
    return launch_pdl(kern, (n + per - 1) / per, 256, 0, s, x, n, cols, kb, fp8_ld(cols), q, scales);
  };
  if (cols % 8 == 0 && aligned16(x))
    return bf16 ? go(quantize_kernel<true, GATED>, kPer) : go(quantize_kernel<false, GATED>, kPer);
  return bf16 ? go(quantize_any_kernel<true, GATED>, 16) : go(quantize_any_kernel<false, GATED>, 16);
}

// CTAs of `kern` with t threads and smem bytes of dynamic shared memory that
// are resident on the current device at once, asked once for each (which also
// lets the kernel have that much shared memory).
cudaError_t resident(const void* kern, int t, size_t smem, int64_t* ctas) {
  struct Known {
    int device;
    const void* kern;
    int t;
    size_t smem;
    int64_t ctas;
  };
  static std::mutex mu;
  static std::vector<Known> known;
  int dev = 0, per = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (const Known& k : known)
    if (k.device == dev && k.kern == kern && k.t == t && k.smem == smem) {
      *ctas = k.ctas;
      return cudaSuccess;
    }
  if ((e = allow_max_smem(kern)) != cudaSuccess ||
      (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, t, smem)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  *ctas = (int64_t)std::max(1, per) * sms;
  try {
    known.push_back({dev, kern, t, smem, *ctas});
  } catch (const std::bad_alloc&) {  // asked again next time
  }
  return cudaSuccess;
}

template <bool XB, bool RB, bool VEC, bool CAREFUL>
cudaError_t launch_norm_as(const NormArgs& a, int64_t rows, cudaStream_t s) {
  // `pieces` of 8 columns per thread, `depth` rows in shared memory, as many
  // CTAs as fit at once
  const int ch = pieces_of(a.cols);
  auto go = [&](auto kern, int t, int pieces, int depth) -> cudaError_t {
    t = (t + 31) / 32 * 32;
    const size_t smem = (size_t)depth * pieces * t * ((XB ? 16 : 32) + (a.res ? RB ? 16 : 32 : 0));
    int64_t fit = 0;
    const cudaError_t e = resident(reinterpret_cast<const void*>(kern), t, smem, &fit);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, (unsigned)std::min(rows, fit), (unsigned)t, smem, s, a, rows);
  };
  if constexpr (VEC && XB && RB) {
    const int t = fp8_blocks(a.cols) * (kLanesPerBlock / kPieces);
    if (a.cols <= 16384) return go(rmsnorm_bf16_kernel<CAREFUL>, t, kPieces, kBf16Slots);
  } else if constexpr (VEC) {
    if (ch <= 256) return go(rmsnorm_kernel<XB, RB, 1, 4, CAREFUL>, ch, 1, 4);
    if (ch <= 1024) return go(rmsnorm_kernel<XB, RB, 2, 3, CAREFUL>, (ch + 1) / 2, 2, 3);
    if (ch <= 2048) return go(rmsnorm_kernel<XB, RB, 2, 1, CAREFUL>, (ch + 1) / 2, 2, 1);
  }
  return launch_pdl(rmsnorm_long_kernel<XB, RB, VEC, CAREFUL>, (unsigned)rows,
                    (unsigned)std::min(1024, (ch + 31) / 32 * 32), 0, s, a);
}
template <bool XB, bool RB, bool VEC>
cudaError_t launch_norm(const NormArgs& a, int64_t rows, cudaStream_t s) {
  return a.eps == 0.f || a.cols % 16 ? launch_norm_as<XB, RB, VEC, true>(a, rows, s)
                                     : launch_norm_as<XB, RB, VEC, false>(a, rows, s);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* x, int bf16, int64_t rows, int cols, uint8_t* q, float* scales,
                                cudaStream_t s) {
  return launch_quant<false>(x, bf16, rows, cols, q, scales, s);
}
cudaError_t launch_fp8_swiglu(const void* x, int bf16, int64_t rows, int cols, uint8_t* q, float* scales,
                              cudaStream_t s) {
  return launch_quant<true>(x, bf16, rows, cols, q, scales, s);
}

cudaError_t launch_rmsnorm(const NormArgs& a, int x_bf16, int res_bf16, int64_t rows, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && aligned16(a.x) && aligned16(a.res) && aligned16(a.sum) && aligned16(a.weight) &&
                   aligned16(a.y);
  if (x_bf16) {
    if (res_bf16) return vec ? launch_norm<true, true, true>(a, rows, s) : launch_norm<true, true, false>(a, rows, s);
    return vec ? launch_norm<true, false, true>(a, rows, s) : launch_norm<true, false, false>(a, rows, s);
  }
  if (res_bf16) return vec ? launch_norm<false, true, true>(a, rows, s) : launch_norm<false, true, false>(a, rows, s);
  return vec ? launch_norm<false, false, true>(a, rows, s) : launch_norm<false, false, false>(a, rows, s);
}

cudaError_t launch_fp8_encode(const void* w, int bf16, int n_experts, int N, int K, uint8_t* q, float* scales,
                              cudaStream_t s) {
  const int nb = fp8_blocks(N), kb = fp8_blocks(K);
  const int64_t n = (int64_t)n_experts * nb * kb;
  auto go = [&](auto kern, int threads, size_t smem) -> cudaError_t {
    int64_t fit = 0;
    const cudaError_t e = resident(reinterpret_cast<const void*>(kern), threads, smem, &fit);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, (unsigned)std::min(n, fit), (unsigned)threads, smem, s, w, N, K, nb, kb, n, q, scales);
  };
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q);
  if (bf16) {
    if (K % 8 == 0 && aligned16(w) && qa % 8 == 0)
      return go(encode_kernel<true>, Enc<true>::kThreads, (size_t)Enc<true>::kSlots * Enc<true>::kSlot);
    return launch_pdl(encode_any_kernel<true>, (unsigned)n, 256, 0, s, w, N, K, nb, kb, q, scales);
  }
  if (K % 4 == 0 && aligned16(w) && qa % 4 == 0)
    return go(encode_kernel<false>, Enc<false>::kThreads, (size_t)Enc<false>::kSlots * Enc<false>::kSlot);
  return launch_pdl(encode_any_kernel<false>, (unsigned)n, 256, 0, s, w, N, K, nb, kb, q, scales);
}

cudaError_t launch_fp8_retile(const uint8_t* src, uint8_t* dst, int N, int K, cudaStream_t s) {
  const int kb = fp8_blocks(K);
  const int64_t n16 = (int64_t)fp8_blocks(N) * kb * (kFp8TileBytes / 16);
  retile_kernel<<<(unsigned)((n16 + 255) / 256), 256, 0, s>>>(src, dst, N, K, kb, n16);
  return cudaGetLastError();
}

}  // namespace hxq
