// Row-wise operators that write 8-bit-float activations, and the weight
// encoder:
//   quantize  q = e4m3(x / s), one scale s per row and 128 columns
//   swiglu    the same of silu(gate) * up
//   rmsnorm   t = x + residual;  h = t / sqrt(mean(t^2) + eps) * weight;
//             the same of h, and / or h as bf16
//   encode    q = e4m3(w / s), one scale per 128 x 128 block
// All are bound by HBM: each element is read once and written once, the
// block maximum and the row's sum of squares are taken from registers.
//
// Scales are powers of two, so the division is exact and a byte depends only
// on the value that is rounded: one rounding, to nearest even, to 4
// significand bits. Values of h and silu(g) * u are formed in fp32 (a few
// 2^-24, far below that rounding); where such an error could move a block to
// the next scale the block is formed again in 64 bits (fp8_scale_unsure).
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>

#include "hxq_fp8.cuh"

namespace hxq {
namespace {

constexpr int kVec = 8;                        // elements per thread and block of 128: 16 lanes share a block
constexpr int kLanesPerBlock = kFp8Block / kVec;

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

// e4m3 bytes of 4 values already divided by their scale. Infinities become
// NaN (e4m3 has none), like NaN: 0 * v adds NaN exactly then.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo =
      __nv_cvt_float2_to_fp8x2(make_float2(fmaf(a, 0.f, a), fmaf(b, 0.f, b)), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi =
      __nv_cvt_float2_to_fp8x2(make_float2(fmaf(c, 0.f, c), fmaf(d, 0.f, d)), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
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

// The 8 bytes of one lane (8 values of its block) and, from the block's first
// lane, the scale. `c` is the lane's first column: bytes are written up to
// the row's padded length.
__device__ __forceinline__ void put8(uint8_t* row, int64_t ld, int c, const float (&v)[8], float inv) {
  if (c >= ld) return;
  const uint2 w = make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                             e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  *reinterpret_cast<uint2*>(row + c) = w;
}

// silu(g) * u. The fp32 form is off by a few 2^-24 relative: one rounding
// each in the exponential (2 ulp), the sum, the quotient and the product.
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + expf(-g)) * u; }
__device__ __forceinline__ double swiglu64(float g, float u) { return (double)g / (1.0 + exp(-(double)g)) * (double)u; }

// One half-warp per block of 128, blocks numbered row-major; GATED: x is
// gate|up of 2 * cols columns.
template <bool BF16, bool VEC, bool GATED>
__global__ void __launch_bounds__(256) quantize_kernel(const void* __restrict__ x, uint32_t n_all, int cols, int kb,
                                                      int64_t ld, uint8_t* __restrict__ q,
                                                      float* __restrict__ scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x & (kLanesPerBlock - 1);
  // whole warps take part in the shuffles: a warp covers two blocks, the second may be past the end
  const uint32_t step = gridDim.x * (blockDim.x / kLanesPerBlock);
  for (uint32_t i0 = blockIdx.x * (blockDim.x / kLanesPerBlock) + (threadIdx.x / 32) * 2; i0 < n_all; i0 += step) {
    const uint32_t i = i0 + ((threadIdx.x >> 4) & 1);
    const bool live = i < n_all;
    const int64_t row = live ? i / (uint32_t)kb : 0;
    const int b = live ? (int)(i - (uint32_t)row * kb) : 0;
    const int c = b * kFp8Block + sub * kVec;
    const int n = live ? cols - c : 0;
    float v[8];
    if (GATED) {
      float g[8], u[8];
      load8<BF16, VEC>(x, row * 2 * cols + c, n, g);
      load8<BF16, VEC>(x, row * 2 * cols + cols + c, n, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = swiglu(g[j], u[j]);
      float inv, amax = block_max(absmax8(v));
      float s = fp8_scale(amax, &inv);
      if (__any_sync(0xffffffffu, live && fp8_scale_unsure(amax))) {
        double m = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double d = swiglu64(g[j], u[j]);
          m = fmax(m, fabs(d));
          v[j] = (float)d;
        }
        s = fp8_scale(block_max(m), &inv);
      }
      if (live) {
        put8(q + row * ld, ld, c, v, inv);
        if (sub == 0) scales[i] = s;
      }
    } else {
      load8<BF16, VEC>(x, row * cols + c, n, v);
      float inv;
      const float s = fp8_scale(block_max(absmax8(v)), &inv);
      if (live) {
        put8(q + row * ld, ld, c, v, inv);
        if (sub == 0) scales[i] = s;
      }
    }
  }
}

// One CTA per row. Thread t holds the columns 8 (i T + t) .. + 7, i < NCH, in
// registers between the sum of squares and the output; NCH = 0: rows longer
// than the registers hold, read twice.
template <bool XBF16, bool RBF16, bool VEC, int NCH>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(NormArgs a) {
  const int64_t row = blockIdx.x;
  const int T = blockDim.x, tid = threadIdx.x, cols = a.cols;
  const int64_t ld = fp8_ld(cols);
  const int kb = fp8_blocks(cols), n_ch = (cols + kVec - 1) / kVec;
  const int iters = NCH ? NCH : (n_ch + T - 1) / T;
  __shared__ double part[32];
  pdl_launch_dependents();
  pdl_wait();
  float t[NCH ? NCH : 1][8];

  // t = x + res, rounded to the residual's type: what the next layer's
  // residual holds and what the norm of the unfused sequence would read
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
  // the sum of squares in 64 bits: the scales follow from it
  double ss = 0.0;
  if (NCH) {
#pragma unroll
    for (int i = 0; i < (NCH ? NCH : 1); ++i) load_t(i, t[i]);
#pragma unroll
    for (int i = 0; i < (NCH ? NCH : 1); ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fma((double)t[i][j], (double)t[i][j], ss);
  } else {
    for (int i = 0; i < iters; ++i) {
      load_t(i, t[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fma((double)t[0][j], (double)t[0][j], ss);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((tid & 31) == 0) part[tid >> 5] = ss;
  __syncthreads();
  ss = (tid & 31) < T / 32 ? part[tid & 31] : 0.0;
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const double mean = ss / cols + (double)a.eps;
  // (sums of squares beyond the range of fp32: the root in 64 bits)
  const float rstd = mean > 1e37 || mean < 1e-37 ? (float)(1.0 / sqrt(mean)) : rsqrtf((float)mean);

#pragma unroll
  for (int i = 0; i < (NCH ? NCH : 1); ++i) {
    for (int ii = i; ii < (NCH ? i + 1 : iters); ++ii) {
      if (!NCH) load_t(ii, t[0]);
      const int c = (ii * T + tid) * kVec, n = cols - c;
      float (&tv)[8] = t[NCH ? i : 0];
      if (a.sum) store8<RBF16, VEC>(a.sum, row * cols + c, n, tv);
      float g[8], h[8];
      if (a.weight) {
        load8<false, VEC>(a.weight, c, n, g);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = 1.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = tv[j] * rstd * g[j];
      if (a.q) {
        float inv;
        const float amax = block_max(absmax8(h));
        float s = fp8_scale(amax, &inv);
        const bool live = c - (tid & (kLanesPerBlock - 1)) * kVec < cols;  // the block has columns
        if (__any_sync(0xffffffffu, live && fp8_scale_unsure(amax))) {
          const double r = 1.0 / sqrt(mean);
          double m = 0.0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const double d = (double)tv[j] * r * (double)g[j];
            m = fmax(m, fabs(d));
            h[j] = (float)d;
          }
          s = fp8_scale(block_max(m), &inv);
        }
        put8(a.q + row * ld, ld, c, h, inv);
        const int b = c / kFp8Block;
        if ((tid & (kLanesPerBlock - 1)) == 0 && b < kb) a.scales[row * kb + b] = s;
      }
      if (a.y) store8<true, VEC>(a.y, row * cols + c, n, h);
    }
  }
}

// One CTA per 128 x 128 block: warp w holds rows w, w + 8, ... (16 of them),
// lane l the columns 4 l .. 4 l + 3, in registers between the maximum and the
// output.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) encode_kernel(const void* __restrict__ w, int N, int K, int nb, int kb,
                                                    uint8_t* __restrict__ q, float* __restrict__ scales) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t blk = blockIdx.x;  // (expert, row block, column block)
  const int b = (int)(blk % kb);
  const int64_t en = blk / kb;
  const int rb = (int)(en % nb);
  const int64_t e = en / nb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = b * kFp8Block + lane * 4;
  float v[16][4];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = rb * kFp8Block + i * 8 + warp;
    const int64_t at = (e * N + r) * (int64_t)K + c;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = 0.f;
    if (r < N) {
      if (VEC) {
        if (c < K) {
          if (BF16) {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + at);
            v[i][0] = __uint_as_float(u.x << 16);
            v[i][1] = __uint_as_float(u.x & 0xFFFF0000u);
            v[i][2] = __uint_as_float(u.y << 16);
            v[i][3] = __uint_as_float(u.y & 0xFFFF0000u);
          } else {
            const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
            v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < K)
            v[i][j] = BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(w)[at + j] << 16)
                           : static_cast<const float*>(w)[at + j];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(v[i][j]));
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
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = rb * kFp8Block + i * 8 + warp;
    if (r >= N) continue;
    const uint32_t u = e4m3x4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
    uint8_t* p = q + (e * N + r) * (int64_t)K + c;
    if (VEC) {
      if (c < K) *reinterpret_cast<uint32_t*>(p) = u;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < K) p[j] = (uint8_t)(u >> (8 * j));
    }
  }
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
  const int kb = fp8_blocks(cols);
  const uint32_t n = (uint32_t)(rows * kb);  // < 2^31, checked by the caller
  // 16 blocks of 128 per CTA; beyond 2^20 CTAs they loop
  const unsigned grid = std::min<uint32_t>((n + 15) / 16, 1u << 20);
  const bool vec = cols % 8 == 0 && aligned16(x);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, 256, 0, s, x, n, cols, kb, fp8_ld(cols), q, scales); };
  if (bf16) return vec ? go(quantize_kernel<true, true, GATED>) : go(quantize_kernel<true, false, GATED>);
  return vec ? go(quantize_kernel<false, true, GATED>) : go(quantize_kernel<false, false, GATED>);
}

template <bool XB, bool RB, bool VEC>
cudaError_t launch_norm(const NormArgs& a, int64_t rows, cudaStream_t s) {
  // chunks of 8 per row, over at most 512 threads of up to 4 chunks, then
  // 1024 threads of 4, then rows that are read twice
  const int ch = (a.cols + kVec - 1) / kVec;
  auto go = [&](auto kern, int nch) {
    const int t = std::min(1024, ((ch + nch - 1) / nch + 31) / 32 * 32);
    return launch_pdl(kern, (unsigned)rows, (unsigned)t, 0, s, a);
  };
  if (ch <= 512) return go(rmsnorm_kernel<XB, RB, VEC, 1>, 1);
  if (ch <= 1024) return go(rmsnorm_kernel<XB, RB, VEC, 2>, 2);
  if (ch <= 4096) return go(rmsnorm_kernel<XB, RB, VEC, 4>, 4);
  return go(rmsnorm_kernel<XB, RB, VEC, 0>, 4);
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
  const bool vec = K % 8 == 0 && aligned16(w) && (reinterpret_cast<uintptr_t>(q) & 3) == 0;
  auto go = [&](auto kern) {
    return launch_pdl(kern, (unsigned)((int64_t)n_experts * nb * kb), 256, 0, s, w, N, K, nb, kb, q, scales);
  };
  if (bf16) return vec ? go(encode_kernel<true, true>) : go(encode_kernel<true, false>);
  return vec ? go(encode_kernel<false, true>) : go(encode_kernel<false, false>);
}

cudaError_t launch_fp8_retile(const uint8_t* src, uint8_t* dst, int N, int K, cudaStream_t s) {
  const int kb = fp8_blocks(K);
  const int64_t n16 = (int64_t)fp8_blocks(N) * kb * (kFp8TileBytes / 16);
  retile_kernel<<<(unsigned)((n16 + 255) / 256), 256, 0, s>>>(src, dst, N, K, kb, n16);
  return cudaGetLastError();
}

}  // namespace hxq
