// Definitions shared by the 8-bit-float translation units: the scale rule,
// the weight handle with its tile layout, and the launchers.
//
// Format: e4m3 values (largest 448) with one fp32 scale per block, one row x
// 128 columns for activations and 128 x 128 for weights.
#pragma once

#include <cuda.h>

#include "hxq_internal.cuh"

namespace hxq {

constexpr int kFp8Block = 128;          // columns (and weight rows) per scale
constexpr int kFp8MaxExperts = HXQ_FP8_MAX_EXPERTS;  // per handle: the kernels keep every expert's row range in shared memory
constexpr int kFp8TileBytes = kFp8Block * kFp8Block;

// Row length in bytes of an 8-bit activation: a multiple of 16, which the
// tensor maps need.
__host__ __device__ inline int64_t fp8_ld(int K) { return ((int64_t)K + 15) / 16 * 16; }
__host__ __device__ inline int fp8_blocks(int n) { return n / kFp8Block + (n % kFp8Block != 0); }

}  // namespace hxq

// Weights of one layer, or of the experts of one layer. Expert e's rows are
// cut into tiles of 128 rows x 128 columns, zero padded; tile (e, t, b) is
// 16 KB of row-major bytes at ((e * n_tiles + t) * n_blocks + b) * 16 KB, so
// that the tiles of one row panel are read front to back and every tile has
// one scale, ws[(e * n_tiles + t) * n_blocks + b].
struct hxq_fp8 {
  int n_experts, N, K;
  int n_tiles;       // ceil(N / 128)
  int n_blocks;      // ceil(K / 128)
  int device, num_sms;
  uint8_t* d_w;
  float* d_ws;
  int* d_status;     // device-side error word (bounded waits that gave up)
  // the tiles as rows of 128 bytes in the 128-byte swizzle, boxes of 128, 64 and 32 rows
  CUtensorMap tm_w, tm_w64, tm_w32;
};

namespace hxq {

// 2D tensor map of bytes, 128-byte rows of the box in the 128-byte swizzle.
cudaError_t fp8_tensor_map(CUtensorMap* tm, const void* base, uint64_t cols, uint64_t rows, uint64_t ld,
                           uint32_t box_rows);

struct Fp8Out {
  void* y;
  const float* bias;  // [n_experts][N] fp32, or null
  int bf16;
};

// offsets: device int32 [n_experts + 1], or null for one expert with all M
// rows. wait_cycles bounds every pipeline wait (about 2 s by default);
// withhold >= 0 is a test hook (that stage of each CTA never gets its
// activations).
constexpr long long kFp8WaitCycles = 4000000000ll;
cudaError_t launch_fp8_mm(const hxq_fp8& h, const uint8_t* xq, const float* xs, const int* offsets, const Fp8Out& out,
                          int M, cudaStream_t s, long long wait_cycles = kFp8WaitCycles, int withhold = -1);
cudaError_t launch_fp8_retile(const uint8_t* src, uint8_t* dst, int N, int K, cudaStream_t s);
cudaError_t launch_fp8_quantize(const void* x, int bf16, int64_t rows, int cols, uint8_t* q, float* scales,
                                cudaStream_t s);
cudaError_t launch_fp8_swiglu(const void* gate_up, int bf16, int64_t rows, int cols, uint8_t* q, float* scales,
                              cudaStream_t s);
cudaError_t launch_fp8_encode(const void* w, int bf16, int n_experts, int N, int K, uint8_t* q, float* scales,
                              cudaStream_t s);
struct NormArgs {
  const void* x;
  const void* res;      // or null
  void* sum;            // x + res, in res's type, or null
  const float* weight;  // or null for ones
  float eps;
  int cols;
  uint16_t* y;          // bf16, or null
  uint8_t* q;           // or null (then scales is null too)
  float* scales;
};
cudaError_t launch_rmsnorm(const NormArgs& a, int x_bf16, int res_bf16, int64_t rows, cudaStream_t s);

#if defined(__CUDACC__)

// The scale of a block whose largest magnitude is amax: the smallest power of
// two s with amax <= 448 s, kept in [2^-126, 2^120]; 1 for a block of zeros.
// With amax = m 2^E, m in [1, 2), and 448 = 1.75 2^8 the exponent is E - 8,
// plus one when m > 1.75: adding 0x1FFFFF to the bits carries into the
// exponent exactly then. *inv receives 1 / s, also a power of two, so that
// x * inv is exact (up to underflow). Infinity is scaled as the largest
// finite number.
__device__ __forceinline__ float fp8_scale(float amax, float* inv) {
  const uint32_t b = __float_as_uint(fminf(amax, 3.402823466e38f));
  int e = (int)((b + 0x1FFFFFu) >> 23) - 8;  // biased by 127
  e = b == 0 ? 127 : max(e, 1);
  *inv = __uint_as_float((uint32_t)(254 - e) << 23);
  return __uint_as_float((uint32_t)e << 23);
}
// The same for an amax held in 64 bits.
__device__ __forceinline__ float fp8_scale(double amax, float* inv) {
  const uint64_t b = (uint64_t)__double_as_longlong(fmin(amax, 3.402823466e38));
  int e = (int)((b + 0x3FFFFFFFFFFFFull) >> 52) - 1023 + 127 - 8;
  e = b == 0 ? 127 : max(e, 1);
  *inv = __uint_as_float((uint32_t)(254 - e) << 23);
  return __uint_as_float((uint32_t)e << 23);
}
// Whether an amax computed in fp32 with a relative error of a few 2^-24 could
// belong to the next scale (its significand is next to 1.75), or its terms may
// have under- or overflowed on the way: such a block is computed again in 64
// bits, so that a scale never depends on fp32 rounding.
__device__ __forceinline__ bool fp8_far(float v) { return !(v >= 1e-30f && v < 1e37f); }
__device__ __forceinline__ bool fp8_scale_unsure(float amax) {
  return ((__float_as_uint(amax) & 0x7FFFFFu) - (0x600000u - 32u)) <= 64u || fp8_far(amax);
}

#endif  // __CUDACC__

}  // namespace hxq
