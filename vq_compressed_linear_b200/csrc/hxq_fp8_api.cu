// C ABI of the 8-bit-float layers: argument checks, the weight handle and
// kernel dispatch.
#include <climits>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <new>

#include "hxq_fp8.cuh"

namespace {

int fp8_status(cudaError_t e) {
  if (e == cudaSuccess) return HXQ_OK;
  cudaGetLastError();
  if (e == cudaErrorMemoryAllocation) return HXQ_ENOMEM;
  return e == cudaErrorInvalidValue ? HXQ_EINVAL : HXQ_ECUDA;
}

bool is_type(int t) { return t == HXQ_TYPE_F32 || t == HXQ_TYPE_BF16; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The current device must be the one whose memory each pointer is (pinned host
// memory and managed memory are reachable from any): a kernel launched
// elsewhere would fault. NULL is passed over.
int check_pointers(std::initializer_list<const void*> all) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return HXQ_ECUDA;
  }
  for (const void* p : all) {
    if (!p) continue;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
      cudaGetLastError();
      return HXQ_EINVAL;
    }
    if (a.type == cudaMemoryTypeUnregistered || (a.type == cudaMemoryTypeDevice && a.device != dev)) return HXQ_EINVAL;
  }
  return HXQ_OK;
}

int check_current(int device) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return HXQ_ECUDA;
  }
  return dev == device ? HXQ_OK : HXQ_EINVAL;
}

constexpr int64_t kMaxBlocks = (int64_t)1 << 31;  // blocks of 128 per call: block numbers are 32-bit

bool rows_ok(int64_t rows, int cols) {
  return rows >= 0 && rows < kMaxBlocks && cols >= 1 && rows * (int64_t)hxq::fp8_blocks(cols) < kMaxBlocks;
}

void free_fp8(hxq_fp8* h) {
  if (!h) return;
  cudaFree(h->d_w);
  cudaFree(h->d_ws);
  cudaFree(h->d_status);
  delete h;
}

int mm_impl(hxq_fp8_t h, const uint8_t* xq, const float* xs, const int32_t* offsets, const float* bias, void* y,
            int out_type, int M, void* stream, long long wait_cycles = hxq::kFp8WaitCycles, int withhold = -1) {
  if (!is_type(out_type) || M < 0) return HXQ_EINVAL;
  if (M == 0) return check_current(h->device);
  if (!xq || !xs || !y) return HXQ_EINVAL;
  if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(offsets, 4) || !aligned(bias, 4) ||
      !aligned(y, out_type == HXQ_TYPE_BF16 ? 2 : 4))
    return HXQ_EINVAL;
  // rows are counted up to whole blocks of 256, and (row tile, weight tile) units numbered, in 32 bits
  if (M > INT_MAX - 255 || ((int64_t)M + h->n_experts) * h->n_tiles >= kMaxBlocks) return HXQ_EINVAL;
  if (const int rc = check_current(h->device)) return rc;
  const hxq::Fp8Out out{y, bias, out_type == HXQ_TYPE_BF16 ? 1 : 0};
  return fp8_status(hxq::launch_fp8_mm(*h, xq, xs, offsets, out, M, static_cast<cudaStream_t>(stream), wait_cycles,
                                       withhold));
}

}  // namespace

extern "C" {

int64_t hxq_fp8_ld(int K) { return K < 1 ? HXQ_EINVAL : hxq::fp8_ld(K); }

int hxq_fp8_quantize(const void* x, int x_type, int64_t rows, int cols, uint8_t* q, float* scales, void* stream) {
  if (!is_type(x_type) || !rows_ok(rows, cols)) return HXQ_EINVAL;
  if (rows == 0) return HXQ_OK;
  if (!x || !q || !scales) return HXQ_EINVAL;
  if (!aligned(q, 16) || !aligned(scales, 4) || !aligned(x, x_type == HXQ_TYPE_BF16 ? 2 : 4)) return HXQ_EINVAL;
  if (const int rc = check_pointers({q})) return rc;
  return fp8_status(hxq::launch_fp8_quantize(x, x_type == HXQ_TYPE_BF16, rows, cols, q, scales,
                                             static_cast<cudaStream_t>(stream)));
}

int hxq_fp8_swiglu(const void* gate_up, int type, int64_t rows, int cols, uint8_t* q, float* scales, void* stream) {
  if (!is_type(type) || !rows_ok(rows, cols)) return HXQ_EINVAL;
  if (rows == 0) return HXQ_OK;
  if (!gate_up || !q || !scales) return HXQ_EINVAL;
  if (!aligned(q, 16) || !aligned(scales, 4) || !aligned(gate_up, type == HXQ_TYPE_BF16 ? 2 : 4)) return HXQ_EINVAL;
  if (const int rc = check_pointers({q})) return rc;
  return fp8_status(hxq::launch_fp8_swiglu(gate_up, type == HXQ_TYPE_BF16, rows, cols, q, scales,
                                           static_cast<cudaStream_t>(stream)));
}

int hxq_fp8_encode(const void* W, int type, int n_experts, int N, int K, uint8_t* q, float* scales, void* stream) {
  if (!W || !q || !scales || !is_type(type) || n_experts < 1 || N < 1 || K < 1) return HXQ_EINVAL;
  if ((int64_t)hxq::fp8_blocks(N) * hxq::fp8_blocks(K) >= kMaxBlocks / n_experts) return HXQ_EINVAL;
  if (!aligned(scales, 4) || !aligned(W, type == HXQ_TYPE_BF16 ? 2 : 4)) return HXQ_EINVAL;
  if (const int rc = check_pointers({q})) return rc;
  return fp8_status(hxq::launch_fp8_encode(W, type == HXQ_TYPE_BF16, n_experts, N, K, q, scales,
                                           static_cast<cudaStream_t>(stream)));
}

int hxq_rmsnorm(const void* x, int x_type, const void* residual, void* sum, int residual_type, const float* weight,
                float eps, int64_t rows, int cols, void* y_bf16, uint8_t* q, float* scales, void* stream) {
  if (!is_type(x_type) || !is_type(residual_type) || !rows_ok(rows, cols)) return HXQ_EINVAL;
  if (!(eps >= 0.f) || std::isinf(eps)) return HXQ_EINVAL;
  if (rows == 0) return HXQ_OK;
  if (!x || (!y_bf16 && !q) || !q != !scales || (sum && !residual)) return HXQ_EINVAL;
  const uintptr_t rt = residual_type == HXQ_TYPE_BF16 ? 2 : 4;
  if (!aligned(x, x_type == HXQ_TYPE_BF16 ? 2 : 4) || !aligned(residual, rt) || !aligned(sum, rt) ||
      !aligned(weight, 4) || !aligned(y_bf16, 2) || !aligned(q, 16) || !aligned(scales, 4))
    return HXQ_EINVAL;
  if (const int rc = check_pointers({y_bf16, q, scales, sum})) return rc;
  const hxq::NormArgs a{x, residual, sum, weight, eps, cols, static_cast<uint16_t*>(y_bf16), q, scales};
  return fp8_status(hxq::launch_rmsnorm(a, x_type == HXQ_TYPE_BF16, residual_type == HXQ_TYPE_BF16, rows,
                                        static_cast<cudaStream_t>(stream)));
}

int hxq_fp8_create(const uint8_t* W, const float* scales, int n_experts, int N, int K, hxq_fp8_t* out) {
  if (!out) return HXQ_EINVAL;
  *out = nullptr;
  if (!W || !scales || n_experts < 1 || n_experts > HXQ_FP8_MAX_EXPERTS || N < 1 || K < 1) return HXQ_EINVAL;
  const int nt = hxq::fp8_blocks(N), kb = hxq::fp8_blocks(K);
  // rows of 128 bytes are addressed with 32-bit coordinates
  if ((int64_t)nt * kb >= kMaxBlocks / hxq::kFp8Block / n_experts) return HXQ_EINVAL;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return HXQ_EUNSUPPORTED;
  }
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return HXQ_ECUDA;
  }
  if (major != 10 || minor != 0) return HXQ_EUNSUPPORTED;

  hxq_fp8* h = new (std::nothrow) hxq_fp8();
  if (!h) return HXQ_ENOMEM;
  h->n_experts = n_experts;
  h->N = N;
  h->K = K;
  h->n_tiles = nt;
  h->n_blocks = kb;
  h->device = dev;
  h->num_sms = sms;
  const size_t tiles = (size_t)n_experts * nt * kb, per = (size_t)nt * kb * hxq::kFp8TileBytes;
  const size_t src = (size_t)N * K;
  uint8_t* d_src = nullptr;  // one expert's weights as given
  // (whatever writes W and scales on other streams of the device is waited for)
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->d_w), tiles * hxq::kFp8TileBytes);
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->d_ws), tiles * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&h->d_status), sizeof(int));
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&d_src), src);
  if (e == cudaSuccess) e = cudaMemset(h->d_status, 0, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpy(h->d_ws, scales, tiles * sizeof(float), cudaMemcpyDefault);
  for (int i = 0; e == cudaSuccess && i < n_experts; ++i) {
    e = cudaMemcpy(d_src, W + i * src, src, cudaMemcpyDefault);
    if (e == cudaSuccess) e = hxq::launch_fp8_retile(d_src, h->d_w + i * per, N, K, nullptr);
  }
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  cudaFree(d_src);
  CUtensorMap* const maps[] = {&h->tm_w, &h->tm_w64, &h->tm_w32};
  for (int i = 0; e == cudaSuccess && i < 3; ++i)
    e = hxq::fp8_tensor_map(maps[i], h->d_w, hxq::kFp8Block, tiles * hxq::kFp8Block, hxq::kFp8Block, 128u >> i);
  if (e != cudaSuccess) {
    free_fp8(h);
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? HXQ_ENOMEM : HXQ_ECUDA;
  }
  *out = h;
  return HXQ_OK;
}

int hxq_fp8_forward(hxq_fp8_t h, const uint8_t* xq, const float* xs, const float* bias, void* y, int out_type, int M,
                    void* stream) {
  if (!h || h->n_experts != 1) return HXQ_EINVAL;
  return mm_impl(h, xq, xs, nullptr, bias, y, out_type, M, stream);
}

int hxq_fp8_forward_grouped(hxq_fp8_t h, const uint8_t* xq, const float* xs, const int32_t* offsets, const float* bias,
                            void* y, int out_type, int M, void* stream) {
  if (!h || !offsets) return HXQ_EINVAL;
  return mm_impl(h, xq, xs, offsets, bias, y, out_type, M, stream);
}

int hxq_fp8_info(hxq_fp8_t h, int* n_experts, int* N, int* K) {
  if (!h) return HXQ_EINVAL;
  if (n_experts) *n_experts = h->n_experts;
  if (N) *N = h->N;
  if (K) *K = h->K;
  return HXQ_OK;
}

int hxq_fp8_check(hxq_fp8_t h) {
  if (!h) return HXQ_EINVAL;
  if (const int rc = check_current(h->device)) return rc;
  int status = 0;
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(&status, h->d_status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) {
    cudaGetLastError();
    return HXQ_ECUDA;
  }
  if (status == 0) return HXQ_OK;
  cudaMemset(h->d_status, 0, sizeof(int));
  cudaDeviceSynchronize();
  return HXQ_ETIMEOUT;
}

int hxq_test_fp8_forward_withheld(hxq_fp8_t h, const uint8_t* xq, const float* xs, const int32_t* offsets, float* y,
                                  int M, int withhold_stage, unsigned wait_limit_us, void* stream) {
  if (!h || (!offsets && h->n_experts != 1)) return HXQ_EINVAL;
  if (withhold_stage < -1 || wait_limit_us < 1 || wait_limit_us > 2000000u) return HXQ_EINVAL;
  return mm_impl(h, xq, xs, offsets, nullptr, y, HXQ_TYPE_F32, M, stream, wait_limit_us * 2000ll, withhold_stage);
}

void hxq_fp8_destroy(hxq_fp8_t h) {
  if (!h) return;
  cudaDeviceSynchronize();
  free_fp8(h);
}

}  // extern "C"
