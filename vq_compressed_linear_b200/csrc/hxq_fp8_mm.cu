// Block-scaled product of 8-bit-float activations and weights on the sm_100a
// tensor cores, for one layer or for the experts of one:
//
//   y[m][n] = sum_b xs[m][b] ws[n / 128][b] P_b[m][n] (+ bias[n]),
//   P_b[m][n] = sum_{k in block b} xq[m][k] wq[n][k],   blocks of 128 columns.
//
// P_b is one 128-deep step of tcgen05.mma kind::f8f6f4 (e4m3 x e4m3, fp32 in
// tensor memory); the scales differ from block to block, so every P_b is read
// back and added to fp32 accumulators in registers, times its two scales.
// Products of e4m3 values carry 8 significand bits and are exact in fp32.
//
// fp8_skinny_kernel: D = W . x^T, lanes = 128 output features, columns = BN
// tokens. Bound by the weights' bytes for few tokens. The unit of work is
// (expert, 128-row tile of W, block of BN tokens); a cluster of CTAs shares a
// unit's K, each CTA streaming its part of the tile row with TMA, and the
// partial sums meet in distributed shared memory: rank r adds the columns it
// owns in rank order, so results are bitwise repeatable and no global
// workspace exists. The units are numbered token block fastest (token blocks
// of one tile run side by side and share it in L2) and taken round robin by a
// persistent grid.
//
// Warps: 0 TMA loads, 1 MMA issue, 2 TMEM, 3 activation scales (cp.async
// into the ring slot of their block), 4..7 epilogue. Every wait is bounded:
// on timeout the CTA sets a status bit, drains what it issued, frees TMEM
// and returns.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>

#include "hxq_fp8.cuh"

namespace hxq {
namespace {

struct MmArgs {
  const float* xs;
  const float* ws;
  const int* offsets;  // or null: one expert with all M rows
  Fp8Out out;
  int M, N, K, n_tiles, n_blocks, n_experts;
  int* status;
};

// ---- PTX that only these kernels use ----------------------------------------

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Shared-memory descriptor of a K-major operand in the 128-byte swizzle
// layout: rows of 128 bytes, 8-row atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor: D fp32, A and B e4m3, both K-major, M x N.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// One arrival on `bar` once this thread's earlier cp.async have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Arrival on the barrier at `bar` (this CTA's address) of the cluster's CTA `rank`.
__device__ __forceinline__ void mbar_arrive_rank(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
               ::"r"(map_to_rank(smem_u32(bar), rank)) : "memory");
}
// mbar_wait for barriers that other CTAs of the cluster arrive on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 63) == 63) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort = 1;
        return false;
      }
    }
  }
}

// ---- row ranges of the experts ------------------------------------------------

// In shared memory: first[e], rows[e] of expert e, and unit0[e] = the number
// of token blocks before expert e (unit0[E] = all). Offsets outside [0, M] or
// falling are clamped to empty ranges, so that no row outside x or y is
// touched whatever the array holds.
struct Ranges {
  int* first;
  int* rows;
  int* unit0;
};
__device__ __forceinline__ Ranges ranges_at(void* p, int E) {
  int* i = static_cast<int*>(p);
  return {i, i + E, i + 2 * E};
}
constexpr size_t ranges_bytes(int E) { return ((size_t)(3 * E + 1) * sizeof(int) + 15) / 16 * 16; }

// All threads of the CTA; ends with a barrier.
template <int BN>
__device__ __forceinline__ void load_ranges(const Ranges& R, const MmArgs& a) {
  const int E = a.n_experts;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int lo = 0, hi = a.M;
    if (a.offsets) {
      lo = min(max(__ldg(a.offsets + e), 0), a.M);
      hi = min(max(__ldg(a.offsets + e + 1), lo), a.M);
    }
    R.first[e] = lo;
    R.rows[e] = hi - lo;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + (int)threadIdx.x;
      const int n = e < E ? (R.rows[e] + BN - 1) / BN : 0;
      int s = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if ((int)threadIdx.x >= o) s += t;
      }
      if (e < E) R.unit0[e] = base + s - n;
      base += __shfl_sync(0xffffffffu, s, 31);
    }
    if (threadIdx.x == 0) R.unit0[E] = base;
  }
  __syncthreads();
}

// A walk over the units of one cluster: u, u + step, ... The expert only moves
// forward.
template <int BN>
struct Walk {
  int u, step, total, e = 0;
  int tile, row, ntok;  // of the current unit: tile of W, first row, rows
  __device__ __forceinline__ Walk(const Ranges& R, const MmArgs& a, int first, int stride)
      : u(first), step(stride), total(R.unit0[a.n_experts] * a.n_tiles) {}
  __device__ __forceinline__ bool get(const Ranges& R, const MmArgs& a) {
    if (u >= total) return false;
    while (R.unit0[e + 1] * a.n_tiles <= u) ++e;
    const int n_tb = R.unit0[e + 1] - R.unit0[e];
    const int local = u - R.unit0[e] * a.n_tiles;
    tile = local / n_tb;
    const int tb = local - tile * n_tb;
    row = R.first[e] + tb * BN;
    ntok = min(BN, R.rows[e] - tb * BN);
    return true;
  }
  __device__ __forceinline__ void next() { u += step; }
};

// ---- few tokens ---------------------------------------------------------------

constexpr int kSkThreads = 256;
template <int BN>
struct Sk {
  static constexpr int kXBytes = BN * kFp8Block;
  static constexpr int kStage = kFp8TileBytes + kXBytes;
  static constexpr int kSlots = BN <= 16 ? 9 : BN <= 32 ? 8 : BN <= 64 ? 7 : 4;  // TMA ring
  static constexpr int kAcc = BN <= 64 ? 4 : 4;                                  // P_b ring in TMEM
  static constexpr int kCols = kAcc * BN < 32 ? 32 : kAcc * BN;                  // a power of two
  static constexpr int kRecv = BN * kFp8Block * 4;                               // cluster sums
  static constexpr size_t smem(int E) { return 1024 + (size_t)kSlots * kStage + kRecv + ranges_bytes(E); }
};

template <int BN>
__global__ void __launch_bounds__(kSkThreads, 1)
fp8_skinny_kernel(const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmx, MmArgs a,
                  int cluster) {
  using C = Sk<BN>;
  constexpr int S = C::kSlots, A = C::kAcc;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
  float* recv = reinterpret_cast<float*>(ring + S * C::kStage);  // [source rank][own column][128 rows]
  const Ranges R = ranges_at(reinterpret_cast<uint8_t*>(recv) + C::kRecv, a.n_experts);
  __shared__ uint64_t bar_full[S], bar_empty[S], bar_p[A], bar_pfree[A], bar_s[A], bar_drain;
  __shared__ uint64_t bar_recv[4], bar_rfree[4];  // per quadrant of rows
  __shared__ __align__(16) float sc[A][BN + 4];   // the block's activation scales, then the tile's scale
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster > 1 ? (int)cluster_rank() : 0;
  const int my = blockIdx.x / cluster, n_clusters = gridDim.x / cluster;
  const int kb0 = rank * a.n_blocks / cluster, kb1 = (rank + 1) * a.n_blocks / cluster;
  volatile int* abrt = &abort_sh;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
    }
    for (int i = 0; i < A; ++i) {
      mbar_init(&bar_p[i], 1);
      mbar_init(&bar_pfree[i], 4);
      mbar_init(&bar_s[i], 32);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar_recv[i], cluster);
      mbar_init(&bar_rfree[i], cluster);
    }
    mbar_init(&bar_drain, 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmw);
    prefetch_tmap(&tmx);
  }
  if (warp == 2) {
    tmem_alloc(&tmem_sh, C::kCols);
    tmem_relinquish();
  }
  // everything the previous kernel may have written (x, scales, offsets) or
  // still read (y) is touched after this
  pdl_wait();
  tc_fence_before();
  load_ranges<BN>(R, a);  // (has the CTA's barriers)
  tc_fence_after();
  if (cluster > 1) {  // the others' barriers exist before they are arrived on
    cluster_arrive_release();
    cluster_wait();
  }
  const uint32_t tmem = tmem_sh;

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0, b = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (Walk<BN> w(R, a, my, n_clusters); ok && w.get(R, a); w.next()) {
        const int t0 = (w.e * a.n_tiles + w.tile) * a.n_blocks;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = mbar_wait(&bar_empty[b], ph ^ 1, abrt, 32))) break;
          uint8_t* slot = ring + b * C::kStage;
          mbar_arrive_expect_tx(&bar_full[b], C::kStage);
          tma_load_2d(slot, &tmw, &bar_full[b], 0, (t0 + kb) * kFp8Block);
          tma_load_2d(slot + kFp8TileBytes, &tmx, &bar_full[b], kb * kFp8Block, w.row);
          ++issued;
          if (++b == S) b = 0, ph ^= 1;
        }
      }
      if (*abrt) {  // let the copies this thread issued land before the CTA ends
        volatile int never = 0;
        for (int i = max(0, issued - S); i < issued; ++i) mbar_wait(&bar_full[i % S], (i / S) & 1, &never);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int b = 0, p = 0;
      uint32_t ph = 0, pph = 0;
      bool ok = true;
      for (Walk<BN> w(R, a, my, n_clusters); ok && w.get(R, a); w.next()) {
        const uint32_t idesc = idesc_e4m3(128, (w.ntok + 15) / 16 * 16);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = mbar_wait(&bar_pfree[p], pph ^ 1, abrt) && mbar_wait(&bar_full[b], ph, abrt))) break;
          tc_fence_after();
          const uint32_t wa = smem_u32(ring + b * C::kStage);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f8(tmem + p * BN, smem_desc(wa + kk * 32), smem_desc(wa + kFp8TileBytes + kk * 32), idesc, kk > 0);
          tc_commit(&bar_empty[b]);
          tc_commit(&bar_p[p]);
          if (++b == S) b = 0, ph ^= 1;
          if (++p == A) p = 0, pph ^= 1;
        }
      }
      if (*abrt) {  // let issued MMAs finish before TMEM is freed
        volatile int never = 0;
        tc_commit(&bar_drain);
        mbar_wait(&bar_drain, 0, &never);
      }
    }
  } else if (warp == 3) {
    int p = 0;
    uint32_t pph = 0;
    bool ok = true;
    for (Walk<BN> w(R, a, my, n_clusters); ok && w.get(R, a); w.next()) {
      const float* ws = a.ws + (size_t)(w.e * a.n_tiles + w.tile) * a.n_blocks;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait(&bar_pfree[p], pph ^ 1, abrt, 32))) break;
#pragma unroll
        for (int c = lane; c < BN; c += 32)  // columns past the tokens take the last one's scale
          cp_async4(&sc[p][c], a.xs + (size_t)(w.row + min(c, w.ntok - 1)) * a.n_blocks + kb);
        if (lane == 0) cp_async4(&sc[p][BN], ws + kb);
        cp_async_arrive(&bar_s[p]);
        if (++p == A) p = 0, pph ^= 1;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 4) {
    const int q = warp & 3, r = q * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    const int cpr = BN / cluster;  // columns each rank adds up
    int p = 0;
    uint32_t pph = 0, uph = 0;
    bool ok = true;
    for (Walk<BN> w(R, a, my, n_clusters); ok && w.get(R, a); w.next()) {
      float acc[BN];
#pragma unroll
      for (int c = 0; c < BN; ++c) acc[c] = 0.f;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait(&bar_s[p], pph, abrt) && mbar_wait(&bar_p[p], pph, abrt))) break;
        tc_fence_after();
        const float wsc = sc[p][BN];
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 16) {
          if (c0 < w.ntok) {
            uint32_t d[16];
            tmem_ld16(lane_base + p * BN + c0, d);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 s4 = *reinterpret_cast<const float4*>(&sc[p][c0 + j]);
              acc[c0 + j] = fmaf(__uint_as_float(d[j]) * s4.x, wsc, acc[c0 + j]);
              acc[c0 + j + 1] = fmaf(__uint_as_float(d[j + 1]) * s4.y, wsc, acc[c0 + j + 1]);
              acc[c0 + j + 2] = fmaf(__uint_as_float(d[j + 2]) * s4.z, wsc, acc[c0 + j + 2]);
              acc[c0 + j + 3] = fmaf(__uint_as_float(d[j + 3]) * s4.w, wsc, acc[c0 + j + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_pfree[p]);
        if (++p == A) p = 0, pph ^= 1;
      }
      if (!ok) break;
      const int n = w.tile * kFp8Block + r;
      Out o{a.out.y, a.out.bias ? a.out.bias + (size_t)w.e * a.N : nullptr, a.out.bf16};
      if (cluster == 1) {
        if (n < a.N) {
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (c < w.ntok) store_out(o, (size_t)(w.row + c) * a.N + n, n, acc[c]);
        }
        continue;
      }
      // this rank's sums of column c to slot [rank][c % cpr] of the rank that owns c
      if (!(ok = mbar_wait_cluster(&bar_rfree[q], uph ^ 1, abrt))) break;
      const uint32_t mine = smem_u32(recv) + (uint32_t)(rank * cpr * kFp8Block + r) * 4u;
#pragma unroll
      for (int c = 0; c < BN; ++c)
        if (c < w.ntok) {
          const int dst = c / cpr;
          st_cluster_f32(map_to_rank(mine + (uint32_t)((c - dst * cpr) * kFp8Block) * 4u, dst), acc[c]);
        }
      __syncwarp();
      if (lane < cluster) mbar_arrive_rank(&bar_recv[q], lane);
      if (!(ok = mbar_wait_cluster(&bar_recv[q], uph, abrt))) break;
      for (int c = 0; c < cpr; ++c) {
        const int col = rank * cpr + c;
        if (col >= w.ntok) break;
        float v = 0.f;
        for (int s = 0; s < cluster; ++s) v += recv[(s * cpr + c) * kFp8Block + r];
        if (n < a.N) store_out(o, (size_t)(w.row + col) * a.N + n, n, v);
      }
      __syncwarp();
      if (lane < cluster) mbar_arrive_rank(&bar_rfree[q], lane);
      uph ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if (*abrt && threadIdx.x == 0) atomicOr(a.status, kStatusWaitTimeout);
  if (cluster > 1) {  // no CTA leaves while another may still store into its shared memory
    cluster_arrive_release();
    cluster_wait();
  }
}

template <int BN>
cudaError_t launch_skinny(const hxq_fp8& h, const uint8_t* xq, const MmArgs& a, cudaStream_t s) {
  CUtensorMap tmx;
  cudaError_t e = fp8_tensor_map(&tmx, xq, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)fp8_ld(a.K), BN);
  if (e != cudaSuccess) return e;
  auto kern = fp8_skinny_kernel<BN>;
  if ((e = allow_max_smem(reinterpret_cast<const void*>(kern))) != cudaSuccess) return e;
  // units: exact for one layer; for experts every expert with rows has at
  // least one token block and at most one that is not full
  const int64_t most = (int64_t)a.n_tiles * (std::min(a.n_experts, a.M) + (a.n_experts > 1 ? a.M / BN : (a.M - 1) / BN));
  // as many CTAs on a unit as leave the GPU's SMs one each, and every CTA two blocks of K
  int c = 1;
  while (c < 8 && most * c * 2 <= h.num_sms && c * 4 <= a.n_blocks) c *= 2;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(most, h.num_sms / c)) * c;
  if (c == 1) return launch_pdl(kern, (unsigned)grid, kSkThreads, Sk<BN>::smem(a.n_experts), s, h.tm_w, tmx, a, c);
  return launch_pdl_cluster(kern, (unsigned)grid, kSkThreads, Sk<BN>::smem(a.n_experts), (unsigned)c, s, h.tm_w, tmx,
                            a, c);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

}  // namespace

cudaError_t fp8_tensor_map(CUtensorMap* tm, const void* base, uint64_t cols, uint64_t rows, uint64_t ld,
                           uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {(cuuint32_t)kFp8Block, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

cudaError_t launch_fp8_mm(const hxq_fp8& h, const uint8_t* xq, const float* xs, const int* offsets, const Fp8Out& out,
                          int M, cudaStream_t s) {
  const MmArgs a{xs, h.d_ws, offsets, out, M, h.N, h.K, h.n_tiles, h.n_blocks, h.n_experts, h.d_status};
  // tokens an expert gets on average decide the block of tokens
  const int per = (M + h.n_experts - 1) / h.n_experts;
  if (per <= 16) return launch_skinny<16>(h, xq, a, s);
  if (per <= 32) return launch_skinny<32>(h, xq, a, s);
  if (per <= 64) return launch_skinny<64>(h, xq, a, s);
  return launch_skinny<128>(h, xq, a, s);
}

}  // namespace hxq
