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
// Two kernels: fp8_skinny_kernel for few tokens, bound by the weights' bytes,
// fp8_wide_kernel for many, bound by the tensor cores and the adding; which one
// runs is estimated from the call's sizes (launch_mm). In both, one warp loads
// by TMA, one issues MMAs, one owns TMEM, one brings the activation scales
// (cp.async into a ring), and the others read P_b, add and store. The issuing
// warps run converged and issue through one elected lane: from `if (lane ==
// 0)`, an MMA took 72 cycles to issue instead of 35. Every wait is bounded: on
// timeout the CTA sets a status bit, drains what it issued, frees TMEM and
// returns.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <memory>
#include <mutex>
#include <new>
#include <vector>

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
  long long wait_cycles;  // limit of every wait, in cycles of the SM's clock
  int withhold;           // test hook: that stage of each CTA never gets its activations (-1: none)
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
// The same without ordering any memory but the tensor core's own (the
// tcgen05 fences do that): a release at cluster scope waits for the thread's
// stores and costs about a thousand cycles.
__device__ __forceinline__ void mbar_signal_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits, bounded: false, with *abort set, when the limit passes or another
// thread of the CTA gave up.
struct Patience {
  volatile int* abort;
  long long limit;  // cycles of the SM's clock
};

template <bool CLUSTER>
__device__ __forceinline__ bool try_bar(uint64_t* bar, uint32_t parity) {
  if (!CLUSTER) return mbar_try_wait(bar, parity);
  uint32_t ok;  // for barriers that other CTAs of the cluster arrive on
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Patience w) {
  if (try_bar<CLUSTER>(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (try_bar<CLUSTER>(bar, parity)) return true;
    if ((i & 31) == 0) {
      if (*w.abort) return false;
      if (clock64() - t0 > w.limit) {
        *w.abort = 1;
        return false;
      }
    }
  }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// wait_bar of a whole warp, which takes the same way afterwards. The lanes may
// wait for different barriers: what one of them acquired is ordered for all by
// the __syncwarp (a vote orders no memory).
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, Patience w) {
  const bool ok = __all_sync(0xffffffffu, wait_bar(bar, parity, w));
  __syncwarp();
  return ok;
}
// After an abort: a wait of its own for what this CTA still has in flight.
__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity, long long limit) {
  volatile int mine = 0;
  wait_bar(bar, parity, Patience{&mine, limit});
}
// After an abort, when every CTA of the cluster has stopped: what is in flight
// between them (arrivals, sums, copies counted in another CTA) has no barrier
// that this CTA could wait for. A millisecond is a thousand times what it takes.
__device__ __forceinline__ void settle() {
  const long long t0 = clock64();
  while (clock64() - t0 < 2000000ll) __nanosleep(10000);
}

__device__ __forceinline__ void put_out(const Fp8Out& o, size_t at, float v) {
  if (o.bf16)
    static_cast<__nv_bfloat16*>(o.y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(o.y)[at] = v;
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

// All threads of the CTA; ends with a barrier. Nothing to do for one layer.
template <int BN, bool GROUPED>
__device__ __forceinline__ void load_ranges(const Ranges& R, const MmArgs& a) {
  if (GROUPED) {
    const int E = a.n_experts;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      const int lo = min(max(a.offsets[e], 0), a.M);
      R.first[e] = lo;
      R.rows[e] = min(max(a.offsets[e + 1], lo), a.M) - lo;
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
  }
  __syncthreads();
}

// A walk over the units u, u + step, ... of one cluster. The expert only
// moves forward.
template <int BN, bool GROUPED>
struct Walk {
  int u, step, total, e = 0;
  int tile, row, ntok;  // of the current unit: tile of W, first row, rows
  __device__ __forceinline__ Walk(const Ranges& R, const MmArgs& a, int first, int stride)
      : u(first), step(stride), total((GROUPED ? R.unit0[a.n_experts] : (a.M + BN - 1) / BN) * a.n_tiles) {}
  __device__ __forceinline__ bool get(const Ranges& R, const MmArgs& a) {
    if (u >= total) return false;
    int n_tb = (a.M + BN - 1) / BN, local = u, first = 0, rows = a.M;
    if (GROUPED) {
      while (R.unit0[e + 1] * a.n_tiles <= u) ++e;
      n_tb = R.unit0[e + 1] - R.unit0[e];
      local = u - R.unit0[e] * a.n_tiles;
      first = R.first[e];
      rows = R.rows[e];
    }
    tile = local / n_tb;
    const int tb = local - tile * n_tb;
    row = first + tb * BN;
    ntok = min(BN, rows - tb * BN);
    return true;
  }
  __device__ __forceinline__ void next() { u += step; }
};

// ---- few tokens ---------------------------------------------------------------
//
// fp8_skinny_kernel: D = W . x^T, lanes = 128 output features, columns = BN
// tokens. The unit of work is (expert, 128-row tile of W, block of BN tokens),
// token blocks fastest (those of one tile run side by side and share it in
// L2), taken round robin by a persistent grid. A cluster of CTAs shares a
// unit's K; the partial sums meet in distributed shared memory, where rank r
// adds the columns it owns in rank order: bitwise repeatable, and no global
// workspace. The scale of a column (its token's) comes from shared memory, four
// columns a load, the tile's is one factor more.
// 1 x 11008 x 2048 in 7.0 us (3.2 TB/s of weights), 29 x 2048 x 11008 in 9.3:
// the start (1 us to the first bytes), the last stage's way out and the
// cluster's exchange (2 us) weigh as much as the 3.5 us that HBM needs.

template <int BN>
struct Sk {
  static constexpr int kPer = 2;                 // blocks of K per stage
  // groups of four adding warps, each with every other 16 columns: one group
  // alone takes 1000 cycles for a stage of 64 columns, the MMAs 450
  static constexpr int kGroups = BN >= 32 ? 2 : 1;
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kXBytes = BN * kFp8Block;
  static constexpr int kStage = kPer * (kFp8TileBytes + kXBytes);
  static constexpr int kSlots = BN <= 16 ? 5 : BN <= 32 ? 4 : 3;               // operands in, P out (TMEM)
  static constexpr int kUsed = kSlots * kPer * BN;
  static constexpr int kCols = kUsed <= 256 ? 256 : 512;                       // allocated: a power of two
  static constexpr int kSc = 8;                                                // ring of activation scales
  static constexpr int kMaxCluster = 16;
  static constexpr int kRecv = (BN + kMaxCluster) * kFp8Block * 4;             // cluster sums
  static constexpr size_t smem(int E) { return 1024 + (size_t)kSlots * kStage + kRecv + ranges_bytes(E); }
};

template <int BN, bool GROUPED>
__global__ void __launch_bounds__(Sk<BN>::kThreads, 1)
fp8_skinny_kernel(const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmx, MmArgs a,
                  int cluster, int own, int own_inv) {
  using C = Sk<BN>;
  constexpr int S = C::kSlots, KP = C::kPer, SC = C::kSc, G = C::kGroups;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
  float* recv = reinterpret_cast<float*>(ring + S * C::kStage);  // [source rank][own column][128 rows]
  const Ranges R = ranges_at(reinterpret_cast<uint8_t*>(recv) + C::kRecv, a.n_experts);
  // stage i: operands landed (full), their products are in TMEM (p: the
  // operands' slot is free too), the products have been read (pfree)
  __shared__ uint64_t bar_full[S], bar_p[S], bar_pfree[S], bar_s[SC], bar_sfree[SC], bar_drain;
  __shared__ uint64_t bar_recv[4], bar_rfree[4];  // per quadrant of rows
  __shared__ __align__(16) float sc[SC][KP][BN + 4];  // a block's activation scales, then the tile's scale
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh, issued_sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster > 1 ? (int)cluster_rank() : 0;
  const int my = blockIdx.x / cluster, n_clusters = gridDim.x / cluster;
  const int kb0 = rank * a.n_blocks / cluster, kb1 = (rank + 1) * a.n_blocks / cluster;
  const Patience pat{&abort_sh, a.wait_cycles};

  pdl_launch_dependents();
  // a stage's weights and activations into its slot
  auto load_w = [&](int tile0, int kb, int slot) {
    uint8_t* p = ring + slot * C::kStage;
    const int nk = min(KP, kb1 - kb);
    mbar_arrive_expect_tx(&bar_full[slot], nk * (kFp8TileBytes + C::kXBytes));
    for (int j = 0; j < nk; ++j)
      tma_load_2d(p + j * kFp8TileBytes, &tmw, &bar_full[slot], 0, (tile0 + kb + j) * kFp8Block);
  };
  auto load_x = [&](int row, int kb, int slot) {
    uint8_t* p = ring + slot * C::kStage + KP * kFp8TileBytes;
    for (int j = 0; j < min(KP, kb1 - kb); ++j)
      tma_load_2d(p + j * C::kXBytes, &tmx, &bar_full[slot], (kb + j) * kFp8Block, row);
  };
  // One layer: the first stages' weights are on their way before the rest is
  // set up, and before the previous kernel has finished.
  const int ahead = !GROUPED && my < a.n_tiles * ((a.M + BN - 1) / BN) ? min(S, (kb1 - kb0 + KP - 1) / KP) : 0;
  if (warp == 0) {
    if (elect_one()) {
      for (int i = 0; i < S; ++i) mbar_init(&bar_full[i], 1);
      fence_mbar_init();
      prefetch_tmap(&tmx);
      const int tile = my / ((a.M + BN - 1) / BN);
      for (int i = 0; i < ahead; ++i) load_w(tile * a.n_blocks, kb0 + i * KP, i);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      for (int i = 0; i < S; ++i) {
        mbar_init(&bar_p[i], 1);
        mbar_init(&bar_pfree[i], 4 * G);
      }
      for (int i = 0; i < SC; ++i) {
        mbar_init(&bar_s[i], 32);
        mbar_init(&bar_sfree[i], 4 * G);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(&bar_recv[i], cluster * G);
        mbar_init(&bar_rfree[i], cluster * G);
      }
      mbar_init(&bar_drain, 1);
      abort_sh = 0;
      fence_mbar_init();
    }
  } else if (warp == 2) {
    tmem_alloc(&tmem_sh, C::kCols);
    tmem_relinquish();
  }
  __syncwarp();
  // what the previous kernel may have written (x, scales, offsets) or still
  // read (y) is touched after pdl_wait
  if (GROUPED) pdl_wait();
  tc_fence_before();
  load_ranges<BN, GROUPED>(R, a);  // (has the CTA's barrier)
  tc_fence_after();
  if (cluster > 1) {  // the others' barriers exist before they are arrived on
    cluster_arrive_relaxed();
    cluster_wait();
  }
  const uint32_t tmem = tmem_sh;

  if (warp == 0) {
    int issued = ahead, b = ahead;
    uint32_t ph = 0;
    if (b == S) b = 0, ph ^= 1;
    bool ok = true, first = true;
    pdl_wait();
    for (Walk<BN, GROUPED> w(R, a, my, n_clusters); ok && w.get(R, a); w.next()) {
      const int t0 = (w.e * a.n_tiles + w.tile) * a.n_blocks;
      int kb = kb0;
      if (first) {
        first = false;
        if (elect_one())
          for (int i = 0; i < ahead; ++i)
            if (i != a.withhold) load_x(w.row, kb0 + i * KP, i);
        __syncwarp();
        kb += ahead * KP;
      }
      for (; kb < kb1; kb += KP) {
        if (!(ok = wait_bar_warp(&bar_p[b], ph ^ 1, pat))) break;
        if (elect_one()) {
          load_w(t0, kb, b);
          if (issued != a.withhold) load_x(w.row, kb, b);
        }
        __syncwarp();
        ++issued;
        if (++b == S) b = 0, ph ^= 1;
      }
    }
    if (lane == 0) issued_sh = issued;
  } else if (warp == 1) {
    int b = 0;
    uint32_t ph = 0;
    bool ok = true;
    pdl_wait();  // x is loaded after it: the previous kernel's time does not count against the first wait
    for (Walk<BN, GROUPED> w(R, a, my, n_clusters); ok && w.get(R, a); w.next()) {
      const uint32_t idesc = idesc_e4m3(128, (w.ntok + 15) / 16 * 16);
      for (int kb = kb0; kb < kb1; kb += KP) {
        // (odd lanes wait for the operands, even lanes for the TMEM slot)
        if (!(ok = wait_bar_warp(lane & 1 ? &bar_full[b] : &bar_pfree[b], lane & 1 ? ph : ph ^ 1, pat))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t wd = smem_desc(smem_u32(ring + b * C::kStage));
          const uint64_t xd = smem_desc(smem_u32(ring + b * C::kStage + KP * kFp8TileBytes));
#pragma unroll
          for (int j = 0; j < KP; ++j) {
            if (kb + j < kb1) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // 32 columns of K each: 2 units of 16 bytes
                tc_mma_f8(tmem + (b * KP + j) * BN, wd + (j * kFp8TileBytes >> 4) + kk * 2,
                          xd + (j * C::kXBytes >> 4) + kk * 2, idesc, kk > 0);
            }
          }
          tc_commit(&bar_p[b]);
        }
        __syncwarp();
        if (++b == S) b = 0, ph ^= 1;
      }
    }
  } else if (warp == 3) {
    int p = 0;
    uint32_t ph = 0;
    bool ok = true;
    pdl_wait();
    for (Walk<BN, GROUPED> w(R, a, my, n_clusters); ok && w.get(R, a); w.next()) {
      const float* ws = a.ws + (size_t)(w.e * a.n_tiles + w.tile) * a.n_blocks;
      const float* xs = a.xs + (size_t)w.row * a.n_blocks;
      for (int kb = kb0; kb < kb1; kb += KP) {
        if (!(ok = wait_bar_warp(&bar_sfree[p], ph ^ 1, pat))) break;
#pragma unroll
        for (int i = lane; i < BN * KP; i += 32) {  // (columns past the tokens are never used)
          const int c = i / KP, j = i % KP;
          if (c < w.ntok && kb + j < kb1) cp_async4(&sc[p][j][c], xs + (size_t)c * a.n_blocks + kb + j);
        }
        if (lane < KP && kb + lane < kb1) cp_async4(&sc[p][lane][BN], ws + kb + lane);
        cp_async_arrive(&bar_s[p]);
        if (++p == SC) p = 0, ph ^= 1;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 4) {
    const int q = warp & 3, r = q * 32 + lane, grp = G > 1 ? (warp - 4) >> 2 : 0;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    int p = 0, sp = 0;
    uint32_t pph = 0, sph = 0, uph = 0;
    bool ok = true;
    pdl_wait();  // y
    constexpr int NC = BN / 16 / G;  // pieces of 16 columns: piece i is columns 16 (i G + grp) ..
    for (Walk<BN, GROUPED> w(R, a, my, n_clusters); ok && w.get(R, a); w.next()) {
      const int n_out = w.tile * kFp8Block + r;
      const float bias = a.out.bias && n_out < a.N ? a.out.bias[(size_t)w.e * a.N + n_out] : 0.f;
      float acc[NC][16];
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
      auto live = [&](int i) { return 16 * (i * G + grp) < w.ntok; };
      for (int kb = kb0; kb < kb1; kb += KP) {
        const int nk = min(KP, kb1 - kb);
        if (!(ok = wait_bar_warp(lane & 1 ? &bar_p[p] : &bar_s[sp], lane & 1 ? pph : sph, pat))) break;
        tc_fence_after();
        // the next block's P loads while this one's is added
        uint32_t d[2][NC][16];
        auto load = [&](int k) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (live(i)) tmem_ld16(lane_base + (p * KP + k) * BN + 16 * (i * G + grp), d[k & 1][i]);
        };
        load(0);
#pragma unroll
        for (int k = 0; k < KP; ++k) {
          if (k < nk) {
            tmem_wait_ld();
            if (k + 1 < nk) {
              load(k + 1);
            } else {  // all of the stage has been read
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar_pfree[p]);
            }
            const float* s = sc[sp][k];
            const float ws = s[BN];  // (times the token's first: P times one scale alone may leave fp32)
#pragma unroll
            for (int i = 0; i < NC; ++i)
              if (live(i)) {
                const uint32_t(&v)[16] = d[k & 1][i];
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                  const float4 s4 = *reinterpret_cast<const float4*>(s + 16 * (i * G + grp) + j);
                  acc[i][j] = fmaf(__uint_as_float(v[j]), s4.x * ws, acc[i][j]);
                  acc[i][j + 1] = fmaf(__uint_as_float(v[j + 1]), s4.y * ws, acc[i][j + 1]);
                  acc[i][j + 2] = fmaf(__uint_as_float(v[j + 2]), s4.z * ws, acc[i][j + 2]);
                  acc[i][j + 3] = fmaf(__uint_as_float(v[j + 3]), s4.w * ws, acc[i][j + 3]);
                }
              }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_sfree[sp]);
        if (++p == S) p = 0, pph ^= 1;
        if (++sp == SC) sp = 0, sph ^= 1;
      }
      if (!ok) break;
      if (cluster == 1) {
        if (n_out < a.N) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int c = 16 * (i * G + grp) + j;
              if (c < w.ntok) put_out(a.out, (size_t)(w.row + c) * a.N + n_out, acc[i][j] + bias);
            }
        }
        continue;
      }
      // this rank's sums of column c to slot [rank][c % own] of the rank c / own that adds column c
      if (!(ok = __all_sync(0xffffffffu, wait_bar<true>(&bar_rfree[q], uph ^ 1, pat)))) break;
      const uint32_t mine = smem_u32(recv) + (uint32_t)(rank * own * kFp8Block + r) * 4u;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int c = 16 * (i * G + grp) + j;
          if (c < w.ntok) {
            const int dst = (c * own_inv) >> 16;
            st_cluster_f32(map_to_rank(mine + (uint32_t)((c - dst * own) * kFp8Block) * 4u, dst), acc[i][j]);
          }
        }
      __syncwarp();
      if (lane < cluster) mbar_arrive_rank(&bar_recv[q], lane);
      if (!(ok = __all_sync(0xffffffffu, wait_bar<true>(&bar_recv[q], uph, pat)))) break;
      const int mine_n = min(own, w.ntok - rank * own);
#pragma unroll 2
      for (int c = grp; c < mine_n; c += G) {
        float v = 0.f;
#pragma unroll 4
        for (int s = 0; s < cluster; ++s) v += recv[(s * own + c) * kFp8Block + r];
        if (n_out < a.N) put_out(a.out, (size_t)(w.row + rank * own + c) * a.N + n_out, v + bias);
      }
      if (w.u + w.step < w.total) {  // nobody waits for the last unit's
        __syncwarp();
        if (lane < cluster) mbar_arrive_rank(&bar_rfree[q], lane);
      }
      uph ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  // Every warp has stopped, and what they issued is known: after an abort the
  // copies land and the MMAs finish before shared memory and TMEM are let go.
  const bool aborted = *pat.abort != 0;
  if (aborted) {
    if (warp == 0) {
      const int n = issued_sh;
      for (int i = max(0, n - S); i < n; ++i) drain_bar(&bar_full[i % S], (i / S) & 1, a.wait_cycles);
    } else if (warp == 1) {
      if (elect_one()) tc_commit(&bar_drain);
      __syncwarp();
      drain_bar(&bar_drain, 0, a.wait_cycles);
    }
    if (threadIdx.x == 0) atomicOr(a.status, kStatusWaitTimeout);
    tc_fence_before();
    __syncthreads();
  }
  if (cluster > 1) cluster_arrive_relaxed();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if (cluster > 1) {  // no CTA leaves while another may still reach into its shared memory
    __syncwarp();
    cluster_wait();
    if (aborted) settle();
  }
}

// Clusters of c CTAs of `kern` that fit on the GPU at once, for c = 1 .. 16
// (0: none). Asked once per (device, kernel).
struct ClusterFit {
  const void* kern;
  int device;
  int fit[17];
};
cudaError_t cluster_fit(const void* kern, int device, int threads, size_t smem, const int** fit) {
  static std::mutex mu;
  static std::vector<std::unique_ptr<ClusterFit>> known;
  std::lock_guard<std::mutex> lock(mu);
  for (const auto& k : known)
    if (k->kern == kern && k->device == device) {
      *fit = k->fit;
      return cudaSuccess;
    }
  cudaError_t e = allow_max_smem(kern);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  std::unique_ptr<ClusterFit> f(new (std::nothrow) ClusterFit{kern, device, {}});
  if (!f) return cudaErrorMemoryAllocation;
  for (int c = 1; c <= 16; ++c) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&f->fit[c], kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      f->fit[c] = 0;
    }
  }
  try {
    known.push_back(std::move(f));
  } catch (const std::bad_alloc&) {
    return cudaErrorMemoryAllocation;
  }
  *fit = known.back()->fit;
  return cudaSuccess;
}

cudaError_t fp8_out_map(CUtensorMap* tm, const Fp8Out& out, uint64_t N, uint64_t M);

// Blocks of `tokens` rows that the experts have, exact for one expert. For
// several the host knows only M: about min(experts, M) of them have rows, and
// the last block of each is half full.
template <bool GROUPED>
int64_t token_blocks(const MmArgs& a, int tokens) {
  if (!GROUPED || a.n_experts == 1) return (a.M + tokens - 1) / tokens;
  const int64_t used = std::min(a.n_experts, a.M);
  return std::max<int64_t>(used, (a.M + used * tokens / 2) / tokens);
}

// How a call runs: the cluster size and the microseconds it may take. The
// model is a kernel's start and end, and for each round of units the blocks of
// K that one CTA works through, fitted to measurements of N x K = 2048 x 2048,
// 11008 x 2048, 3584 x 14336 and of 8 and 64 experts at M = 8 .. 12288, which
// it meets within some 20 %; it only has to rank the kernels.
struct Plan {
  int cluster;
  double us;
};
template <int BN, bool GROUPED>
cudaError_t plan_skinny(const hxq_fp8& h, const MmArgs& a, Plan* plan, const int** fit) {
  cudaError_t e = cluster_fit(reinterpret_cast<const void*>(fp8_skinny_kernel<BN, GROUPED>), h.device, Sk<BN>::kThreads,
                              Sk<BN>::smem(GROUPED ? kFp8MaxExperts : 0), fit);
  if (e != cudaSuccess) return e;
  constexpr double kBlock = BN == 16 ? 0.2 : BN == 32 ? 0.26 : 0.43, kExchange = BN <= 32 ? 0.9 : 1.3;
  const int64_t units = a.n_tiles * token_blocks<GROUPED>(a, BN);
  *plan = {1, 1e30};
  for (int c = 1; c <= Sk<BN>::kMaxCluster && c <= a.n_blocks; ++c) {
    if ((*fit)[c] < 1) continue;
    // (the units of several experts are a guess: a third of a round's loss on average)
    const double rounds = GROUPED && a.n_experts > 1 ? std::max(1.0, (double)units / (*fit)[c] + 0.3)
                                                     : (double)((units + (*fit)[c] - 1) / (*fit)[c]);
    const double us = 4.0 + rounds * ((a.n_blocks + c - 1) / c) * kBlock + (c > 1 ? 1.0 + kExchange * rounds : 0.0);
    if (us < plan->us) *plan = {c, us};
    if (units * c > 2 * h.num_sms) break;  // larger clusters only add rounds
  }
  return cudaSuccess;
}

template <int BN, bool GROUPED>
cudaError_t launch_skinny(const hxq_fp8& h, const uint8_t* xq, const MmArgs& a, const Plan& plan, const int* fit,
                          cudaStream_t s) {
  CUtensorMap tmx;
  const cudaError_t e = fp8_tensor_map(&tmx, xq, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)fp8_ld(a.K), BN);
  if (e != cudaSuccess) return e;
  auto kern = fp8_skinny_kernel<BN, GROUPED>;
  const size_t smem = Sk<BN>::smem(GROUPED ? a.n_experts : 0);
  // no more clusters than there can be units
  const int64_t most =
      (int64_t)a.n_tiles * (GROUPED ? std::min(a.n_experts, a.M) + a.M / BN : (a.M + BN - 1) / BN);
  const int c = plan.cluster, own = (BN + c - 1) / c;
  const int own_inv = (65536 + own - 1) / own;  // (x * own_inv) >> 16 = x / own for x < BN
  const unsigned grid = (unsigned)(std::min<int64_t>(most, fit[c]) * c);
  if (c == 1) return launch_pdl(kern, grid, Sk<BN>::kThreads, smem, s, h.tm_w, tmx, a, c, own, own_inv);
  return launch_pdl_cluster(kern, grid, Sk<BN>::kThreads, smem, (unsigned)c, s, h.tm_w, tmx, a, c, own, own_inv);
}

// ---- many tokens ----------------------------------------------------------------
//
// fp8_wide_kernel: D = x . W^T, lanes = tokens, columns = features, by pairs
// of CTAs (tcgen05 cta_group::2): 256 tokens x 256 features a pair, each CTA
// with 128 of the tokens, in shared memory as in TMEM. With tokens on the
// lanes a thread needs one scale per block of K (its token's times its
// tile's), so adding P_b is one multiply-add per element.
//
// P_b has two buffers in TMEM. Eight warps read it, each 32 tokens x half the
// features, 64 columns at a time, and hand it back before they add the last
// ones. A block of K takes 775 cycles against the MMAs' 512: the way round a
// buffer (MMA, commit, read, arrival in the leading CTA, issue) takes 1550.
// 2048 x 14336 x 3584 runs in 107 us, 1.96 PFLOP/s. Tried and slower there (at
// 113 us):
// halves of 128 features with an MMA and buffers of their own, 126 us (their
// MMAs read the 256 tokens from shared memory twice); 16 adding warps, 127;
// reads of 32 columns, each under way while the last one is added, 122.
//
// The units are (expert, 256 tokens, two tiles of W), one after another on
// each pair, in groups of 8 token blocks that walk the features together (so
// that the pairs at work share both operands in L2); what does not fill the
// last round of all pairs is cut into pieces of 128 or 64 features.

constexpr int kWideTokens = 256;
constexpr int kWideSlots = 4;
constexpr int kWideSc = 8;                     // ring of activation scales
constexpr int kWideGroup = 8;                  // token blocks that walk the features together
constexpr int kWideStage = 2 * kFp8TileBytes;  // 128 tokens and up to 128 features of one block of K
constexpr int kWideAdders = 8;                 // warps that add and store: 32 tokens x half the features each
constexpr int kWideThreads = 128 + 32 * kWideAdders;
constexpr int kWideLaunchRegs = 168;           // a thread's at launch: 65536 / 384, a multiple of 8
constexpr int kWideCtlRegs = 40, kWideAddRegs = 224;
static_assert(128 * kWideCtlRegs + 32 * kWideAdders * kWideAddRegs <= kWideThreads * kWideLaunchRegs,
              "register split: setmaxnreg draws on what the block was launched with");
constexpr int kWideOut = 2 * 32 * 128;         // per adding warp: two pieces of 32 rows x 128 bytes on their way out
constexpr size_t wide_smem(int E) { return 1024 + (size_t)kWideSlots * kWideStage + kWideAdders * kWideOut + ranges_bytes(E); }

struct WideWalk {
  int item, step, items, full, cut, cu_n, e = 0;
  int cu, row, ntok;     // of the current unit: pair of tiles, first row, rows
  int width, piece;      // features of the piece, and which
  __device__ __forceinline__ WideWalk(const Ranges& R, const MmArgs& a, bool grouped, int first, int pairs)
      : item(first), step(pairs), cu_n((a.n_tiles + 1) / 2) {
    const int units = (grouped ? R.unit0[a.n_experts] : (a.M + kWideTokens - 1) / kWideTokens) * cu_n;
    full = units / pairs * pairs;
    const int rest = units - full;
    cut = rest * 4 <= pairs ? 4 : rest * 2 <= pairs ? 2 : 1;
    items = full + rest * cut;
  }
  // The next item with work, or false.
  __device__ __forceinline__ bool get(const Ranges& R, const MmArgs& a, bool grouped) {
    for (;; item += step) {
      if (item >= items) return false;
      int u = item;
      width = 256;
      piece = 0;
      if (u >= full) {
        u = full + (item - full) / cut;
        piece = (item - full) % cut;
        width = 256 / cut;
      }
      int n_tb = (a.M + kWideTokens - 1) / kWideTokens, local = u, first = 0, rows = a.M;
      if (grouped) {
        while (R.unit0[e + 1] * cu_n <= u) ++e;
        n_tb = R.unit0[e + 1] - R.unit0[e];
        local = u - R.unit0[e] * cu_n;
        first = R.first[e];
        rows = R.rows[e];
      }
      const int g = local / (kWideGroup * cu_n), in = local - g * kWideGroup * cu_n;
      const int tbs = min(kWideGroup, n_tb - g * kWideGroup);
      cu = in / tbs;
      const int tb = g * kWideGroup + in - cu * tbs;
      row = first + tb * kWideTokens;
      ntok = min(kWideTokens, rows - tb * kWideTokens);
      const int have = 2 * cu + 1 < a.n_tiles ? 256 : 128;  // an odd last tile stands alone
      width = min(width, have);
      if (piece * width < have) return true;
    }
  }
  // Tile of W and row in it of the piece's feature `off`.
  __device__ __forceinline__ int tile(int off) const { return 2 * cu + (piece * width + off) / kFp8Block; }
  __device__ __forceinline__ int tile_row(int off) const { return (piece * width + off) % kFp8Block; }
};

__device__ __forceinline__ void tmem_alloc2(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               ::"r"(smem_u32(dst_smem)), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_mma2_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this address in both CTAs of the pair.
__device__ __forceinline__ void tc_commit2(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
      ::"r"(smem_u32(bar)), "h"((uint16_t)3)
      : "memory");
}
// The same on this CTA's barrier alone.
__device__ __forceinline__ void tc_commit2_own(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(smem_u32(bar)) : "memory");
}
// This CTA's shared memory <- global; the bytes are counted on the barrier `bar` (an address from map_to_rank) of
// either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* tmap, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];"
      ::"r"(smem_u32(dst)), "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
// (a0, a1) += (d0, d1) * (s, s)
__device__ __forceinline__ void fma2(float2& a, uint32_t d0, uint32_t d1, float s) {
  a = __ffma2_rn(make_float2(__uint_as_float(d0), __uint_as_float(d1)), make_float2(s, s), a);
}
// Outputs of a warp, one row per lane: w holds 128 bytes of it, columns n0 ..,
// n of which exist. The rows go through `buf` (swizzled as the tensor map
// has it: 16-byte chunk c of row r at c ^ (r & 7)) and, where all of them exist,
// out as one TMA store that nobody waits for. Stored from the registers, or by a
// bulk copy per lane, a tile's rows took 3500 cycles of 28 blocks' 22000.
__device__ __forceinline__ void store_rows(const Fp8Out& o, const CUtensorMap* tmap, uint8_t* buf, int row, int N,
                                           int n_rows, int n0, int n, int lane, bool tma, const uint32_t (&w)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  // (a box reaches past n only where y ends)
  if (tma && n_rows >= 32 && (n >= 128 / (o.bf16 ? 2 : 4) || n0 + n == N)) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                   ::"l"(tmap), "r"(n0), "r"(row), "r"(smem_u32(buf))
                   : "memory");
    }
  } else {
    __syncwarp();
    const int esz = o.bf16 ? 2 : 4;
    n = min(n, 128 / esz);
    uint8_t* y = static_cast<uint8_t*>(o.y) + ((size_t)row * N + n0) * esz;
    if (tma) {  // rows of whole 16-byte pieces
      const int c = lane & 7;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        if (r < n_rows && c * 16 < n * esz)
          *reinterpret_cast<uint4*>(y + (size_t)r * N * esz + c * 16) =
              *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
      }
    } else {
#pragma unroll 4
      for (int r = 0; r < min(n_rows, 32); ++r)
        for (int b = lane * esz; b < n * esz; b += 32 * esz) {
          const uint8_t* src = buf + r * 128 + (((b >> 4) ^ (r & 7)) << 4) + (b & 15);
          uint8_t* dst = y + (size_t)r * N * esz + b;
          if (o.bf16)
            *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
          else
            *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
        }
    }
    __syncwarp();
  }
  if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The pieces that this warp stored before the last `left` have left `buf`.
template <int LEFT>
__device__ __forceinline__ void stores_read(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
  __syncwarp();
}

struct WideMaps {
  CUtensorMap x;      // 128 tokens
  CUtensorMap y;      // 32 rows x 128 bytes
  CUtensorMap w[3];   // 128, 64, 32 rows of a tile
};

template <bool GROUPED>
__global__ void __launch_bounds__(kWideThreads, 1)
fp8_wide_kernel(const __grid_constant__ WideMaps maps, MmArgs a, int tma_out) {
  constexpr int S = kWideSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
  uint8_t* outs = ring + S * kWideStage;
  const Ranges R = ranges_at(outs + kWideAdders * kWideOut, a.n_experts);
  // full and pfree are used in the leading CTA only; empty and p arrive in both
  __shared__ uint64_t bar_full[S], bar_empty[S], bar_p[2], bar_pfree[2], bar_drain;
  __shared__ uint64_t bar_s[kWideSc], bar_sfree[kWideSc];
  __shared__ float sc[kWideSc][128 + 2];  // a block's activation scales, then the two tiles' scales
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh, issued_sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const Patience pat{&abort_sh, a.wait_cycles};

  pdl_launch_dependents();
  if (warp == 0 && elect_one()) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_p[i], 1);
      mbar_init(&bar_pfree[i], 2 * kWideAdders);
    }
    for (int i = 0; i < kWideSc; ++i) {
      mbar_init(&bar_s[i], 32);
      mbar_init(&bar_sfree[i], kWideAdders);
    }
    mbar_init(&bar_drain, 1);
    abort_sh = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.x);
    prefetch_tmap(&maps.w[0]);
  }
  __syncwarp();
  if (warp == 2) {
    tmem_alloc2(&tmem_sh, 512);
    tmem_relinquish2();
  }
  if (GROUPED) pdl_wait();
  tc_fence_before();
  load_ranges<kWideTokens, GROUPED>(R, a);
  tc_fence_after();
  cluster_arrive_relaxed();
  cluster_wait();
  const uint32_t tmem = tmem_sh;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideCtlRegs));
    if (warp == 0) {
      int issued = 0, b = 0;
      uint32_t ph = 0;
      bool ok = true;
      pdl_wait();
      for (WideWalk w(R, a, GROUPED, pair, pairs); ok && w.get(R, a, GROUPED); w.item += w.step) {
        // of the piece's features each CTA holds one half
        const int rows = w.width / 2, off = rank * rows;
        const CUtensorMap* tw = rows == 128 ? &maps.w[0] : rows == 64 ? &maps.w[1] : &maps.w[2];
        const int w0 = (w.e * a.n_tiles + w.tile(off)) * a.n_blocks * kFp8Block + w.tile_row(off);
        const int x0 = w.row + rank * 128;
        for (int kb = 0; kb < a.n_blocks; ++kb) {
          if (!(ok = wait_bar_warp(&bar_empty[b], ph ^ 1, pat))) break;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(&bar_full[b], 2 * (kFp8TileBytes + rows * kFp8Block));
            const uint32_t bar = map_to_rank(smem_u32(&bar_full[b]), 0);
            uint8_t* slot = ring + b * kWideStage;
            if (issued != a.withhold) tma_load_2d_pair(slot, &maps.x, bar, kb * kFp8Block, x0);
            tma_load_2d_pair(slot + kFp8TileBytes, tw, bar, 0, w0 + kb * kFp8Block);
          }
          __syncwarp();
          ++issued;
          if (++b == S) b = 0, ph ^= 1;
        }
      }
      // The leading CTA's tensor core arrives on this CTA's bar_empty after bar_p, which the adders wait for: the last
      // stages' arrivals land before the CTA leaves its shared memory.
      for (int i = max(0, issued - S); ok && i < issued; ++i)
        ok = wait_bar_warp(&bar_empty[i % S], (i / S) & 1, pat);
      if (lane == 0) issued_sh = issued;
    } else if (warp == 1 && rank == 0) {
      int b = 0, p = 0, issued = 0;
      uint32_t ph = 0, pph = 0;
      bool ok = true;
      pdl_wait();  // x is loaded after it: the previous kernel's time does not count against the first wait
      for (WideWalk w(R, a, GROUPED, pair, pairs); ok && w.get(R, a, GROUPED); w.item += w.step) {
        const uint32_t idesc = idesc_e4m3(256, w.width);
        for (int kb = 0; kb < a.n_blocks; ++kb) {
          const uint64_t xd = smem_desc(smem_u32(ring + b * kWideStage)), wd = xd + (kFp8TileBytes >> 4);
          if (!(ok = wait_bar_warp(lane & 1 ? &bar_full[b] : &bar_pfree[p], lane & 1 ? ph : pph ^ 1, pat))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc_mma2_f8(tmem + p * 256, xd + kk * 2, wd + kk * 2, idesc, kk > 0);
            tc_commit2(&bar_p[p]);
            tc_commit2(&bar_empty[b]);
          }
          __syncwarp();
          ++issued;
          if (++b == S) b = 0, ph ^= 1;
          if (++p == 2) p = 0, pph ^= 1;
        }
      }
      // and so do the other CTA's last arrivals on bar_pfree (relaxed: no barrier at the end orders them)
      for (int i = max(0, issued - 2); ok && i < issued; ++i)
        ok = wait_bar_warp(&bar_pfree[i % 2], (i / 2) & 1, pat);
    } else if (warp == 3) {
      int sp = 0;
      uint32_t sph = 0;
      bool ok = true;
      pdl_wait();
      for (WideWalk w(R, a, GROUPED, pair, pairs); ok && w.get(R, a, GROUPED); w.item += w.step) {
        const float* ws = a.ws + (size_t)(w.e * a.n_tiles + w.tile(lane * w.width / 2)) * a.n_blocks;
        for (int kb = 0; kb < a.n_blocks; ++kb) {
          if (!(ok = wait_bar_warp(&bar_sfree[sp], sph ^ 1, pat))) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = i * 32 + lane, tok = rank * 128 + t;  // (rows past the tokens are never stored)
            if (tok < w.ntok) cp_async4(&sc[sp][t], a.xs + (size_t)(w.row + tok) * a.n_blocks + kb);
          }
          if (lane < 2) cp_async4(&sc[sp][128 + lane], ws + kb);
          cp_async_arrive(&bar_s[sp]);
          if (++sp == kWideSc) sp = 0, sph ^= 1;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWideAddRegs));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t pfree0 = map_to_rank(smem_u32(&bar_pfree[0]), 0);  // in the leading CTA
    int p = 0, sp = 0;
    uint32_t pph = 0, sph = 0;
    bool ok = true;
    pdl_wait();
    for (WideWalk w(R, a, GROUPED, pair, pairs); ok && w.get(R, a, GROUPED); w.item += w.step) {
      const int cols = w.width / 2, col0 = half * cols;
      float2 acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
      for (int kb = 0; kb < a.n_blocks; ++kb) {
        if (!(ok = wait_bar_warp(lane & 1 ? &bar_p[p] : &bar_s[sp], lane & 1 ? pph : sph, pat))) break;
        tc_fence_after();
        const uint32_t at = lane_base + p * 256 + col0;
        const float s = sc[sp][q * 32 + lane] * sc[sp][128 + half];
        uint32_t d[64];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i * 64 < cols) {
            tmem_ld32(at + i * 64, d);
            tmem_ld32(at + i * 64 + 32, d + 32);  // (columns past a narrow width hold nothing that is stored)
            tmem_wait_ld();
            if (i == 1 || cols <= 64) {  // the last read of this buffer and of its scales
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                mbar_signal_at(pfree0 + p * 8);
                mbar_arrive(&bar_sfree[sp]);
              }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) fma2(acc[i * 32 + j], d[2 * j], d[2 * j + 1], s);
          }
        }
        if (++p == 2) p = 0, pph ^= 1;
        if (++sp == kWideSc) sp = 0, sph ^= 1;
      }
      if (!ok) break;
      const int n0 = w.cu * 256 + w.piece * w.width + col0;
      const int n = min(cols, a.N - n0), n_rows = w.ntok - (rank * 128 + q * 32);
      if (n <= 0 || n_rows <= 0) continue;
      const int row = w.row + rank * 128 + q * 32;
      uint8_t* buf = outs + (warp - 4) * kWideOut;
      if (a.out.bias) {
        const float* bias = a.out.bias + (size_t)w.e * a.N + n0;
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          if (2 * j < n) acc[j].x += bias[2 * j];
          if (2 * j + 1 < n) acc[j].y += bias[2 * j + 1];
        }
      }
      uint32_t v[32];
      stores_read<0>(lane);
      if (a.out.bf16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i * 64 >= n) break;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(acc[i * 32 + j].x, acc[i * 32 + j].y);
            v[j] = *reinterpret_cast<const uint32_t*>(&t);
          }
          store_rows(a.out, &maps.y, buf + i * 4096, row, a.N, n_rows, n0 + i * 64, n - i * 64, lane, tma_out, v);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i * 32 >= n) break;
          if (i >= 2) stores_read<1>(lane);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[2 * j] = __float_as_uint(acc[i * 16 + j].x);
            v[2 * j + 1] = __float_as_uint(acc[i * 16 + j].y);
          }
          store_rows(a.out, &maps.y, buf + (i & 1) * 4096, row, a.N, n_rows, n0 + i * 32, n - i * 32, lane, tma_out, v);
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the rows have arrived
  }

  tc_fence_before();
  __syncthreads();
  // as in fp8_skinny_kernel; the other CTA's copies are counted here, too
  const bool aborted = *pat.abort != 0;
  if (aborted) {
    if (warp == 0 && rank == 0) {
      const int n = issued_sh;
      for (int i = max(0, n - S); i < n; ++i) drain_bar(&bar_full[i % S], (i / S) & 1, a.wait_cycles);
    } else if (warp == 1 && rank == 0) {
      if (elect_one()) tc_commit2_own(&bar_drain);
      __syncwarp();
      drain_bar(&bar_drain, 0, a.wait_cycles);
    }
    if (threadIdx.x == 0) atomicOr(a.status, kStatusWaitTimeout);
    tc_fence_before();
    __syncthreads();
  }
  // neither CTA frees TMEM or leaves while the other may still use its memory
  __syncwarp();
  cluster_arrive_relaxed();
  cluster_wait();
  if (aborted) settle();
  __syncwarp();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

template <bool GROUPED>
cudaError_t launch_wide(const hxq_fp8& h, const uint8_t* xq, const MmArgs& a, cudaStream_t s) {
  WideMaps m;
  cudaError_t e = fp8_tensor_map(&m.x, xq, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)fp8_ld(a.K), 128);
  if (e != cudaSuccess) return e;
  m.w[0] = h.tm_w;
  m.w[1] = h.tm_w64;
  m.w[2] = h.tm_w32;
  auto kern = fp8_wide_kernel<GROUPED>;
  if ((e = allow_max_smem(reinterpret_cast<const void*>(kern))) != cudaSuccess) return e;
  // (the register split assumes what the block is launched with)
  static const int regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, reinterpret_cast<const void*>(kern)) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs < kWideLaunchRegs) return cudaErrorLaunchOutOfResources;
  // whole pieces of y leave by TMA where its rows allow a tensor map
  const size_t esz = a.out.bf16 ? 2 : 4;
  const int tma_out = (reinterpret_cast<uintptr_t>(a.out.y) | (uintptr_t)(a.N * esz)) % 16 == 0;
  m.y = m.x;
  if (tma_out && (e = fp8_out_map(&m.y, a.out, (uint64_t)a.N, (uint64_t)a.M)) != cudaSuccess) return e;
  return launch_pdl_cluster(kern, (unsigned)(h.num_sms / 2 * 2), kWideThreads, wide_smem(GROUPED ? a.n_experts : 0), 2,
                            s, m, a, tma_out);
}

template <bool GROUPED>
double wide_us(const hxq_fp8& h, const MmArgs& a) {
  const int64_t units = (a.n_tiles + 1) / 2 * token_blocks<GROUPED>(a, kWideTokens), pairs = h.num_sms / 2;
  const int64_t rest = units % pairs;  // cut as the kernel cuts them
  const double last = rest == 0 ? 0.0 : rest * 4 <= pairs ? 0.355 : rest * 2 <= pairs ? 0.43 : 0.55;
  return 5.0 + (units / pairs * 0.55 + last) * a.n_blocks;
}

template <bool GROUPED>
cudaError_t launch_mm(const hxq_fp8& h, const uint8_t* xq, const MmArgs& a, cudaStream_t s) {
  Plan p16, p32, p64;
  const int *f16, *f32, *f64;
  cudaError_t e = plan_skinny<16, GROUPED>(h, a, &p16, &f16);
  if (e != cudaSuccess) return e;
  // up to 16 rows in all, wider blocks only add work
  if (a.M <= 16) return launch_skinny<16, GROUPED>(h, xq, a, p16, f16, s);
  if ((e = plan_skinny<32, GROUPED>(h, a, &p32, &f32)) != cudaSuccess ||
      (e = plan_skinny<64, GROUPED>(h, a, &p64, &f64)) != cudaSuccess)
    return e;
  const double best = std::min({p16.us, p32.us, p64.us});
  if (wide_us<GROUPED>(h, a) <= best) return launch_wide<GROUPED>(h, xq, a, s);
  if (p16.us <= best) return launch_skinny<16, GROUPED>(h, xq, a, p16, f16, s);
  if (p32.us <= best) return launch_skinny<32, GROUPED>(h, xq, a, p32, f32, s);
  return launch_skinny<64, GROUPED>(h, xq, a, p64, f64, s);
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

// y [M][N], boxes of 32 rows x 128 bytes in the 128-byte swizzle.
cudaError_t fp8_out_map(CUtensorMap* tm, const Fp8Out& out, uint64_t N, uint64_t M) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint32_t esz = out.bf16 ? 2 : 4;
  cuuint64_t dims[2] = {N, M};
  cuuint64_t strides[1] = {N * esz};
  cuuint32_t box[2] = {128 / esz, 32};
  cuuint32_t estr[2] = {1, 1};
  return fn(tm, out.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, out.y, dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
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
                          int M, cudaStream_t s, long long wait_cycles, int withhold) {
  const MmArgs a{xs,     h.d_ws,     offsets,    out,         M,          h.N,        h.K,
                 h.n_tiles, h.n_blocks, h.n_experts, h.d_status, wait_cycles, withhold};
  return offsets ? launch_mm<true>(h, xq, a, s) : launch_mm<false>(h, xq, a, s);
}

}  // namespace hxq
