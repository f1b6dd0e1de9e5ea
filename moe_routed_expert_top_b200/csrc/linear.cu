// linear.cu - the linear product on tcgen05 tensor cores, and what its backward
// pass needs beside it:
//
//   forward   y[m,n]  = act(sum_k x[m,k] w[n,k] + bias[n]) + residual[m,n]
//   backward  dz = dy * act'(z);  dx[m,k] = sum_n dz[m,n] w[n,k];
//             dw[n,k] = sum_m dz[m,n] x[m,k];  dbias[n] = sum_m dz[m,n]
//
// One kernel serves the three products C[m,n] = sum_k A(m,k) B(n,k). What differs
// is which index of A and B is contiguous in memory: k (x and w in the forward,
// dz in dx) or the output index ("MN": w in dx, dz and x in dw). The MMA takes
// either, by a bit of its instruction descriptor and another reading of the
// shared-memory tile, so no operand is transposed in memory.
//
// What bounds it: the tensor cores at training sizes. A CTA pair (cluster of two
// on one TPC) computes a 256 x BN tile with 256-row MMAs (cta_group::2): each CTA
// fetches its 128 rows of A and its half of B's rows, 16 KB + BN/2*128 B per 64
// of k against the 16 KB + BN*128 B that a tile of its own would take. Two
// accumulators in tensor memory let a tile's epilogue run under the next one's
// main loop. Few tiles (a narrow output, few rows): the k range is split over
// the idle pairs, each part leaves fp32 sums in the workspace and a second kernel
// adds them in order and applies the epilogue. An fp32 result is always made of
// parts of at most 2048 k: the tensor core's fp32 accumulator drops the low bits
// of each product sum it adds (about 1e-5 of the result at k = 7168, measured),
// and adding parts in full fp32 keeps an fp32 result near 4e-6.
//
// Operand tiles in shared memory (128-byte swizzle, written by TMA):
//   k contiguous   rows of 64 k = 128 bytes, 8-row groups 1024 B apart; a K = 16
//                  step is 32 bytes along the row;
//   MN contiguous  boxes of 64 output indices (128 bytes) x 64 k rows = 8 KB: 8-k
//                  groups 1024 B apart (stride offset), the next 64 indices 8 KB
//                  on (leading offset); a K = 16 step is two groups, 2 KB.
// Rows and columns past the operands' ends are filled with zeros by TMA and
// masked at the store. Every wait is bounded and sets MOE_DEV_TIMEOUT on expiry.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "internal.h"
#include "linear.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kLinThreads = 320;  // TMA, MMA, two groups of 4 epilogue warps

struct LinParams {
  int M, N, K;
  int tiles_m, tiles_n, splits;
  int kb_total, kb_split;  // 64-wide k blocks: all, and of one split
  float* partial;          // [splits][M][N] when splits > 1
  int32_t* status;
  int wide;                // every row of y, z, residual (and partial) takes 32-byte accesses
  LinearEpilogue e;
};

template <int BN>
struct LCfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = (BN / 2) * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 5 : 7;
  static constexpr int NUM_ACC = 2;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * NUM_ACC + 1;
  // each epilogue warp's 32 x 32 block, its rows 33 apart
  static constexpr int BLOCK_BYTES = 32 * 33 * 4;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + 8 * BLOCK_BYTES + NUM_BARS * 8 + 32;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// Descriptor of an operand tile whose output index is contiguous (see above).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;  // to the next 64 output indices
  d |= static_cast<uint64_t>(1024 >> 4) << 32;  // to the next 8 k
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Work item -> tile. Tiles go in bands of 8 along M, so that the tiles that run
// together share operands in both directions (8 x 9 of them on 74 pairs read 17
// operand strips instead of 75).
__device__ __forceinline__ void lin_decode(const LinParams& p, int t, int& tm, int& tn, int& sp) {
  const int tiles = p.tiles_m * p.tiles_n;
  sp = t / tiles;
  const int i = t - sp * tiles;
  const int band = i / (8 * p.tiles_n);
  const int h = min(8, p.tiles_m - 8 * band);
  const int r = i - band * 8 * p.tiles_n;
  tn = r / h;
  tm = 8 * band + (r - tn * h);
}

__device__ __forceinline__ void lin_st8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void lin_ld8(uint32_t* v, const void* p) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void lin_store32_f32(float* dst, const uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) lin_st8(dst + i, v + i);
}
__device__ __forceinline__ void lin_store32_bf16(__nv_bfloat16* dst, const uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      o[j] = pack_bf16x2(__uint_as_float(v[i + 2 * j]), __uint_as_float(v[i + 2 * j + 1]));
    lin_st8(dst + i, o);
  }
}

template <int kAct>
__device__ __forceinline__ void lin_act32(uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(linear_act(__uint_as_float(v[i]), kAct));
}

// The epilogue of 32 columns n.. of row m, all accesses 32 bytes wide.
__device__ __forceinline__ void lin_store32(const LinearEpilogue& e, long long m, int n, uint32_t (&v)[32]) {
  if (e.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + linear_bias(e, n + i));
  }
  if (e.z != nullptr) lin_store32_bf16(static_cast<__nv_bfloat16*>(e.z) + m * e.ldz + n, v);
  if (e.act == kActRelu)
    lin_act32<kActRelu>(v);
  else if (e.act == kActSilu)
    lin_act32<kActSilu>(v);
  else if (e.act == kActGelu)
    lin_act32<kActGelu>(v);
  if (e.res != nullptr) {
    uint32_t r[8];
    if (e.res_f32) {
      const float* src = static_cast<const float*>(e.res) + m * e.ldr + n;
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        lin_ld8(r, src + i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i + j] = __float_as_uint(__uint_as_float(v[i + j]) + __uint_as_float(r[j]));
      }
    } else {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(e.res) + m * e.ldr + n;
#pragma unroll
      for (int i = 0; i < 32; i += 16) {
        lin_ld8(r, src + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i + 2 * j] = __float_as_uint(__uint_as_float(v[i + 2 * j]) + bf16lo_to_f32(r[j]));
          v[i + 2 * j + 1] = __float_as_uint(__uint_as_float(v[i + 2 * j + 1]) + bf16hi_to_f32(r[j]));
        }
      }
    }
  }
  if (e.y_f32)
    lin_store32_f32(static_cast<float*>(e.y) + m * e.ldy + n, v);
  else
    lin_store32_bf16(static_cast<__nv_bfloat16*>(e.y) + m * e.ldy + n, v);
}

template <bool AMN, bool BMN, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLinThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB, const LinParams p) {
  using Cfg = LCfg<BN>;
  constexpr int STAGES = Cfg::STAGES;
  constexpr int NUM_ACC = Cfg::NUM_ACC;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * Cfg::A_BYTES;
  float* sBlock = reinterpret_cast<float*>(sB + STAGES * Cfg::B_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sBlock) + 8 * Cfg::BLOCK_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * STAGES;
  const uint32_t tfull0 = empty0 + 8 * STAGES;
  const uint32_t tempty0 = tfull0 + 8 * NUM_ACC;
  const uint32_t drain_bar = tempty0 + 8 * NUM_ACC;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < NUM_ACC; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 16);  // 8 epilogue warps in each CTA of the pair
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), Cfg::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrive or load completion
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int items = p.tiles_m * p.tiles_n * p.splits;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0;
      bool ok = true;
      for (int t = pair; ok && t < items; t += npairs) {
        int tm, tn, sp;
        lin_decode(p, t, tm, tn, sp);
        const int m0 = tm * 256 + static_cast<int>(rank) * 128;
        const int n0 = tn * BN + static_cast<int>(rank) * (BN / 2);
        const int kb1 = min(p.kb_total, (sp + 1) * p.kb_split);
        for (int kb = sp * p.kb_split; kb < kb1; ++kb) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = full0 + 8 * stage;
          const uint32_t fb = cluster_map_shared(fb_local, 0);
          if (leader) mbar_arrive_expect_tx(fb_local, 2u * Cfg::STAGE_BYTES);
          const uint32_t a_dst = smem_u32(sA + stage * Cfg::A_BYTES);
          const uint32_t b_dst = smem_u32(sB + stage * Cfg::B_BYTES);
          if constexpr (AMN) {
            tma_load_2d_pair(a_dst, &tmA, m0, kb * 64, fb, pol);
            tma_load_2d_pair(a_dst + 8192, &tmA, m0 + 64, kb * 64, fb, pol);
          } else {
            tma_load_2d_pair(a_dst, &tmA, kb * 64, m0, fb, pol);
          }
          if constexpr (BMN) {
#pragma unroll
            for (int i = 0; i < BN / 128; ++i)
              tma_load_2d_pair(b_dst + 8192 * i, &tmB, n0 + 64 * i, kb * 64, fb, pol);
          } else {
            tma_load_2d_pair(b_dst, &tmB, kb * 64, n0, fb, pol);
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // A wait gave up: copies of the last stages may still be in flight. The
        // leader waits for their arrival on its own `full` barriers (armed with
        // both halves' bytes); the other CTA waits for the stages' release. One
        // deadline bounds the drain, the cluster barrier at the end keeps both
        // CTAs alive until both have drained.
        const uint32_t n = issued < static_cast<uint32_t>(STAGES) ? issued : STAGES;
        const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
        int s = stage;
        uint32_t ph = phase;
        for (uint32_t i = 0; i < n; ++i) {
          if (--s < 0) {
            s = STAGES - 1;
            ph ^= 1u;
          }
          mbar_wait_until((leader ? full0 : empty0) + 8 * s, ph, deadline);
        }
      } else {
        // every load this CTA issued has been consumed (its stage released) before leaving
        for (int i = 0; i < STAGES; ++i) {
          mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag, p.status);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, BN) | (AMN ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u);
      constexpr uint64_t a_step = AMN ? 2048 >> 4 : 32 >> 4;
      constexpr uint64_t b_step = BMN ? 2048 >> 4 : 32 >> 4;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int t = pair; ok && t < items; t += npairs) {
        const int sp = t / (p.tiles_m * p.tiles_n);
        const int kbs = min(p.kb_total, (sp + 1) * p.kb_split) - sp * p.kb_split;
        if (!mbar_wait(tempty0 + 8 * acc, acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = 0; kb < kbs; ++kb) {
          if (!mbar_wait(full0 + 8 * stage, phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_at = smem_u32(sA + stage * Cfg::A_BYTES);
          const uint32_t b_at = smem_u32(sB + stage * Cfg::B_BYTES);
          const uint64_t adesc = AMN ? smem_desc_mn(a_at) : smem_desc_sw128(a_at);
          const uint64_t bdesc = BMN ? smem_desc_mn(b_at) : smem_desc_sw128(b_at);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_pair(d, adesc + a_step * k, bdesc + b_step * k, idesc, (kb | k) != 0 ? 1u : 0u);
          mma_commit_pair_mc(empty0 + 8 * stage, 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair_mc(tfull0 + 8 * acc, 0x3);
        if (++acc == NUM_ACC) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain_bar)
          : "memory");
      mbar_wait_drain(drain_bar, 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // Group g takes the tile's columns [g BN/2, (g+1) BN/2) in runs of 32; a
    // warp has 32 rows. Tensor memory gives a thread 32 columns of one row.
    //   32-byte accesses possible: it stores them as they are (32 rows at a time,
    //     whole sectors);
    //   else (odd pitches, the last columns): through shared memory, so that the
    //     lanes lie along the row (a 2-byte store to 32 rows at a time would cost
    //     more than the main loop).
    const int grp = (warp - 2) >> 2;
    const int q = warp & 3;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    float* block = sBlock + (warp - 2) * (32 * 33);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = pair; t < items; t += npairs) {
      int tm, tn, sp;
      lin_decode(p, t, tm, tn, sp);
      bool got = true;
      if (lane == 0) got = mbar_wait(tfull0 + 8 * acc, acc_phase, abort_flag, p.status);
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) break;
      tc_fence_after();
      const long long m0 = static_cast<long long>(tm) * 256 + static_cast<int>(rank) * 128 + q * 32;
      const int rows = static_cast<int>(min(32ll, p.M - m0));
      const int c0 = tn * BN + grp * (BN / 2);
#pragma unroll 1
      for (int j = 0; j < BN / 2; j += 32) {
        const int n = c0 + j;
        if (rows <= 0 || n >= p.N) break;
        uint32_t v[32];
        tmem_ld32(lane_base + static_cast<uint32_t>(acc * BN + grp * (BN / 2) + j), v);
        tmem_ld_wait();
        const int cols = min(32, p.N - n);
        if (p.wide && cols == 32) {
          if (lane < rows) {
            if (p.splits > 1)
              lin_store32_f32(p.partial + (static_cast<long long>(sp) * p.M + m0 + lane) * p.N + n, v);
            else
              lin_store32(p.e, m0 + lane, n, v);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) block[lane * 33 + i] = __uint_as_float(v[i]);
          __syncwarp();
          if (lane < cols) {
            if (p.splits > 1) {
              float* dst = p.partial + (static_cast<long long>(sp) * p.M + m0) * p.N + n + lane;
              for (int i = 0; i < rows; ++i) dst[static_cast<long long>(i) * p.N] = block[i * 33 + lane];
            } else {
              const float bias = linear_bias(p.e, n + lane);
              for (int i0 = 0; i0 < rows; i0 += 8) {
                float res[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  res[i] = p.e.res != nullptr && i0 + i < rows ? linear_res(p.e, m0 + i0 + i, n + lane) : 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (i0 + i < rows) {
                    float z;
                    const float y = linear_result(p.e, block[(i0 + i) * 33 + lane], bias, res[i], &z);
                    linear_put(p.e, m0 + i0 + i, n + lane, y, z);
                  }
              }
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_map_shared(tempty0 + 8 * acc, 0));
      if (++acc == NUM_ACC) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }

  __syncthreads();
  cluster_sync();  // neither CTA frees tensor memory or exits while its pair still runs
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
  }
}

// y from the splits' sums, in split order. A block has 64 columns x 4 rows.
__global__ void __launch_bounds__(256) linear_join_kernel(const float* partial, int splits, int M, int N,
                                                          const LinearEpilogue e) {
  const int n = blockIdx.x * 64 + threadIdx.x;
  if (n >= N) return;
  const long long total = static_cast<long long>(M) * N;
  const float bias = linear_bias(e, n);
  for (long long m = blockIdx.y * 4 + threadIdx.y; m < M; m += gridDim.y * 4) {
    const float* src = partial + m * N + n;
    const float res = e.res != nullptr ? linear_res(e, m, n) : 0.0f;
    float s = 0.0f;
#pragma unroll 8
    for (int k = 0; k < splits; ++k) s += src[k * total];
    float z;
    const float y = linear_result(e, s, bias, res, &z);
    linear_put(e, m, n, y, z);
  }
}

// dz = dy * act'(z), rounded to bf16 (the MMA's operand type; dbias takes the
// unrounded values), and the column sums of a block's rows. A thread has V
// columns, a block's 8 warps every eighth row. Bound by HBM: one pass.
constexpr int kDzRows = 64;      // rows of a block, while kDzLines blocks cover M
constexpr int kDzLines = 1024;
template <int V, bool kF32>
__global__ void __launch_bounds__(256) linear_dz_kernel(const LinearDzLaunch p) {
  using Dy = typename std::conditional<kF32, float, __nv_bfloat16>::type;
  struct alignas(sizeof(Dy) * V > 16 ? 16 : sizeof(Dy) * V) DyV {
    Dy v[V];
  };
  struct alignas(2 * V) ZV {
    __nv_bfloat16 v[V];
  };
  __shared__ float sum[8][32 * V + 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int n = (blockIdx.x * 32 + lane) * V;
  const long long m0 = static_cast<long long>(p.M) * blockIdx.y / gridDim.y;
  const long long m1 = static_cast<long long>(p.M) * (blockIdx.y + 1) / gridDim.y;
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.0f;
  if (n < p.N) {
    const Dy* dy = static_cast<const Dy*>(p.dy) + n;
    const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(p.z) + n;
#pragma unroll 4
    for (long long m = m0 + w; m < m1; m += 8) {
      const DyV d = *reinterpret_cast<const DyV*>(dy + m * p.lddy);
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = static_cast<float>(d.v[i]);
      if (p.z != nullptr) {
        const ZV zv = *reinterpret_cast<const ZV*>(z + m * p.ldz);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= linear_slope(__bfloat162float(zv.v[i]), p.act);
      }
      if (p.dz != nullptr) {
        ZV o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = __float2bfloat16(f[i]);
        *reinterpret_cast<ZV*>(static_cast<__nv_bfloat16*>(p.dz) + m * p.lddz + n) = o;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] += f[i];
    }
  }
  if (p.lines == nullptr) return;
#pragma unroll
  for (int i = 0; i < V; ++i) sum[w][i * 32 + lane] = s[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * V; i += 256) {
    const int c = (blockIdx.x * 32 + (i & 31)) * V + (i >> 5);
    if (c < p.N) {
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) t += sum[j][i];
      p.lines[static_cast<long long>(blockIdx.y) * p.N + c] = t;
    }
  }
}

PFN_cuTensorMapEncodeTiled_v12000 lin_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Tensor map of a bf16 matrix of `rows` rows of `inner` elements, `ld` apart, in
// boxes of 64 elements x box_rows rows.
bool lin_encode(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows,
                uint64_t ld) {
  auto fn = lin_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct LinPlan {
  int bn, tiles_m, tiles_n, splits, kb_split;
};

// Tile width and k split. 256-wide tiles move the fewest operand bytes per MMA;
// 128-wide ones (full MMA rate too) where 256 would leave pairs idle or the
// output is that narrow. k is split while that fills idle pairs and a part keeps
// at least 4 blocks of 64.
LinPlan lin_plan(int M, int N, int K, int y_f32) {
  const int pairs = device_sm_count() / 2;
  const int kb = (K + 63) / 64;
  LinPlan p;
  p.tiles_m = (M + 255) / 256;
  p.bn = N > 128 && static_cast<long long>(p.tiles_m) * ((N + 255) / 256) * 4 >= 3ll * pairs ? 256 : 128;
  p.tiles_n = (N + p.bn - 1) / p.bn;
  const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
  long long s = tiles > 0 ? pairs / tiles : 1;
  if (s > kb / 4) s = kb / 4;
  if (y_f32 && s < (kb + 31) / 32) s = (kb + 31) / 32;
  if (s < 1) s = 1;
  p.kb_split = static_cast<int>((kb + s - 1) / s);
  p.splits = (kb + p.kb_split - 1) / p.kb_split;
  return p;
}

template <bool AMN, bool BMN, int BN>
cudaError_t run_gemm(const LinearLaunch& L, const LinPlan& plan, cudaStream_t stream) {
  using Cfg = LCfg<BN>;
  static int max_pairs_cache[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (max_pairs_cache[dev] == 0) {
    e = cudaFuncSetAttribute(linear_gemm_kernel<AMN, BMN, BN>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(device_sm_count() & ~1));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, linear_gemm_kernel<AMN, BMN, BN>, &cfg);
    if (e != cudaSuccess) return e;
    max_pairs_cache[dev] = n > 0 ? n : 1;
  }
  CUtensorMap tmA, tmB;
  const bool okA = AMN ? lin_encode(&tmA, L.A, L.M, L.K, 64, L.lda) : lin_encode(&tmA, L.A, L.K, L.M, 128, L.lda);
  const bool okB = BMN ? lin_encode(&tmB, L.B, L.N, L.K, 64, L.ldb)
                       : lin_encode(&tmB, L.B, L.K, L.N, BN / 2, L.ldb);
  if (!okA || !okB) return cudaErrorInvalidValue;
  LinParams p{};
  p.M = L.M;
  p.N = L.N;
  p.K = L.K;
  p.tiles_m = plan.tiles_m;
  p.tiles_n = plan.tiles_n;
  p.splits = plan.splits;
  p.kb_total = (L.K + 63) / 64;
  p.kb_split = plan.kb_split;
  p.partial = L.partial;
  p.status = L.status;
  if (plan.splits > 1) {
    p.wide = L.N % 8 == 0 && (reinterpret_cast<uintptr_t>(L.partial) & 31u) == 0;
  } else {
    auto rows32 = [](const void* at, long long ld, int size) {
      return at == nullptr || (ld * size % 32 == 0 && (reinterpret_cast<uintptr_t>(at) & 31u) == 0);
    };
    p.wide = rows32(L.e.y, L.e.ldy, L.e.y_f32 ? 4 : 2) && rows32(L.e.z, L.e.ldz, 2) &&
             rows32(L.e.res, L.e.ldr, L.e.res_f32 ? 4 : 2);
  }
  p.e = L.e;
  const long long items = static_cast<long long>(plan.tiles_m) * plan.tiles_n * plan.splits;
  const int pairs = items < max_pairs_cache[dev] ? static_cast<int>(items) : max_pairs_cache[dev];
  linear_gemm_kernel<AMN, BMN, BN><<<2 * pairs, kLinThreads, Cfg::SMEM_BYTES, stream>>>(tmA, tmB, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || plan.splits == 1) return e;
  const unsigned rows = (static_cast<unsigned>(L.M) + 3) / 4;
  linear_join_kernel<<<dim3((static_cast<unsigned>(L.N) + 63) / 64, rows < 16384 ? rows : 16384), dim3(64, 4), 0,
                       stream>>>(L.partial, plan.splits, L.M, L.N, L.e);
  return cudaGetLastError();
}

}  // namespace

long long linear_gemm_partial(int M, int N, int K, int y_f32) {
  const LinPlan p = lin_plan(M, N, K, y_f32);
  return p.splits > 1 ? static_cast<long long>(p.splits) * M * N : 0;
}

cudaError_t launch_linear_gemm(const LinearLaunch& L, cudaStream_t stream) {
  const LinPlan p = lin_plan(L.M, L.N, L.K, L.e.y_f32);
  if (L.a_mn)
    return p.bn == 256 ? run_gemm<true, true, 256>(L, p, stream) : run_gemm<true, true, 128>(L, p, stream);
  if (L.b_mn)
    return p.bn == 256 ? run_gemm<false, true, 256>(L, p, stream) : run_gemm<false, true, 128>(L, p, stream);
  return p.bn == 256 ? run_gemm<false, false, 256>(L, p, stream) : run_gemm<false, false, 128>(L, p, stream);
}

int linear_dz_lines(int M) {
  const int n = (M + kDzRows - 1) / kDzRows;
  return n < kDzLines ? n : kDzLines;
}

cudaError_t launch_linear_dz(const LinearDzLaunch& L, cudaStream_t stream) {
  const int lines = linear_dz_lines(L.M);
  auto rows16 = [](const void* at, long long ld, int size) {
    return at == nullptr || (ld * size % 16 == 0 && (reinterpret_cast<uintptr_t>(at) & 15u) == 0);
  };
  const bool wide = L.N % 8 == 0 && rows16(L.dy, L.lddy, L.dy_f32 ? 4 : 2) && rows16(L.z, L.ldz, 2) &&
                    rows16(L.dz, L.lddz, 2);
  const int cols = wide ? 256 : 32;
  const dim3 grid((static_cast<unsigned>(L.N) + cols - 1) / cols, static_cast<unsigned>(lines));
  if (wide)
    L.dy_f32 ? linear_dz_kernel<8, true><<<grid, 256, 0, stream>>>(L)
             : linear_dz_kernel<8, false><<<grid, 256, 0, stream>>>(L);
  else
    L.dy_f32 ? linear_dz_kernel<1, true><<<grid, 256, 0, stream>>>(L)
             : linear_dz_kernel<1, false><<<grid, 256, 0, stream>>>(L);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || L.lines == nullptr) return e;
  return launch_sum_lines(L.lines, 1, lines, L.N, L.dbias, nullptr, stream);
}

}  // namespace moe
