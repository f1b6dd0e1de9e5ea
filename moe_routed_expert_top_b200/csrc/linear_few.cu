// linear_few.cu - the linear product y = act(x W^T + bias) + residual for 1..64
// rows of x (a decode step's projections and router logits).
//
// What bounds it: the weight's N*K values, read once from HBM. The layout is the
// few-token layer's (few.cuh): every CTA takes an equal share of the weight's
// rows, its warps split k, their sums meet in shared memory and the epilogue
// follows there. Two shapes of tile:
//   32 rows x 64 k a warp and step, where a CTA has more than 8 rows;
//   8 rows x 256 k, where it has fewer (a router: 256 rows over 296 CTAs). The
//     wide tile would then load 128 bytes a warp and step and the time is k's
//     length in memory latencies; with four chunks of the same rows at once it
//     is a quarter of that.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "few.cuh"
#include "internal.h"
#include "linear.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

struct LinearFewParams {
  int M, N, K;
  long long ldx, ldw;
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  LinearEpilogue e;
  int32_t* status;
};

// 16 values of a weight row from k on; kWhole: 32-byte aligned and K % 16 == 0,
// else two 16-byte loads (K % 8 == 0).
template <bool kWhole>
__device__ __forceinline__ void linear_ldw(FewW& v, const __nv_bfloat16* row, int k, int K, bool on,
                                           uint64_t policy) {
  if constexpr (kWhole) {
    few_ldw(v, row + k, on && k < K, policy);
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (on && k + 8 * s < K)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.r[4 * s]), "=r"(v.r[4 * s + 1]), "=r"(v.r[4 * s + 2]),
                       "=r"(v.r[4 * s + 3])
                     : "l"(row + k + 8 * s));
      else
#pragma unroll
        for (int i = 0; i < 4; ++i) v.r[4 * s + i] = 0u;
    }
  }
}

template <int NT, bool kTall, bool kWhole>
__global__ void __launch_bounds__(kFewThreads, 2) linear_few_kernel(const LinearFewParams p) {
  constexpr int kRows = kTall ? 32 : 8;
  constexpr int kSpan = kTall ? 64 : 256;  // k of a warp's step
  constexpr int kBlocks = kTall ? 2 : 1;
  extern __shared__ __align__(16) uint8_t few_smem[];
  float4* red = reinterpret_cast<float4*>(few_smem);  // [warp][token tile][block][lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int row0 = static_cast<int>(static_cast<int64_t>(p.N) * blockIdx.x / gridDim.x);
  const int row1 = static_cast<int>(static_cast<int64_t>(p.N) * (blockIdx.x + 1) / gridDim.x);
  const int steps = (p.K + kFewWarps * kSpan - 1) / (kFewWarps * kSpan);
  const int nt = (p.M + 7) >> 3;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;  // nothing here waits on a barrier in memory

  const __nv_bfloat16* xr[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    xr[j] = j * 8 + g < p.M ? p.x + static_cast<int64_t>(j * 8 + g) * p.ldx : nullptr;

  const uint64_t policy = l2_policy_evict_first();
  auto load = [&](FewA& a, int rb, int step) {
    const int k0 = (step * kFewWarps + warp) * kSpan + q * 16;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = rb + g + (kTall ? 16 * m + 8 * half : 0);
        const int k = k0 + (kTall ? 0 : 64 * (2 * m + half));
        linear_ldw<kWhole>(a.v[m][half], p.w + static_cast<int64_t>(row) * p.ldw, k, p.K, row < row1,
                           policy);
      }
  };

  FewA a0, a1;
  load(a0, row0, 0);
  for (int rb = row0; rb < row1; rb += kRows) {
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
    for (int step = 0; step < steps; ++step) {
      const bool last = step + 1 == steps;
      load(a1, last ? rb + kRows : rb, last ? 0 : step + 1);
      const int kofs = (step * kFewWarps + warp) * kSpan + q * 16;
      if constexpr (kTall) {
        few_mul<NT>(acc, a0, xr, nt, kofs, p.K);
      } else {
        // the four chunks lie behind one another in k; rows 8..15 of the MMA are empty
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (j < nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const int k = kofs + 64 * i + 8 * s;
                const uint4 b = few_ldx(xr[j] + k, xr[j] != nullptr && k < p.K);
                const uint32_t* lo = a0.v[i >> 1][i & 1].r + 4 * s;
                few_mma(acc[0][j], lo[0], 0u, lo[1], 0u, b.x, b.y);
                few_mma(acc[0][j], lo[2], 0u, lo[3], 0u, b.z, b.w);
              }
          }
      }
      a0 = a1;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (j < nt)
#pragma unroll
        for (int m = 0; m < kBlocks; ++m)
          red[((warp * NT + j) * kBlocks + m) * 32 + lane] =
              make_float4(acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3]);
    __syncthreads();
    // value (lane l, register v) of a block: row l/4 + 8*(v/2), token 2*(l%4) + v%2
    const float* rf = reinterpret_cast<const float*>(red);
    for (int i = threadIdx.x; i < nt * kBlocks * 128; i += kFewThreads) {
      const int j = i / (kBlocks * 128), m = (i >> 7) % kBlocks, l = (i >> 2) & 31, v = i & 3;
      const int row = rb + 16 * m + (l >> 2) + 8 * (v >> 1);
      const int col = j * 8 + 2 * (l & 3) + (v & 1);
      if ((kTall || v < 2) && row < row1 && col < p.M) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) s += rf[((w * NT + j) * kBlocks + m) * 128 + (i & 127)];
        linear_store(p.e, col, row, s);
      }
    }
    __syncthreads();
  }
}

template <int NT, bool kTall, bool kWhole>
cudaError_t run(const LinearFewParams& p, int grid, cudaStream_t stream) {
  const int smem = kFewWarps * NT * (kTall ? 2 : 1) * 32 * static_cast<int>(sizeof(float4));
  static bool set[64] = {};  // the attribute holds for the process: once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(linear_few_kernel<NT, kTall, kWhole>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  linear_few_kernel<NT, kTall, kWhole><<<grid, kFewThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <int NT>
cudaError_t run_few(const LinearFewParams& p, cudaStream_t stream) {
  const int most = 2 * device_sm_count();
  const int grid = p.N < most ? p.N : most;
  const bool tall = p.N > 8 * grid;
  const bool whole = p.K % 16 == 0 && p.ldw % 16 == 0 && (reinterpret_cast<uintptr_t>(p.w) & 31u) == 0;
  if (tall)
    return whole ? run<NT, true, true>(p, grid, stream) : run<NT, true, false>(p, grid, stream);
  return whole ? run<NT, false, true>(p, grid, stream) : run<NT, false, false>(p, grid, stream);
}

}  // namespace

cudaError_t launch_linear_few(const LinearLaunch& L, cudaStream_t stream) {
  LinearFewParams p;
  p.M = L.M;
  p.N = L.N;
  p.K = L.K;
  p.ldx = L.lda;
  p.ldw = L.ldb;
  p.x = static_cast<const __nv_bfloat16*>(L.A);
  p.w = static_cast<const __nv_bfloat16*>(L.B);
  p.e = L.e;
  p.status = L.status;
  if (p.M <= 8) return run_few<1>(p, stream);
  if (p.M <= 16) return run_few<2>(p, stream);
  if (p.M <= 32) return run_few<4>(p, stream);
  return run_few<8>(p, stream);
}

}  // namespace moe
