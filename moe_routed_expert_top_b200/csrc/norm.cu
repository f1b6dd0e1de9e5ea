// norm.cu - layer norm, forward and backward (no counterpart on the pages; the
// norm in front of a feed-forward block's router and experts).
//
//   forward   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps),
//             y = (x - m) r gamma + beta
//   backward  xh = (x - m) r, g = dy gamma,
//             dx = r (g - mean(g) - xh mean(g xh)),
//             dgamma = sum_rows dy xh, dbeta = sum_rows dy
//
// What bounds it: HBM. A row is read once, held in registers through its
// reductions, and written once (forward 2, backward 3 values moved per
// element). The variance is taken around the mean of the registers' values, not
// from a difference of squares, so a large mean costs no digits. All sums are
// fp32.
//
// A block is blockDim.y rows of blockDim.x threads (a multiple of 32); a thread
// holds 16 values of its row, as vectors of V values where the row's length,
// pitch and addresses allow 16-byte accesses, narrower ones where they do not.
// Blocks stay and take every gridDim-th group of rows, and the next rows' values
// are on their way while a row goes through its reductions.
// Rows longer than 16 * 1024 (backward: 16 * 512) values do not fit the block's
// registers and go to the *_wide kernels, which read a row again for each step
// (from L2: a row is far smaller).
//
// The weight gradients are sums over the rows: each block keeps its rows' sums
// in registers, leaves them as one line of a [2][blocks][H] table and a second
// kernel adds the lines in order. No atomics: the same bits every time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kEpt = 16;            // values of a row held by one thread
constexpr int kNormMaxThreads = 1024;
constexpr int kNormBwdMaxThreads = 512;

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float& o, float v) { o = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& o, float v) { o = __float2bfloat16(v); }

// gamma or beta (fp32 or bf16, or absent) at column c
__device__ __forceinline__ float weight_at(const void* w, int w_f32, int c, float absent) {
  if (w == nullptr) return absent;
  return w_f32 ? __ldg(static_cast<const float*>(w) + c)
               : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
}

// Sum of v over the threadIdx.x of this threadIdx.y; `slot` [2][blockDim.y][32]
// floats, `flip` alternates so that one barrier a reduction is enough. All
// threads of the block call it together.
__device__ __forceinline__ float2 row_sum2(float2 v, float2* slot, int flip) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float2* s = slot + (flip * blockDim.y + threadIdx.y) * 32;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = lane < nw ? s[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

// The same for one value; `slot` [2][blockDim.y][32] floats.
__device__ __forceinline__ float row_sum(float v, float* slot, int flip) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float* s = slot + (flip * blockDim.y + threadIdx.y) * 32;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = lane < nw ? s[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// V weights (gamma or beta) at column c as fp32.
template <typename WT, int V>
__device__ __forceinline__ void load_weights(const void* w, int c, float absent, float (&o)[V]) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = absent;
    return;
  }
  const Vec<WT, V> v = *reinterpret_cast<const Vec<WT, V>*>(static_cast<const WT*>(w) + c);
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = to_f32(v.v[j]);
}

// The thread's values of a row (on: there is one).
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int H, bool on, Vec<T, V> (&v)[kEpt / V]) {
#pragma unroll
  for (int i = 0; i < kEpt / V; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (on && c < H) v[i] = *reinterpret_cast<const Vec<T, V>*>(row + c);
  }
}

// Mean and 1 / standard deviation of the row that the block's threadIdx.x hold in
// xv (values past the row: anything).
template <typename T, int V>
__device__ __forceinline__ void row_stats(const Vec<T, V> (&xv)[kEpt / V], int H, float inv, float eps,
                                          float* slot, float& mean, float& rstd) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kEpt / V; ++i) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) t += to_f32(xv[i].v[j]);
    s += (i * blockDim.x + threadIdx.x) * V < H ? t : 0.0f;
  }
  mean = row_sum(s, slot, 0) * inv;
  float d2 = 0.0f;
#pragma unroll
  for (int i = 0; i < kEpt / V; ++i) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = to_f32(xv[i].v[j]) - mean;
      t = fmaf(d, d, t);
    }
    d2 += (i * blockDim.x + threadIdx.x) * V < H ? t : 0.0f;
  }
  rstd = 1.0f / sqrtf(row_sum(d2, slot, 1) * inv + eps);
}

template <typename T, typename WT, int V>
__device__ __forceinline__ void store_row(const NormLaunch& p, long long row, const Vec<T, V> (&xv)[kEpt / V],
                                          float mean, float rstd) {
  T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < kEpt / V; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < p.H) {
      float g[V], b[V];
      load_weights<WT, V>(p.gamma, c, 1.0f, g);
      load_weights<WT, V>(p.beta, c, 0.0f, b);
      Vec<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) from_f32(o.v[j], (to_f32(xv[i].v[j]) - mean) * rstd * g[j] + b[j]);
      *reinterpret_cast<Vec<T, V>*>(y + c) = o;
    }
  }
}

constexpr int kNormStages = 8;

// One row of `bytes` (a multiple of 16) into shared memory, counted on `bar`;
// `first`: of the copies that this phase of the barrier counts, two in all with
// `both`.
__device__ __forceinline__ void norm_copy(void* dst, const void* src, uint32_t bytes, uint32_t bar, bool first,
                                          bool both = false) {
  if (first) mbar_arrive_expect_tx(bar, both ? 2 * bytes : bytes);
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

template <typename T, typename WT, int V>
__global__ void __launch_bounds__(kNormMaxThreads) norm_kernel(const NormLaunch p) {
  constexpr int NV = kEpt / V;
  using VT = Vec<T, V>;
  __shared__ float slot[2 * 32 * 8];
  const float inv = 1.0f / static_cast<float>(p.H);
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.y;
  const T* x = static_cast<const T*>(p.x);
  long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  VT next[NV];
  load_row<T, V>(x + (row < p.M ? row : 0) * p.ldx, p.H, row < p.M, next);
  // every row group of the block runs the same number of turns (barriers inside)
  for (long long base = row - threadIdx.y; base < p.M; base += stride, row += stride) {
    const bool on = row < p.M;
    VT xv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) xv[i] = next[i];
    const long long ahead = row + stride;
    load_row<T, V>(x + (ahead < p.M ? ahead : 0) * p.ldx, p.H, ahead < p.M, next);
    float mean, rstd;
    row_stats<T, V>(xv, p.H, inv, p.eps, slot, mean, rstd);
    if (!on) continue;
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    store_row<T, WT, V>(p, row, xv, mean, rstd);
  }
}

// The same for rows of 2 KB and more whose accesses are 16 bytes wide: whole rows
// come through a ring in shared memory, a bulk copy each, so that 100 KB an SM and
// more are on their way whatever the threads do (registers hold one row ahead). The
// block's barrier of a row's first sum tells that all have taken their values; its
// first thread then asks for the row that goes in that place.
template <typename T, typename WT>
__global__ void __launch_bounds__(kNormMaxThreads) norm_ring_kernel(const NormLaunch p, int stages) {
  constexpr int V = 16 / sizeof(T);
  constexpr int NV = kEpt / V;
  using VT = Vec<T, V>;
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ float slot[2 * 32];
  __shared__ uint64_t bars[kNormStages];
  const float inv = 1.0f / static_cast<float>(p.H);
  const uint32_t bytes = static_cast<uint32_t>(p.H) * sizeof(T);
  const T* x = static_cast<const T*>(p.x);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(bars + s), 1);
    mbar_fence_init();
    for (int s = 0; s < stages; ++s) {
      const long long row = blockIdx.x + static_cast<long long>(s) * gridDim.x;
      if (row < p.M) norm_copy(norm_smem + s * bytes, x + row * p.ldx, bytes, smem_u32(bars + s), true);
    }
  }
  __syncthreads();
  int stage = 0;
  uint32_t phase = 0;
  for (long long row = blockIdx.x; row < p.M; row += gridDim.x) {
    mbar_wait_drain(smem_u32(bars + stage), phase);
    VT xv[NV];
    const T* in = reinterpret_cast<const T*>(norm_smem + stage * bytes);
    load_row<T, V>(in, p.H, true, xv);
    float mean, rstd;
    row_stats<T, V>(xv, p.H, inv, p.eps, slot, mean, rstd);
    __syncwarp();
    if (threadIdx.x == 0) {
      const long long ahead = row + static_cast<long long>(stages) * gridDim.x;
      if (ahead < p.M)
        norm_copy(norm_smem + stage * bytes, x + ahead * p.ldx, bytes, smem_u32(bars + stage), true);
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    store_row<T, WT, V>(p, row, xv, mean, rstd);
  }
}

// Rows too long for the registers: one block a row, three passes over it.
template <typename T>
__global__ void __launch_bounds__(kNormMaxThreads) norm_wide_kernel(const NormLaunch p) {
  __shared__ float2 slot[2 * 32];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  float s = 0.0f;
  for (int c = threadIdx.x; c < p.H; c += blockDim.x) s += to_f32(x[c]);
  const float inv = 1.0f / static_cast<float>(p.H);
  const float mean = row_sum2(make_float2(s, 0.0f), slot, 0).x * inv;
  float d2 = 0.0f;
  for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
    const float d = to_f32(x[c]) - mean;
    d2 += d * d;
  }
  const float rstd = 1.0f / sqrtf(row_sum2(make_float2(d2, 0.0f), slot, 1).x * inv + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(p.y) + row * p.ldy;
  for (int c = threadIdx.x; c < p.H; c += blockDim.x)
    from_f32(y[c], (to_f32(x[c]) - mean) * rstd * weight_at(p.gamma, p.w_f32, c, 1.0f) +
                       weight_at(p.beta, p.w_f32, c, 0.0f));
}

// A thread's weights (as stored: bf16 ones take half the registers) and zeros for
// its sums of the weight gradients.
template <typename WT, int V>
__device__ __forceinline__ void bwd_start(const NormLaunch& p, Vec<WT, V> (&gw)[kEpt / V], float (&dg)[kEpt / V][V],
                                          float (&db)[kEpt / V][V]) {
#pragma unroll
  for (int i = 0; i < kEpt / V; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      dg[i][j] = db[i][j] = 0.0f;
      from_f32(gw[i].v[j], 1.0f);
    }
    if (p.gamma != nullptr && c < p.H)
      gw[i] = *reinterpret_cast<const Vec<WT, V>*>(static_cast<const WT*>(p.gamma) + c);
  }
}

// The thread's part of sum(g), sum(g xh); adds to its weight gradients.
template <typename T, typename WT, int V>
__device__ __forceinline__ float2 bwd_sums(const Vec<T, V> (&xv)[kEpt / V], const Vec<T, V> (&gv)[kEpt / V],
                                           const Vec<WT, V> (&gw)[kEpt / V], float mean, float rstd, int H,
                                           float (&dg)[kEpt / V][V], float (&db)[kEpt / V][V]) {
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kEpt / V; ++i) {
    if ((i * blockDim.x + threadIdx.x) * V < H)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = to_f32(gv[i].v[j]);
        const float xh = (to_f32(xv[i].v[j]) - mean) * rstd;
        const float g = d * to_f32(gw[i].v[j]);
        s.x += g;
        s.y = fmaf(g, xh, s.y);
        dg[i][j] = fmaf(d, xh, dg[i][j]);
        db[i][j] += d;
      }
  }
  return s;
}

template <typename T, typename WT, int V>
__device__ __forceinline__ void bwd_store(const NormLaunch& p, long long row, const Vec<T, V> (&xv)[kEpt / V],
                                          const Vec<T, V> (&gv)[kEpt / V], const Vec<WT, V> (&gw)[kEpt / V],
                                          float mean, float rstd, float c1, float c2) {
  T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
  for (int i = 0; i < kEpt / V; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < p.H) {
      Vec<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = (to_f32(xv[i].v[j]) - mean) * rstd;
        from_f32(o.v[j], rstd * (to_f32(gv[i].v[j]) * to_f32(gw[i].v[j]) - c1 - xh * c2));
      }
      *reinterpret_cast<Vec<T, V>*>(dx + c) = o;
    }
  }
}

// One line of the [2][lines][H] table.
template <int V>
__device__ __forceinline__ void bwd_lines(const NormLaunch& p, long long line, long long lines,
                                          const float (&dg)[kEpt / V][V], const float (&db)[kEpt / V][V]) {
  float* pg = p.partial + line * p.H;
  float* pb = p.partial + (lines + line) * p.H;
  constexpr int W = V < 4 ? V : 4;  // (a line starts at a multiple of V floats)
#pragma unroll
  for (int i = 0; i < kEpt / V; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < p.H)
#pragma unroll
      for (int j = 0; j < V; j += W) {
        Vec<float, W> a, b;
#pragma unroll
        for (int q = 0; q < W; ++q) {
          a.v[q] = dg[i][j + q];
          b.v[q] = db[i][j + q];
        }
        *reinterpret_cast<Vec<float, W>*>(pg + c + j) = a;
        *reinterpret_cast<Vec<float, W>*>(pb + c + j) = b;
      }
  }
}

// A row's values of the backward pass, as they are loaded.
template <typename T, int V>
struct BwdRow {
  Vec<T, V> x[kEpt / V], g[kEpt / V];
  float mean, rstd;
};
template <typename T, int V>
__device__ __forceinline__ void load_bwd_row(const NormLaunch& p, long long row, BwdRow<T, V>& r) {
  const bool on = row < p.M;
  const long long at = on ? row : 0;
  load_row<T, V>(static_cast<const T*>(p.x) + at * p.ldx, p.H, on, r.x);
  load_row<T, V>(static_cast<const T*>(p.dy) + at * p.ldy, p.H, on, r.g);
  r.mean = on ? __ldg(p.mean + at) : 0.0f;
  r.rstd = on ? __ldg(p.rstd + at) : 0.0f;
}

template <typename T, typename WT, int V>
__global__ void __launch_bounds__(kNormBwdMaxThreads) norm_bwd_kernel(const NormLaunch p) {
  constexpr int NV = kEpt / V;
  __shared__ float2 slot[2 * 32 * 8];
  const float inv = 1.0f / static_cast<float>(p.H);
  float dg[NV][V], db[NV][V];
  Vec<WT, V> gw[NV];
  bwd_start<WT, V>(p, gw, dg, db);
  int flip = 0;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.y;
  long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  BwdRow<T, V> next;
  load_bwd_row<T, V>(p, row, next);
  // every row group of the block runs the same number of turns (barriers inside)
  for (long long base = row - threadIdx.y; base < p.M; base += stride, row += stride) {
    const bool on = row < p.M;
    const BwdRow<T, V> cur = next;
    load_bwd_row<T, V>(p, row + stride, next);
    float2 s = bwd_sums<T, WT, V>(cur.x, cur.g, gw, cur.mean, cur.rstd, on ? p.H : 0, dg, db);
    if (p.dx == nullptr) continue;
    s = row_sum2(s, slot, flip);
    flip ^= 1;
    if (on) bwd_store<T, WT, V>(p, row, cur.x, cur.g, gw, cur.mean, cur.rstd, s.x * inv, s.y * inv);
  }
  if (p.partial != nullptr)
    bwd_lines<V>(p, static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y,
                 static_cast<long long>(gridDim.x) * blockDim.y, dg, db);
}

// The same through a ring of whole rows (see norm_ring_kernel), x's and dy's.
template <typename T, typename WT>
__global__ void __launch_bounds__(kNormBwdMaxThreads) norm_bwd_ring_kernel(const NormLaunch p, int stages) {
  constexpr int V = 16 / sizeof(T);
  constexpr int NV = kEpt / V;
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ float2 slot[2 * 32];
  __shared__ uint64_t bars[kNormStages];
  const float inv = 1.0f / static_cast<float>(p.H);
  const uint32_t bytes = static_cast<uint32_t>(p.H) * sizeof(T);
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  auto ask = [&](int s, long long row) {
    if (row >= p.M) return;
    norm_copy(norm_smem + 2 * s * bytes, x + row * p.ldx, bytes, smem_u32(bars + s), true, true);
    norm_copy(norm_smem + (2 * s + 1) * bytes, dy + row * p.ldy, bytes, smem_u32(bars + s), false);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(bars + s), 1);
    mbar_fence_init();
    for (int s = 0; s < stages; ++s) ask(s, blockIdx.x + static_cast<long long>(s) * gridDim.x);
  }
  float dg[NV][V], db[NV][V];
  Vec<WT, V> gw[NV];
  bwd_start<WT, V>(p, gw, dg, db);
  __syncthreads();
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  for (long long row = blockIdx.x; row < p.M; row += gridDim.x) {
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    mbar_wait_drain(smem_u32(bars + stage), phase);
    Vec<T, V> xv[NV], gv[NV];
    load_row<T, V>(reinterpret_cast<const T*>(norm_smem + 2 * stage * bytes), p.H, true, xv);
    load_row<T, V>(reinterpret_cast<const T*>(norm_smem + (2 * stage + 1) * bytes), p.H, true, gv);
    float2 s = bwd_sums<T, WT, V>(xv, gv, gw, mean, rstd, p.H, dg, db);
    s = row_sum2(s, slot, flip);
    flip ^= 1;
    __syncwarp();
    if (threadIdx.x == 0) ask(stage, row + static_cast<long long>(stages) * gridDim.x);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    if (p.dx != nullptr) bwd_store<T, WT, V>(p, row, xv, gv, gw, mean, rstd, s.x * inv, s.y * inv);
  }
  if (p.partial != nullptr) bwd_lines<V>(p, blockIdx.x, gridDim.x, dg, db);
}

// dx of rows too long for the registers: one block a row, two passes.
template <typename T>
__global__ void __launch_bounds__(kNormMaxThreads) norm_bwd_wide_kernel(const NormLaunch p) {
  __shared__ float2 slot[2 * 32];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* dy = static_cast<const T*>(p.dy) + row * p.ldy;
  const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
  const float inv = 1.0f / static_cast<float>(p.H);
  float2 s = make_float2(0.0f, 0.0f);
  for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
    const float g = to_f32(dy[c]) * weight_at(p.gamma, p.w_f32, c, 1.0f);
    s.x += g;
    s.y += g * ((to_f32(x[c]) - mean) * rstd);
  }
  s = row_sum2(s, slot, 0);
  const float c1 = s.x * inv, c2 = s.y * inv;
  T* dx = static_cast<T*>(p.dx) + row * p.lddx;
  for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
    const float g = to_f32(dy[c]) * weight_at(p.gamma, p.w_f32, c, 1.0f);
    from_f32(dx[c], rstd * (g - c1 - (to_f32(x[c]) - mean) * rstd * c2));
  }
}

// Their weight gradients: a thread sums one column over a strided set of rows,
// one line of the table for each blockIdx.y.
template <typename T>
__global__ void __launch_bounds__(256) norm_bwd_cols_kernel(const NormLaunch p) {
  const long long c = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= p.H) return;
  float dg = 0.0f, db = 0.0f;
  for (long long row = blockIdx.y; row < p.M; row += gridDim.y) {
    const float d = to_f32(static_cast<const T*>(p.dy)[row * p.ldy + c]);
    const float xh = (to_f32(static_cast<const T*>(p.x)[row * p.ldx + c]) - __ldg(p.mean + row)) *
                     __ldg(p.rstd + row);
    dg += d * xh;
    db += d;
  }
  p.partial[static_cast<long long>(blockIdx.y) * p.H + c] = dg;
  p.partial[(static_cast<long long>(gridDim.y) + blockIdx.y) * p.H + c] = db;
}

int round32(int v) { return (v + 31) & ~31; }

// Widest vector (in values) every access allows: 16 bytes, 2 values or one.
int norm_vec(const NormLaunch& L, bool backward) {
  const int size = L.x_f32 ? 4 : 2, wsize = L.w_f32 ? 4 : 2;
  long long any = L.H | L.ldx | L.ldy;
  uintptr_t at = reinterpret_cast<uintptr_t>(L.x);
  if (backward) {
    at |= reinterpret_cast<uintptr_t>(L.dy);
    if (L.dx != nullptr) {
      any |= L.lddx;
      at |= reinterpret_cast<uintptr_t>(L.dx);
    }
  } else {
    at |= reinterpret_cast<uintptr_t>(L.y);
  }
  const uintptr_t w = reinterpret_cast<uintptr_t>(L.gamma) | (backward ? 0 : reinterpret_cast<uintptr_t>(L.beta));
  for (int v : {16 / size, 2})
    if (any % v == 0 && at % (static_cast<uintptr_t>(v) * size) == 0 &&
        w % (static_cast<uintptr_t>(v) * wsize) == 0)
      return v;
  return 1;
}

// Threads of a row and rows of a block: whole warps for the row, at least 128
// threads a block so that short rows still fill an SM.
dim3 norm_block(int H) {
  const int tx = round32((H + kEpt - 1) / kEpt);
  int ty = 1;
  while (tx * ty * 2 <= 256 && ty < 8) ty *= 2;
  return dim3(static_cast<unsigned>(tx), static_cast<unsigned>(ty));
}

bool norm_bwd_wide(int H) { return H > kEpt * kNormBwdMaxThreads; }

// Blocks that stay: what an SM holds at 64 registers a thread (forward), at 128
// (backward, where a block's sums are a line of the table each).
int norm_blocks(int M, const dim3& b, int registers) {
  const long long need = (static_cast<long long>(M) + b.y - 1) / b.y;
  const int threads = static_cast<int>(b.x * b.y);
  const int per_sm = 65536 / (registers * threads) > 0 ? 65536 / (registers * threads) : 1;
  const long long cap = static_cast<long long>(device_sm_count()) * per_sm;
  return static_cast<int>(need < cap ? need : cap);
}

// The ring's stages for a block (0: rows too short or not 16 bytes wide).
// room: shared memory of a block; rows: rows of a stage.
int norm_ring_stages(int v, int size, int H, int room, int rows) {
  if (v * size != 16 || H * size < 2048) return 0;
  const int n = room / (rows * H * size);
  return n < kNormStages ? n : kNormStages;
}

template <void (*kernel)(const NormLaunch, int)>
cudaError_t norm_ring_launch(const NormLaunch& L, int grid, int threads, int stages, int rows,
                             cudaStream_t stream) {
  static bool set[64] = {};  // the attribute holds for the process: once per device and kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const size_t smem = static_cast<size_t>(stages) * rows * L.H * (L.x_f32 ? 4 : 2);
  kernel<<<grid, threads, smem, stream>>>(L, stages);
  return cudaGetLastError();
}

template <typename T, typename WT>
cudaError_t norm_forward_launch(const NormLaunch& L, cudaStream_t stream) {
  const dim3 b = norm_block(L.H);
  const int v = norm_vec(L, false);
  // blocks an SM: at least two for the ring, so that one's sums run under the other's stores
  const int per_sm = 65536 / (64 * static_cast<int>(b.x)) > 1 ? 65536 / (64 * static_cast<int>(b.x)) : 1;
  const int ring_blocks = per_sm < 4 ? per_sm : 4;
  const int stages = norm_ring_stages(v, sizeof(T), L.H, 200 * 1024 / ring_blocks, 1);
  if (stages >= 2) {
    const long long most = static_cast<long long>(device_sm_count()) * ring_blocks;
    return norm_ring_launch<norm_ring_kernel<T, WT>>(L, static_cast<int>(L.M < most ? L.M : most),
                            static_cast<int>(b.x), stages, 1, stream);
  }
  const unsigned grid = static_cast<unsigned>(norm_blocks(L.M, b, 64));
  if (v == 16 / static_cast<int>(sizeof(T)))
    norm_kernel<T, WT, 16 / sizeof(T)><<<grid, b, 0, stream>>>(L);
  else if (v == 2)
    norm_kernel<T, WT, 2><<<grid, b, 0, stream>>>(L);
  else
    norm_kernel<T, WT, 1><<<grid, b, 0, stream>>>(L);
  return cudaGetLastError();
}

// `lines` receives the table's lines.
template <typename T, typename WT>
cudaError_t norm_backward_launch(const NormLaunch& L, int* lines, cudaStream_t stream) {
  const dim3 b = norm_block(L.H);
  const int v = norm_vec(L, true);
  const int per_sm = 65536 / (128 * static_cast<int>(b.x)) > 1 ? 65536 / (128 * static_cast<int>(b.x)) : 1;
  const int ring_blocks = per_sm < 2 ? per_sm : 2;
  const int stages = norm_ring_stages(v, sizeof(T), L.H, 200 * 1024 / ring_blocks, 2);
  if (stages >= 2) {
    const long long most = static_cast<long long>(device_sm_count()) * ring_blocks;
    *lines = static_cast<int>(L.M < most ? L.M : most);
    return norm_ring_launch<norm_bwd_ring_kernel<T, WT>>(L, *lines, static_cast<int>(b.x), stages, 2, stream);
  }
  const unsigned grid = static_cast<unsigned>(norm_blocks(L.M, b, 128));
  *lines = static_cast<int>(grid * b.y);
  if (v == 16 / static_cast<int>(sizeof(T)))
    norm_bwd_kernel<T, WT, 16 / sizeof(T)><<<grid, b, 0, stream>>>(L);
  else if (v == 2)
    norm_bwd_kernel<T, WT, 2><<<grid, b, 0, stream>>>(L);
  else
    norm_bwd_kernel<T, WT, 1><<<grid, b, 0, stream>>>(L);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_norm(const NormLaunch& L, cudaStream_t stream) {
  if (L.H > kEpt * kNormMaxThreads) {
    norm_wide_kernel<T><<<L.M, kNormMaxThreads, 0, stream>>>(L);
    return cudaGetLastError();
  }
  return L.w_f32 ? norm_forward_launch<T, float>(L, stream) : norm_forward_launch<T, __nv_bfloat16>(L, stream);
}

template <typename T>
cudaError_t run_norm_backward(const NormLaunch& L, cudaStream_t stream) {
  int lines = 0;
  cudaError_t e = cudaSuccess;
  if (norm_bwd_wide(L.H)) {
    lines = norm_partial_rows(L.M, L.H);
    if (L.partial != nullptr) {
      const dim3 grid((static_cast<unsigned>(L.H) + 255) / 256, static_cast<unsigned>(lines));
      norm_bwd_cols_kernel<T><<<grid, 256, 0, stream>>>(L);
    }
    // last: dx may take dy's or x's place
    if (L.dx != nullptr) norm_bwd_wide_kernel<T><<<L.M, kNormMaxThreads, 0, stream>>>(L);
    e = cudaGetLastError();
  } else {
    e = L.w_f32 ? norm_backward_launch<T, float>(L, &lines, stream)
                : norm_backward_launch<T, __nv_bfloat16>(L, &lines, stream);
  }
  if (e != cudaSuccess || L.partial == nullptr) return e;
  return launch_sum_lines(L.partial, 2, lines, L.H, L.dgamma, L.dbeta, stream);
}

// A table's lines added up (weight and bias gradients): 8 warps take every eighth
// line of 32 columns, then one warp adds the eight sums in order.
__global__ void __launch_bounds__(256) sum_lines_kernel(const float* partial, int lines, int H,
                                                        float* out0, float* out1) {
  __shared__ float sum[8][33];
  float* out = blockIdx.y == 0 ? out0 : out1;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  const float* src = partial + static_cast<long long>(blockIdx.y) * lines * H + c;
  float s = 0.0f;
  if (c < H)
#pragma unroll 8
    for (int l = w; l < lines; l += 8) s += src[static_cast<long long>(l) * H];
  sum[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < H) {
    for (int i = 1; i < 8; ++i) s += sum[i][lane];
    out[c] = s;
  }
}

}  // namespace

cudaError_t launch_sum_lines(const float* table, int tables, int lines, int H, float* out0,
                             float* out1, cudaStream_t stream) {
  const dim3 grid((static_cast<unsigned>(H) + 31) / 32, static_cast<unsigned>(tables));
  sum_lines_kernel<<<grid, 256, 0, stream>>>(table, lines, H, out0, out1);
  return cudaGetLastError();
}

int norm_partial_rows(int M, int H) {
  if (norm_bwd_wide(H)) return M < 32 ? M : 32;
  const dim3 b = norm_block(H);
  const int lines = norm_blocks(M, b, 128) * static_cast<int>(b.y);
  const long long ring = 2ll * device_sm_count();  // the ring's blocks, at most
  const int most = static_cast<int>(M < ring ? M : ring);
  return lines > most ? lines : most;
}

cudaError_t launch_norm(const NormLaunch& L, cudaStream_t stream) {
  return L.x_f32 ? run_norm<float>(L, stream) : run_norm<__nv_bfloat16>(L, stream);
}

cudaError_t launch_norm_backward(const NormLaunch& L, cudaStream_t stream) {
  return L.x_f32 ? run_norm_backward<float>(L, stream) : run_norm_backward<__nv_bfloat16>(L, stream);
}

}  // namespace moe
