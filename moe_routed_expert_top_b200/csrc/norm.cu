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
// Rows longer than 16 * 1024 (backward: 16 * 512) values do not fit the block's
// registers and go to the *_wide kernels, which read a row again for each step
// (from L2: a row is far smaller).
//
// The weight gradients are sums over the rows: each of a few hundred blocks
// keeps its rows' sums in registers (its rows are strided over the grid), leaves
// them as one line of a [2][blocks][H] table and a second kernel adds the
// lines in order. No atomics: the same bits every time.
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

template <typename T, int V>
__global__ void __launch_bounds__(kNormMaxThreads) norm_kernel(const NormLaunch p) {
  constexpr int NV = kEpt / V;
  using VT = Vec<T, V>;
  __shared__ float2 slot[2 * 32 * 8];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool on = row < p.M;
  const T* x = static_cast<const T*>(p.x) + (on ? row : 0) * p.ldx;
  VT xv[NV];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < p.H) xv[i] = *reinterpret_cast<const VT*>(x + c);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < p.H)
#pragma unroll
      for (int j = 0; j < V; ++j) s += to_f32(xv[i].v[j]);
  }
  const float inv = 1.0f / static_cast<float>(p.H);
  const float mean = row_sum2(make_float2(s, 0.0f), slot, 0).x * inv;
  float d2 = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < p.H)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = to_f32(xv[i].v[j]) - mean;
        d2 += d * d;
      }
  }
  const float var = row_sum2(make_float2(d2, 0.0f), slot, 1).x * inv;
  const float rstd = 1.0f / sqrtf(var + p.eps);
  if (!on) return;
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < p.H) {
      VT o;
#pragma unroll
      for (int j = 0; j < V; ++j)
        from_f32(o.v[j], (to_f32(xv[i].v[j]) - mean) * rstd *
                                 weight_at(p.gamma, p.w_f32, c + j, 1.0f) +
                             weight_at(p.beta, p.w_f32, c + j, 0.0f));
      *reinterpret_cast<VT*>(y + c) = o;
    }
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

template <typename T, int V>
__global__ void __launch_bounds__(kNormBwdMaxThreads) norm_bwd_kernel(const NormLaunch p) {
  constexpr int NV = kEpt / V;
  using VT = Vec<T, V>;
  __shared__ float2 slot[2 * 32 * 8];
  const float inv = 1.0f / static_cast<float>(p.H);
  float gw[NV][V], dg[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      gw[i][j] = c < p.H ? weight_at(p.gamma, p.w_f32, c + j, 1.0f) : 0.0f;
      dg[i][j] = 0.0f;
      db[i][j] = 0.0f;
    }
  }
  int flip = 0;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.y;
  // every row group of the block runs the same number of turns (barriers inside)
  for (long long base = static_cast<long long>(blockIdx.x) * blockDim.y; base < p.M; base += stride) {
    const long long row = base + threadIdx.y;
    const bool on = row < p.M;
    const T* x = static_cast<const T*>(p.x) + (on ? row : 0) * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + (on ? row : 0) * p.ldy;
    const float mean = on ? __ldg(p.mean + row) : 0.0f;
    const float rstd = on ? __ldg(p.rstd + row) : 0.0f;
    VT xv[NV], gv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V;
      if (on && c < p.H) {
        xv[i] = *reinterpret_cast<const VT*>(x + c);
        gv[i] = *reinterpret_cast<const VT*>(dy + c);
      }
    }
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V;
      if (on && c < p.H)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = to_f32(gv[i].v[j]);
          const float xh = (to_f32(xv[i].v[j]) - mean) * rstd;
          const float g = d * gw[i][j];
          s.x += g;
          s.y += g * xh;
          dg[i][j] += d * xh;
          db[i][j] += d;
        }
    }
    if (p.dx == nullptr) continue;
    s = row_sum2(s, slot, flip);
    flip ^= 1;
    const float c1 = s.x * inv, c2 = s.y * inv;
    if (on) {
      T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < p.H) {
          VT o;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float xh = (to_f32(xv[i].v[j]) - mean) * rstd;
            from_f32(o.v[j], rstd * (to_f32(gv[i].v[j]) * gw[i][j] - c1 - xh * c2));
          }
          *reinterpret_cast<VT*>(dx + c) = o;
        }
      }
    }
  }
  if (p.partial == nullptr) return;
  // one line of the table for each row group of the block
  const long long line = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const long long lines = static_cast<long long>(gridDim.x) * blockDim.y;
  float* pg = p.partial + line * p.H;
  float* pb = p.partial + (lines + line) * p.H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < p.H)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        pg[c + j] = dg[i][j];
        pb[c + j] = db[i][j];
      }
  }
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

// Widest vector (in values) every row access allows: 16 bytes, 4 bytes (8 in
// fp32) or one value.
int norm_vec(const NormLaunch& L, bool backward) {
  const int size = L.x_f32 ? 4 : 2;
  long long any = L.H | L.ldx;
  uintptr_t at = reinterpret_cast<uintptr_t>(L.x);
  if (backward) {
    any |= L.ldy;
    at |= reinterpret_cast<uintptr_t>(L.dy);
    if (L.dx != nullptr) {
      any |= L.lddx;
      at |= reinterpret_cast<uintptr_t>(L.dx);
    }
  } else {
    any |= L.ldy;
    at |= reinterpret_cast<uintptr_t>(L.y);
  }
  for (int v : {16 / size, 2})
    if (any % v == 0 && at % (static_cast<uintptr_t>(v) * size) == 0) return v;
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

// Blocks of the backward pass: as many as run at once (2 a SM at 448 threads and
// more, 4 below), so that few lines are left to add.
int norm_bwd_blocks(int M, const dim3& b) {
  const long long need = (static_cast<long long>(M) + b.y - 1) / b.y;
  const long long cap = static_cast<long long>(device_sm_count()) * (b.x * b.y > 256 ? 2 : 4);
  return static_cast<int>(need < cap ? need : cap);
}

template <typename T>
cudaError_t run_norm(const NormLaunch& L, cudaStream_t stream) {
  if (L.H > kEpt * kNormMaxThreads) {
    norm_wide_kernel<T><<<L.M, kNormMaxThreads, 0, stream>>>(L);
    return cudaGetLastError();
  }
  const dim3 b = norm_block(L.H);
  const unsigned grid = (static_cast<unsigned>(L.M) + b.y - 1) / b.y;
  const int v = norm_vec(L, false);
  if (v == 16 / static_cast<int>(sizeof(T)))
    norm_kernel<T, 16 / sizeof(T)><<<grid, b, 0, stream>>>(L);
  else if (v == 2)
    norm_kernel<T, 2><<<grid, b, 0, stream>>>(L);
  else
    norm_kernel<T, 1><<<grid, b, 0, stream>>>(L);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_norm_backward(const NormLaunch& L, cudaStream_t stream) {
  int lines;
  if (norm_bwd_wide(L.H)) {
    lines = norm_partial_rows(L.M, L.H);
    if (L.partial != nullptr) {
      const dim3 grid((static_cast<unsigned>(L.H) + 255) / 256, static_cast<unsigned>(lines));
      norm_bwd_cols_kernel<T><<<grid, 256, 0, stream>>>(L);
    }
    // last: dx may take dy's or x's place
    if (L.dx != nullptr) norm_bwd_wide_kernel<T><<<L.M, kNormMaxThreads, 0, stream>>>(L);
  } else {
    const dim3 b = norm_block(L.H);
    const int grid = norm_bwd_blocks(L.M, b);
    lines = grid * static_cast<int>(b.y);
    const int v = norm_vec(L, true);
    if (v == 16 / static_cast<int>(sizeof(T)))
      norm_bwd_kernel<T, 16 / sizeof(T)><<<grid, b, 0, stream>>>(L);
    else if (v == 2)
      norm_bwd_kernel<T, 2><<<grid, b, 0, stream>>>(L);
    else
      norm_bwd_kernel<T, 1><<<grid, b, 0, stream>>>(L);
  }
  cudaError_t e = cudaGetLastError();
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
  return norm_bwd_blocks(M, b) * static_cast<int>(b.y);
}

cudaError_t launch_norm(const NormLaunch& L, cudaStream_t stream) {
  return L.x_f32 ? run_norm<float>(L, stream) : run_norm<__nv_bfloat16>(L, stream);
}

cudaError_t launch_norm_backward(const NormLaunch& L, cudaStream_t stream) {
  return L.x_f32 ? run_norm_backward<float>(L, stream) : run_norm_backward<__nv_bfloat16>(L, stream);
}

}  // namespace moe
