// few.cu - the whole routed mixture-of-experts layer for 1..64 tokens in two
// kernels (the same path as the forward in api.cu, TileLang tutorial "Example
// 07" section 2: routed grouped GEMM -> SiLU -> down -> weighted write-back):
//
//   out[t] = residual[t] + shared(x_t)
//          + scale * sum_j p[t,j] * Wd[e] bf16( silu(Wg[e] x_t) * (Wu[e] x_t) ),  e = id[t,j]
//
// What bounds it: with so few tokens every touched expert's 3*H*F weights are
// read once from HBM and meet 1..64 rows each, so the time is the weights'
// bytes over the memory rate plus the fixed cost of the launches. The kernels
// therefore (a) give every CTA the same number of weight ROWS, to within one
// row, whatever the routing; (b) read each row exactly once, straight into the
// registers of the warp that multiplies it (32 bytes a lane, the next chunk in
// flight while this one is multiplied); (c) rebuild the routing in every CTA
// from the logits, which costs less than a third launch and lets the second
// kernel start its weight loads before the first has ended (programmatic
// dependent launch).
//
// The products themselves (mma.sync from registers) are in few.cuh.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "few.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "route.cuh"

namespace moe {

namespace {

struct FewParams {
  int T, H, F, E, k, Fs;
  int score_fn, renormalize;
  float scale;
  const float* logits;       // null: topk_ids / topk_weights are inputs
  int32_t* topk_ids;
  float* topk_weights;
  const __nv_bfloat16* x;
  const __nv_bfloat16* w_gate_up;
  const __nv_bfloat16* w_down;
  const __nv_bfloat16* ws_gate_up;
  const __nv_bfloat16* ws_down;
  const __nv_bfloat16* residual;
  __nv_bfloat16* h;   // [pairs, F] in expert order, then the shared expert's [T, Fs]
  __nv_bfloat16* hs;
  __nv_bfloat16* out;
  int32_t* status;
};

// The routing of all tokens, in shared memory.
struct FewRoute {
  unsigned long long* mask;  // [E] tokens of each expert, as bits
  float* weight;             // [P] weight of a pair, in expert order
  int* act_e;                // [E] experts with tokens, in index order
  int* act_off;              // [E + 1] first pair of each of them
  short* ids;                // [P] expert of pair (t, j), -1 = none
  float* raw;                // [P] weight of pair (t, j)
  uint8_t* tok;              // [P] token of a pair, in expert order
  int* n_act;
  int* bad;
};

__host__ __device__ inline size_t few_up16(size_t v) { return (v + 15) & ~static_cast<size_t>(15); }

__host__ __device__ inline size_t few_route_bytes(int E, int P) {
  return few_up16(8ull * E) + few_up16(4ull * P) + few_up16(4ull * E) + few_up16(4ull * (E + 1)) +
         few_up16(2ull * P) + few_up16(4ull * P) + few_up16(P) + 64;
}

__device__ __forceinline__ FewRoute few_route_layout(uint8_t* s, int E, int P) {
  FewRoute r;
  r.mask = reinterpret_cast<unsigned long long*>(s);
  s += few_up16(8ull * E);
  r.weight = reinterpret_cast<float*>(s);
  s += few_up16(4ull * P);
  r.act_e = reinterpret_cast<int*>(s);
  s += few_up16(4ull * E);
  r.act_off = reinterpret_cast<int*>(s);
  s += few_up16(4ull * (E + 1));
  r.ids = reinterpret_cast<short*>(s);
  s += few_up16(2ull * P);
  r.raw = reinterpret_cast<float*>(s);
  s += few_up16(4ull * P);
  r.tok = s;
  s += few_up16(P);
  r.n_act = reinterpret_cast<int*>(s);
  r.bad = r.n_act + 1;
  return r;
}

// float -> unsigned with the same order (+0 and -0 equal); 0 is below every float.
__device__ __forceinline__ uint32_t few_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return key > 0u ? key : 1u;  // a NaN's bits never read as "taken"
}
__device__ __forceinline__ float few_unkey(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// Top-k of one token by one warp, with the weights of route_topk_kernel bit for
// bit (largest logit first, then the lowest index; sums in slot order). Lane
// l holds experts l, l + 32, ...; the result of slot j is lane j's.
__device__ __forceinline__ void few_topk(const float* row, int E, int k, int score_fn,
                                         int renormalize, int& my_id, float& my_w) {
  const int lane = threadIdx.x & 31;
  uint32_t key[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    key[i] = 0;
    if (32 * i < E && lane + 32 * i < E) key[i] = few_key(__ldg(row + lane + 32 * i));
  }
  uint32_t my_key = 0x80000000u;
  my_id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (32 * i < E) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    int at = INT_MAX;
#pragma unroll
    for (int i = 31; i >= 0; --i)
      if (32 * i < E && key[i] == best) at = lane + 32 * i;
    at = __reduce_min_sync(0xffffffffu, at);
    if ((at & 31) == lane) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if ((at >> 5) == i) key[i] = 0;
    }
    if (lane == j) {
      my_key = best;
      my_id = at;
    }
  }
  const float val = few_unkey(my_key);
  const float top = __shfl_sync(0xffffffffu, val, 0);
  if (score_fn == 0) {
    const float ev = moe_expf(__fsub_rn(val, top));
    float den = 0.0f;
    if (renormalize) {
      for (int j = 0; j < k; ++j) den = __fadd_rn(den, __shfl_sync(0xffffffffu, ev, j));
    } else {
      // over all experts in index order
      for (int e0 = 0; e0 < E; e0 += 32) {
        const float v = e0 + lane < E ? __ldg(row + e0 + lane) : 0.0f;
        const float x = moe_expf(__fsub_rn(v, top));
        for (int l = 0; l < 32 && e0 + l < E; ++l)
          den = __fadd_rn(den, __shfl_sync(0xffffffffu, x, l));
      }
    }
    my_w = __fdiv_rn(ev, den);
  } else {
    const float sv = __fdiv_rn(1.0f, __fadd_rn(1.0f, moe_expf(-val)));
    my_w = sv;
    if (renormalize) {
      float den = 0.0f;
      for (int j = 0; j < k; ++j) den = __fadd_rn(den, __shfl_sync(0xffffffffu, sv, j));
      my_w = __fdiv_rn(sv, den);
    }
  }
}

// Builds the routing in shared memory. A token that names an expert twice gets
// one pair with the sum of both weights, so an expert has at most T <= 64 rows
// and its tokens fit one 64-bit mask: a pair's place in expert order is then a
// bit count, with no atomics deciding an order. `publish`: this CTA also writes
// the ids, the weights and the status word to global memory.
__device__ void few_route(const FewParams& p, const FewRoute& r, bool publish, int* scratch) {
  const int P = p.T * p.k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kFewThreads) r.mask[e] = 0ull;
  if (threadIdx.x == 0) *r.bad = 0;
  if (p.logits != nullptr) {
    for (int t = warp; t < p.T; t += kFewWarps) {
      int id;
      float w;
      few_topk(p.logits + static_cast<int64_t>(t) * p.E, p.E, p.k, p.score_fn, p.renormalize, id, w);
      if (lane < p.k) {
        r.ids[t * p.k + lane] = static_cast<short>(id);
        r.raw[t * p.k + lane] = w;
        if (publish && p.topk_ids != nullptr) p.topk_ids[t * p.k + lane] = id;
        if (publish && p.topk_weights != nullptr) p.topk_weights[t * p.k + lane] = w;
      }
    }
    __syncthreads();
  } else {
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += kFewThreads) {
      const int id = __ldg(p.topk_ids + i);
      const bool ok = id >= 0 && id < p.E;
      r.ids[i] = ok ? static_cast<short>(id) : static_cast<short>(-1);
      r.raw[i] = __ldg(p.topk_weights + i);
      if (!ok) *r.bad = 1;  // every writer writes the same value
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < P; i += kFewThreads) {
    const int id = r.ids[i];
    if (id >= 0) atomicOr(&r.mask[id], 1ull << (i / p.k));
  }
  __syncthreads();
  // exclusive scan over the experts of (pairs, experts with pairs)
  const int per = (p.E + kFewThreads - 1) / kFewThreads;
  const int beg = threadIdx.x * per;
  uint32_t local = 0;
  for (int i = 0; i < per && beg + i < p.E; ++i) {
    const int n = __popcll(r.mask[beg + i]);
    local += (static_cast<uint32_t>(n) << 12) + (n > 0 ? 1u : 0u);
  }
  uint32_t inc = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 31) scratch[warp] = static_cast<int>(inc);
  __syncthreads();
  uint32_t run = inc - local;
  for (int w = 0; w < warp; ++w) run += static_cast<uint32_t>(scratch[w]);
  for (int i = 0; i < per && beg + i < p.E; ++i) {
    const unsigned long long m = r.mask[beg + i];
    const int n = __popcll(m);
    if (n > 0) {
      const int a = static_cast<int>(run & 0xFFFu), off = static_cast<int>(run >> 12);
      r.act_e[a] = beg + i;
      r.act_off[a] = off;
      // the pairs of this expert, in token order
      unsigned long long left = m;
      for (int c = 0; c < n; ++c) {
        const int t = __ffsll(static_cast<long long>(left)) - 1;
        left &= left - 1;
        float w = 0.0f;
        for (int j = 0; j < p.k; ++j)
          if (r.ids[t * p.k + j] == beg + i) w += r.raw[t * p.k + j];
        r.tok[off + c] = static_cast<uint8_t>(t);
        r.weight[off + c] = w;
      }
    }
    run += (static_cast<uint32_t>(n) << 12) + (n > 0 ? 1u : 0u);
  }
  if (threadIdx.x == kFewThreads - 1) {
    *r.n_act = static_cast<int>(run & 0xFFFu);
    r.act_off[run & 0xFFFu] = static_cast<int>(run >> 12);
  }
  if (publish && threadIdx.x == 0) *p.status = *r.bad ? MOE_DEV_BAD_EXPERT_ID_FLAG : 0;
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Kernel 1: h = bf16(silu(Wg x) * (Wu x)) for every pair.
// The rows of all active experts (and of the shared expert) form one list of
// gate/up row pairs; CTA c takes an equal share of it, in tiles of up to 16
// pairs of one expert. In a tile the warps split k in chunks of 64 and add
// their sums through shared memory.
// ---------------------------------------------------------------------------
struct UpTile {
  const __nv_bfloat16* gate;  // first gate row (row pitch H); null: no tile
  int64_t up;                 // elements from a gate row to its up row
  int rows;                   // 1..16
  int off, n;                 // the expert's pairs (shared: off -1, n = T)
  int f0;
};

__device__ __forceinline__ UpTile up_tile(const FewParams& p, const FewRoute& r, int n_act, int64_t u,
                                          int64_t u1) {
  UpTile t;
  t.gate = nullptr;
  t.rows = 0;
  t.n = 0;
  t.off = 0;
  t.f0 = 0;
  t.up = 0;
  if (u >= u1) return t;
  const int64_t routed = static_cast<int64_t>(n_act) * p.F;
  int F;
  const __nv_bfloat16* w;
  if (u < routed) {
    const int a = static_cast<int>(u / p.F);
    t.f0 = static_cast<int>(u - static_cast<int64_t>(a) * p.F);
    F = p.F;
    t.off = r.act_off[a];
    t.n = r.act_off[a + 1] - t.off;
    w = p.w_gate_up + static_cast<int64_t>(r.act_e[a]) * 2 * p.F * p.H;
  } else {
    t.f0 = static_cast<int>(u - routed);
    F = p.Fs;
    t.off = -1;
    t.n = p.T;
    w = p.ws_gate_up;
  }
  const int64_t room = min(static_cast<int64_t>(F - t.f0), u1 - u);
  t.rows = room < 16 ? static_cast<int>(room) : 16;
  t.gate = w + static_cast<int64_t>(t.f0) * p.H;
  t.up = static_cast<int64_t>(F) * p.H;
  return t;
}

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 2) few_up_kernel(const FewParams p) {
  extern __shared__ __align__(16) uint8_t few_smem[];
  __shared__ int scratch[kFewWarps];
  const int P = p.T * p.k;
  const FewRoute r = few_route_layout(few_smem, p.E, P);
  // [warp][token tile][gate/up][lane] sums of the warps
  float4* red = reinterpret_cast<float4*>(few_smem + few_route_bytes(p.E, P));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  few_route(p, r, blockIdx.x == 0, scratch);
  const int n_act = *r.n_act;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int64_t units = static_cast<int64_t>(n_act) * p.F + p.Fs;
  int64_t u = units * blockIdx.x / gridDim.x;
  const int64_t u1 = units * (blockIdx.x + 1) / gridDim.x;
  const int chunks = p.H / 64;
  const int steps = (chunks + kFewWarps - 1) / kFewWarps;

  auto load = [&](FewA& a, const UpTile& t, int step) {
    const int c = step * kFewWarps + warp;
    const bool on = t.gate != nullptr && c < chunks;
    const __nv_bfloat16* base = t.gate + static_cast<int64_t>(c) * 64 + q * 16;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = g + 8 * half;
      const __nv_bfloat16* pr = base + static_cast<int64_t>(row) * p.H;
      const bool have = on && row < t.rows;
      few_ldw(a.v[0][half], pr, have);
      few_ldw(a.v[1][half], pr + t.up, have);
    }
  };

  UpTile cur = up_tile(p, r, n_act, u, u1);
  FewA a0, a1;
  load(a0, cur, 0);
  while (cur.gate != nullptr) {
    u += cur.rows;
    const UpTile next = up_tile(p, r, n_act, u, u1);
    const int nt = (cur.n + 7) >> 3;
    const __nv_bfloat16* xr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int c = j * 8 + g;
      xr[j] = c < cur.n ? p.x + static_cast<int64_t>(cur.off < 0 ? c : r.tok[cur.off + c]) * p.H
                        : nullptr;
    }
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
    for (int step = 0; step < steps; ++step) {
      const bool last = step + 1 == steps;
      load(a1, last ? next : cur, last ? 0 : step + 1);
      const int c = step * kFewWarps + warp;
      few_mul<NT>(acc, a0, xr, nt, c * 64 + q * 16, p.H);
      a0 = a1;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (j < nt) {
        float4* dst = red + ((warp * NT + j) * 2) * 32 + lane;
        dst[0] = make_float4(acc[0][j][0], acc[0][j][1], acc[0][j][2], acc[0][j][3]);
        dst[32] = make_float4(acc[1][j][0], acc[1][j][1], acc[1][j][2], acc[1][j][3]);
      }
    __syncthreads();
    // value (lane l, register i) of a tile: row l/4 + 8*(i/2), token 2*(l%4) + i%2
    const float* rf = reinterpret_cast<const float*>(red);
    for (int i = threadIdx.x; i < nt * 128; i += kFewThreads) {
      const int j = i >> 7, l = (i >> 2) & 31, v = i & 3;
      const int row = (l >> 2) + 8 * (v >> 1);
      const int col = j * 8 + 2 * (l & 3) + (v & 1);
      if (row < cur.rows && col < cur.n) {
        float gs = 0.0f, us = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
          const float* s = rf + ((w * NT + j) * 2) * 128 + (i & 127);
          gs += s[0];
          us += s[128];
        }
        const __nv_bfloat16 hv = __float2bfloat16(few_silu(gs) * us);
        if (cur.off < 0)
          p.hs[static_cast<int64_t>(col) * p.Fs + cur.f0 + row] = hv;
        else
          p.h[static_cast<int64_t>(cur.off + col) * p.F + cur.f0 + row] = hv;
      }
    }
    __syncthreads();
    cur = next;
  }
}

// ---------------------------------------------------------------------------
// Kernel 2: out = residual + sum over the experts of weight * (Wd h).
// CTA c owns an equal share of the H output rows, for every expert, so a
// token's sum over its experts stays in one CTA. The (expert, 64-wide chunk)
// items are split evenly over the warps; a warp adds its weighted sums into
// its own fp32 table [token][row] in shared memory, and the tables are added
// in warp order at the end: no atomics, the same bits every time.
// ---------------------------------------------------------------------------
struct DownItem {
  const __nv_bfloat16* w;  // row 0 of this CTA's rows, at the item's chunk; null: none
  int64_t ld;
  int a;                   // active expert, n_act = the shared expert
  int c;                   // chunk
};

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 2) few_down_kernel(const FewParams p) {
  extern __shared__ __align__(16) uint8_t few_smem[];
  __shared__ int scratch[kFewWarps];
  const int P = p.T * p.k;
  const FewRoute r = few_route_layout(few_smem, p.E, P);
  float* table = reinterpret_cast<float*>(few_smem + few_route_bytes(p.E, P));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  constexpr int kRows = 32;
  constexpr int TP = NT * 8;
  float* mine = table + warp * TP * kRows;

  few_route(p, r, false, scratch);
  const int n_act = *r.n_act;
  const int row0 = static_cast<int>(static_cast<int64_t>(p.H) * blockIdx.x / gridDim.x);
  const int row1 = static_cast<int>(static_cast<int64_t>(p.H) * (blockIdx.x + 1) / gridDim.x);
  const int chF = p.F / 64, chS = p.Fs / 64;
  const int items = n_act * chF + chS;
  const int i0 = static_cast<int>(static_cast<int64_t>(items) * warp / kFewWarps);
  const int i1 = static_cast<int>(static_cast<int64_t>(items) * (warp + 1) / kFewWarps);
  bool waited = false;

  for (int rb = row0; rb < row1; rb += kRows) {
    const int rows = min(kRows, row1 - rb);
    for (int i = lane; i < TP * kRows; i += 32) mine[i] = 0.0f;
    __syncwarp();
    auto item = [&](int i) {
      DownItem d;
      d.w = nullptr;
      d.ld = p.F;
      d.a = -1;
      d.c = 0;
      if (i >= i1) return d;
      if (i < n_act * chF) {
        d.a = i / chF;
        d.c = i - d.a * chF;
        d.w = p.w_down + (static_cast<int64_t>(r.act_e[d.a]) * p.H + rb) * p.F + d.c * 64;
      } else {
        d.a = n_act;
        d.c = i - n_act * chF;
        d.ld = p.Fs;
        d.w = p.ws_down + static_cast<int64_t>(rb) * p.Fs + d.c * 64;
      }
      return d;
    };
    auto load = [&](FewA& a, const DownItem& d) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = 16 * m + 8 * half + g;
          const bool have = d.w != nullptr && row < rows;
          few_ldw(a.v[m][half], d.w + row * d.ld + q * 16, have);
        }
    };
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
    DownItem cur = item(i0);
    FewA a0, a1;
    load(a0, cur);
    if (!waited) {
      // the weights are on their way; h comes from kernel 1
      asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
    }
    for (int i = i0; i < i1; ++i) {
      const DownItem next = item(i + 1);
      load(a1, next);
      const bool shared = cur.a == n_act;
      const int off = shared ? 0 : r.act_off[cur.a];
      const int n = shared ? p.T : r.act_off[cur.a + 1] - off;
      const int nt = (n + 7) >> 3;
      const __nv_bfloat16* xr[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = j * 8 + g;
        xr[j] = c < n ? (shared ? p.hs + static_cast<int64_t>(c) * p.Fs
                                : p.h + static_cast<int64_t>(off + c) * p.F)
                      : nullptr;
      }
      few_mul<NT>(acc, a0, xr, nt, cur.c * 64 + q * 16, static_cast<int>(cur.ld));
      if (next.a != cur.a) {
        // the expert ends here (or its other chunks are another warp's)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (j < nt) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int col = j * 8 + 2 * q + (v & 1);
              if (col < n) {
                const int t = shared ? col : r.tok[off + col];
                const float w = shared ? 1.0f : p.scale * r.weight[off + col];
#pragma unroll
                for (int m = 0; m < 2; ++m)
                  mine[t * kRows + 16 * m + 8 * (v >> 1) + g] += w * acc[m][j][v];
              }
              acc[0][j][v] = 0.0f;
              acc[1][j][v] = 0.0f;
            }
          }
        __syncwarp();
      }
      cur = next;
      a0 = a1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * kRows; i += kFewThreads) {
      const int t = i / kRows, row = i % kRows;
      if (row < rows) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) s += table[(w * TP + t) * kRows + row];
        const int64_t at = static_cast<int64_t>(t) * p.H + rb + row;
        if (p.residual != nullptr) s += __bfloat162float(p.residual[at]);
        p.out[at] = __float2bfloat16(s);
      }
    }
    __syncthreads();
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int NT>
cudaError_t run_few(const FewParams& p, cudaStream_t stream) {
  const size_t route = few_route_bytes(p.E, p.T * p.k);
  const size_t up_smem = route + sizeof(float4) * kFewWarps * NT * 2 * 32;
  const size_t down_smem = route + sizeof(float) * kFewWarps * NT * 8 * 32;
  static bool set[64] = {};  // the attributes hold for the process: once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    const size_t most = few_route_bytes(1024, 32 * NT * 8);
    e = cudaFuncSetAttribute(few_up_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(most + up_smem - route));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(few_down_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(most + down_smem - route));
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const int grid = 2 * device_sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = up_smem;
  cfg.stream = stream;
  e = cudaLaunchKernelEx(&cfg, few_up_kernel<NT>, p);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.dynamicSmemBytes = down_smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_down_kernel<NT>, p);
}

}  // namespace

cudaError_t launch_few(const FewLaunch& L, cudaStream_t stream) {
  FewParams p;
  p.T = L.T;
  p.H = L.H;
  p.F = L.F;
  p.E = L.E;
  p.k = L.k;
  p.Fs = L.F_shared;
  p.score_fn = L.score_fn;
  p.renormalize = L.renormalize;
  p.scale = L.scale;
  p.logits = L.logits;
  p.topk_ids = L.topk_ids;
  p.topk_weights = L.topk_weights;
  p.x = static_cast<const __nv_bfloat16*>(L.hidden);
  p.w_gate_up = static_cast<const __nv_bfloat16*>(L.w_gate_up);
  p.w_down = static_cast<const __nv_bfloat16*>(L.w_down);
  p.ws_gate_up = static_cast<const __nv_bfloat16*>(L.ws_gate_up);
  p.ws_down = static_cast<const __nv_bfloat16*>(L.ws_down);
  p.residual = static_cast<const __nv_bfloat16*>(L.residual);
  p.h = static_cast<__nv_bfloat16*>(L.h);
  p.hs = static_cast<__nv_bfloat16*>(L.hs);
  p.out = static_cast<__nv_bfloat16*>(L.out);
  p.status = L.status;
  if (p.T <= 8) return run_few<1>(p, stream);
  if (p.T <= 16) return run_few<2>(p, stream);
  if (p.T <= 32) return run_few<4>(p, stream);
  return run_few<8>(p, stream);
}

}  // namespace moe
