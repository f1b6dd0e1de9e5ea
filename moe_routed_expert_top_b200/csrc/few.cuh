// few.cuh - products of streamed weight rows with a few token rows, shared by
// the few-token layer (few.cu) and the few-row linear product (linear_few.cu).
//
// mma.sync m16n8k16, 16 weight rows against 8 tokens. With 1..64 tokens the
// weights' arrival from HBM is the bound and the tensor pipe is idle most of the
// time (8 tokens use 1/20 of what the arrival allows), so both operands go
// straight from global memory to registers, without a trip through shared
// memory. A dot product may sum its k indices in any order, so lane q of a row
// group takes the 16 consecutive elements at k0 + 16q of its row AND of its
// token: a weight row's 128 bytes are one 32-byte load of four lanes, and
// fragment register r of A meets register r of B.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace moe {

constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;

__device__ __forceinline__ void few_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 bytes of a weight row (four lanes take a whole 128-byte line): read once by
// one lane, so it is kept out of L1; `policy` says what L2 does with it. A row
// that is not there reads as zero.
struct FewW {
  uint32_t r[8];
};
__device__ __forceinline__ void few_ldw(FewW& v, const __nv_bfloat16* p, bool on, uint64_t policy) {
  if (on) {
    asm volatile(
        "ld.global.nc.L1::no_allocate.L2::cache_hint.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
        : "=r"(v.r[0]), "=r"(v.r[1]), "=r"(v.r[2]), "=r"(v.r[3]), "=r"(v.r[4]), "=r"(v.r[5]),
          "=r"(v.r[6]), "=r"(v.r[7])
        : "l"(p), "l"(policy));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.r[i] = 0u;
  }
}
__device__ __forceinline__ uint4 few_ldx(const __nv_bfloat16* p, bool on) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (on) v = *reinterpret_cast<const uint4*>(p);
  return v;
}

__device__ __forceinline__ float few_silu(float g) { return g / (1.0f + expf(-g)); }

// One 64-wide chunk of k: rows g and g + 8 of two 16-row blocks.
struct FewA {
  FewW v[2][2];  // [block][row half]
};

}  // namespace moe
