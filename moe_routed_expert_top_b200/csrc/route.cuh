// route.cuh - the routing arithmetic shared by the routing kernel
// (route_permute.cu) and the few-token layer (few.cu): one fixed float32 exp
// and one fixed order of sums, so both give the same weights bit for bit.
// Only explicitly rounded operations are used, so the result does not depend on
// the translation unit's FMA setting.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

// exp(x) in float32 (Cody & Waite, "Software Manual for the Elementary
// Functions", 1980, range reduction; Taylor polynomial of degree 7):
//   n = rint(x * log2 e); r = (x - n*ln2_hi) - n*ln2_lo, ln2_hi = 355/512
//   (exact product for |n| < 2^15); p = sum_{i<=7} r^i / i! by Horner;
//   result = (p * 2^(n - floor(n/2))) * 2^floor(n/2): the first product is
//   exact, the second is the single final rounding (also into subnormals).
// The argument is clamped to [-104, 89] first (exp underflows to 0 below and
// overflows to +inf above). NaN inputs are outside the supported domain.
__device__ __forceinline__ float moe_expf(float x) {
  const float kLog2e = 0x1.715476p+0f;
  const float kLn2Hi = 0x1.630000p-1f;  // 0.693359375
  const float kLn2Lo = -0x1.bd0106p-13f;
  x = fminf(fmaxf(x, -104.0f), 89.0f);
  const float n = rintf(__fmul_rn(x, kLog2e));
  float r = __fsub_rn(x, __fmul_rn(n, kLn2Hi));
  r = __fsub_rn(r, __fmul_rn(n, kLn2Lo));
  float p = 0x1.a01a02p-13f;                     // 1/7!
  p = __fadd_rn(__fmul_rn(p, r), 0x1.6c16c2p-10f);  // 1/6!
  p = __fadd_rn(__fmul_rn(p, r), 0x1.111112p-7f);   // 1/5!
  p = __fadd_rn(__fmul_rn(p, r), 0x1.555556p-5f);   // 1/4!
  p = __fadd_rn(__fmul_rn(p, r), 0x1.555556p-3f);   // 1/3!
  p = __fadd_rn(__fmul_rn(p, r), 0.5f);             // 1/2!
  p = __fadd_rn(__fmul_rn(p, r), 1.0f);             // 1/1!
  p = __fadd_rn(__fmul_rn(p, r), 1.0f);             // 1/0!
  const int ni = static_cast<int>(n);
  const int lo = ni >> 1;  // floor(n/2)
  const int hi = ni - lo;
  const float s_hi = __int_as_float((hi + 127) << 23);
  const float s_lo = __int_as_float((lo + 127) << 23);
  return __fmul_rn(__fmul_rn(p, s_hi), s_lo);
}

}  // namespace moe
