// What every kernel of the 8-bit integer layers does to an exact sum: one place,
// and intrinsics that are not contracted, so that an output has the same bits
// whichever kernel computes it.
#pragma once

#include "common.cuh"

namespace ffn {

__device__ __forceinline__ float int8_scaled(int sum, float xs, float ws) {
  return __fmul_rn(__fmul_rn(__int2float_rn(sum), xs), ws);
}

// exp(v) and 1 / v by the hardware's approximations, two steps of fp32 off (exp one
// more for each unit of |v|).  Results below fp32's normal range are zeros.
__device__ __forceinline__ float exp_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmul_rn(v, 1.44269504f)));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// h before its rounding to bf16, which drops 16 bits right after.
__device__ __forceinline__ float int8_silu_mul(float gate, float up) {
  return __fmul_rn(__fmul_rn(gate, rcp_approx(__fadd_rn(1.0f, exp_approx(-gate)))), up);
}

// Quantisation of a row by the largest magnitude among its bf16 bits.  Factors
// are fp32 numbers rounded once: a row of values below 2^-100, where 127 / a may
// be infinite, is scaled by 2^64 on the way.
struct Int8Row {
  float scale, pre, inv;  // code = rint((x * pre) * inv)
  __device__ __forceinline__ explicit Int8Row(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits << 16);
    const bool finite = amax_bits < 0x7f80u;
    scale = finite ? __fdiv_rn(a, 127.0f) : __uint_as_float(0x7fc00000u);
    pre = a < 7.8886091e-31f ? 18446744073709551616.0f : 1.0f;  // 2^-100, 2^64
    inv = finite && a > 0.0f ? __fdiv_rn(127.0f, __fmul_rn(a, pre)) : 0.0f;
  }
  __device__ __forceinline__ uint32_t code(float x) const {  // (in the low byte)
    return (uint32_t)__float2int_rn(__fmul_rn(__fmul_rn(x, pre), inv)) & 0xffu;
  }
};

// Codes of 8 bf16 values.
__device__ __forceinline__ uint2 int8_encode8(const Int8Row& q, uint4 v) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = q.code(__uint_as_float(in[i] << 16)) | (q.code(__uint_as_float(in[i] & 0xffff0000u)) << 8);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The larger magnitude in each half: NaN is above infinity, and that above all numbers.
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t top, uint32_t pair) {
  return __vmaxu2(top, pair & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t amax8_bf16(uint32_t top, uint4 v) {
  return amax_bf16x2(amax_bf16x2(amax_bf16x2(amax_bf16x2(top, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint32_t amax_of_pair(uint32_t top) { return max(top & 0xffffu, top >> 16); }

}  // namespace ffn
