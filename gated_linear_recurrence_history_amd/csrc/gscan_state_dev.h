// Device helpers shared by the matrix-state scan and its single-token step.
#pragma once

#include <cstdint>
#include <hip/hip_runtime.h>

#include "gscan_state.h"

namespace gscan {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float bf_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float bf_hi(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

__device__ __forceinline__ uint16_t to_bf16(float a)
{
    return __builtin_bit_cast(uint16_t, (__bf16)a);
}

// element i of an operand of type dtype (0: fp32, 1: bf16)
__device__ __forceinline__ float load_scalar(const void *p, int64_t i, int dtype)
{
    return dtype ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16)
                 : reinterpret_cast<const float *>(p)[i];
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// log of the gate: x itself (log form), or log sigmoid(x) = min(x, 0) -
// log1p(e), e = exp(-|x|), without cancellation at either end: log1p(e) =
// 2 atanh(s), s = e / (2 + e) <= 1/3, by its power series to s^15 (the next
// term is below 2^-26 of the sum).  Below -1000 the gate is zero in fp32 and
// far beyond; the clamp keeps sums of log gates finite, so that differences
// behind a closed gate stay exact.  NaN passes.
__device__ __forceinline__ float log_gate(float x, int form)
{
    float l = x;
    if (!form) {
        const float e = exp2_(-1.44269504f * fabsf(x));
        const float s = e * __builtin_amdgcn_rcpf(2.f + e), z = s * s;
        float p = fmaf(z, 1.f / 15.f, 1.f / 13.f);
        p = fmaf(z, p, 1.f / 11.f);
        p = fmaf(z, p, 1.f / 9.f);
        p = fmaf(z, p, 1.f / 7.f);
        p = fmaf(z, p, 1.f / 5.f);
        p = fmaf(z, p, 1.f / 3.f);
        p = fmaf(z, p, 1.f);
        l = (x < 0.f ? x : 0.f) - 2.f * s * p;
    }
    return l < -1000.f ? -1000.f : l;
}

// d(log gate)/dx: 1 - sigmoid(x) = sigmoid(-x), or 1
__device__ __forceinline__ float log_gate_slope(float x, int form)
{
    return form ? 1.f : 1.f / (1.f + expf(x));
}

}  // namespace
}  // namespace gscan
