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

// log of the gate: x itself (log form), or log sigmoid(x) without
// cancellation at either end.  Below -1000 the gate is zero in fp32 and far
// beyond; the clamp keeps sums of log gates finite, so that differences
// behind a closed gate stay exact.  NaN passes.
__device__ __forceinline__ float log_gate(float x, int form)
{
    const float l = form ? x : fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
    const float y = x != x ? x : l;  // fminf would drop a NaN
    return y < -1000.f ? -1000.f : y;
}

// d(log gate)/dx: 1 - sigmoid(x) = sigmoid(-x), or 1
__device__ __forceinline__ float log_gate_slope(float x, int form)
{
    return form ? 1.f : 1.f / (1.f + expf(x));
}

}  // namespace
}  // namespace gscan
