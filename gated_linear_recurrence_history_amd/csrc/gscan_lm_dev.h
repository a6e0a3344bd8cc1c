// Device helpers shared by the token embedding, the gated projection and the
// vocabulary's cross entropy.
#pragma once

#include "gscan_lm.h"
#include "gscan_state_dev.h"

namespace gscan {
namespace {

// A launch has fewer than 2^32 threads: workgroups of what may be more go on in strides.
constexpr int64_t kMaxGroups = int64_t(1) << 20;
inline dim3 groups_of(int64_t n) { return dim3((unsigned)(n < kMaxGroups ? n : kMaxGroups)); }

// Eight elements of a row (fp32 or bf16, 16-byte aligned), widened.
struct Oct {
    float v[8];
};

template <bool BF>
struct OctRaw;
template <>
struct OctRaw<true> {
    u4 a;
};
template <>
struct OctRaw<false> {
    f4 a, b;
};

template <bool BF>
__device__ __forceinline__ OctRaw<BF> load_oct(const void *p, int64_t i)
{
    if constexpr (BF) {
        return OctRaw<true>{*reinterpret_cast<const u4 *>(reinterpret_cast<const uint16_t *>(p) + i)};
    } else {
        const f4 *s = reinterpret_cast<const f4 *>(reinterpret_cast<const float *>(p) + i);
        return OctRaw<false>{s[0], s[1]};
    }
}

__device__ __forceinline__ Oct widen(const OctRaw<true> &r)
{
    return Oct{bf_lo(r.a[0]), bf_hi(r.a[0]), bf_lo(r.a[1]), bf_hi(r.a[1]),
               bf_lo(r.a[2]), bf_hi(r.a[2]), bf_lo(r.a[3]), bf_hi(r.a[3])};
}
__device__ __forceinline__ Oct widen(const OctRaw<false> &r)
{
    return Oct{r.a[0], r.a[1], r.a[2], r.a[3], r.b[0], r.b[1], r.b[2], r.b[3]};
}

template <bool BF>
__device__ __forceinline__ void store_oct(void *p, int64_t i, const Oct &x)
{
    if constexpr (BF) {
        *reinterpret_cast<u4 *>(reinterpret_cast<uint16_t *>(p) + i) =
            u4{pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[2], x.v[3]), pack_bf16(x.v[4], x.v[5]),
               pack_bf16(x.v[6], x.v[7])};
    } else {
        f4 *d = reinterpret_cast<f4 *>(reinterpret_cast<float *>(p) + i);
        d[0] = f4{x.v[0], x.v[1], x.v[2], x.v[3]};
        d[1] = f4{x.v[4], x.v[5], x.v[6], x.v[7]};
    }
}

// Token or target i; anything outside 0 .. V - 1 is -1.
__device__ __forceinline__ int64_t token_at(const void *tokens, int64_t i, int tok64, int64_t V)
{
    const int64_t t = tok64 ? reinterpret_cast<const int64_t *>(tokens)[i]
                            : (int64_t) reinterpret_cast<const int32_t *>(tokens)[i];
    return t >= 0 && t < V ? t : -1;
}

// Tokens i0 + 64 j, the lanes' behind each other, as keys: anything outside 0 .. V - 1
// is V, what lies behind the last of the n tokens ~0.
template <int ITEMS>
__device__ __forceinline__ void token_keys(const void *tokens, int tok64, int64_t V, int64_t i0, int64_t n,
                                           uint32_t (&key)[ITEMS])
{
    if (tok64) {  // (not by token: the loads of one lane are to be under way together)
        int64_t t[ITEMS];
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            t[j] = -1;
            if (i0 + 64 * j < n) t[j] = reinterpret_cast<const int64_t *>(tokens)[i0 + 64 * j];
        }
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) key[j] = t[j] >= 0 && t[j] < V ? (uint32_t)t[j] : (uint32_t)V;
    } else {
        int32_t t[ITEMS];
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            t[j] = -1;
            if (i0 + 64 * j < n) t[j] = reinterpret_cast<const int32_t *>(tokens)[i0 + 64 * j];
        }
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) key[j] = t[j] >= 0 && t[j] < V ? (uint32_t)t[j] : (uint32_t)V;
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j)
        if (i0 + 64 * j >= n) key[j] = ~0u;
}

}  // namespace
}  // namespace gscan
