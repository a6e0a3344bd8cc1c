// Products of few tokens with a large weight, for the gated projection and the
// forward of the cross entropy: bound by reading the weight once.
//
// A workgroup takes 16 R rows of the weight (of both weights, gated) at a time; its
// eight wavefronts divide k.  A wavefront's share of the rows goes from memory into
// registers in the layout of the 16 x 16 products, a good part of it requested before the
// first product (1 kB a load; the tokens' rows come from L2 the same way, lanes past the
// last token load nothing: R rows of the weight share them), and the eight partial sums
// meet in LDS.  One token, 2048 x 2 x 5504: 11.6 us, 3.9 TB/s; 19 tokens, 2048 x 32000: 30 us, 4.4
// TB/s (both as tiles of 128 x 64: 22 and 50, which take as long for one token as for 64).
#pragma once

#include "gscan_mm.h"

namespace gscan {
namespace {

constexpr int kFewThreads = 512, kFewWaves = 8;
constexpr int kFewGrid = 512;  // workgroups: two per CU

template <bool BF>
__device__ __forceinline__ f4 multiply16(const u4 &x, const u4 &y, f4 acc)
{
    if constexpr (BF) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, x), __builtin_bit_cast(bf8, y), acc, 0,
                                                       0, 0);
    } else {
        const f4 a = __builtin_bit_cast(f4, x), b = __builtin_bit_cast(f4, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
        return acc;
    }
}

// EPI_GATE: out[n][m].  EPI_LSE: part[n][workgroup], the maximum and the sum of
// powers of two of the workgroup's logits, and the targets' logits.
// R: groups of 16 rows of a weight taken together.  (Losses of 1, 8 and 16 tokens, 2048 x
// 32000, other weights each time: with one group 33.9, 38.3 and 44.1 us, with two 32.7,
// 35.6 and 41.6, with four 34.7, 35.7 and 39.5.)
template <Epi E, int NT>
constexpr int kFewRows = E == EPI_GATE ? NT : 2 * NT;

template <Epi E, bool BF, int NT>
__global__ void __launch_bounds__(kFewThreads, 4) gscan_few_kernel(MmArgs a, int groups)
{
    constexpr int kMats = E == EPI_GATE ? 2 : 1, R = kFewRows<E, NT>, kAhead = NT > 1 ? 2 : E == EPI_GATE ? 8 : 4;
    constexpr int kIn = BF ? 8 : 4, kBlock = 4 * kIn, kSz = kSize<BF>;  // elements of 16 bytes, k of a product
    __shared__ f4 red[2][kFewWaves][kMats][NT][64];
    __shared__ float2 ends[E == EPI_LSE ? kFewThreads / 2 : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int blocks = (int)ceil_div(a.K, kBlock), share = (int)ceil_div(blocks, kFewWaves);
    const int b0 = wave * share, b1 = b0 + share < blocks ? b0 + share : blocks;
    const int k0 = kIn * (lane >> 4), K = (int)a.K;  // of a block
    const char *const w[2] = {reinterpret_cast<const char *>(a.a), reinterpret_cast<const char *>(a.a2)};
    const float unit = a.scale * 1.4426950408889634f;
    // the output element of a thread: row r of 16, token n of 16
    const int r = tid & 15, n = (tid >> 4) & 15;
    float top[NT], sum[NT];
    int64_t target[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        top[t] = -INFINITY;
        sum[t] = 0.f;
        target[t] = -1;
        if (E == EPI_LSE && 16 * t + n < a.N) target[t] = token_at(a.tokens, 16 * t + n, a.tok64, a.M);
    }
    int odd = 0;
    for (int g = blockIdx.x; g < groups; g += gridDim.x) {
        const int64_t row = 16 * R * (int64_t)g + (lane & 15);
        f4 acc[R][kMats][NT];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[i][m][t] = f4{};
        for (int b = b0; b < b1; b += kAhead) {
            u4 x[R][kMats][kAhead], y[NT][kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int k = (b + u) * kBlock + k0;
                const bool in = b + u < b1 && k < K;
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int m = 0; m < kMats; ++m) {
                        x[i][m][u] = u4{};
                        if (in && row + 16 * i < a.M)
                            x[i][m][u] = *reinterpret_cast<const u4 *>(
                                w[m] + ((row + 16 * i) * (m ? a.lda2 : a.lda) + k) * kSz);
                    }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int token = 16 * t + (lane & 15);
                    y[t][u] = u4{};
                    if (in && token < a.N)
                        y[t][u] = *reinterpret_cast<const u4 *>(reinterpret_cast<const char *>(a.b) +
                                                                (token * a.ldb + k) * kSz);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int m = 0; m < kMats; ++m)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            acc[i][m][t] = multiply16<BF>(x[i][m][u], y[t][u], acc[i][m][t]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i, odd ^= 1) {
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) red[odd][wave][m][t][lane] = acc[i][m][t];
            __syncthreads();  // (the other buffer's readers are behind the next one)
            if (tid >= 256) continue;
            const int64_t m1 = 16 * (R * (int64_t)g + i) + r;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float z[kMats];
#pragma unroll
                for (int m = 0; m < kMats; ++m) {
                    z[m] = 0.f;
#pragma unroll
                    for (int v = 0; v < kFewWaves; ++v) z[m] += red[odd][v][m][t][16 * (r >> 2) + n][r & 3];
                }
                const int64_t token = 16 * t + n;
                if (m1 >= a.M || token >= a.N) continue;
                if constexpr (E == EPI_GATE) {
                    float f, slope;
                    activation<BF>(z[0], a.act, f, slope);
                    const float o = f * z[1];
                    if constexpr (BF)
                        reinterpret_cast<uint16_t *>(a.out)[token * a.ldo + m1] = to_bf16(o);
                    else
                        reinterpret_cast<float *>(a.out)[token * a.ldo + m1] = o;
                } else {
                    const float q = z[0] * unit;
                    if (target[t] == m1) a.picked[token] = q;
                    join_lse(top[t], sum[t], q, 1.f);
                }
            }
        }
    }
    if constexpr (E == EPI_LSE) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            __syncthreads();
            if (tid < 256) ends[tid] = float2{top[t], sum[t]};
            __syncthreads();
            if (tid < 16 && 16 * t + tid < a.N) {
                float m = -INFINITY, s = 0.f;
                for (int i = 0; i < 16; ++i) join_lse(m, s, ends[16 * tid + i].x, ends[16 * tid + i].y);
                a.part[(int64_t)(16 * t + tid) * gridDim.x + blockIdx.x] = float2{m, s};
            }
        }
    }
}

constexpr int64_t kFew = 32;  // tokens, at most

template <Epi E>
int few_groups(const MmArgs &a)
{
    return (int)ceil_div(a.M, 16 * (a.N <= 16 ? kFewRows<E, 1> : kFewRows<E, 2>));
}

int few_grid(int groups) { return groups < kFewGrid ? groups : kFewGrid; }

template <Epi E, bool BF>
hipError_t launch_few_of(const MmArgs &a, hipStream_t st)
{
    const int groups = few_groups<E>(a);
    auto *k = a.N <= 16 ? gscan_few_kernel<E, BF, 1> : gscan_few_kernel<E, BF, 2>;
    hipLaunchKernelGGL(k, dim3((unsigned)few_grid(groups)), dim3(kFewThreads), 0, st, a, groups);
    return hipGetLastError();
}

template <Epi E>
hipError_t launch_few(const MmArgs &a, int dtype, hipStream_t st)
{
    return dtype ? launch_few_of<E, true>(a, st) : launch_few_of<E, false>(a, st);
}

}  // namespace
}  // namespace gscan
