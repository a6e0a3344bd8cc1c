// RMS norm of every query and key head with the position rotation in the
// same pass, forward and backward, for gfx950 (MI355X).
//
// Per row x (one head of one token), r = rsqrt(mean(x^2) + eps):
//   n = x r w;  the first `rot` elements are turned in pairs by the angles
//   pos * freq_i, (a, b) -> m (a cos - b sin, b cos + a sin), with the pairs
//   (2i, 2i + 1) (interleaved) or (i, i + rot/2) (half).
// Backward, with G the upstream gradient turned back (the rotation's
// transpose):
//   dw = sum over rows of G x r,   dx = r (G w) - x r^3 mean(G w x).
// Every row is read and written once and that is all the time there is, so
// rows stay in registers: a group of lanes holds a row, eight elements per
// lane in two pieces of four.  The pieces follow each other, but in the
// rotated part of the half layout, where a lane takes the two members of four
// pairs: either way a rotation stays inside the lane, and sums are lane
// exchanges inside the group.  All heads of a token share its angles: a
// workgroup forms the sines and cosines of its tokens once, in LDS, from the
// angle reduced to [-pi, pi] in fp64, so positions of any size keep fp32
// accuracy.
// dw: every workgroup keeps its sums in registers over its tokens and leaves
// one partial, which a second kernel adds in a fixed order in fp64.
// Rows are requested a few at a time as raw words, before the angles are formed
// (one at a time: 88 us where this takes 81; four bf16 rows widened to fp32 as they
// come: 106, for fewer wavefronts fit).  Measured (a profiler's means over 40 calls):
// forward, 16384 tokens, 40 bf16 heads of 128: 336 MB in 81 us, 4.1 TB/s (a large
// copy: 4.8; a whole call without the profiler, caches cold: 75 us); 8192 tokens in
// fp32: 70; backward, 8191 tokens, 32 fp32 heads of 80: 252 MB in 46 us and 7 us for
// the 1024 partials of dw; the 16384 tokens in bf16: 503 MB in 122 and 8; one token:
// 4 us.
#include <type_traits>

#include "gscan_state_dev.h"

namespace gscan {
namespace {

constexpr int kNThreads = 256;
constexpr int kNMaxTok = 8;       // tokens whose angles are in LDS at a time
constexpr int kNMaxPairs = 128;
constexpr int64_t kNMaxGrid = 1024;  // workgroups of the backward (partials of dw)
constexpr int kNBatch = 4, kNBatchBwd = 2;  // rows of a lane group requested together

// Eight elements of a row as loaded: two pieces of four.
template <bool BF>
struct Raw;
template <>
struct Raw<true> {
    uint2 a, b;
};
template <>
struct Raw<false> {
    f4 a, b;
};

struct Vec {
    float v[8];
};

__device__ __forceinline__ Vec widen(const Raw<true> &r)
{
    return Vec{bf_lo(r.a.x), bf_hi(r.a.x), bf_lo(r.a.y), bf_hi(r.a.y),
               bf_lo(r.b.x), bf_hi(r.b.x), bf_lo(r.b.y), bf_hi(r.b.y)};
}
__device__ __forceinline__ Vec widen(const Raw<false> &r)
{
    return Vec{r.a[0], r.a[1], r.a[2], r.a[3], r.b[0], r.b[1], r.b[2], r.b[3]};
}

// Pieces at elements i and i + hop of p.
template <bool BF>
__device__ __forceinline__ Raw<BF> load_raw(const void *p, int64_t i, int hop)
{
    typedef typename std::conditional<BF, uint16_t, float>::type S;
    typedef decltype(Raw<BF>::a) P;
    const S *s = reinterpret_cast<const S *>(p) + i;
    return Raw<BF>{*reinterpret_cast<const P *>(s), *reinterpret_cast<const P *>(s + hop)};
}

template <bool BF>
__device__ __forceinline__ void store_vec(void *p, int64_t i, int hop, const Vec &x)
{
    if constexpr (BF) {
        uint16_t *d = reinterpret_cast<uint16_t *>(p) + i;
        *reinterpret_cast<uint2 *>(d) = uint2{pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[2], x.v[3])};
        *reinterpret_cast<uint2 *>(d + hop) = uint2{pack_bf16(x.v[4], x.v[5]), pack_bf16(x.v[6], x.v[7])};
    } else {
        float *d = reinterpret_cast<float *>(p) + i;
        *reinterpret_cast<f4 *>(d) = f4{x.v[0], x.v[1], x.v[2], x.v[3]};
        *reinterpret_cast<f4 *>(d + hop) = f4{x.v[4], x.v[5], x.v[6], x.v[7]};
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// Sum over groups of lpr lanes, in every lane: exchanges of neighbours, of
// pairs, then mirrors of 8 and of 16 lanes (whose parts are sums already).
__device__ __forceinline__ float group_sum(float x, int lpr)
{
    if (lpr > 1) x += dpp<0xb1>(x);    // lanes 1 0 3 2
    if (lpr > 2) x += dpp<0x4e>(x);    // lanes 2 3 0 1
    if (lpr > 4) x += dpp<0x141>(x);   // 7 .. 0
    if (lpr > 8) x += dpp<0x140>(x);   // 15 .. 0
    if (lpr > 16) x += __shfl_xor(x, 16);
    return x;
}

// Where a lane's pieces are: elements at and at + hop, the angles of its four
// pairs from `pair` (turned: it has any).
struct Place {
    int at, hop, pair;
    bool in, turned;
};
template <bool HALF>
__device__ __forceinline__ Place place_of(const NormArgs &a, int sub)
{
    Place p;
    p.in = 8 * sub < a.D;
    p.turned = 8 * sub < a.rot;
    p.at = 8 * sub;
    p.hop = 4;
    p.pair = 4 * sub;
    if (HALF && p.turned) {
        p.at = 4 * sub;
        p.hop = a.rot / 2;
    }
    return p;
}

// cos and sin of the angles of `n` tokens from `t0`, times the magnitude
__device__ __forceinline__ void angles(const NormArgs &a, float2 (*cs)[kNMaxPairs], int64_t t0,
                                       int n, int tid)
{
    const int half = a.rot / 2;
    for (int i = tid; i < n * half; i += kNThreads) {
        const int t = i / half, e = i % half;
        const double pos = a.pos64 ? (double)reinterpret_cast<const int64_t *>(a.pos)[t0 + t]
                                   : (double)reinterpret_cast<const int32_t *>(a.pos)[t0 + t];
        const double w = pos * (double)a.freq[e];
        const double turns = rint(w * 0.15915494309189533577);
        // 2 pi in two fp64 parts
        const double r = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586232, w));
        float s, c;
        sincosf((float)r, &s, &c);
        cs[t][e] = float2{a.magnitude * c, a.magnitude * s};
    }
}

// x turned by the angles (sign 1) or back (sign -1)
template <bool HALF>
__device__ __forceinline__ Vec turn(const Vec &x, const float2 *cs, const Place &p, float sign)
{
    Vec y = x;
    if (p.turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = cs[p.pair + j];
            const int u = HALF ? j : 2 * j, w = HALF ? 4 + j : 2 * j + 1;
            const float sn = sign * t.y;
            y.v[u] = x.v[u] * t.x - x.v[w] * sn;
            y.v[w] = x.v[w] * t.x + x.v[u] * sn;
        }
    }
    return y;
}

// Rows of a workgroup: row r of its tokens is head r - t heads of token t =
// r / heads = floor(2 r inv / 2^32) with inv = ceil(2^31 / heads), which fits 32
// bits for one head too and is exact for r heads < 2^31 (r is below 2048 where a
// workgroup has more than one token).  inv 0: one token.
struct Row {
    int t, which, h;
    bool ok;
};
__device__ __forceinline__ Row row_of(const NormArgs &a, int row, int rows, int heads, uint32_t inv,
                                      bool in)
{
    Row r;
    r.ok = row < rows && in;
    row = row < rows ? row : 0;
    r.t = inv ? (int)__umulhi(2u * (uint32_t)row, inv) : 0;
    const int hh = row - r.t * heads;
    r.which = hh >= a.heads[0];
    r.h = hh - r.which * a.heads[0];
    return r;
}

// Weights of the lane's elements, of queries and keys.
__device__ __forceinline__ void load_weights(const NormArgs &a, const Place &p, Vec (&w)[2])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i].v[e] = 1.f;
        if (p.in && a.w[i]) w[i] = widen(load_raw<false>(a.w[i], p.at, p.hop));
    }
}

// Rows of a lane group requested together: the angles are formed, and one row
// is finished, while the others are on their way.
template <bool BF, bool HALF>
__global__ void __launch_bounds__(kNThreads) gscan_norm_fwd_kernel(NormArgs a, int lpr, int tpb, uint32_t inv)
{
    __shared__ __align__(16) float2 cs[kNMaxTok][kNMaxPairs];
    const int tid = threadIdx.x, grp = tid / lpr;
    const Place p = place_of<HALF>(a, tid & (lpr - 1));
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
    const int n = (int)(a.tokens - t0 < tpb ? a.tokens - t0 : tpb);
    const int heads = a.heads[0] + a.heads[1], rows = n * heads, rpp = kNThreads / lpr;
    const float mean = 1.f / (float)a.D;
    Vec w[2];
    Raw<BF> x[kNBatch];
    for (int b = 0; b < rows; b += kNBatch * rpp) {  // all lanes take part in the exchanges
#pragma unroll
        for (int i = 0; i < kNBatch; ++i) {
            const Row r = row_of(a, b + grp + i * rpp, rows, heads, inv, p.in);
            x[i] = Raw<BF>{};
            if (r.ok)
                x[i] = load_raw<BF>(r.which ? a.x[1] : a.x[0],
                                    (t0 + r.t) * (r.which ? a.xn[1] : a.xn[0]) +
                                        r.h * (r.which ? a.xh[1] : a.xh[0]) + p.at, p.hop);
        }
        if (b == 0) {
            load_weights(a, p, w);
            angles(a, cs, t0, n, tid);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kNBatch; ++i) {
            const Row r = row_of(a, b + grp + i * rpp, rows, heads, inv, p.in);
            Vec v = widen(x[i]);
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(v.v[e], v.v[e], s);
            const float f = __builtin_amdgcn_rsqf(group_sum(s, lpr) * mean + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] *= f * (r.which ? w[1].v[e] : w[0].v[e]);
            v = turn<HALF>(v, cs[r.t], p, 1.f);
            if (r.ok)
                store_vec<BF>(r.which ? a.y[1] : a.y[0],
                              ((t0 + r.t) * (r.which ? a.heads[1] : a.heads[0]) + r.h) * a.D + p.at, p.hop, v);
        }
    }
}

template <bool BF, bool HALF>
__global__ void __launch_bounds__(kNThreads) gscan_norm_bwd_kernel(NormArgs a, int lpr, int tpb, uint32_t inv)
{
    __shared__ __align__(16) float2 cs[2][kNMaxTok][kNMaxPairs];
    __shared__ float red[2][256];
    const int tid = threadIdx.x, grp = tid / lpr;
    const Place p = place_of<HALF>(a, tid & (lpr - 1));
    const int heads = a.heads[0] + a.heads[1], rpp = kNThreads / lpr;
    const float mean = 1.f / (float)a.D;
    Vec dw[2] = {}, w[2];
    load_weights(a, p, w);
    int odd = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * tpb; t0 < a.tokens; t0 += (int64_t)gridDim.x * tpb, odd ^= 1) {
        const int n = (int)(a.tokens - t0 < tpb ? a.tokens - t0 : tpb), rows = n * heads;
        for (int b = 0; b < rows; b += kNBatchBwd * rpp) {
            Raw<BF> xr[kNBatchBwd], gr[kNBatchBwd];
#pragma unroll
            for (int i = 0; i < kNBatchBwd; ++i) {
                const Row r = row_of(a, b + grp + i * rpp, rows, heads, inv, p.in);
                xr[i] = gr[i] = Raw<BF>{};
                if (r.ok) {
                    xr[i] = load_raw<BF>(r.which ? a.x[1] : a.x[0],
                                         (t0 + r.t) * (r.which ? a.xn[1] : a.xn[0]) +
                                             r.h * (r.which ? a.xh[1] : a.xh[0]) + p.at, p.hop);
                    gr[i] = load_raw<BF>(r.which ? a.dy[1] : a.dy[0],
                                         (t0 + r.t) * (r.which ? a.dn[1] : a.dn[0]) +
                                             r.h * (r.which ? a.dh[1] : a.dh[0]) + p.at, p.hop);
                }
            }
            if (b == 0) {  // (the other buffer's readers may still be at work)
                angles(a, cs[odd], t0, n, tid);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kNBatchBwd; ++i) {
                const Row r = row_of(a, b + grp + i * rpp, rows, heads, inv, p.in);
                const Vec x = widen(xr[i]), g = turn<HALF>(widen(gr[i]), cs[odd][r.t], p, -1.f);
                Vec gw;
                float s = 0.f, m = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    gw.v[e] = g.v[e] * (r.which ? w[1].v[e] : w[0].v[e]);
                    s = fmaf(x.v[e], x.v[e], s);
                    m = fmaf(gw.v[e], x.v[e], m);
                }
                const float f = __builtin_amdgcn_rsqf(group_sum(s, lpr) * mean + a.eps);
                const float c = group_sum(m, lpr) * mean * f * f;
                if (r.ok) {
                    Vec dx;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float q = g.v[e] * (x.v[e] * f);
                        dw[0].v[e] += r.which ? 0.f : q;
                        dw[1].v[e] += r.which ? q : 0.f;
                        dx.v[e] = f * (gw.v[e] - x.v[e] * c);
                    }
                    store_vec<BF>(r.which ? a.y[1] : a.y[0],
                                  ((t0 + r.t) * (r.which ? a.heads[1] : a.heads[0]) + r.h) * a.D + p.at, p.hop, dx);
                }
            }
        }
    }
    if (!a.ws) return;
    // lane groups add theirs one after the other
    for (int k = 0; k < rpp; ++k) {
        __syncthreads();
        if (grp == k && p.in)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float *q = &red[i][p.at + (e < 4 ? e : p.hop + e - 4)];
                    *q = (k ? *q : 0.f) + dw[i].v[e];
                }
    }
    __syncthreads();
    float *part = reinterpret_cast<float *>(a.ws) + (int64_t)blockIdx.x * 2 * a.D;
    for (int i = tid; i < 2 * a.D; i += kNThreads) part[i] = i < a.D ? red[0][i] : red[1][i - a.D];
}

// dw[i][d] = sum over the partials in a fixed order: 16 columns per workgroup,
// 64 partials apart per thread
__global__ void __launch_bounds__(1024) gscan_norm_dw_kernel(const float *part, int grid, int D, float *dwq,
                                                             float *dwk)
{
    __shared__ double red[64][17];
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4, i = blockIdx.x * 16 + c;
    double s = 0.0;
    if (i < 2 * D)
        for (int b = r; b < grid; b += 64) s += (double)part[(int64_t)b * 2 * D + i];
    red[r][c] = s;
    __syncthreads();
    for (int h = 32; h > 0; h /= 2) {
        if (r < h) red[r][c] += red[r + h][c];
        __syncthreads();
    }
    float *o = i < D ? dwq : dwk;
    if (r == 0 && i < 2 * D && o) o[i < D ? i : i - D] = (float)red[0][c];
}

struct NormGeom {
    int lpr, tpb;
    uint32_t inv;  // ceil(2^31 / heads), 0 where a workgroup has one token
    int64_t blocks;
};

// Tokens per workgroup: the fewest that come within 2 per cent of filling the
// lane groups' batches best, up to two batches.  (Relative: few narrow heads fill
// little of a workgroup even together; 32768 tokens of 2 bf16 heads of 32 take 15
// us, with a workgroup per token 82.)
NormGeom geom(int64_t tokens, int heads, int D)
{
    NormGeom g;
    g.lpr = 1;
    while (g.lpr * 8 < D) g.lpr *= 2;
    const int rpp = kNThreads / g.lpr, full = kNBatch * rpp;
    g.tpb = 1;
    double best = 0.0;
    for (int t = 1; t <= kNMaxTok && (t == 1 || t * (int64_t)heads <= 2 * full); ++t) {
        const int64_t rows = t * (int64_t)heads;
        const double use = (double)rows / (double)((rows + rpp - 1) / rpp * rpp) *
                           (rows < full ? (double)rows / full : 1.0);
        if (use > best * 1.02) {
            best = use;
            g.tpb = t;
        }
    }
    g.inv = g.tpb > 1 ? (uint32_t)((0x80000000ull + heads - 1) / heads) : 0u;
    g.blocks = (tokens + g.tpb - 1) / g.tpb;
    return g;
}

int64_t bwd_grid(int64_t blocks) { return blocks < kNMaxGrid ? blocks : kNMaxGrid; }

}  // namespace

// A partial of both weights' gradients per workgroup.
size_t norm_workspace_bytes(int64_t tokens, int heads, int D)
{
    const int64_t n = bwd_grid(geom(tokens, heads, D).blocks);
    return (size_t)(n > 0 ? n : 1) * 2u * (size_t)D * sizeof(float);
}

hipError_t launch_norm_forward(const NormArgs &a, hipStream_t st)
{
    const NormGeom g = geom(a.tokens, a.heads[0] + a.heads[1], a.D);
    const dim3 grid((unsigned)g.blocks), blk(kNThreads);
    if (!g.blocks) return hipSuccess;
    const bool half = a.layout == 0;
    auto *k = a.dtype ? (half ? gscan_norm_fwd_kernel<true, true> : gscan_norm_fwd_kernel<true, false>)
                      : (half ? gscan_norm_fwd_kernel<false, true> : gscan_norm_fwd_kernel<false, false>);
    hipLaunchKernelGGL(k, grid, blk, 0, st, a, g.lpr, g.tpb, g.inv);
    return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs &a, hipStream_t st)
{
    const NormGeom g = geom(a.tokens, a.heads[0] + a.heads[1], a.D);
    const int64_t n = bwd_grid(g.blocks);
    if (n) {  // without tokens dw is zero
        const bool half = a.layout == 0;
        auto *k = a.dtype ? (half ? gscan_norm_bwd_kernel<true, true> : gscan_norm_bwd_kernel<true, false>)
                          : (half ? gscan_norm_bwd_kernel<false, true> : gscan_norm_bwd_kernel<false, false>);
        hipLaunchKernelGGL(k, dim3((unsigned)n), dim3(kNThreads), 0, st, a, g.lpr, g.tpb, g.inv);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.ws) return hipSuccess;  // no weight gradient wanted
    hipLaunchKernelGGL(gscan_norm_dw_kernel, dim3((unsigned)((2 * a.D + 15) / 16)), dim3(1024), 0, st,
                       reinterpret_cast<const float *>(a.ws), (int)n, a.D, a.dw[0], a.dw[1]);
    return hipGetLastError();
}

}  // namespace gscan
