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
// rows stay in registers: a group of lanes holds a row, VE consecutive
// elements per lane, sums are lane exchanges inside the group, and the
// partner of a pair is in the same lane (interleaved) or one exchange away
// (half).  All heads of a token share its angles: a workgroup forms the
// sines and cosines of its tokens once, in LDS, from the angle reduced to
// [-pi, pi] in fp64, so positions of any size keep fp32 accuracy.
// dw: every workgroup keeps its sums in registers over its tokens and leaves
// one partial, which a second kernel adds in a fixed order in fp64.
#include "gscan_state_dev.h"

namespace gscan {
namespace {

constexpr int kNThreads = 256;
constexpr int kNMaxTok = 8;       // tokens whose angles are in LDS at a time
constexpr int kNMaxPairs = 128;
constexpr int64_t kNMaxGrid = 1024;  // workgroups of the backward (partials of dw)

template <int VE>
struct Vec {
    float v[VE];
};

template <int VE>
__device__ __forceinline__ Vec<VE> load_vec(const void *p, int64_t i, int dtype)
{
    Vec<VE> x;
    if (dtype) {
        const uint2 *s = reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + i);
        uint2 u[VE / 4];
        if constexpr (VE == 8) {
            const u4 t = *reinterpret_cast<const u4 *>(s);
            u[0] = uint2{t[0], t[1]};
            u[1] = uint2{t[2], t[3]};
        } else {
            u[0] = *s;
        }
#pragma unroll
        for (int j = 0; j < VE / 4; ++j) {
            x.v[4 * j] = bf_lo(u[j].x);
            x.v[4 * j + 1] = bf_hi(u[j].x);
            x.v[4 * j + 2] = bf_lo(u[j].y);
            x.v[4 * j + 3] = bf_hi(u[j].y);
        }
    } else {
        const f4 *s = reinterpret_cast<const f4 *>(reinterpret_cast<const float *>(p) + i);
#pragma unroll
        for (int j = 0; j < VE / 4; ++j) {
            const f4 t = s[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) x.v[4 * j + e] = t[e];
        }
    }
    return x;
}

template <int VE>
__device__ __forceinline__ void store_vec(void *p, int64_t i, int dtype, const Vec<VE> &x)
{
    if (dtype) {
        uint32_t u[VE / 2];
#pragma unroll
        for (int j = 0; j < VE / 2; ++j) u[j] = pack_bf16(x.v[2 * j], x.v[2 * j + 1]);
        uint16_t *d = reinterpret_cast<uint16_t *>(p) + i;
        if constexpr (VE == 8) *reinterpret_cast<u4 *>(d) = u4{u[0], u[1], u[2], u[3]};
        else *reinterpret_cast<uint2 *>(d) = uint2{u[0], u[1]};
    } else {
        f4 *d = reinterpret_cast<f4 *>(reinterpret_cast<float *>(p) + i);
#pragma unroll
        for (int j = 0; j < VE / 4; ++j)
            d[j] = f4{x.v[4 * j], x.v[4 * j + 1], x.v[4 * j + 2], x.v[4 * j + 3]};
    }
}

__device__ __forceinline__ float group_sum(float x, int lpr)
{
    for (int d = 1; d < lpr; d *= 2) x += __shfl_xor(x, d);
    return x;
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

// x turned by the angles (SIGN 1) or back (SIGN -1); d0: the lane's first
// element, half layout: `hop` lanes to the partner
template <int VE, bool HALF>
__device__ __forceinline__ Vec<VE> turn(const Vec<VE> &x, const float2 *cs, int d0, int rot,
                                        float sign)
{
    Vec<VE> y = x;
    if constexpr (HALF) {
        const int half = rot / 2, lane = threadIdx.x & 63;
        const bool low = d0 < half, in = d0 < rot;
        const int from = in ? (low ? lane + half / VE : lane - half / VE) : lane;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float other = __shfl(x.v[e], from);
            if (in) {
                const float2 t = cs[low ? d0 + e : d0 + e - half];
                y.v[e] = x.v[e] * t.x + (low ? -sign : sign) * (other * t.y);
            }
        }
    } else if (d0 < rot) {
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
            const float2 t = cs[(d0 + e) / 2];
            y.v[e] = x.v[e] * t.x - sign * (x.v[e + 1] * t.y);
            y.v[e + 1] = x.v[e + 1] * t.x + sign * (x.v[e] * t.y);
        }
    }
    return y;
}

template <int VE, bool HALF>
__global__ void __launch_bounds__(kNThreads) gscan_norm_fwd_kernel(NormArgs a, int lpr, int tpb)
{
    __shared__ float2 cs[kNMaxTok][kNMaxPairs];
    const int tid = threadIdx.x, sub = tid & (lpr - 1), d0 = sub * VE;
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
    const int n = (int)(a.tokens - t0 < tpb ? a.tokens - t0 : tpb);
    const int heads = a.heads[0] + a.heads[1], rows = n * heads, rpp = kNThreads / lpr;
    const bool in = d0 < a.D;
    angles(a, cs, t0, n, tid);
    __syncthreads();
    for (int b = 0; b < rows; b += rpp) {  // every lane takes part in the exchanges
        const int row = b + tid / lpr;
        const bool ok = row < rows && in;
        const int t = row < rows ? row / heads : 0, hh = row < rows ? row % heads : 0;
        const int which = hh >= a.heads[0], h = hh - which * a.heads[0];
        Vec<VE> x = {}, wv;
        if (ok) x = load_vec<VE>(a.x[which], (t0 + t) * a.xn[which] + h * a.xh[which] + d0, a.dtype);
#pragma unroll
        for (int e = 0; e < VE; ++e) wv.v[e] = 1.f;
        if (ok && a.w[which]) wv = load_vec<VE>(a.w[which], d0, 0);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) s += x.v[e] * x.v[e];
        const float r = 1.f / sqrtf(group_sum(s, lpr) / (float)a.D + a.eps);
#pragma unroll
        for (int e = 0; e < VE; ++e) x.v[e] *= r * wv.v[e];
        const Vec<VE> y = turn<VE, HALF>(x, cs[t], d0, a.rot, 1.f);
        if (ok) store_vec<VE>(a.y[which], ((t0 + t) * a.heads[which] + h) * a.D + d0, a.dtype, y);
    }
}

template <int VE, bool HALF>
__global__ void __launch_bounds__(kNThreads) gscan_norm_bwd_kernel(NormArgs a, int lpr, int tpb)
{
    __shared__ float2 cs[kNMaxTok][kNMaxPairs];
    __shared__ float red[2][kNThreads * VE];
    const int tid = threadIdx.x, sub = tid & (lpr - 1), d0 = sub * VE;
    const int heads = a.heads[0] + a.heads[1], rpp = kNThreads / lpr;
    const bool in = d0 < a.D;
    Vec<VE> dw[2] = {};
    for (int64_t t0 = (int64_t)blockIdx.x * tpb; t0 < a.tokens; t0 += (int64_t)gridDim.x * tpb) {
        const int n = (int)(a.tokens - t0 < tpb ? a.tokens - t0 : tpb), rows = n * heads;
        __syncthreads();
        angles(a, cs, t0, n, tid);
        __syncthreads();
        for (int b = 0; b < rows; b += rpp) {
            const int row = b + tid / lpr;
            const bool ok = row < rows && in;
            const int t = row < rows ? row / heads : 0, hh = row < rows ? row % heads : 0;
            const int which = hh >= a.heads[0], h = hh - which * a.heads[0];
            Vec<VE> x = {}, g = {}, wv;
            if (ok) {
                x = load_vec<VE>(a.x[which], (t0 + t) * a.xn[which] + h * a.xh[which] + d0, a.dtype);
                g = load_vec<VE>(a.dy[which], (t0 + t) * a.dn[which] + h * a.dh[which] + d0, a.dtype);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) wv.v[e] = 1.f;
            if (ok && a.w[which]) wv = load_vec<VE>(a.w[which], d0, 0);
            g = turn<VE, HALF>(g, cs[t], d0, a.rot, -1.f);
            float s = 0.f, m = 0.f;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                s += x.v[e] * x.v[e];
                m += g.v[e] * wv.v[e] * x.v[e];
            }
            const float r = 1.f / sqrtf(group_sum(s, lpr) / (float)a.D + a.eps);
            const float f = group_sum(m, lpr) / (float)a.D * r * r;
            if (ok) {
                Vec<VE> dx;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float p = g.v[e] * (x.v[e] * r);
                    dw[0].v[e] += which ? 0.f : p;
                    dw[1].v[e] += which ? p : 0.f;
                    dx.v[e] = r * (g.v[e] * wv.v[e] - x.v[e] * f);
                }
                store_vec<VE>(a.y[which], ((t0 + t) * a.heads[which] + h) * a.D + d0, a.dtype, dx);
            }
        }
    }
    if (!a.ws) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) red[i][tid * VE + e] = dw[i].v[e];
    __syncthreads();
    float *part = reinterpret_cast<float *>(a.ws) + (int64_t)blockIdx.x * 2 * a.D;
    for (int i = tid; i < 2 * a.D; i += kNThreads) {
        const int wh = i / a.D, d = i % a.D;
        float s = 0.f;
        for (int r = 0; r < rpp; ++r) s += red[wh][r * lpr * VE + d];
        part[i] = s;
    }
}

// dw[i][d] = sum over the partials, 64 lanes per element, in a fixed order
__global__ void __launch_bounds__(64) gscan_norm_dw_kernel(const float *part, int grid, int D, float *dwq,
                                                           float *dwk)
{
    const int i = blockIdx.x, lane = threadIdx.x;
    double s = 0.0;
    for (int b = lane; b < grid; b += 64) s += (double)part[(int64_t)b * 2 * D + i];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    float *o = i < D ? dwq : dwk;
    if (lane == 0 && o) o[i % D] = (float)s;
}

struct NormGeom {
    int ve, lpr, tpb;
    int64_t blocks;
};

// Eight elements per lane, or four where a pair's halves are not eight apart
// (half layout).  Tokens per workgroup: about four rows per lane group.
NormGeom geom(int64_t tokens, int heads, int D, int rot, int layout)
{
    NormGeom g;
    g.ve = layout == 0 && (rot / 2) % 8 != 0 ? 4 : 8;
    g.lpr = 1;
    while (g.lpr * g.ve < D) g.lpr *= 2;
    const int rpp = kNThreads / g.lpr;
    int t = 4 * rpp / heads;
    g.tpb = t < 1 ? 1 : t > kNMaxTok ? kNMaxTok : t;
    g.blocks = (tokens + g.tpb - 1) / g.tpb;
    return g;
}

int64_t bwd_grid(int64_t blocks) { return blocks < kNMaxGrid ? blocks : kNMaxGrid; }

}  // namespace

// Enough for either layout: the grid is at most kNMaxGrid and the tokens.
size_t norm_workspace_bytes(int64_t tokens, int D)
{
    return (size_t)(tokens > 0 ? bwd_grid(tokens) : 1) * 2u * (size_t)D * sizeof(float);
}

hipError_t launch_norm_forward(const NormArgs &a, hipStream_t st)
{
    const NormGeom g = geom(a.tokens, a.heads[0] + a.heads[1], a.D, a.rot, a.layout);
    const dim3 grid((unsigned)g.blocks), blk(kNThreads);
    if (!g.blocks) return hipSuccess;
    if (a.layout) hipLaunchKernelGGL((gscan_norm_fwd_kernel<8, false>), grid, blk, 0, st, a, g.lpr, g.tpb);
    else if (g.ve == 8) hipLaunchKernelGGL((gscan_norm_fwd_kernel<8, true>), grid, blk, 0, st, a, g.lpr, g.tpb);
    else hipLaunchKernelGGL((gscan_norm_fwd_kernel<4, true>), grid, blk, 0, st, a, g.lpr, g.tpb);
    return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs &a, hipStream_t st)
{
    const NormGeom g = geom(a.tokens, a.heads[0] + a.heads[1], a.D, a.rot, a.layout);
    const int64_t n = bwd_grid(g.blocks);
    const dim3 grid((unsigned)n), blk(kNThreads);
    if (!n) {}  // no tokens: dw is zero
    else if (a.layout) hipLaunchKernelGGL((gscan_norm_bwd_kernel<8, false>), grid, blk, 0, st, a, g.lpr, g.tpb);
    else if (g.ve == 8) hipLaunchKernelGGL((gscan_norm_bwd_kernel<8, true>), grid, blk, 0, st, a, g.lpr, g.tpb);
    else hipLaunchKernelGGL((gscan_norm_bwd_kernel<4, true>), grid, blk, 0, st, a, g.lpr, g.tpb);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.ws) return e;  // no weight gradient wanted
    hipLaunchKernelGGL(gscan_norm_dw_kernel, dim3((unsigned)(2 * a.D)), dim3(64), 0, st,
                       reinterpret_cast<const float *>(a.ws), (int)n, a.D, a.dw[0], a.dw[1]);
    return hipGetLastError();
}

}  // namespace gscan
