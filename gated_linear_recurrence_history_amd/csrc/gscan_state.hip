// Matrix-state gated scan, forward and backward, for gfx950 (MI355X).
//
// Per sequence and head, with a state S [Dk][Dv]:
//   g_t = sigmoid(a_t + shift) (or exp(a_t)),  S_t = g_t S_{t-1} + k_t v_t^T,
//   o_t = scale S_t^T q_t
// and its gradients, with dS_t the whole gradient of S_t:
//   dS_{t-1} = g_t dS_t + scale q_{t-1} do_{t-1}^T,
//   dq_t = scale S_t do_t,  dk_t = dS_t v_t,  dv_t = dS_t^T k_t,
//   dlog g_t = g_t <S_{t-1}, dS_t>.
//
// Chunks of C tokens turn the recurrence into matrix products.  With L the
// running sum of log g inside the chunk and S the state before it,
//   O  = scale [ ((Q K^T) . D) V + e^L Q S ],     D_ts = e^(L_t - L_s), t >= s
//   S' = e^(L_C) S + sum_s e^(L_C - L_s) k_s v_s^T
//   dQ = (dP . D) K + scale e^L dO S^T            dP = scale dO V^T
//   dK = (dP . D)^T Q + e^(L_C - L) V dS^T        (dS: after the chunk)
//   dV = (P . D)^T dO + e^(L_C - L) K dS          P = scale Q K^T
// and with W = P . D . (dO V^T), A_u = scale e^(L_u) q_u^T S do_u,
// B_s = e^(L_C - L_s) k_s^T dS v_s, F = e^(L_C) <S, dS>:
//   dlog g_t = sum_{u>=t, s<t} W_us + sum_{u>=t} A_u + sum_{s<t} B_s + F,
// every term of which carries the gate g_t itself, so that a closed gate
// gives zero and not a difference of large sums (the shorter form, running
// sums of q . dq - k . dk, cancels); nothing is summed over more than a chunk.
//
// Operands.  A chunk's tensors are staged in LDS row-major.  Every product is
// MFMA 16x16 with 32 contracted elements a step: lane l holds row (or column)
// l % 16 and, with g = l / 16, the elements 4g .. 4g+3 and 16+4g .. 16+4g+3.
// That order is what two 16-row accumulators hold of a column, so a state
// kept in accumulators is an operand without moving; it is two 8-byte LDS
// reads along a row, or two transposed reads (ds_read_b64_tr_b16) down a
// column.  bf16: one v_mfma_f32_16x16x32_bf16.  fp32: eight
// v_mfma_f32_16x16x4_f32 over the same elements (exact fp32 products).
//
// Roundings (bf16): P . D, dP . D and the states are rounded to bf16 where
// they enter a product as operands, once, with fp32 accumulation; the state
// itself stays fp32 in registers, and what is added to it, decay * v, is
// split in three bf16 parts (24 bits), so a state carried over a long
// sequence has fp32 accuracy.
#include <cstdint>
#include <cstdlib>
#include <type_traits>

#include "gscan_state_dev.h"

namespace gscan {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));

constexpr int kSThreads = 256;
constexpr int kSlice = 64;  // columns of a state that one workgroup walks

__device__ __forceinline__ f4 zf4() { return f4{0.f, 0.f, 0.f, 0.f}; }
__device__ __forceinline__ u4 zu4() { return u4{0u, 0u, 0u, 0u}; }

// ------------------------------------------------------- operand types

struct BF {
    typedef uint16_t S;   // storage
    typedef u4 Frag;      // eight bf16
    static constexpr int kDtype = 1, C = 64, VE = 8, kPad = 8;
};
struct FP {
    typedef float S;
    struct Frag {
        f4 a, b;
    };
    static constexpr int kDtype = 0, C = 32, VE = 4, kPad = 4;
};

__device__ __forceinline__ f4 mma(const u4 &a, const u4 &b, f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                    __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ f4 mma(const FP::Frag &a, const FP::Frag &b, f4 c)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[j], b.a[j], c, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[j], b.b[j], c, 0, 0, 0);
    return c;
}

// Row r0 + l%16 of a row-major tile, elements k0 + {4g.., 16+4g..}.
__device__ __forceinline__ u4 ld_row(const uint16_t *t, int pitch, int r0, int k0, int lane)
{
    const uint16_t *p = t + (r0 + (lane & 15)) * pitch + k0 + 4 * (lane >> 4);
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    const uint2 y = *reinterpret_cast<const uint2 *>(p + 16);
    return u4{x.x, x.y, y.x, y.y};
}
__device__ __forceinline__ FP::Frag ld_row(const float *t, int pitch, int r0, int k0, int lane)
{
    const float *p = t + (r0 + (lane & 15)) * pitch + k0 + 4 * (lane >> 4);
    return FP::Frag{*reinterpret_cast<const f4 *>(p), *reinterpret_cast<const f4 *>(p + 16)};
}

// Column c0 + l%16, elements of rows k0 + {4g.., 16+4g..}.  The transposed
// read gives lane i of a 16-lane group element i%4 of the 8-byte pieces that
// lanes 4j + i/4 address, j = 0..3: with lane p addressing row 4g + p/4,
// columns 4(p%4).., it receives column p of rows 4g .. 4g+3.
__device__ __forceinline__ uint2 read_tr(const uint16_t *p)
{
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s4v *)(p)));
}
__device__ __forceinline__ u4 ld_col(const uint16_t *t, int pitch, int k0, int c0, int lane)
{
    const int p = lane & 15;
    const uint16_t *a = t + (k0 + 4 * (lane >> 4) + (p >> 2)) * pitch + c0 + 4 * (p & 3);
    const uint2 x = read_tr(a), y = read_tr(a + 16 * pitch);
    return u4{x.x, x.y, y.x, y.y};
}
__device__ __forceinline__ FP::Frag ld_col(const float *t, int pitch, int k0, int c0, int lane)
{
    const float *a = t + (k0 + 4 * (lane >> 4)) * pitch + c0 + (lane & 15);
    FP::Frag f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f.a[j] = a[j * pitch];
        f.b[j] = a[(16 + j) * pitch];
    }
    return f;
}

// Two accumulators (rows 0..15 and 16..31 of a column) as an operand.
__device__ __forceinline__ void to_frag(f4 x, f4 y, u4 *f)
{
    *f = u4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(y[0], y[1]),
            pack_bf16(y[2], y[3])};
}
__device__ __forceinline__ void to_frag(f4 x, f4 y, FP::Frag *f) { *f = FP::Frag{x, y}; }

__device__ __forceinline__ void from_frag(const u4 &f, f4 *x, f4 *y)
{
    *x = f4{bf_lo(f[0]), bf_hi(f[0]), bf_lo(f[1]), bf_hi(f[1])};
    *y = f4{bf_lo(f[2]), bf_hi(f[2]), bf_lo(f[3]), bf_hi(f[3])};
}
__device__ __forceinline__ void from_frag(const FP::Frag &f, f4 *x, f4 *y)
{
    *x = f.a;
    *y = f.b;
}

// acc + A (x | y) with every bit of the fp32 values x, y: three bf16 parts,
// each the rounding of what the parts before it leave (the differences are
// exact in fp32).
struct Parts {
    u4 p[3];
};
__device__ __forceinline__ void to_parts(f4 x, f4 y, Parts *s)
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        to_frag(x, y, &s->p[i]);
        f4 hx, hy;
        from_frag(s->p[i], &hx, &hy);
        x -= hx;
        y -= hy;
    }
}
__device__ __forceinline__ void to_parts(f4 x, f4 y, FP::Frag *s) { *s = FP::Frag{x, y}; }
__device__ __forceinline__ f4 mma_parts(const u4 &a, const Parts &b, f4 c)
{
    return mma(a, b.p[0], mma(a, b.p[1], mma(a, b.p[2], c)));
}
__device__ __forceinline__ f4 mma_parts(const FP::Frag &a, const FP::Frag &b, f4 c)
{
    return mma(a, b, c);
}
template <class T>
struct PartsOf {
    typedef Parts type;
};
template <>
struct PartsOf<FP> {
    typedef FP::Frag type;
};

__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ void narrow(float x, uint16_t *p) { *p = to_bf16(x); }
__device__ __forceinline__ void narrow(float x, float *p) { *p = x; }

// Operands kept in device memory: 16 bytes (bf16) or two planes of 16 bytes
// (fp32) per lane.
__device__ __forceinline__ void put_frag(void *base, int64_t i, int lane, const u4 &f)
{
    reinterpret_cast<u4 *>(base)[i * 64 + lane] = f;
}
__device__ __forceinline__ void put_frag(void *base, int64_t i, int lane, const FP::Frag &f)
{
    reinterpret_cast<f4 *>(base)[i * 128 + lane] = f.a;
    reinterpret_cast<f4 *>(base)[i * 128 + 64 + lane] = f.b;
}
__device__ __forceinline__ void get_frag(const void *base, int64_t i, int lane, u4 *f)
{
    *f = reinterpret_cast<const u4 *>(base)[i * 64 + lane];
}
__device__ __forceinline__ void get_frag(const void *base, int64_t i, int lane, FP::Frag *f)
{
    f->a = reinterpret_cast<const f4 *>(base)[i * 128 + lane];
    f->b = reinterpret_cast<const f4 *>(base)[i * 128 + 64 + lane];
}

// An infinity or NaN in sixteen bytes.
__device__ __forceinline__ bool nonfinite(const u4 &x, const BF &)
{
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (x[i] & 0x7f80u) == 0x7f80u || (x[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
}
__device__ __forceinline__ bool nonfinite(const u4 &x, const FP &)
{
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (x[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
}

// A masked product (entries of m where k > r, or k < r, are zero) must not
// carry an infinity or NaN of b's row k to the rows r that the mask keeps
// from it, as 0 * b would.  Chunks that hold one take the product of b's
// finite elements (the others as zeros, which leaves the other rows' bits
// as they are) and then add the terms left out one by one.
__device__ __forceinline__ u4 finite_part(u4 f)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((f[i] & 0x7f80u) == 0x7f80u) f[i] &= 0xffff0000u;
        if ((f[i] & 0x7f800000u) == 0x7f800000u) f[i] &= 0xffffu;
    }
    return f;
}
__device__ __forceinline__ FP::Frag finite_part(FP::Frag f)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!isfinite(f.a[i])) f.a[i] = 0.f;
        if (!isfinite(f.b[i])) f.b[i] = 0.f;
    }
    return f;
}

// The terms left out, for rows r0 .. r0+3 and column col: sum over the k of
// non-finite b[k][col] with k <= r (LOWER) or k >= r of m[r][k] (TRANS:
// m[k][r]) times it.
template <bool LOWER, bool TRANS, class S>
__device__ f4 other_terms(const S *m, int pm, const S *b, int pb, int r0, int col, int C)
{
    f4 x = zf4();
    for (int k = 0; k < C; ++k) {
        const float v = widen(b[k * pb + col]);
        if (isfinite(v)) continue;
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + j;
            if (LOWER ? k <= r : k >= r) x[j] += widen(TRANS ? m[k * pm + r] : m[r * pm + k]) * v;
        }
    }
    return x;
}

// ------------------------------------------------------ sequences and units

// Sequences are cut into units of `per` tokens (a sequence without tokens is
// one unit, which passes its state on).  Unit u of the call belongs to
// sequence `seq`, is its `part`-th, and the chunk slots of the sequence start
// at `slot0`.
struct Unit {
    int64_t tok0;  // first token of the sequence in [tokens][H][..] outputs
    int64_t in0;   // the same where inputs have a batch stride: packed first token, else 0
    int seq, part, parts, len, slot0;
};

// Whether unit u exists.  Offsets are clamped to the tokens there are, so
// wrong ones read and write nothing out of range.  Called by whole wavefronts.
__device__ __forceinline__ bool find_unit(const StateArgs &a, int64_t u, int64_t per, int C,
                                          int lane, Unit *w)
{
    if (!a.off) {
        const int64_t n = a.T > per ? (a.T + per - 1) / per : 1;
        const int64_t nc = a.T > C ? (a.T + C - 1) / C : 1;
        const int64_t seq = u / n;
        if (seq >= a.B) return false;
        w->seq = (int)seq;
        w->part = (int)(u - seq * n);
        w->parts = (int)n;
        w->len = (int)a.T;
        w->slot0 = (int)(seq * nc);
        w->tok0 = seq * a.T;
        w->in0 = 0;
        return true;
    }
    int64_t ub = 0, cb = 0;
    for (int64_t i0 = 0; i0 < a.B; i0 += 64) {
        const int64_t i = i0 + lane;
        int64_t s = 0, e = 0;
        int nu = 0, nc = 0;
        if (i < a.B) {
            s = a.off[i];
            e = a.off[i + 1];
            s = s < 0 ? 0 : s > a.T ? a.T : s;
            e = e < s ? s : e > a.T ? a.T : e;
            nu = e - s > per ? (int)((e - s + per - 1) / per) : 1;
            nc = e - s > C ? (int)((e - s + C - 1) / C) : 1;
        }
        int su = nu, sc = nc;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int x = __shfl_up(su, d), y = __shfl_up(sc, d);
            if (lane >= d) {
                su += x;
                sc += y;
            }
        }
        const uint64_t hit = __ballot(u < ub + su);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            const int64_t seq = i0 + l;
            if (seq >= a.B) return false;
            w->seq = (int)seq;
            w->parts = __shfl(nu, l);
            w->part = (int)(u - (ub + __shfl(su, l) - w->parts));
            w->slot0 = (int)(cb + __shfl(sc, l) - __shfl(nc, l));
            // offsets that overlap could ask for more chunks than there are
            if (w->slot0 + __shfl(nc, l) > a.chunks) return false;
            const int start = __shfl((int)s, l);
            w->len = __shfl((int)(e - s), l);
            w->tok0 = w->in0 = start;
            return true;
        }
        ub += __shfl(su, 63);
        cb += __shfl(sc, 63);
    }
    return false;
}

// First element of a sequence's rows of head h.
template <class S>
__device__ __forceinline__ const S *rows_of(const void *p, const Strides &s, const Unit &w,
                                            bool packed, int h)
{
    return reinterpret_cast<const S *>(p) + (packed ? w.in0 * s.t : (int64_t)w.seq * s.b) +
           (int64_t)h * s.h;
}

// ---------------------------------------------------------- staged tiles

// C rows of NKU 32-wide units, 16 bytes at a time: NKU pieces per thread.
template <class T, int NKU>
struct Stage {
    u4 r[NKU];
    static constexpr int kPpr = NKU * 32 / T::VE;  // pieces per row

    // rows t0 .. of `base` (stride st), those before `len` and columns before
    // `cols`; zero elsewhere
    __device__ __forceinline__ void load(const typename T::S *base, int64_t st, int t0, int len,
                                         int cols, int tid)
    {
#pragma unroll
        for (int i = 0; i < NKU; ++i) {
            const int p = tid + kSThreads * i, row = p / kPpr, col = p % kPpr * T::VE;
            r[i] = t0 + row < len && col < cols
                       ? *reinterpret_cast<const u4 *>(base + (int64_t)(t0 + row) * st + col)
                       : zu4();
        }
    }
    __device__ __forceinline__ void store(typename T::S *tile, int pitch, int tid) const
    {
#pragma unroll
        for (int i = 0; i < NKU; ++i) {
            const int p = tid + kSThreads * i;
            *reinterpret_cast<u4 *>(tile + p / kPpr * pitch + p % kPpr * T::VE) = r[i];
        }
    }
    __device__ __forceinline__ bool bad() const
    {
        bool b = false;
#pragma unroll
        for (int i = 0; i < NKU; ++i) b |= nonfinite(r[i], T());
        return b;
    }
};

// Decays of one chunk, in LDS: L in units of log 2 (as a sum of two floats,
// so that differences of far-down values keep fp32 accuracy), e^L,
// e^(L_end - L), e^(L_end).
template <int C>
struct __align__(16) Decay {
    float hi[C], lo[C], e[C], d[C], g;
};

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// x: the gate argument of token `lane` (ok: there is one).  One wavefront.
template <int C>
__device__ __forceinline__ void gate_scan(Decay<C> &s, float x, bool ok, int form, int lane)
{
    double L = ok ? (double)log_gate(x, form) * 1.44269504088896340736 : 0.0;
#pragma unroll
    for (int d = 1; d < C; d *= 2) {
        const double y = __shfl_up(L, d);
        if (lane >= d) L += y;
    }
    const double end = __shfl(L, C - 1);
    if (lane < C) {
        const float h = (float)L;
        s.hi[lane] = h;
        s.lo[lane] = (float)(L - (double)h);
        s.e[lane] = exp2_(h);
        s.d[lane] = exp2_((float)(end - L));
        if (lane == C - 1) s.g = exp2_((float)end);
    }
}

// e^(L_t - L_s)
template <int C>
__device__ __forceinline__ float decay(const Decay<C> &s, int t, int u)
{
    return exp2_((s.hi[t] - s.hi[u]) + (s.lo[t] - s.lo[u]));
}

// --------------------------------------------------------------- forward

// One workgroup walks a unit's chunks for one head and 64 columns of its
// state: wavefront w keeps columns 16w .. 16w+15 of every row in
// accumulators, which are operands of Q S as they are; Q K^T is split over
// the wavefronts by rows and passes through LDS.  The next chunk's rows are
// requested while this one is computed, its decays are formed by the
// wavefront that has least of Q K^T to do, and the outputs leave through LDS
// in 16-byte pieces while the next chunk is staged.
template <class T, int NK>
__global__ void __launch_bounds__(kSThreads)
gscan_state_fwd_kernel(StateArgs a, int slices, int64_t per, size_t st_part)
{
    typedef typename T::S S;
    typedef typename T::Frag Frag;
    constexpr int C = T::C, RT = C / 16, CS = 4 / RT, KS = C / 32;
    constexpr int PK = NK * 32 + T::kPad, PV = kSlice + T::kPad, PP = C + T::kPad;
    constexpr int GW = CS == 1 ? 0 : RT;  // the wavefront of the decays
    __shared__ __align__(16) S qt[C * PK], kt[C * PK], vt[C * PV], pt[C * PP], ot[C * PV];
    __shared__ Decay<C> dcs[2];
    __shared__ int bad[2];

    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int l16 = lane & 15, g4 = 4 * (lane >> 4);
    const int slice = blockIdx.x % slices;
    const int h = blockIdx.x / slices % a.H;
    const int64_t unit = blockIdx.x / slices / a.H;
    Unit un;
    if (!find_unit(a, unit, per, C, lane, &un)) return;
    const bool packed = a.off != nullptr;
    const int hk = h / (a.H / a.Hk), c0 = slice * kSlice, vcols = a.Dv - c0;
    const S *qp = rows_of<S>(a.q, a.qs, un, packed, hk), *kp = rows_of<S>(a.k, a.ks, un, packed, hk);
    const S *vp = rows_of<S>(a.v, a.vs, un, packed, h) + c0;
    const int64_t g0 = (packed ? un.in0 * a.gs.t : (int64_t)un.seq * a.gs.b) + (int64_t)h * a.gs.h;
    S *op = reinterpret_cast<S *>(a.out) + (un.tok0 * a.H + h) * a.Dv + c0;
    const int64_t ost = (int64_t)a.H * a.Dv;
    const int col = w * 16 + l16;  // this lane's column of the slice
    const int tb = (int)(un.part * per);
    const int te = un.len - tb > per ? (int)(tb + per) : un.len;

    // the state: row 16i + 4g + j of column `col`
    const int64_t srow = ((int64_t)un.seq * a.H + h) * a.Dk;
    const float *init = a.s0 ? a.s0 + srow * a.Dv : nullptr;
    if (un.part)
        init = reinterpret_cast<const float *>(reinterpret_cast<const char *>(a.ws) + st_part) +
               (unit * a.H + h) * a.Dk * a.Dv;
    f4 st[2 * NK];
#pragma unroll
    for (int i = 0; i < 2 * NK; ++i) {
        st[i] = zf4();
        if (init && col < vcols)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (16 * i + g4 + j < a.Dk) st[i][j] = init[(16 * i + g4 + j) * a.Dv + c0 + col];
    }

    Stage<T, NK> sq, sk;
    Stage<T, 2> sv;
    float gx = 0.f;
    auto request = [&](int t0) {
        sq.load(qp, a.qs.t, t0, te, a.Dk, tid);
        sk.load(kp, a.ks.t, t0, te, a.Dk, tid);
        sv.load(vp, a.vs.t, t0, te, vcols, tid);
    };
    auto request_gate = [&](int t0) {
        if (w == GW && lane < C && t0 + lane < te)
            gx = load_scalar(a.gate, g0 + (int64_t)(t0 + lane) * a.gs.t, a.gate_dtype) + a.gate_shift;
    };
    // outputs of the chunk at t0, from LDS
    auto flush = [&](int t0) {
        constexpr int ppr = kSlice / T::VE;
#pragma unroll
        for (int i = 0; i < C * ppr / kSThreads; ++i) {
            const int p = tid + kSThreads * i, row = p / ppr, cc = p % ppr * T::VE;
            if (t0 + row < te && cc < vcols)
                *reinterpret_cast<u4 *>(op + (t0 + row) * ost + cc) =
                    *reinterpret_cast<const u4 *>(ot + row * PV + cc);
        }
    };
    if (tid < 2) bad[tid] = 0;
    request_gate(tb);
    request(tb);
    if (w == GW) gate_scan<C>(dcs[0], gx, tb + lane < te, a.gate_form, lane);
    request_gate(tb + C);
    __syncthreads();

    int odd = 0;
    for (int t0 = tb; t0 < te; t0 += C, odd ^= 1) {
        const Decay<C> &dc = dcs[odd];
        sq.store(qt, PK, tid);
        sk.store(kt, PK, tid);
        sv.store(vt, PV, tid);
        if (sv.bad()) bad[odd] = 1;
        if (t0 > tb) flush(t0 - C);
        __syncthreads();
        if (tid == 0) bad[odd ^ 1] = 0;
        if (t0 + C < te) request(t0 + C);

        // P . D, rows 16rt .. of wavefront (rt, ct % CS)
        {
            const int rt = w % RT;
#pragma unroll
            for (int ct = w / RT; ct < RT; ct += CS) {
                f4 x = zf4();
                if (ct <= rt) {
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk)
                        x = mma(ld_row(qt, PK, 16 * rt, 32 * kk, lane),
                                ld_row(kt, PK, 16 * ct, 32 * kk, lane), x);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = 16 * rt + g4 + j, s = 16 * ct + l16;
                    narrow(t >= s ? x[j] * decay(dc, t, s) : 0.f, &pt[t * PP + s]);
                }
            }
            if (w == GW && t0 + C < te) {
                gate_scan<C>(dcs[odd ^ 1], gx, t0 + C + lane < te, a.gate_form, lane);
                request_gate(t0 + 2 * C);
            }
        }
        __syncthreads();

        const bool slow = bad[odd] != 0;
        Frag vf[KS], pf[KS];
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) vf[kk] = pf[kk] = ld_col(vt, PV, 32 * kk, 16 * w, lane);
        if (slow)
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) pf[kk] = finite_part(pf[kk]);
        {
            f4 o[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) o[r] = zf4();
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) {
                Frag sf;
                to_frag(st[2 * kk], st[2 * kk + 1], &sf);
#pragma unroll
                for (int r = 0; r < RT; ++r) o[r] = mma(ld_row(qt, PK, 16 * r, 32 * kk, lane), sf, o[r]);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
#pragma unroll
                for (int j = 0; j < 4; ++j) o[r][j] *= dc.e[16 * r + g4 + j];
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
                    if (2 * kk <= r) o[r] = mma(ld_row(pt, PP, 16 * r, 32 * kk, lane), pf[kk], o[r]);
            }
            if (slow)
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    o[r] += other_terms<true, false>(pt, PP, vt, PV, 16 * r + g4, col, C);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) narrow(a.scale * o[r][j], &ot[(16 * r + g4 + j) * PV + col]);
        }
        // S' = e^(L_end) S + K^T (e^(L_end - L) V)
        typename PartsOf<T>::type vs[KS];
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            f4 x, y;
            from_frag(vf[kk], &x, &y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] *= dc.d[32 * kk + g4 + j];
                y[j] *= dc.d[32 * kk + 16 + g4 + j];
            }
            to_parts(x, y, &vs[kk]);
        }
        const float ge = dc.g;
#pragma unroll
        for (int i = 0; i < 2 * NK; ++i) {
            st[i] *= ge;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
                st[i] = mma_parts(ld_col(kt, PK, 32 * kk, 16 * i, lane), vs[kk], st[i]);
        }
        __syncthreads();
    }
    if (te > tb) flush(tb + (te - tb - 1) / C * C);

    if (a.sT && te == un.len && col < vcols) {
#pragma unroll
        for (int i = 0; i < 2 * NK; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (16 * i + g4 + j < a.Dk)
                    a.sT[(srow + 16 * i + g4 + j) * a.Dv + c0 + col] = st[i][j];
    }
}

// ------------------------------------------------- backward: chunk states

// A walk over a unit's chunks that keeps the state (REV false) or the gradient
// of the state (REV true) of one head: X rows, 64 columns of Y, acc += X^T
// (decay . Y).  STORE: before every chunk (after it, REV) the accumulators are
// left as operands: column tile n and 32-row unit kk of chunk slot c and head
// h are operand ((c H + h) 2NY + n) NX + kk of `dst`.
struct PassJob {
    const void *x, *y;
    Strides xs, ys;
    int xh, yh;          // heads of x, y
    int xd, yd;          // widths
    const float *init;   // the state to begin with, or null
    float *fin;          // for the state at the end, or null
    float *dec;          // for the product of the unit's gates, or null
    int rstr, cstr;      // strides of a row and a column in init and fin
    void *dst;
    float mul;           // factor of what is added
};

template <class T, int NX, bool REV, bool STORE>
__device__ __forceinline__ void pass_walk(const StateArgs &a, const PassJob &jb, int ny, int slice,
                                          int h, const Unit &un, int tb, int te, char *smem,
                                          Decay<T::C> (&dcs)[2])
{
    typedef typename T::S S;
    typedef typename T::Frag Frag;
    constexpr int C = T::C, KS = C / 32, PX = NX * 32 + T::kPad, PY = kSlice + T::kPad;
    S *xt = reinterpret_cast<S *>(smem), *yt = xt + C * PX;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int l16 = lane & 15, g4 = 4 * (lane >> 4);
    const bool packed = a.off != nullptr;
    const int c0 = slice * kSlice, ycols = jb.yd - c0, col = 16 * w + l16;
    const S *xp = rows_of<S>(jb.x, jb.xs, un, packed, jb.xh);
    const S *yp = rows_of<S>(jb.y, jb.ys, un, packed, jb.yh) + c0;
    const int64_t g0 = (packed ? un.in0 * a.gs.t : (int64_t)un.seq * a.gs.b) + (int64_t)h * a.gs.h;
    const int sb = (c0 + col) * jb.cstr;
    f4 st[2 * NX];
#pragma unroll
    for (int i = 0; i < 2 * NX; ++i) {
        st[i] = zf4();
        if (jb.init && col < ycols)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (16 * i + g4 + j < jb.xd) st[i][j] = jb.init[sb + (16 * i + g4 + j) * jb.rstr];
    }
    const int cb = tb / C, ce = te > tb ? (te + C - 1) / C : cb + 1;  // chunks
    Stage<T, NX> sx;
    Stage<T, 2> sy;
    float gx = 0.f, gall = 1.f;
    auto request = [&](int c) {
        sx.load(xp, jb.xs.t, c * C, te, jb.xd, tid);
        sy.load(yp, jb.ys.t, c * C, te, ycols, tid);
    };
    auto request_gate = [&](int c) {
        if (w == 0 && lane < C && c >= cb && c * C + lane < te)
            gx = load_scalar(a.gate, g0 + (int64_t)(c * C + lane) * a.gs.t, a.gate_dtype) + a.gate_shift;
    };
    constexpr int step = REV ? -1 : 1;
    int c = REV ? ce - 1 : cb;
    request_gate(c);
    request(c);
    if (w == 0) gate_scan<C>(dcs[0], gx, c * C + lane < te, a.gate_form, lane);
    request_gate(c + step);
    int odd = 0;
    for (int n = ce - cb; n > 0; --n, c += step, odd ^= 1) {
        const Decay<C> &dc = dcs[odd];
        sx.store(xt, PX, tid);
        sy.store(yt, PY, tid);
        if constexpr (STORE) {  // the operands of this chunk, before its own tokens enter
#pragma unroll
            for (int kk = 0; kk < NX; ++kk) {
                Frag f;
                to_frag(st[2 * kk], st[2 * kk + 1], &f);
                put_frag(jb.dst, (((int64_t)(un.slot0 + c) * a.H + h) * 2 * ny + slice * 4 + w) * NX + kk,
                         lane, f);
            }
        }
        __syncthreads();
        if (n > 1) {
            request(c + step);
            if (w == 0) {
                gate_scan<C>(dcs[odd ^ 1], gx, (c + step) * C + lane < te, a.gate_form, lane);
                request_gate(c + 2 * step);
            }
        }
        typename PartsOf<T>::type ys[KS];
        const float *m = REV ? dc.e : dc.d;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            f4 x, y;
            from_frag(ld_col(yt, PY, 32 * kk, 16 * w, lane), &x, &y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] *= jb.mul * m[32 * kk + g4 + j];
                y[j] *= jb.mul * m[32 * kk + 16 + g4 + j];
            }
            to_parts(x, y, &ys[kk]);
        }
        const float ge = dc.g;
        gall *= ge;
#pragma unroll
        for (int i = 0; i < 2 * NX; ++i) {
            st[i] *= ge;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
                st[i] = mma_parts(ld_col(xt, PX, 32 * kk, 16 * i, lane), ys[kk], st[i]);
        }
        __syncthreads();
    }
    if (jb.fin && col < ycols) {
#pragma unroll
        for (int i = 0; i < 2 * NX; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (16 * i + g4 + j < jb.xd) jb.fin[sb + (16 * i + g4 + j) * jb.rstr] = st[i][j];
    }
    if (jb.dec && slice == 0 && tid == 0) *jb.dec = gall;
}

template <class T, int NM>
struct PassLds {
    static constexpr size_t bytes = T::C * (NM * 32 + kSlice + 2 * T::kPad) * sizeof(typename T::S);
};

// Units of split sequences, by themselves: what a unit adds to the state after
// it (REV: to the gradient of the state before it) and the product of its
// gates.  fp32 [units][H][Dk][Dv] and [units][H] at st_part, st_dec.
template <class T, int NK, bool REV>
__global__ void __launch_bounds__(kSThreads)
gscan_state_part_kernel(StateArgs a, int slices, int64_t per, size_t st_part, size_t st_dec)
{
    __shared__ __align__(16) char smem[PassLds<T, NK>::bytes];
    __shared__ Decay<T::C> dcs[2];
    const int lane = threadIdx.x & 63, slice = blockIdx.x % slices;
    const int h = blockIdx.x / slices % a.H, hk = h / (a.H / a.Hk);
    const int64_t unit = blockIdx.x / slices / a.H;
    Unit un;
    if (!find_unit(a, unit, per, T::C, lane, &un)) return;
    if (un.part == (REV ? 0 : un.parts - 1)) return;  // nothing comes after it
    const int tb = (int)(un.part * per);
    const int te = un.len - tb > per ? (int)(tb + per) : un.len;
    char *ws = reinterpret_cast<char *>(a.ws);
    float *fin = reinterpret_cast<float *>(ws + st_part) + (unit * a.H + h) * a.Dk * a.Dv;
    float *dec = reinterpret_cast<float *>(ws + st_dec) + unit * a.H + h;
    const PassJob jb = {REV ? a.q : a.k, REV ? a.dout : a.v, REV ? a.qs : a.ks, REV ? a.ds : a.vs, hk, h,
                        a.Dk, a.Dv, nullptr, fin, dec, a.Dv, 1, nullptr, REV ? a.scale : 1.f};
    pass_walk<T, NK, REV, false>(a, jb, 0, slice, h, un, tb, te, smem, dcs);
}

// Joins the units of split sequences: in place, what each adds becomes the
// state it begins with (REV: the gradient of the state it ends with).
template <bool REV>
__global__ void __launch_bounds__(kSThreads)
gscan_state_join_kernel(StateArgs a, int64_t per, size_t st_part, size_t st_dec)
{
    const int n4 = a.Dk * a.Dv / 4, blocks = (n4 + kSThreads - 1) / kSThreads;
    const int part = blockIdx.x % blocks, h = blockIdx.x / blocks % a.H;
    const int seq = blockIdx.x / blocks / a.H;
    int64_t u0 = 0;
    int n;
    if (!a.off) {
        n = (int)((a.T + per - 1) / per);
        u0 = (int64_t)seq * n;
    } else {  // units of the sequences before it
        int64_t sum = 0;
        n = 1;
        for (int i = threadIdx.x & 63; i <= seq; i += 64) {
            int64_t s = a.off[i], e = a.off[i + 1];
            s = s < 0 ? 0 : s > a.T ? a.T : s;
            e = e < s ? s : e > a.T ? a.T : e;
            const int nu = e - s > per ? (int)((e - s + per - 1) / per) : 1;
            if (i < seq) sum += nu;
            else n = nu;
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
        u0 = sum;
        n = __shfl(n, seq & 63);
    }
    const int64_t units = a.off ? a.T / per + a.B : u0 + n;  // what the workspace holds
    const int i4 = part * kSThreads + threadIdx.x;
    if (n < 2 || i4 >= n4 || u0 + n > units) return;
    char *ws = reinterpret_cast<char *>(a.ws);
    f4 *p = reinterpret_cast<f4 *>(ws + st_part) + (u0 * a.H + h) * n4 + i4;
    const float *dec = reinterpret_cast<const float *>(ws + st_dec) + u0 * a.H + h;
    const int64_t ps = (int64_t)a.H * n4;
    const float *from = REV ? a.dsT : a.s0;
    f4 st = from ? reinterpret_cast<const f4 *>(from)[((int64_t)seq * a.H + h) * n4 + i4] : zf4();
    constexpr int B = 8;  // units in flight
    for (int b = 0; b < n; b += B) {
        f4 x[B];
        float g[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int i = REV ? n - 1 - b - j : b + j;
            if (b + j < n - 1) {
                x[j] = p[i * ps];
                g[j] = dec[(int64_t)i * a.H];
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int i = REV ? n - 1 - b - j : b + j;
            if (b + j < n) {
                p[i * ps] = st;
                if (b + j < n - 1) st = g[j] * st + x[j];
            }
        }
    }
}

// Three walks per unit and head that leave operands: the states for dO S^T,
// and the gradients of the states for V dS^T and for K dS.
struct PassWs {
    size_t kv, gt, g;      // operands
    size_t part_f, part_r; // units' states and gradients of states (split sequences)
};

template <class T, int NK, int NV>
__global__ void __launch_bounds__(kSThreads)
gscan_state_pass_kernel(StateArgs a, int64_t tokens, PassWs o)
{
    constexpr int NM = NK > NV ? NK : NV;
    __shared__ __align__(16) char smem[PassLds<T, NM>::bytes];
    __shared__ Decay<T::C> dcs[2];
    constexpr int ks = NK / 2, vs = NV / 2, per = 2 * ks + vs;
    const int lane = threadIdx.x & 63;
    const int j = blockIdx.x % per;
    const int h = blockIdx.x / per % a.H, hk = h / (a.H / a.Hk);
    const int64_t unit = blockIdx.x / per / a.H;
    Unit un;
    if (!find_unit(a, unit, tokens, T::C, lane, &un)) return;
    const int tb = (int)(un.part * tokens);
    const int te = un.len - tb > tokens ? (int)(tb + tokens) : un.len;
    char *ws = reinterpret_cast<char *>(a.ws);
    const int64_t one = (int64_t)a.Dk * a.Dv, mine = (unit * a.H + h) * one;
    const int64_t whole = ((int64_t)un.seq * a.H + h) * one;
    const float *s0 = un.part ? reinterpret_cast<const float *>(ws + o.part_f) + mine
                              : a.s0 ? a.s0 + whole : nullptr;
    const float *ds = un.part + 1 < un.parts ? reinterpret_cast<const float *>(ws + o.part_r) + mine
                                             : a.dsT ? a.dsT + whole : nullptr;
    if (j < ks) {
        const PassJob jb = {a.v, a.k, a.vs, a.ks, h, hk, a.Dv, a.Dk, s0, nullptr, nullptr, 1, a.Dv,
                            ws + o.kv, 1.f};
        pass_walk<T, NV, false, true>(a, jb, NK, j, h, un, tb, te, smem, dcs);
    } else if (j < 2 * ks) {
        const PassJob jb = {a.dout, a.q, a.ds, a.qs, h, hk, a.Dv, a.Dk, ds, nullptr, nullptr, 1, a.Dv,
                            ws + o.gt, a.scale};
        pass_walk<T, NV, true, true>(a, jb, NK, j - ks, h, un, tb, te, smem, dcs);
    } else {
        const PassJob jb = {a.q, a.dout, a.qs, a.ds, hk, h, a.Dk, a.Dv, ds,
                            a.ds0 && un.part == 0 ? a.ds0 + whole : nullptr, nullptr, a.Dv, 1,
                            ws + o.g, a.scale};
        pass_walk<T, NK, true, true>(a, jb, NV, j - 2 * ks, h, un, tb, te, smem, dcs);
    }
}

// ---------------------------------------------------- backward: gradients

// x of the lane N below in its group of 16, 0 in the first N lanes
template <int N>
__device__ __forceinline__ float row_shr(float x)
{
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x110 + N, 0xf, 0xf, false));
}

__device__ __forceinline__ float sum16(float x)
{
#pragma unroll
    for (int d = 1; d < 16; d *= 2) x += __shfl_xor(x, d);
    return x;
}

// One workgroup per chunk and key head: its queries and keys stay in LDS
// while it takes the value heads that share them one by one, so dQ and dK of
// shared heads are summed in registers in a fixed order.  Wavefront (rt, cs)
// owns token rows 16rt .. 16rt+15 and every CS-th 16-column tile.
template <class T, int NK, int NV>
__global__ void __launch_bounds__(kSThreads)
gscan_state_grad_kernel(StateArgs a, size_t st_kv, size_t st_gt, size_t st_g)
{
    typedef typename T::S S;
    typedef typename T::Frag Frag;
    constexpr int C = T::C, RT = C / 16, CS = 4 / RT, KS = C / 32;
    constexpr int PK = NK * 32 + T::kPad, PV = NV * 32 + T::kPad, PP = C + T::kPad;
    constexpr int TK = 2 * NK / CS, TV = 2 * NV / CS;  // column tiles per wavefront
    __shared__ __align__(16) S qt[C * PK], kt[C * PK], vt[C * PV], ot[C * PV], pt[C * PP], dt[C * PP];
    __shared__ Decay<C> dc;
    __shared__ float rsum[C][RT], csum[RT][C], asum[CS][C], bsum[CS][C], fsum[4];
    __shared__ int bad_q, bad_o;

    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int l16 = lane & 15, g4 = 4 * (lane >> 4);
    const int rt = w % RT, cs = w / RT;
    const int hk = blockIdx.x % a.Hk;
    Unit un;
    if (!find_unit(a, blockIdx.x / a.Hk, C, C, lane, &un)) return;
    const bool packed = a.off != nullptr;
    const int t0 = un.part * C, reps = a.H / a.Hk;
    if (t0 >= un.len) return;  // a sequence without tokens
    const int64_t slot = un.slot0 + un.part;
    const char *ws = reinterpret_cast<const char *>(a.ws);

    if (tid == 0) bad_q = bad_o = 0;
    __syncthreads();
    {
        Stage<T, NK> sq, sk;
        sq.load(rows_of<S>(a.q, a.qs, un, packed, hk), a.qs.t, t0, un.len, a.Dk, tid);
        sk.load(rows_of<S>(a.k, a.ks, un, packed, hk), a.ks.t, t0, un.len, a.Dk, tid);
        sq.store(qt, PK, tid);
        sk.store(kt, PK, tid);
        if (sq.bad() || sk.bad()) bad_q = 1;
    }
    f4 dq[TK], dk[TK];
#pragma unroll
    for (int i = 0; i < TK; ++i) dq[i] = dk[i] = zf4();

    for (int hr = 0; hr < reps; ++hr) {
        const int h = hk * reps + hr;
        {
            Stage<T, NV> sv, so;
            sv.load(rows_of<S>(a.v, a.vs, un, packed, h), a.vs.t, t0, un.len, a.Dv, tid);
            so.load(rows_of<S>(a.dout, a.ds, un, packed, h), a.ds.t, t0, un.len, a.Dv, tid);
            sv.store(vt, PV, tid);
            so.store(ot, PV, tid);
            if (so.bad()) bad_o = 1;
        }
        float gx = 0.f;
        if (w == 0) {
            const int64_t g0 = (packed ? un.in0 * a.gs.t : (int64_t)un.seq * a.gs.b) + (int64_t)h * a.gs.h;
            const bool ok = lane < C && t0 + lane < un.len;
            if (ok) gx = load_scalar(a.gate, g0 + (int64_t)(t0 + lane) * a.gs.t, a.gate_dtype) + a.gate_shift;
            gate_scan<C>(dc, gx, ok, a.gate_form, lane);
        }
        __syncthreads();
        const bool bq = bad_q != 0, bo = bad_o != 0;

        // P . D and dP . D, and the sums of W: over s < t inside a tile's
        // columns and u >= t (csum), and each row's whole tile (rsum)
        {
#pragma unroll
            for (int ct = cs; ct < RT; ct += CS) {
                f4 x = zf4(), y = zf4();
                float cp = 0.f;
                if (ct <= rt) {
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk)
                        x = mma(ld_row(qt, PK, 16 * rt, 32 * kk, lane),
                                ld_row(kt, PK, 16 * ct, 32 * kk, lane), x);
#pragma unroll
                    for (int kk = 0; kk < NV; ++kk)
                        y = mma(ld_row(ot, PV, 16 * rt, 32 * kk, lane),
                                ld_row(vt, PV, 16 * ct, 32 * kk, lane), y);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u = 16 * rt + g4 + j, s = 16 * ct + l16;
                    const float f = a.scale * decay(dc, u, s);
                    narrow(u >= s ? x[j] * f : 0.f, &pt[u * PP + s]);
                    narrow(u >= s ? y[j] * f : 0.f, &dt[u * PP + s]);
                    float wv = u > s ? x[j] * y[j] * f : 0.f;
                    wv += row_shr<1>(wv);
                    wv += row_shr<2>(wv);
                    wv += row_shr<4>(wv);
                    wv += row_shr<8>(wv);
                    const float before = row_shr<1>(wv);
                    cp += u >= s ? before : 0.f;
                    if (l16 == 15) rsum[u][ct] = wv;
                }
                cp += __shfl_xor(cp, 16);
                cp += __shfl_xor(cp, 32);
                if (lane < 16) csum[rt][16 * ct + lane] = cp;
            }
        }
        __syncthreads();

        if (tid == 0) bad_o = 0;  // read by all before this barrier, set again after the last one
        const void *Sf = ws + st_kv, *Gt = ws + st_gt, *Gf = ws + st_g;
        const int64_t fh = (slot * a.H + h) * 2 * NK * NV;  // operands before this head's
        // dQ: (dP . D) K + scale e^L dO S^T
        {
            Frag of[NV];
            f4 as = zf4();
#pragma unroll
            for (int kk = 0; kk < NV; ++kk) of[kk] = ld_row(ot, PV, 16 * rt, 32 * kk, lane);
#pragma unroll
            for (int i = 0; i < TK; ++i) {
                const int n = i * CS + cs;
                f4 x = zf4();
#pragma unroll
                for (int kk = 0; kk < NV; ++kk) {
                    Frag sf;
                    get_frag(Sf, fh + n * NV + kk, lane, &sf);
                    x = mma(of[kk], sf, x);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] *= a.scale * dc.e[16 * rt + g4 + j];
                    as[j] += x[j] * widen(qt[(16 * rt + g4 + j) * PK + 16 * n + l16]);
                }
                dq[i] += x;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
                    if (2 * kk <= rt) {
                        Frag f = ld_col(kt, PK, 32 * kk, 16 * n, lane);
                        if (bq) f = finite_part(f);
                        dq[i] = mma(ld_row(dt, PP, 16 * rt, 32 * kk, lane), f, dq[i]);
                    }
                if (bq) dq[i] += other_terms<true, false>(dt, PP, kt, PK, 16 * rt + g4, 16 * n + l16, C);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float r = sum16(as[j]);
                if (l16 == 0) asum[cs][16 * rt + g4 + j] = r;
            }
        }
        // dK: (dP . D)^T Q + e^(L_end - L) V dS^T
        {
            Frag vf[NV];
            f4 bs = zf4();
#pragma unroll
            for (int kk = 0; kk < NV; ++kk) vf[kk] = ld_row(vt, PV, 16 * rt, 32 * kk, lane);
#pragma unroll
            for (int i = 0; i < TK; ++i) {
                const int n = i * CS + cs;
                f4 x = zf4();
#pragma unroll
                for (int kk = 0; kk < NV; ++kk) {
                    Frag gf;
                    get_frag(Gt, fh + n * NV + kk, lane, &gf);
                    x = mma(vf[kk], gf, x);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] *= dc.d[16 * rt + g4 + j];
                    bs[j] += x[j] * widen(kt[(16 * rt + g4 + j) * PK + 16 * n + l16]);
                }
                dk[i] += x;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
                    if (2 * kk + 1 >= rt) {
                        Frag f = ld_col(qt, PK, 32 * kk, 16 * n, lane);
                        if (bq) f = finite_part(f);
                        dk[i] = mma(ld_col(dt, PP, 32 * kk, 16 * rt, lane), f, dk[i]);
                    }
                if (bq) dk[i] += other_terms<false, true>(dt, PP, qt, PK, 16 * rt + g4, 16 * n + l16, C);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float r = sum16(bs[j]);
                if (l16 == 0) bsum[cs][16 * rt + g4 + j] = r;
            }
        }
        // dV: (P . D)^T dO + e^(L_end - L) K dS
        {
            Frag kf[NK];
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) kf[kk] = ld_row(kt, PK, 16 * rt, 32 * kk, lane);
#pragma unroll
            for (int i = 0; i < TV; ++i) {
                const int n = i * CS + cs, col = 16 * n + l16;
                f4 x = zf4();
#pragma unroll
                for (int kk = 0; kk < NK; ++kk) {
                    Frag gf;
                    get_frag(Gf, fh + n * NK + kk, lane, &gf);
                    x = mma(kf[kk], gf, x);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] *= dc.d[16 * rt + g4 + j];
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
                    if (2 * kk + 1 >= rt) {
                        Frag f = ld_col(ot, PV, 32 * kk, 16 * n, lane);
                        if (bo) f = finite_part(f);
                        x = mma(ld_col(pt, PP, 32 * kk, 16 * rt, lane), f, x);
                    }
                if (bo) x += other_terms<false, true>(pt, PP, ot, PV, 16 * rt + g4, col, C);
                if (col < a.Dv)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = t0 + 16 * rt + g4 + j;
                        if (t < un.len)
                            narrow(x[j], reinterpret_cast<S *>(a.dv) + ((un.tok0 + t) * a.H + h) * a.Dv + col);
                    }
            }
        }
        // F = e^(L_end) <S, dS>
        {
            float f = 0.f;
            for (int i = w; i < 2 * NK * NV; i += 4) {
                Frag x, y;
                f4 x0, x1, y0, y1;
                get_frag(Sf, fh + i, lane, &x);
                get_frag(Gt, fh + i, lane, &y);
                from_frag(x, &x0, &x1);
                from_frag(y, &y0, &y1);
#pragma unroll
                for (int j = 0; j < 4; ++j) f += x0[j] * y0[j] + x1[j] * y1[j];
            }
#pragma unroll
            for (int d = 1; d < 64; d *= 2) f += __shfl_xor(f, d);
            if (lane == 0) fsum[w] = f;
        }
        __syncthreads();
        if (w == 0) {
            float x = 0.f, b = 0.f, in = 0.f, rs[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) rs[i] = 0.f;
            if (lane < C) {
#pragma unroll
                for (int i = 0; i < CS; ++i) {
                    x += asum[i][lane];
                    b += bsum[i][lane];
                }
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    in += csum[i][lane];
                    rs[i] = rsum[lane][i];
                }
            }
            float pb = b;
#pragma unroll
            for (int d = 1; d < C; d *= 2) {
                const float y = __shfl_down(x, d), z = __shfl_up(pb, d);
                if (lane + d < 64) x += y;
                if (lane >= d) pb += z;
#pragma unroll
                for (int i = 0; i + 1 < RT; ++i) {
                    const float r = __shfl_down(rs[i], d);
                    if (lane + d < 64) rs[i] += r;
                }
            }
            x += in;
#pragma unroll
            for (int i = 0; i + 1 < RT; ++i)
                if (lane >= 16 * (i + 1)) x += rs[i];
            const float F = dc.g * ((fsum[0] + fsum[1]) + (fsum[2] + fsum[3]));
            const float before = __shfl_up(pb, 1);
            if (lane < C && t0 + lane < un.len) {
                const float dl = x + (lane ? before : 0.f) + F;
                const float r = dl * log_gate_slope(gx, a.gate_form);
                const int64_t at = (un.tok0 + t0 + lane) * a.H + h;
                if (a.gate_dtype) reinterpret_cast<uint16_t *>(a.dgate)[at] = to_bf16(r);
                else reinterpret_cast<float *>(a.dgate)[at] = r;
            }
        }
        __syncthreads();
    }

#pragma unroll
    for (int i = 0; i < TK; ++i) {
        const int col = 16 * (i * CS + cs) + l16;
        if (col < a.Dk)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t0 + 16 * rt + g4 + j;
                if (t < un.len) {
                    const int64_t at = ((un.tok0 + t) * a.Hk + hk) * a.Dk + col;
                    narrow(dq[i][j], reinterpret_cast<S *>(a.dq) + at);
                    narrow(dk[i][j], reinterpret_cast<S *>(a.dk) + at);
                }
            }
    }
}

template <class T, int NK, bool REV>
hipError_t part_launch(const StatePlan &p, const StateArgs &a, size_t st_part, size_t st_dec,
                       hipStream_t st)
{
    const int slices = (a.Dv + kSlice - 1) / kSlice;
    hipLaunchKernelGGL((gscan_state_part_kernel<T, NK, REV>), dim3((unsigned)(p.units * a.H * slices)),
                       dim3(kSThreads), 0, st, a, slices, p.per, st_part, st_dec);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = (a.Dk * a.Dv / 4 + kSThreads - 1) / kSThreads;
    hipLaunchKernelGGL((gscan_state_join_kernel<REV>), dim3((unsigned)(a.B * a.H * blocks)),
                       dim3(kSThreads), 0, st, a, p.per, st_part, st_dec);
    return hipGetLastError();
}

template <class T, int NK>
hipError_t fwd_launch(const StatePlan &p, const StateArgs &a, hipStream_t st)
{
    const int slices = (a.Dv + kSlice - 1) / kSlice;
    if (p.split) {
        const hipError_t e = part_launch<T, NK, false>(p, a, p.st_part, p.st_dec, st);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((gscan_state_fwd_kernel<T, NK>), dim3((unsigned)(p.units * a.H * slices)),
                       dim3(kSThreads), 0, st, a, slices, p.per, p.st_part);
    return hipGetLastError();
}

template <class T, int NK, int NV>
hipError_t bwd_launch(const StatePlan &p, const StateArgs &a, hipStream_t st)
{
    hipError_t e;
    if (p.split) {
        e = part_launch<T, NK, false>(p, a, p.st_part, p.st_dec, st);
        if (e == hipSuccess) e = part_launch<T, NK, true>(p, a, p.st_part_r, p.st_dec_r, st);
        if (e != hipSuccess) return e;
    }
    const PassWs o = {p.st_kv, p.st_gt, p.st_g, p.st_part, p.st_part_r};
    hipLaunchKernelGGL((gscan_state_pass_kernel<T, NK, NV>),
                       dim3((unsigned)(p.units * a.H * (NK + NV / 2))), dim3(kSThreads), 0, st, a, p.per, o);
    e = hipGetLastError();
    if (e != hipSuccess || a.T == 0) return e;
    hipLaunchKernelGGL((gscan_state_grad_kernel<T, NK, NV>), dim3((unsigned)(p.chunks * a.Hk)),
                       dim3(kSThreads), 0, st, a, p.st_kv, p.st_gt, p.st_g);
    return hipGetLastError();
}

template <class T>
hipError_t bwd_widths(const StatePlan &p, const StateArgs &a, hipStream_t st)
{
    if (p.nk == 2) return p.nv == 2 ? bwd_launch<T, 2, 2>(p, a, st) : bwd_launch<T, 2, 4>(p, a, st);
    return p.nv == 2 ? bwd_launch<T, 4, 2>(p, a, st) : bwd_launch<T, 4, 4>(p, a, st);
}

}  // namespace

// Sequences are split into units of `per` tokens, walked in parallel, where
// there are too few of them to fill the card.
StatePlan make_state_plan(const StateArgs &a, bool backward)
{
    StatePlan p;
    p.chunk = a.dtype ? BF::C : FP::C;
    p.nk = a.Dk <= 64 ? 2 : 4;
    p.nv = a.Dv <= 64 ? 2 : 4;
    const int64_t nc = a.T > p.chunk ? (a.T + p.chunk - 1) / p.chunk : 1;
    // packed: sum over sequences of max(1, ceil(len / C)) <= T / C + B
    p.chunks = a.off ? a.T / p.chunk + a.B : a.B * nc;
    const int64_t walks = (int64_t)a.H * (backward ? p.nk + p.nv / 2 : (a.Dv + kSlice - 1) / kSlice);
    static const int64_t tgt = getenv("GS_TGT") ? atoi(getenv("GS_TGT")) : 768;
    static const int64_t mn = getenv("GS_MIN") ? atoi(getenv("GS_MIN")) : 4;
    int64_t pc = p.chunks * walks / tgt;
    pc = pc < mn ? mn : pc;
    p.split = pc < nc;
    p.per = p.split ? pc * p.chunk : (nc > 1 ? nc : 1) * p.chunk;
    p.units = !p.split ? a.B : a.off ? a.T / p.per + a.B : a.B * ((a.T + p.per - 1) / p.per);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t r = at;
        at += (n + 255) / 256 * 256;
        return r;
    };
    if (p.split) {
        const size_t states = (size_t)p.units * (size_t)a.H * (size_t)a.Dk * (size_t)a.Dv * 4u;
        const size_t decs = (size_t)p.units * (size_t)a.H * 4u;
        p.st_part = take(states);
        p.st_dec = take(decs);
        if (backward) {
            p.st_part_r = take(states);
            p.st_dec_r = take(decs);
        }
    }
    if (backward) {
        const size_t one = (size_t)p.chunks * (size_t)a.H * (size_t)(p.nk * p.nv) * 1024u *
                           (a.dtype ? 2u : 4u);
        p.st_kv = take(one);
        p.st_gt = take(one);
        p.st_g = take(one);
    }
    p.bytes = at;
    return p;
}

hipError_t launch_state_forward(const StatePlan &p, const StateArgs &args, hipStream_t st)
{
    StateArgs a = args;
    a.chunks = p.chunks;
    if (a.dtype) return p.nk == 2 ? fwd_launch<BF, 2>(p, a, st) : fwd_launch<BF, 4>(p, a, st);
    return p.nk == 2 ? fwd_launch<FP, 2>(p, a, st) : fwd_launch<FP, 4>(p, a, st);
}

hipError_t launch_state_backward(const StatePlan &p, const StateArgs &args, hipStream_t st)
{
    StateArgs a = args;
    a.chunks = p.chunks;
    return a.dtype ? bwd_widths<BF>(p, a, st) : bwd_widths<FP>(p, a, st);
}

}  // namespace gscan
