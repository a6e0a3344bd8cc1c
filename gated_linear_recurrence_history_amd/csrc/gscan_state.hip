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
// sequence has fp32 accuracy.  The backward's chunk states go through memory as
// fp16 with a power of two per tile (put_state).
#include <cstdint>
#include <type_traits>

#include "gscan_state_dev.h"

namespace gscan {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));

constexpr int kSThreads = 256;
constexpr int kSlice = 64;  // columns of a state that one workgroup walks

// Loads are not moved across this: without it the unrolled steps of a chunk
// are all loaded at its beginning, for more registers than there are.
#define GSCAN_STEP() asm volatile("" ::: "memory")

__device__ __forceinline__ f4 zf4() { return f4{0.f, 0.f, 0.f, 0.f}; }

// ------------------------------------------------------- operand types

struct BF {
    typedef uint16_t S;   // storage
    typedef u4 Frag;      // eight bf16
    static constexpr int C = 64, VE = 8;  // tokens per chunk, elements of 16 bytes
};
struct FP {
    typedef float S;
    struct Frag {
        f4 a, b;
    };
    static constexpr int C = 32, VE = 4;
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

// Tiles in LDS: rows of 64 or 128 elements (W), `bytes` a row apart.  bf16 rows
// are not padded; the 8-byte pieces of each 128 bytes of row r are exchanged
// by XOR with ((r & 3) << 2) | (((r >> 2) ^ r) & 3), which puts the sixteen rows a
// read along rows touches, the four rows times four pieces a transposed read
// touches, and the first (second) halves of eight 16-byte pieces each of two
// neighbouring rows that are stored together on different banks (32 of 4
// bytes; without the "^ r" such stores took each bank twice, and the
// scan of 32771 tokens 125 us where it then took 120).  fp32 rows are 16 bytes
// longer than their elements, which does the same for both reads.
//
// Per lane: byte offsets of the pieces it reads along a row (r[c]: elements
// 16c + 4g of row l % 16) and down a column (c[i]: column 16i + l % 16 of rows
// 4g ..); what a read adds to them is known at compile time.
template <class T, int W>
struct Tile;

template <int W>
struct Tile<BF, W> {
    static constexpr int bytes = W * 2;
    uint32_t r[4], c[4];
    __device__ __forceinline__ explicit Tile(int lane)
    {
        const uint32_t l16 = lane & 15, g = lane >> 4, p4 = l16 >> 2;
        const uint32_t fr = ((l16 & 3) << 2) | ((p4 ^ l16) & 3), fc = (p4 << 2) | (g ^ p4);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            r[i] = l16 * bytes + ((g ^ (4 * i) ^ fr) << 3);
            c[i] = (4 * g + p4) * bytes + (((l16 & 3) ^ (4 * i) ^ fc) << 3);
        }
    }
    // byte offset of an 8-byte piece (four elements)
    static __device__ __forceinline__ uint32_t piece(uint32_t row, uint32_t col)
    {
        const uint32_t f = ((row & 3) << 2) | (((row >> 2) ^ row) & 3), p = col / 4;
        return row * bytes + (p >> 4) * 128 + (((p & 15) ^ f) << 3);
    }
    static __device__ __forceinline__ void put(char *t, uint32_t row, uint32_t col, const u4 &x)
    {
        const uint32_t at = piece(row, col);
        *reinterpret_cast<uint2 *>(t + at) = uint2{x[0], x[1]};
        *reinterpret_cast<uint2 *>(t + (at ^ 8)) = uint2{x[2], x[3]};
    }
    // elements 16c + 4g .. +3 of row r0 + l % 16
    __device__ __forceinline__ uint2 quad_bits(const char *t, int r0, int cc) const
    {
        return *reinterpret_cast<const uint2 *>(t + r[cc & 3] + (r0 * bytes + (cc >> 2) * 128));
    }
    __device__ __forceinline__ f4 quad(const char *t, int r0, int cc) const
    {
        const uint2 x = quad_bits(t, r0, cc);
        return f4{bf_lo(x.x), bf_hi(x.x), bf_lo(x.y), bf_hi(x.y)};
    }
    // row r0 + l%16, elements 32kk + {4g.., 16 + 4g..}
    __device__ __forceinline__ u4 row(const char *t, int r0, int kk) const
    {
        const uint2 x = quad_bits(t, r0, 2 * kk), y = quad_bits(t, r0, 2 * kk + 1);
        return u4{x.x, x.y, y.x, y.y};
    }
    // column 16i + l%16 of rows k0 + {4g.., 16 + 4g..}.  The transposed read
    // gives lane i of a 16-lane group element i % 4 of the 8-byte pieces that
    // lanes 4j + i/4 address, j = 0..3: with lane p addressing row 4g + p/4,
    // columns 4 (p % 4).., it receives column p of rows 4g .. 4g+3.
    __device__ __forceinline__ u4 at_col(const char *t, int k0, uint32_t off) const
    {
        const char *p = t + off + k0 * bytes;
        const uint2 x = tr(p), y = tr(p + 16 * bytes);
        return u4{x.x, x.y, y.x, y.y};
    }
    __device__ __forceinline__ u4 col(const char *t, int k0, int i) const
    {
        return at_col(t + (i >> 2) * 128, k0, c[i & 3]);
    }
    // the offset of a column tile known at run time only
    __device__ __forceinline__ uint32_t col_off(int i) const
    {
        return (c[0] ^ ((i & 3) << 5)) + (i >> 2) * 128;
    }
    static __device__ __forceinline__ uint2 tr(const char *p)
    {
        return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                             (__attribute__((address_space(3))) s4v *)(p)));
    }
    // replaces an infinity or NaN by zero
    static __device__ __forceinline__ bool scrub(char *t, int row, int col)
    {
        uint16_t *x = reinterpret_cast<uint16_t *>(t + piece(row, col)) + (col & 3);
        if ((*x & 0x7f80u) != 0x7f80u) return false;
        *x = 0;
        return true;
    }
};

template <int W>
struct Tile<FP, W> {
    static constexpr int bytes = W * 4 + 16;
    uint32_t r, c;
    __device__ __forceinline__ explicit Tile(int lane)
        : r((lane & 15) * bytes + (lane >> 4) * 16), c((lane >> 4) * 4 * bytes + (lane & 15) * 4)
    {
    }
    static __device__ __forceinline__ void put(char *t, uint32_t row, uint32_t col, const u4 &x)
    {
        *reinterpret_cast<u4 *>(t + row * bytes + col * 4) = x;
    }
    __device__ __forceinline__ f4 quad(const char *t, int r0, int cc) const
    {
        return *reinterpret_cast<const f4 *>(t + r + (r0 * bytes + cc * 64));
    }
    __device__ __forceinline__ FP::Frag row(const char *t, int r0, int kk) const
    {
        return FP::Frag{quad(t, r0, 2 * kk), quad(t, r0, 2 * kk + 1)};
    }
    __device__ __forceinline__ FP::Frag at_col(const char *t, int k0, uint32_t off) const
    {
        const char *p = t + off + k0 * bytes;
        FP::Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.a[j] = *reinterpret_cast<const float *>(p + j * bytes);
            f.b[j] = *reinterpret_cast<const float *>(p + (16 + j) * bytes);
        }
        return f;
    }
    __device__ __forceinline__ FP::Frag col(const char *t, int k0, int i) const
    {
        return at_col(t + i * 64, k0, c);
    }
    __device__ __forceinline__ uint32_t col_off(int i) const { return c + i * 64; }
    static __device__ __forceinline__ bool scrub(char *t, int row, int col)
    {
        float *x = reinterpret_cast<float *>(t + row * bytes + col * 4);
        if (isfinite(*x)) return false;
        *x = 0.f;
        return true;
    }
};

// Rows of N 32-wide units; three are in rows of four.
template <class T, int N>
using Rows = Tile<T, N == 3 ? 128 : N * 32>;

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
// each the rounding of what the parts before it leave.  The remainder of a
// pair is -1 * part + 0 * (the other half) + x, one bf16 dot product per
// element: the products and the difference are exact.  The selectors are
// scalars, as an inline constant would be taken for fp32 -1.0.
struct Parts {
    u4 p[3];
};
__device__ __forceinline__ void to_parts(f4 x, f4 y, Parts *s)
{
    uint32_t m0 = 0x0000bf80u, m1 = 0xbf800000u;
    asm("" : "+s"(m0), "+s"(m1));
    const bf16x2 lo = __builtin_bit_cast(bf16x2, m0), hi = __builtin_bit_cast(bf16x2, m1);
    float r[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t h = pack_bf16(r[2 * j], r[2 * j + 1]);
            s->p[i][j] = h;
            if (i < 2) {
                const bf16x2 hv = __builtin_bit_cast(bf16x2, h);
                r[2 * j] = __builtin_amdgcn_fdot2_f32_bf16(hv, lo, r[2 * j], false);
                r[2 * j + 1] = __builtin_amdgcn_fdot2_f32_bf16(hv, hi, r[2 * j + 1], false);
            }
        }
}
__device__ __forceinline__ void to_parts(f4 x, f4 y, FP::Frag *s) { *s = FP::Frag{x, y}; }
template <int N>
__device__ __forceinline__ void mma_all(f4 (&st)[N], const u4 (&x)[N], const Parts &y)
{
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int i = 0; i < N; ++i) st[i] = mma(x[i], y.p[p], st[i]);
}
template <int N>
__device__ __forceinline__ void mma_all(f4 (&st)[N], const FP::Frag (&x)[N], const FP::Frag &y)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < N; ++i) st[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i].a[j], y.a[j], st[i], 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < N; ++i) st[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i].b[j], y.b[j], st[i], 0, 0, 0);
    }
}

template <class T>
struct PartsOf {
    typedef Parts type;
};
template <>
struct PartsOf<FP> {
    typedef FP::Frag type;
};

// Operands of states kept in device memory: 16 bytes (bf16) or two planes of
// 16 bytes (fp32) per lane.  bf16: fp16 with a power of two per tile of 16
// columns, whose 11 bits <S, dS> needs (with bf16's 8 its gradient of the gate
// was off by 2.9e-3, more than the rounding of the result); they become bf16
// where they are operands.
__device__ __forceinline__ void put_state(void *base, int64_t i, int lane, f4 x, f4 y, float up, const BF &)
{
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    auto pk = [&](float u, float v) {
        return __builtin_bit_cast(uint32_t, h2{(_Float16)(u * up), (_Float16)(v * up)});
    };
    reinterpret_cast<u4 *>(base)[i * 64 + lane] = u4{pk(x[0], x[1]), pk(x[2], x[3]), pk(y[0], y[1]), pk(y[2], y[3])};
}
__device__ __forceinline__ void put_state(void *base, int64_t i, int lane, f4 x, f4 y, float, const FP &)
{
    reinterpret_cast<f4 *>(base)[i * 128 + lane] = x;
    reinterpret_cast<f4 *>(base)[i * 128 + 64 + lane] = y;
}
__device__ __forceinline__ u4 get_state(const u4 &x, float down, const BF &)
{
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    u4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = x[i];  // (a bit cast of the element itself takes the first one)
        const h2 h = __builtin_bit_cast(h2, u);
        r[i] = pack_bf16((float)h[0] * down, (float)h[1] * down);
    }
    return r;
}
__device__ __forceinline__ u4 get_state(const u4 &x, float, const FP &) { return x; }

// Whether sixteen bytes hold an infinity or NaN: the largest magnitude's bits.
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void magnitude(const u4 &x, const BF &, uint32_t *m)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(
                 __builtin_bit_cast(us2, *m), __builtin_bit_cast(us2, x[i] & 0x7fff7fffu)));
}
__device__ __forceinline__ bool nonfinite(uint32_t m, const BF &)
{
    return (m & 0xffffu) >= 0x7f80u || m >= 0x7f800000u;
}
__device__ __forceinline__ void magnitude(const u4 &x, const FP &, uint32_t *m)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t y = x[i] & 0x7fffffffu;
        *m = y > *m ? y : *m;
    }
}
__device__ __forceinline__ bool nonfinite(uint32_t m, const FP &) { return m >= 0x7f800000u; }

// ------------------------------------------------------------ device memory

// A buffer of the 2 GiB from p: offsets of -1 read as zero and write nothing,
// so rows past a sequence's end and columns past a width cost no branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint64_t u = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a);
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(u), 0, 0x80000000, 0x00027000);
}
constexpr uint32_t kNowhere = 0xffffffffu;

__device__ __forceinline__ void put1(uint16_t *p, float x) { *p = to_bf16(x); }
__device__ __forceinline__ void put1(float *p, float x) { *p = x; }

// Four elements at byte offset `at` of a buffer.
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t b, uint32_t at, f4 x, const BF &)
{
    typedef unsigned int u2 __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(u2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])}, b, at, 0, 0);
}
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t b, uint32_t at, f4 x, const FP &)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, x), b, at, 0, 0);
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

__device__ __forceinline__ int first_lane(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Workgroups are dealt to the eight XCDs in turn.  The index this one takes so
// that `share` neighbours, which read the same rows, meet in one XCD's L2.
__device__ __forceinline__ uint32_t neighbours(uint32_t share)
{
    const uint32_t b = blockIdx.x, whole = gridDim.x / (8 * share) * (8 * share);
    return b < whole ? ((b / 8 / share) * 8 + b % 8) * share + b / 8 % share : b;
}

// Whether unit u exists (the same answer, in scalar registers, for every
// lane).  Offsets are clamped to the tokens there are, so
// wrong ones read and write nothing out of range.  Called by whole wavefronts.
__device__ __forceinline__ bool find_unit(const StateArgs &a, int64_t u, int64_t per, int C,
                                          int lane, Unit *w)
{
    if (!a.off) {
        const uint32_t T = (uint32_t)a.T, p = (uint32_t)per;
        const uint32_t n = T > p ? (T + p - 1) / p : 1, nc = T > (uint32_t)C ? (T + C - 1) / C : 1;
        const int64_t seq = (uint32_t)u / n;
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
            const int64_t seq = i0 + first_lane(l);
            if (seq >= a.B) return false;
            w->seq = (int)seq;
            w->parts = first_lane(__shfl(nu, l));
            w->part = first_lane((int)(u - (ub + __shfl(su, l) - w->parts)));
            w->slot0 = first_lane((int)(cb + __shfl(sc, l) - __shfl(nc, l)));
            // offsets that overlap could ask for more chunks than there are
            if (w->slot0 + first_lane(__shfl(nc, l)) > a.chunks) return false;
            const int start = first_lane(__shfl((int)s, l));
            w->len = first_lane(__shfl((int)(e - s), l));
            w->tok0 = w->in0 = start;
            return true;
        }
        ub += first_lane(__shfl(su, 63));
        cb += first_lane(__shfl(sc, 63));
    }
    return false;
}

// The row of token t of a sequence and head h.
template <class S>
__device__ __forceinline__ const S *row_at(const void *p, const Strides &s, const Unit &w, int h,
                                           int64_t t)
{
    return reinterpret_cast<const S *>(p) + (int64_t)w.seq * s.b +
           ((uint64_t)s.h * (uint32_t)h + (uint64_t)s.t * (uint32_t)(w.in0 + t));
}

// Gate arguments of a chunk's tokens, one per lane (those from `left` on: zero),
// either type without a branch, so that the loads in flight can be counted.
struct Gates {
    const char *base;
    uint32_t o32, o16;
    int64_t step;
    __device__ __forceinline__ void begin(const StateArgs &a, const Unit &w, int h, int64_t t0, int C,
                                          int lane)
    {
        const int64_t e = a.gate_dtype ? 2 : 4;
        base = a.gate_dtype ? reinterpret_cast<const char *>(row_at<uint16_t>(a.gate, a.gs, w, h, t0))
                            : reinterpret_cast<const char *>(row_at<float>(a.gate, a.gs, w, h, t0));
        const uint32_t at = (uint32_t)lane * a.gs.t * (uint32_t)e;
        o32 = lane < C && !a.gate_dtype ? at : kNowhere;
        o16 = lane < C && a.gate_dtype ? at : kNowhere;
        step = (int64_t)(C * a.gs.t) * e;
    }
    struct Raw {
        uint32_t x32;
        uint16_t x16;
    };
    // the next chunk's, and on by `dir` chunks
    __device__ __forceinline__ Raw load(int left, int lane, int dir)
    {
        const __amdgpu_buffer_rsrc_t b = buffer(base);
        Raw r;
        r.x32 = __builtin_amdgcn_raw_buffer_load_b32(b, lane < left ? o32 : kNowhere, 0, 0);
        r.x16 = __builtin_amdgcn_raw_buffer_load_b16(b, lane < left ? o16 : kNowhere, 0, 0);
        base += dir * step;
        return r;
    }
    static __device__ __forceinline__ float value(const Raw &r, const StateArgs &a)
    {
        return __uint_as_float(r.x32 | (uint32_t)r.x16 << 16) + a.gate_shift;
    }
};

// ---------------------------------------------------------- staged tiles

// C rows of NKU 32-wide units, 16 bytes at a time, by TH threads.
template <class T, int NKU, int TH = kSThreads>
struct Stage {
    static constexpr int N = NKU * kSThreads / TH;  // pieces per thread
    typedef u4 Regs[N];
    uint32_t off[N];  // of the pieces from the chunk's first row
    const typename T::S *base;  // that row
    static constexpr int kPpr = NKU * 32 / T::VE;  // pieces per row
    // Piece q of the tile.  Two halves of a row (bf16): eight follow each other in a
    // row, then eight of the next row, before the rows' other halves (Tile's banks).
    static constexpr bool kHalves = T::VE == 8 && kPpr == 16;
    static __device__ __forceinline__ int row_of(int q)
    {
        return kHalves ? (q >> 5) * 2 + (q >> 3 & 1) : q / kPpr;
    }
    static __device__ __forceinline__ int col_of(int q)
    {
        return (kHalves ? (q >> 4 & 1) * 8 + (q & 7) : q % kPpr) * T::VE;
    }

    // row 0 of the tile is at `row` (stride st, below 2^23); columns before
    // `cols` are read, the others are zero
    __device__ __forceinline__ void begin(const typename T::S *row0, uint32_t st, int cols, int tid)
    {
        base = row0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int q = tid + TH * i, row = row_of(q), col = col_of(q);
            off[i] = col < cols ? (uint32_t)(row * st + col) * (uint32_t)sizeof(typename T::S) : kNowhere;
        }
    }
    // the first `left` rows of the tile (the others zero), and on by `step`
    // elements to the next
    __device__ __forceinline__ void load(Regs &r, int left, int64_t step, int tid)
    {
        const __amdgpu_buffer_rsrc_t b = buffer(base);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = row_of(tid + TH * i);
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(b, row < left ? off[i] : kNowhere, 0, 0);
        }
        base += step;
    }
    // the same of a tile that is not followed by others
    static __device__ __forceinline__ void fetch(Regs &r, __amdgpu_buffer_rsrc_t b, uint32_t st, int cols,
                                                 int left, int tid)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int q = tid + TH * i, row = row_of(q), col = col_of(q);
            const uint32_t at = (__umul24(row, st) + col) * (uint32_t)sizeof(typename T::S);
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(b, ((row < left) & (col < cols)) ? at : kNowhere, 0, 0);
        }
    }
    template <class TL>
    static __device__ __forceinline__ void store(const Regs &r, char *tile, int tid)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int q = tid + TH * i;
            TL::put(tile, row_of(q), col_of(q), r[i]);
        }
    }
    // Infinities and NaN of the stored tile become zero, and `found(row, column)`
    // is called for each.  A product with scores that are zero above the
    // diagonal would carry them to tokens they do not reach, as 0 * inf.  What
    // they do reach is not finite in any case (the whole column of the state
    // from that token on), so those results become NaN without being computed.
    template <class TL, class F>
    static __device__ __forceinline__ void scrub(const Regs &r, char *tile, int tid, F found)
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) magnitude(r[i], T(), &m);
        if (!nonfinite(m, T())) return;
#pragma unroll 1
        for (int i = 0; i < N * T::VE; ++i) {
            const int q = tid + TH * (i / T::VE), row = row_of(q), col = col_of(q) + i % T::VE;
            if (TL::scrub(tile, row, col)) found(row, col);
        }
    }
};

// Four columns of a row, NaN where one of `where` reaches it (from that row on,
// LAST: up to it), or everywhere (all).
template <bool LAST>
__device__ __forceinline__ f4 poison(f4 x, const int *where, int row, bool all = false)
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (all || (LAST ? row <= where[j] : row >= where[j])) x[j] = __builtin_nanf("");
    return x;
}

// Decays of one chunk, in LDS.  L in units of log 2 (as a sum of two floats,
// so that differences of far-down values keep fp32 accuracy), e^L,
// e^(L_end - L), e^(L_end); and for tiles of 16 x 16 tokens below the
// diagonal the two factors of e^(L_t - L_s) around the last token m of s's
// tile, e^(L_m - L_s) and (zero where t is not below the tile) e^(L_t - L_m),
// neither above what the gates allow.
template <int C>
struct __align__(16) Decay {
    float hi[C], lo[C], e[C], d[C], col[C], row[C / 16][C], g;
};

// x of other lanes, zero where there is none: CTRL 0x110 + n, n lanes below in
// the group of 16; 0x142 and 0x143, the last lane of the group (of the half)
// before, taken by the groups of row mask RM; 0x150 + n, lane n of the group.
template <int CTRL, int RM = 0xf>
__device__ __forceinline__ float dpp(float x)
{
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, RM, 0xf, false));
}
template <int CTRL, int RM = 0xf>
__device__ __forceinline__ double dpp(double x)
{
    const uint2 u = __builtin_bit_cast(uint2, x);
    return __builtin_bit_cast(double, uint2{__builtin_amdgcn_update_dpp(0u, u.x, CTRL, RM, 0xf, false),
                                            __builtin_amdgcn_update_dpp(0u, u.y, CTRL, RM, 0xf, false)});
}
__device__ __forceinline__ double of_lane(double x, int lane)
{
    const uint2 u = __builtin_bit_cast(uint2, x);
    return __builtin_bit_cast(double, uint2{(uint32_t)__builtin_amdgcn_readlane(u.x, lane),
                                            (uint32_t)__builtin_amdgcn_readlane(u.y, lane)});
}

// The running sum of log2 of the gates, of which token `lane` has the argument
// x (ok: there is one).  One wavefront.
template <int C>
__device__ __forceinline__ double gate_sum(float x, bool ok, int form)
{
    double L = ok ? (double)log_gate(x, form) * 1.44269504088896340736 : 0.0;
    L += dpp<0x111>(L);
    L += dpp<0x112>(L);
    L += dpp<0x114>(L);
    L += dpp<0x118>(L);
    L += dpp<0x142, 0xa>(L);
    if constexpr (C > 32) L += dpp<0x143, 0xc>(L);
    return L;
}
// The decays from it.  Factors of scores off the diagonal are multiplied by mul.
template <int C>
__device__ __forceinline__ void gate_decays(Decay<C> &s, double L, int lane, float mul = 1.f)
{
    const double end = of_lane(L, C - 1);
    double m = end, mid[C / 16 - 1];
#pragma unroll
    for (int i = C / 16 - 2; i >= 0; --i) {
        mid[i] = of_lane(L, 16 * i + 15);
        if (lane < 16 * i + 16) m = mid[i];
    }
    if (lane < C) {
        const float h = (float)L;
        s.hi[lane] = h;
        s.lo[lane] = (float)(L - (double)h);
        s.e[lane] = exp2_(h);
        s.d[lane] = exp2_((float)(end - L));
        s.col[lane] = mul * exp2_((float)(m - L));
#pragma unroll
        for (int i = 0; i < C / 16 - 1; ++i)
            s.row[i][lane] = lane >= 16 * i + 16 ? exp2_((float)(L - mid[i])) : 0.f;
        s.row[C / 16 - 1][lane] = 0.f;
        if (lane == C - 1) s.g = exp2_((float)end);
    }
}
template <int C>
__device__ __forceinline__ void gate_scan(Decay<C> &s, float x, bool ok, int form, int lane,
                                          float mul = 1.f)
{
    gate_decays<C>(s, gate_sum<C>(x, ok, form), lane, mul);
}

// Scores of a tile times e^(L_t - L_s), zero where s > t.  Rows s = 16ct + 4g + j
// and columns t = 16rt + l16 (on the diagonal where ct == rt):
template <int C>
__device__ __forceinline__ f4 decayed_st(const Decay<C> &s, f4 x, int rt, int ct, int l16, int g4)
{
    const int t = 16 * rt + l16;
    if (ct < rt) return x * *reinterpret_cast<const f4 *>(&s.col[16 * ct + g4]) * s.row[ct][t];
    const f4 hi = *reinterpret_cast<const f4 *>(&s.hi[16 * ct + g4]);
    const f4 lo = *reinterpret_cast<const f4 *>(&s.lo[16 * ct + g4]);
    const float ht = s.hi[t], lt = s.lo[t];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x[j] = g4 + j <= l16 ? x[j] * exp2_((ht - hi[j]) + (lt - lo[j])) : 0.f;
    return x;
}
// The factors, times mul (Decay's own), of all tiles of a wavefront's 16
// tokens `own`, known at run time only: ST, tokens t = 16own + l16 are the
// columns and s the rows; otherwise the columns are s = 16own + l16 and the
// rows t.  Without a branch, to be read before the products they belong to.
template <bool ST, int C>
__device__ __forceinline__ void factors(const Decay<C> &s, f4 (&f)[C / 16], int own, float mul, int l16,
                                        int g4)
{
    const int me = 16 * own + l16;
    const float c = s.col[me], hm = s.hi[me], lm = s.lo[me];
    const f4 hi = *reinterpret_cast<const f4 *>(&s.hi[16 * own + g4]);
    const f4 lo = *reinterpret_cast<const f4 *>(&s.lo[16 * own + g4]);
#pragma unroll
    for (int i = 0; i < C / 16; ++i)
        f[i] = ST ? *reinterpret_cast<const f4 *>(&s.col[16 * i + g4]) * s.row[i][me]
                  : *reinterpret_cast<const f4 *>(&s.row[own][16 * i + g4]) * c;
    f4 d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = mul * exp2_(ST ? (hm - hi[j]) + (lm - lo[j]) : (hi[j] - hm) + (lo[j] - lm));
        d[j] = (ST ? g4 + j <= l16 : g4 + j >= l16) ? x : 0.f;
    }
#pragma unroll
    for (int i = 0; i < C / 16; ++i) f[i] = i == own ? d : f[i];
}
// Scores times their factors; zero on the wrong side of the diagonal, whatever
// the score.
template <bool ST, int RT>
__device__ __forceinline__ void apply(f4 (&p)[RT], const f4 (&f)[RT], int own, int l16, int g4)
{
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        if (ST ? i <= own : i >= own) {
            p[i] *= f[i];
            if (i == own)
#pragma unroll
                for (int j = 0; j < 4; ++j) p[i][j] = (ST ? g4 + j <= l16 : g4 + j >= l16) ? p[i][j] : 0.f;
        } else {
            p[i] = zf4();
        }
    }
}

// Running sum over the wavefront (the whole sum in its last lane).
__device__ __forceinline__ float scan64(float x)
{
    x += dpp<0x111>(x);
    x += dpp<0x112>(x);
    x += dpp<0x114>(x);
    x += dpp<0x118>(x);
    x += dpp<0x142, 0xa>(x);
    x += dpp<0x143, 0xc>(x);
    return x;
}

// Running sum over groups of 16 lanes.
__device__ __forceinline__ float scan16(float x)
{
    x += dpp<0x111>(x);
    x += dpp<0x112>(x);
    x += dpp<0x114>(x);
    x += dpp<0x118>(x);
    return x;
}

// The sums of v[i] over a group of 16 lanes, that of v[i] in lane i (eight
// values: in i and i + 8): lanes eight apart exchange the halves they do not
// keep, then mirrored ones of eight, then those two apart, then neighbours.
template <int N>
__device__ __forceinline__ float sums_to_lanes(float (&v)[N], int lane)
{
    auto halve = [&](auto ctrl, auto half, int bit) {
        constexpr int M = decltype(half)::value;
        const bool up = lane & bit;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float keep = up ? v[i + M] : v[i], give = up ? v[i] : v[i + M];
            v[i] = keep + dpp<decltype(ctrl)::value>(give);
        }
    };
    if constexpr (N == 16) {
        halve(std::integral_constant<int, 0x128>(), std::integral_constant<int, 8>(), 8);
    } else {
        static_assert(N == 8);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += dpp<0x128>(v[i]);
    }
    halve(std::integral_constant<int, 0x141>(), std::integral_constant<int, 4>(), 4);
    halve(std::integral_constant<int, 0x4e>(), std::integral_constant<int, 2>(), 2);
    halve(std::integral_constant<int, 0xb1>(), std::integral_constant<int, 1>(), 1);
    return v[0];
}

// y[i] += A(i, k) b[k], the operands A of step k + 1 requested before the
// products of step k; those of a step do not wait for each other.
template <int N, int K, class F, class LD>
__device__ __forceinline__ void mma_group(f4 (&y)[N], const F (&b)[K], LD ld)
{
    F x[2][N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[0][i] = ld(i, 0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (k + 1 < K)
#pragma unroll
            for (int i = 0; i < N; ++i) x[(k + 1) & 1][i] = ld(i, k + 1);
        GSCAN_STEP();
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = mma(x[k & 1][i], b[k], y[i]);
    }
}

// The exponent e of the wavefront's largest finite |st| (below 2^e), not below -100.
template <int N>
__device__ __forceinline__ int exponent_of(const f4 (&st)[N])
{
    auto largest = [&](auto part) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fmaxf(m, part(fabsf(st[i][j])));  // (NaN is passed over)
        m = fmaxf(m, dpp<0xb1>(m));
        m = fmaxf(m, dpp<0x4e>(m));
        m = fmaxf(m, dpp<0x141>(m));
        m = fmaxf(m, dpp<0x140>(m));
        auto row = [&](int i) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(m), i)); };
        return fmaxf(fmaxf(row(0), row(16)), fmaxf(row(32), row(48)));
    };
    float m = largest([](float x) { return x; });
    if (m == __builtin_inff()) m = largest([](float x) { return x < __builtin_inff() ? x : 0.f; });
    const int e = __builtin_amdgcn_frexp_expf(m);
    return first_lane(e < -100 ? -100 : e);
}

// st = g st + mul X^T (m . y) of a staged tile X: y is an operand of 16 columns of
// the chunk, m a factor per token.  Accumulators in turn, so that products
// which follow each other do not wait for each other.
template <class T, int NX, class TX, class F>
__device__ __forceinline__ void add_decayed(f4 (&st)[2 * NX], const F (&y)[T::C / 32], const float *m,
                                            float mul, float g, const TX &lx, const char *xt, int g4)
{
    constexpr int KS = T::C / 32;
    typename PartsOf<T>::type ys[KS];
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        f4 a, b;
        from_frag(y[kk], &a, &b);
        a *= mul * *reinterpret_cast<const f4 *>(&m[32 * kk + g4]);
        b *= mul * *reinterpret_cast<const f4 *>(&m[32 * kk + 16 + g4]);
        to_parts(a, b, &ys[kk]);
    }
#pragma unroll
    for (int i = 0; i < 2 * NX; ++i) st[i] *= g;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        F xf[2 * NX];
#pragma unroll
        for (int i = 0; i < 2 * NX; ++i) xf[i] = lx.col(xt, 32 * kk, i);
        mma_all(st, xf, ys[kk]);
    }
}

// --------------------------------------------------------------- forward

// One workgroup walks a unit's chunks for one head and 64 columns of its
// state.  What a chunk needs before its state is known does not wait for it:
// wavefronts 4-7 bring chunk n + 1 (its rows into LDS, its decays, then its
// scores) while wavefronts 0-3 finish chunk n (its outputs, then the state),
// two steps a chunk with a barrier after each; tiles and scores are kept
// twice, decays three times.  (All of it in turn by the same four wavefronts took 3 us a
// chunk, one workgroup per CU, most of it waiting.)  Workgroups that share
// queries and keys sit in one XCD (neighbours): 65 -> 61 us in the case below when it was added.
//
// Measured (bf16; times here and below are a profiler's means over 40 calls on
// the same inputs): 8 sequences of 2048 tokens, 16 heads of 64 x 128, one walk per
// CU: 57 us, 3.6 TB/s of the 206 MB to be moved; a chunk takes 3100 cycles (keys
// of 128: 4500), and 18000 pass before a walk's first (its loads, of all CUs at
// once, come at the memory's rate).  The two steps of a chunk are bound about
// equally by the bringing side (rows into LDS 700 to 1100 cycles, requests 300 to
// 1700, scores 1500 to 2400) and the finishing side (outputs 1250 to 2400, state
// 1500 to 2000); LDS is busy 38 per cent of the time, the matrix units 19.
// One workgroup per CU fits: 154 registers at keys of 64 (73 KB of LDS would leave
// room for two), 248 and 106 KB at keys of 128.  fp32: 16x16x4 products are half of
// a chunk's time; every slice of 64 value columns stages queries and keys and forms
// the scores again.
//
// Wavefront w < 4 keeps columns 16w .. 16w+15 of every row of the state in
// accumulators, which are operands of S^T Q^T as they are.  The ten (three)
// tiles of scores K Q^T on and below the diagonal are shared out to the other
// four; in that order a tile's accumulators are operands of V^T P^T, so they
// pass through LDS as they are, sixteen bytes per lane.  Outputs are formed
// transposed, four columns of a token per lane, stored as they are.
template <class T, int NK>
__global__ void __launch_bounds__(2 * kSThreads, 2)
gscan_state_fwd_kernel(StateArgs a, int slices, int64_t per, size_t st_part)
{
    typedef typename T::S S;
    typedef typename T::Frag Frag;
    typedef Rows<T, NK> TK;
    typedef Tile<T, kSlice> TV;
    constexpr int C = T::C, RT = C / 16, KS = C / 32;
    constexpr int kQ = 0, kK = C * TK::bytes, kV = 2 * C * TK::bytes, kBuf = kV + C * TV::bytes;
    // (the loads in flight are counted in order, so the chunks are walked in
    // pairs without a branch around either)
    __shared__ __align__(16) char tiles[2][kBuf];
    // operands of the scores: columns 16r .. of tokens 32kk .., at r + RT kk
    __shared__ Frag pts[2][RT * KS][64];
    __shared__ Decay<C> dcs[3];  // of chunk n - 1 (its state), n (its scores), n + 1 (being formed)
    __shared__ int bad[2], first[2][kSlice];
    constexpr int GW = 3;  // the wavefront (of its four) that forms the decays

    const int tid = threadIdx.x & (kSThreads - 1), lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool brings = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0;
    const int l16 = lane & 15, g4 = 4 * (lane >> 4);
    const uint32_t block = neighbours(slices * (a.H / a.Hk));
    const int slice = block % slices, h = block / slices % a.H;
    const int64_t unit = block / slices / a.H;
    Unit un;
    if (!find_unit(a, unit, per, C, lane, &un)) return;
    const int c0 = slice * kSlice, vcols = a.Dv - c0;
    const int tb = (int)(un.part * per);
    const int te = un.len - tb > per ? (int)(tb + per) : un.len;
    const int nc = (te - tb + C - 1) / C;
    const TK lk(lane);
    if (threadIdx.x < 2) bad[threadIdx.x] = 0;
    if (threadIdx.x < 2 * kSlice) first[0][threadIdx.x] = C;
    __syncthreads();

    if (brings) {
        const int hk = h / (a.H / a.Hk);
        // rows are requested two chunks ahead, into two sets of registers
        Stage<T, NK> sq, sk;
        Stage<T, 2> sv;
        u4 rq[2][NK], rk[2][NK], rv[2][2];
        Gates gates;
        Gates::Raw gx[2];
        gates.begin(a, un, h, tb, C, lane);
        sq.begin(row_at<S>(a.q, a.qs, un, hk, tb), a.qs.t, a.Dk, tid);
        sk.begin(row_at<S>(a.k, a.ks, un, hk, tb), a.ks.t, a.Dk, tid);
        sv.begin(row_at<S>(a.v, a.vs, un, h, tb) + c0, a.vs.t, vcols, tid);
        auto request = [&](int t0, auto set) {
            constexpr int O = decltype(set)::value;
            sq.load(rq[O], te - t0, (int64_t)(C * a.qs.t), tid);
            sk.load(rk[O], te - t0, (int64_t)(C * a.ks.t), tid);
            sv.load(rv[O], te - t0, (int64_t)(C * a.vs.t), tid);
            gx[O] = gates.load(te - t0, lane, 1);
        };
        request(tb, std::integral_constant<int, 0>());
        request(tb + C, std::integral_constant<int, 1>());
        auto bring = [&](int n, auto set) {
            constexpr int odd = decltype(set)::value;
            const int t0 = tb + n * C;
            char *tile = tiles[odd];
            const Decay<C> &dc = dcs[n % 3];
            sq.template store<TK>(rq[odd], tile + kQ, tid);
            sk.template store<TK>(rk[odd], tile + kK, tid);
            sv.template store<TV>(rv[odd], tile + kV, tid);
            sv.template scrub<TV>(rv[odd], tile + kV, tid, [&](int row, int c) {
                atomicMin(&first[odd][c], row);
                bad[odd] = 1;
            });
            request(t0 + 2 * C, set);
            __syncthreads();
            // scores of columns 16r .. with tokens 32kk ..
            auto score = [&](auto rc, auto kc) {
                constexpr int r = decltype(rc)::value, kk = decltype(kc)::value;
                f4 p[2] = {zf4(), zf4()};
                Frag qf[NK], kf[2][NK], f;
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    qf[k] = lk.row(tile + kQ, 16 * r, k);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (2 * kk + i <= r) kf[i][k] = lk.row(tile + kK, 32 * kk + 16 * i, k);
                }
#pragma unroll
                for (int k = 0; k < NK; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (2 * kk + i <= r) p[i] = mma(kf[i][k], qf[k], p[i]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (2 * kk + i <= r) p[i] = decayed_st(dc, p[i], r, 2 * kk + i, l16, g4);
                to_frag(p[0], p[1], &f);
                pts[odd][r + RT * kk][lane] = f;
            };
            using I0 = std::integral_constant<int, 0>;
            using I1 = std::integral_constant<int, 1>;
            using I2 = std::integral_constant<int, 2>;
            using I3 = std::integral_constant<int, 3>;
            if (w == GW) {
                gate_scan<C>(dcs[(n + 1) % 3], Gates::value(gx[odd ^ 1], a), t0 + C + lane < te, a.gate_form, lane);
            } else if constexpr (RT == 4) {
                if (w == 0) {
                    score(I0(), I0());
                    score(I1(), I0());
                } else if (w == 1) {
                    score(I2(), I0());
                    score(I2(), I1());
                } else {
                    score(I3(), I0());
                    score(I3(), I1());
                }
            } else {
                if (w == 0) score(I0(), I0());
                else if (w == 1) score(I1(), I0());
            }
            __syncthreads();
        };
        if (w == GW) gate_scan<C>(dcs[0], Gates::value(gx[0], a), tb + lane < te, a.gate_form, lane);
        for (int n = 0; n < nc; n += 2) {
            bring(n, std::integral_constant<int, 0>());
            bring(n + 1, std::integral_constant<int, 1>());  // past the end: empty rows
        }
        __syncthreads();
        __syncthreads();
        return;
    }

    // the state: row 16i + 4g + j of column `col` of the slice
    const int col = w * 16 + l16;
    const int64_t srow = ((int64_t)un.seq * a.H + h) * a.Dk;
    const float *init = a.s0 ? a.s0 + srow * a.Dv : nullptr;
    // A divided sequence begins from the workspace in its first part too, where the
    // join has put the initial state: its last part, another workgroup of this
    // launch, may write the final state over that one.
    if (un.parts > 1)
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
    const uint32_t vcol = TV(lane).col_off(w);
    // outputs: token 16r + l16, columns 16w + 4g .. +3
    const S *op = reinterpret_cast<const S *>(a.out) + (un.tok0 + tb) * a.H * a.Dv;
    const uint32_t ost = (uint32_t)(a.H * a.Dv * sizeof(S));
    const uint32_t o0 = 16 * w + g4 < vcols
        ? (uint32_t)(h * a.Dv + c0 + 16 * w + g4) * (uint32_t)sizeof(S) + l16 * ost : kNowhere;
    __syncthreads();
    __syncthreads();
    for (int n = 0; n < (nc + 1) / 2 * 2; ++n) {
        if (n == nc) {  // an empty chunk
            __syncthreads();
            __syncthreads();
            break;
        }
        const int t0 = tb + n * C, odd = n & 1;
        const char *tile = tiles[odd];
        const Decay<C> &dc = dcs[n % 3];
        const bool nan = bad[odd] != 0;
        const bool gone = first[odd][col] < C;
        Frag vf[KS];
        {
            const __amdgpu_buffer_rsrc_t ob = buffer(op);
            f4 x[RT], y[RT];
            Frag qf[2][RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                x[r] = y[r] = zf4();
                qf[0][r] = lk.row(tile + kQ, 16 * r, 0);
            }
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) vf[kk] = TV(lane).at_col(tile + kV, 32 * kk, vcol);
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) {
                Frag sf;
                to_frag(st[2 * kk], st[2 * kk + 1], &sf);
                if (kk + 1 < NK)
#pragma unroll
                    for (int r = 0; r < RT; ++r) qf[(kk + 1) & 1][r] = lk.row(tile + kQ, 16 * r, kk + 1);
#pragma unroll
                for (int r = 0; r < RT; ++r) x[r] = mma(sf, qf[kk & 1][r], x[r]);
            }
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                for (int r = 2 * kk; r < RT; ++r) y[r] = mma(vf[kk], pts[odd][r + RT * kk][lane], y[r]);
#pragma unroll
            for (int r = 0; r < RT; ++r)
                store4(ob, t0 + 16 * r + l16 < te && o0 != kNowhere ? o0 + 16 * r * ost : kNowhere,
                       a.scale * (dc.e[16 * r + l16] * x[r] + y[r]), T());
        }
        if (nan) {
            for (int r = 0; r < RT; ++r)
                for (int j = 0; j < 4; ++j)
                    if (t0 + 16 * r + l16 < te && 16 * w + g4 + j < vcols &&
                        16 * r + l16 >= first[odd][16 * w + g4 + j])
                        put1(const_cast<S *>(op) + (int64_t)(16 * r + l16) * a.H * a.Dv + h * a.Dv + c0 +
                                 16 * w + g4 + j, __builtin_nanf(""));
        }
        op += (int64_t)C * a.H * a.Dv;
        __syncthreads();
        // S' = e^(L_end) S + K^T (e^(L_end - L) V)
        add_decayed<T, NK>(st, vf, dc.d, 1.f, dc.g, lk, tile + kK, g4);
        if (nan) {
            if (gone)
#pragma unroll
                for (int i = 0; i < 2 * NK; ++i) st[i] = zf4() + __builtin_nanf("");
            first[odd][col] = C;
            if (tid == 0) bad[odd] = 0;
        }
        __syncthreads();
    }

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
    float *down;         // bf16: what the operands of a column tile are to be multiplied by,
                         // [chunk slot][H][2][2 NY], the state's and its gradient's
};

// Wavefronts 4-7 bring the next chunk's rows and decays into LDS while
// wavefronts 0-3 add this one's, one barrier a chunk.  Measured (bf16): the two
// walks of 8 x 2048 tokens, 16 heads of 64 x 128, move 344 MB (134 of it the
// stored states) in 67 us, 5.1 TB/s, which is all there is; without storing,
// 32771 tokens of 16 heads of 128 x 64 in 256 walks take 43 us, 1.3 us a chunk,
// bound by the products (three bf16 parts) and the chain of the decays.  The decays, a long chain
// of short steps, are formed by the last two in turn, each over two chunks: the
// sum of log gates in one, the exponentials in the next.
template <class T, int NX>
struct PassLds {
    static constexpr int kX = T::C * Rows<T, NX>::bytes, kBuf = kX + T::C * Tile<T, kSlice>::bytes;
    char tile[2][kBuf];
};

template <class T, int NX, bool REV, bool STORE>
__device__ __forceinline__ void pass_walk(const StateArgs &a, const PassJob &jb, int ny, int slice,
                                          int h, const Unit &un, int tb, int te, void *smem,
                                          Decay<T::C> (&dcs)[2])
{
    typedef typename T::S S;
    typedef typename T::Frag Frag;
    typedef Rows<T, NX> TX;
    typedef Tile<T, kSlice> TY;
    typedef PassLds<T, NX> Lds;
    constexpr int C = T::C, KS = C / 32, step = REV ? -1 : 1;
    Lds &lds = *reinterpret_cast<Lds *>(smem);
    const int tid = threadIdx.x & (kSThreads - 1), lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool brings = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0;
    const int l16 = lane & 15, g4 = 4 * (lane >> 4);
    const int c0 = slice * kSlice, ycols = jb.yd - c0;
    const int cb = tb / C, nc = te > tb ? (te + C - 1) / C - cb : 1;  // chunks, at least one
    const int c1 = REV ? cb + nc - 1 : cb;                           // the first walked

    if (brings) {
        Stage<T, NX> sx;
        Stage<T, 2> sy;
        Gates gates;
        u4 rx[2][NX], ry[2][2];
        Gates::Raw gx[2];
        sx.begin(row_at<S>(jb.x, jb.xs, un, jb.xh, c1 * C), jb.xs.t, jb.xd, tid);
        sy.begin(row_at<S>(jb.y, jb.ys, un, jb.yh, c1 * C) + c0, jb.ys.t, ycols, tid);
        gates.begin(a, un, h, c1 * C, C, lane);
        // chunks past the end (in either direction) have no rows
        auto request = [&](int n, auto set) {
            constexpr int O = decltype(set)::value;
            const int left = n < nc ? te - (c1 + step * n) * C : 0;
            sx.load(rx[O], left, step * (int64_t)(C * jb.xs.t), tid);
            sy.load(ry[O], left, step * (int64_t)(C * jb.ys.t), tid);
            gx[O] = gates.load(left, lane, step);
        };
        double sum = 0.0;
        auto sum_gates = [&](int n, auto set) {
            sum = gate_sum<C>(Gates::value(gx[decltype(set)::value], a), lane < te - (c1 + step * n) * C,
                              a.gate_form);
        };
        auto bring = [&](int n, auto set) {
            constexpr int odd = decltype(set)::value;
            sx.template store<TX>(rx[odd], lds.tile[odd], tid);
            sy.template store<TY>(ry[odd], lds.tile[odd] + Lds::kX, tid);
            if (w == 2 + odd) gate_decays<C>(dcs[odd], sum, lane);
            if (w == 3 - odd) sum_gates(n + 1, std::integral_constant<int, odd ^ 1>());
            request(n + 2, set);
            __syncthreads();
        };
        request(0, std::integral_constant<int, 0>());
        request(1, std::integral_constant<int, 1>());
        if (w == 2) sum_gates(0, std::integral_constant<int, 0>());
        for (int n = 0; n < nc; n += 2) {
            bring(n, std::integral_constant<int, 0>());
            bring(n + 1, std::integral_constant<int, 1>());
        }
        return;
    }

    const int col = 16 * w + l16, sb = (c0 + col) * jb.cstr;
    const TX lx(lane);
    const uint32_t ycol = TY(lane).col_off(w);
    f4 st[2 * NX];
#pragma unroll
    for (int i = 0; i < 2 * NX; ++i) {
        st[i] = zf4();
        if (jb.init && col < ycols)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (16 * i + g4 + j < jb.xd) st[i][j] = jb.init[sb + (16 * i + g4 + j) * jb.rstr];
    }
    float gall = 1.f;
    for (int n = 0; n < (nc + 1) / 2 * 2; ++n) {
        __syncthreads();
        if (n == nc) break;  // the empty chunk of the last pair
        const int odd = n & 1;
        const Decay<C> &dc = dcs[odd];
        if constexpr (STORE) {  // the operands of this chunk, before its own tokens enter
            const int64_t tile = ((int64_t)(un.slot0 + c1 + step * n) * a.H + h) * 2 * ny + slice * 4 + w;
            float up = 1.f;
            if constexpr (sizeof(S) == 2) {
                const int e = exponent_of(st);
                up = ldexpf(1.f, 14 - e);
                const int64_t item = (int64_t)(un.slot0 + c1 + step * n) * a.H + h;
                if (lane == 0) jb.down[(2 * item + REV) * 2 * ny + slice * 4 + w] = ldexpf(1.f, e - 14);
            }
#pragma unroll
            for (int kk = 0; kk < NX; ++kk)
                put_state(jb.dst, tile * NX + kk, lane, st[2 * kk], st[2 * kk + 1], up, T());
        }
        Frag yf[KS];
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) yf[kk] = TY(lane).at_col(lds.tile[odd] + Lds::kX, 32 * kk, ycol);
        gall *= dc.g;
        add_decayed<T, NX>(st, yf, REV ? dc.e : dc.d, jb.mul, dc.g, lx, lds.tile[odd], g4);
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

// Units of split sequences, by themselves: what a unit adds to the state after
// it and, in the backward (ways == 2), to the gradient of the state before it;
// and the product of its gates.  fp32 [units][H][Dk][Dv] and [units][H].
struct Parts2 {
    size_t st[2], dec[2];  // workspace offsets, forwards and backwards
};

template <class T, int NK>
__global__ void __launch_bounds__(2 * kSThreads, 2)
gscan_state_part_kernel(StateArgs a, int slices, int ways, int64_t per, Parts2 o)
{
    __shared__ __align__(16) PassLds<T, NK> smem;
    __shared__ Decay<T::C> dcs[2];
    const uint32_t block = neighbours(slices * ways * (a.H / a.Hk));
    const int lane = threadIdx.x & 63, slice = block % slices, way = block / slices % ways;
    const int64_t b = block / slices / ways;
    const int h = (int)(b % a.H), hk = h / (a.H / a.Hk);
    const int64_t unit = b / a.H;
    Unit un;
    if (!find_unit(a, unit, per, T::C, lane, &un)) return;
    if (un.part == (way ? 0 : un.parts - 1)) return;  // nothing comes after it
    const int tb = (int)(un.part * per);
    const int te = un.len - tb > per ? (int)(tb + per) : un.len;
    char *ws = reinterpret_cast<char *>(a.ws);
    float *fin = reinterpret_cast<float *>(ws + o.st[way]) + (unit * a.H + h) * a.Dk * a.Dv;
    float *dec = reinterpret_cast<float *>(ws + o.dec[way]) + unit * a.H + h;
    if (!way) {
        const PassJob jb = {a.k, a.v, a.ks, a.vs, hk, h, a.Dk, a.Dv, nullptr, fin, dec, a.Dv, 1, nullptr, 1.f,
                            nullptr};
        pass_walk<T, NK, false, false>(a, jb, 0, slice, h, un, tb, te, &smem, dcs);
    } else {
        const PassJob jb = {a.q, a.dout, a.qs, a.ds, hk, h, a.Dk, a.Dv, nullptr, fin, dec, a.Dv, 1, nullptr,
                            a.scale, nullptr};
        pass_walk<T, NK, true, false>(a, jb, 0, slice, h, un, tb, te, &smem, dcs);
    }
}

// Joins the units of split sequences: in place, what each adds becomes the
// state it begins with (backwards: the gradient of the state it ends with).
// Four elements per thread, the units of a sequence in turn, eight requested at a
// time: 5.8 us for 16 units of 16 heads of 128 x 64 (16 MB), most of it latency.
__global__ void __launch_bounds__(kSThreads)
gscan_state_join_kernel(StateArgs a, int ways, int64_t per, Parts2 o)
{
    const int n4 = a.Dk * a.Dv / 4, blocks = (n4 + kSThreads - 1) / kSThreads;
    const int part = blockIdx.x % blocks, way = blockIdx.x / blocks % ways;
    const int h = blockIdx.x / blocks / ways % a.H, seq = blockIdx.x / blocks / ways / a.H;
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
    f4 *p = reinterpret_cast<f4 *>(ws + o.st[way]) + (u0 * a.H + h) * n4 + i4;
    const float *dec = reinterpret_cast<const float *>(ws + o.dec[way]) + u0 * a.H + h;
    const int64_t ps = (int64_t)a.H * n4;
    const float *from = way ? a.dsT : a.s0;
    f4 st = from ? reinterpret_cast<const f4 *>(from)[((int64_t)seq * a.H + h) * n4 + i4] : zf4();
    constexpr int B = 8;  // units in flight
    for (int b = 0; b < n; b += B) {
        f4 x[B];
        float g[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int i = way ? n - 1 - b - j : b + j;
            if (b + j < n - 1) {
                x[j] = p[i * ps];
                g[j] = dec[(int64_t)i * a.H];
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int i = way ? n - 1 - b - j : b + j;
            if (b + j < n) {
                p[i * ps] = st;
                if (b + j < n - 1) st = g[j] * st + x[j];
            }
        }
    }
}

// Two walks per unit and head that leave operands for every chunk: the state
// before it and the gradient of the state after it, both with the columns of
// S^T: operand (n, kk) holds columns (keys) 16n .. and rows (values) 32kk ...
struct PassWs {
    size_t s, ds;  // operands
    size_t down;   // bf16: the factors of their column tiles
    Parts2 parts;  // units' states and gradients of states (split sequences)
};

template <class T, int NK, int NV>
__global__ void __launch_bounds__(2 * kSThreads, 2)
gscan_state_pass_kernel(StateArgs a, int64_t per, PassWs o)
{
    __shared__ __align__(16) PassLds<T, NV> smem;
    __shared__ Decay<T::C> dcs[2];
    constexpr int slices = NK / 2;
    const uint32_t block = neighbours(slices * 2 * (a.H / a.Hk));
    const int lane = threadIdx.x & 63, slice = block % slices, way = block / slices & 1;
    const int64_t b = block / slices / 2;
    const int h = (int)(b % a.H), hk = h / (a.H / a.Hk);
    const int64_t unit = b / a.H;
    Unit un;
    if (!find_unit(a, unit, per, T::C, lane, &un)) return;
    const int tb = (int)(un.part * per);
    const int te = un.len - tb > per ? (int)(tb + per) : un.len;
    char *ws = reinterpret_cast<char *>(a.ws);
    const int64_t one = (int64_t)a.Dk * a.Dv, whole = ((int64_t)un.seq * a.H + h) * one;
    const bool outer = un.part == (way ? un.parts - 1 : 0);  // begins with the caller's
    const float *from = way ? a.dsT : a.s0;
    const float *init = !outer ? reinterpret_cast<const float *>(ws + o.parts.st[way]) + (unit * a.H + h) * one
                               : from ? from + whole : nullptr;
    if (!way) {
        const PassJob jb = {a.v, a.k, a.vs, a.ks, h, hk, a.Dv, a.Dk, init, nullptr, nullptr, 1, a.Dv,
                            ws + o.s, 1.f, reinterpret_cast<float *>(ws + o.down)};
        pass_walk<T, NV, false, true>(a, jb, NK, slice, h, un, tb, te, &smem, dcs);
    } else {
        const PassJob jb = {a.dout, a.q, a.ds, a.qs, h, hk, a.Dv, a.Dk, init,
                            a.ds0 && un.part == 0 ? a.ds0 + whole : nullptr, nullptr, 1, a.Dv,
                            ws + o.ds, a.scale, reinterpret_cast<float *>(ws + o.down)};
        pass_walk<T, NV, true, true>(a, jb, NK, slice, h, un, tb, te, &smem, dcs);
    }
}

// ---------------------------------------------------- backward: gradients

// The operands of a state in LDS: operand (n, kk) at 64 (n NV + kk) lanes of
// sixteen bytes (fp32: two planes), read as they are or, four keys of a value,
// transposed.
template <class T, int NV>
struct States;

template <int NV>
struct States<BF, NV> {
    // keys 16n + l16, values 32kk + {4g.., 16 + 4g..}
    static __device__ __forceinline__ u4 get(const u4 *t, int n, int kk, int lane)
    {
        return t[(n * NV + kk) * 64 + lane];
    }
    // value 16m + l16, keys 32kk + {4g.., 16 + 4g..}
    static __device__ __forceinline__ u4 turned(const u4 *t, int m, int kk, int lane)
    {
        const uint32_t l16 = lane & 15, g = lane >> 4;
        const char *p = reinterpret_cast<const char *>(t) + (2 * kk * NV + m / 2) * 1024 + (m & 1) * 8 +
                        ((l16 & 3) * 16 + 4 * g + (l16 >> 2)) * 16;
        const uint2 x = Tile<BF, 64>::tr(p), y = Tile<BF, 64>::tr(p + NV * 1024);
        return u4{x.x, x.y, y.x, y.y};
    }
};
template <int NV>
struct States<FP, NV> {
    static __device__ __forceinline__ FP::Frag get(const u4 *t, int n, int kk, int lane)
    {
        const f4 *p = reinterpret_cast<const f4 *>(t) + (n * NV + kk) * 128 + lane;
        return FP::Frag{p[0], p[64]};
    }
    static __device__ __forceinline__ FP::Frag turned(const u4 *t, int m, int kk, int lane)
    {
        const uint32_t l16 = lane & 15, g = lane >> 4;
        const float *p = reinterpret_cast<const float *>(t) + (2 * kk * NV + m / 2) * 512 + (m & 1) * 256 + (l16 & 3);
        FP::Frag f;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t at = ((l16 >> 2) * 16 + 4 * g + j) * 4;
            f.a[j] = p[at];
            f.b[j] = p[at + NV * 512];
        }
        return f;
    }
};

// Of stored states (fp32 sums of exact products).
__device__ __forceinline__ float dot16(const u4 &x, const u4 &y, const BF &)
{
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = x[i], v = y[i];
        s = __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, u), __builtin_bit_cast(h2, v), s, false);
    }
    return s;
}
__device__ __forceinline__ float dot16(const u4 &x, const u4 &y, const FP &)
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += __uint_as_float(x[i]) * __uint_as_float(y[i]);
    return s;
}

// Workgroups (one per CU, its registers full) take chunks of a key head in
// turn: its queries and keys stay in LDS while the value heads that share
// them are taken one by one, so dQ and dK of shared heads are summed in
// registers in a fixed order.  The rows and state operands of the next head,
// or of the next chunk's first, are requested while this one is computed
// (one workgroup per chunk, which waits for its own, took 192 us where this
// took 125 at its fastest).
//
// Measured (bf16): 8 x 2048 tokens, 16 heads of 64 x 128: 144 us (the fastest call:
// 125) for 481 MB (by the counters), 3.3 TB/s (a large copy: 4.8); 15233 tokens, 16
// heads of 128 x 64 on 4 key heads: 116 us for 289 MB.  Where chunks times key heads
// are few, CUs idle: one sequence of 2048, 16 heads of 64 x 64 takes 18 us on 16 key
// heads, 24 on 4 and 72 on one, whose 32 workgroups take 16 heads in turn.  Of the
// scores, dO V^T is formed by the query and by the key wavefronts, and all three
// products in all 16 tiles of 16 x 16 (ten are on or below the diagonal).  100 to 114
// scalar registers live in lanes of vector ones.  An item (a chunk of a
// head) takes about 13000 cycles: into LDS 1700, scores 6000 (key wavefronts;
// the others form dQ and dV's part of the state meanwhile), requests 1000 to 2000
// (as fast as the memory takes them), dK or dV 2400.  LDS moves 620 KB in it and
// is busy 36 to 39 per cent of the time, the matrix units 12.
//
// Eight wavefronts: `rt` owns token rows 16rt .. 16rt+15, half of them dQ and
// half dK, each half of dV (and, fp32 with its two rows of tiles, each every
// other column tile).  A wavefront forms the scores it needs itself, in the
// order whose accumulators are operands: dO V^T of its tokens with the tokens
// before them (for dQ), Q K^T and dO V^T of its tokens with those after them
// (for dV and dK).  Gradients are formed transposed, four columns of a token
// per lane.
constexpr int kGThreads = 512;
constexpr int kCus = 256;

template <class T, int NK, int NV>
__global__ void __launch_bounds__(kGThreads, 2)
gscan_state_grad_kernel(StateArgs a, uint32_t units, uint32_t per, PassWs o)
{
    typedef typename T::S S;
    typedef typename T::Frag Frag;
    typedef Tile<T, NK * 32> TK;
    typedef Tile<T, NV * 32> TV;
    typedef States<T, NV> ST;
    constexpr int C = T::C, RT = C / 16, KS = C / 32;
    constexpr int CH = 8 / (2 * RT);                // column halves
    constexpr int NTK = 2 * NK / CH;                // column tiles of dQ, dK per wavefront
    constexpr int G = sizeof(Frag) == 16 && NK * NV < 16 ? 4 : 2;  // of them at a time
    constexpr int kOps = 2 * NK * NV * (int)sizeof(Frag) / 16 * 64;  // 16-byte pieces of a state
    constexpr int NS = kOps / kGThreads;
    __shared__ __align__(16) char qt[C * TK::bytes], kt[C * TK::bytes], vt[C * TV::bytes], ot[C * TV::bytes];
    // the state before the chunk and the gradient of the one after it, side by
    // side where LDS holds both (all but fp32 at the full widths, where the second
    // takes the first one's place between the two steps)
    constexpr bool both = sizeof(Frag) == 16 || NK * NV < 16;
    __shared__ u4 state[kOps], second[both ? kOps : 1];
    const u4 *after = both ? second : state;
    __shared__ Frag scores[RT][KS][64];  // P . D of a tile row's keys, for dV
    __shared__ Decay<C> dcs[2];
    // sums for the gates' gradients, which are finished beside the next item
    struct Sums {
        float row[C][RT], inner[C], a[CH][C], b[CH][C], f[8];
    };
    __shared__ Sums sums[2];
    // what infinities and NaN reach: per column the first row of k and the last
    // of q and d_out that hold one, which rows of k and d_out do, and the last
    // row of q, of d_out, the first of k
    __shared__ int first_k[NK * 32], last_q[NK * 32], last_o[NV * 32], row_k[C], row_o[C], ends[3], bad;

    int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    int l16 = lane & 15, g4 = 4 * (lane >> 4);
    const int rt = w % RT, ch = CH == 1 ? 0 : w / (2 * RT);
    const bool keys = (w / RT) & 1;
    const int reps = a.H / a.Hk;
    const char *ws = reinterpret_cast<const char *>(a.ws);
    const TK lk(lane);
    const TV lv(lane);

    const uint32_t last = (blockIdx.x + 1) * per < units ? (blockIdx.x + 1) * per : units;

    // what is computed: value head `h` of chunk `slot`, and where its tokens are
    struct Item {
        Unit un;
        uint32_t u;  // unit of the grid (chunk and key head)
        int slot, h, hk, t0, left;
    };
    // Lanes 0 .. 4 hold the strides of q, k, v, d_out and the gate and where the
    // sequence last found begins in each, so that an item's five addresses are
    // one computation.
    auto of_tensor = [&](auto q, auto k, auto v, auto o, auto g) {
        return lane == 0 ? q : lane == 1 ? k : lane == 2 ? v : lane == 3 ? o : g;
    };
    const uint32_t ts = of_tensor(a.qs.t, a.ks.t, a.vs.t, a.ds.t, a.gs.t);
    const uint32_t hs = of_tensor(a.qs.h, a.ks.h, a.vs.h, a.ds.h, a.gs.h);
    const int se = sizeof(S) == 2 ? 1 : 2, ge = a.gate_dtype ? 1 : 2;  // element bytes, as shifts
    uint64_t seq0 = 0;
    // the first item from unit u on; u >= last when there is none
    auto find = [&](uint32_t u, Item *it) {
        for (; u < last; ++u) {
            const uint32_t c = u / (uint32_t)a.Hk;
            if (!find_unit(a, c, C, C, lane, &it->un)) continue;
            it->t0 = it->un.part * C;
            it->left = it->un.len - it->t0;
            if (it->left <= 0) continue;  // a sequence without tokens
            it->slot = it->un.slot0 + it->un.part;
            it->hk = (int)(u - c * (uint32_t)a.Hk);
            it->h = it->hk * reps;
            const int64_t b = of_tensor(a.qs.b, a.ks.b, a.vs.b, a.ds.b, a.gs.b);
            const uint64_t p = reinterpret_cast<uint64_t>(of_tensor(a.q, a.k, a.v, a.dout, a.gate));
            seq0 = p + ((uint64_t)(it->un.seq * b + (int64_t)ts * it->un.in0) << (lane < 4 ? se : ge));
            break;
        }
        it->u = u;
    };
    // the one after it: another head, the next chunk, or to be found
    auto advance = [&](Item *it) {
        if (++it->u >= last) return;
        if (++it->hk == a.Hk) {
            it->hk = 0;
            it->t0 += C;
            it->left -= C;
            ++it->slot;
            if (it->left <= 0) return find(it->u, it);
        }
        it->h = it->hk * reps;
    };
    typedef Stage<T, NK, kGThreads> SK;
    typedef Stage<T, NV, kGThreads> SV;
    typename SK::Regs rq, rk;
    typename SV::Regs rv, ro;
    u4 rs[NS], rd[NS];
    uint32_t down = 0;
    // the factor of this thread's i-th piece of the state (of its gradient: from 2NK)
    const int w0 = w;
    auto factor = [&](int i, int from) {
        return __uint_as_float(__builtin_amdgcn_readlane(down, from + (w0 + kGThreads / 64 * i) / NV));
    };
    Gates::Raw gx;
    // requests of an item (`some`: there is one) without a branch, which would
    // wait for what it loads where it ends; `first`: its chunk's queries and keys
    auto request = [&](const Item &it, bool some, bool first) {
        const int rows = some ? it.left : 0, shared = first ? rows : 0;
        const uint64_t at = seq0 + (((uint64_t)hs * (uint32_t)(lane < 2 ? it.hk : it.h) +
                                     (uint64_t)ts * (uint32_t)it.t0) << (lane < 4 ? se : ge));
        auto base = [&](int i) {
            return buffer(reinterpret_cast<const void *>(
                (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(at >> 32), i) << 32 |
                (uint32_t)__builtin_amdgcn_readlane((uint32_t)at, i)));
        };
        auto step = [&](int i) { return (uint32_t)__builtin_amdgcn_readlane(ts, i); };
        SK::fetch(rq, base(0), step(0), a.Dk, shared, tid);
        SK::fetch(rk, base(1), step(1), a.Dk, shared, tid);
        SV::fetch(rv, base(2), step(2), a.Dv, rows, tid);
        SV::fetch(ro, base(3), step(3), a.Dv, rows, tid);
        const __amdgpu_buffer_rsrc_t g = base(4);
        const uint32_t og = __umul24(lane, step(4)) << ge;
        gx.x32 = __builtin_amdgcn_raw_buffer_load_b32(g, lane < rows && lane < C && ge == 2 ? og : kNowhere, 0, 0);
        gx.x16 = __builtin_amdgcn_raw_buffer_load_b16(g, lane < rows && lane < C && ge == 1 ? og : kNowhere, 0, 0);
    };
    auto request_states = [&](const Item &it, bool some) {
        const int64_t at = ((int64_t)it.slot * a.H + it.h) * kOps * 16;
        const __amdgpu_buffer_rsrc_t p = buffer(ws + o.s + at), q = buffer(ws + o.ds + at);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            rs[i] = __builtin_amdgcn_raw_buffer_load_b128(p, some ? (tid + kGThreads * i) * 16 : kNowhere, 0, 0);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            rd[i] = __builtin_amdgcn_raw_buffer_load_b128(q, some ? (tid + kGThreads * i) * 16 : kNowhere, 0, 0);
        if constexpr (sizeof(S) == 2) {  // lane n: of the state's tile n; 2NK + n: of its gradient's
            const __amdgpu_buffer_rsrc_t u = buffer(ws + o.down + ((int64_t)it.slot * a.H + it.h) * 4 * NK * 4);
            down = __builtin_amdgcn_raw_buffer_load_b32(u, some && lane < 4 * NK ? lane * 4 : kNowhere, 0, 0);
        }
    };
    auto keep = [&](const u4 (&r)[NS], u4 *to, int from) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int q = tid + kGThreads * i;
            to[q] = get_state(r[i], factor(i, from), T());
        }
    };
    auto clear = [&] {
        for (int i = tid; i < NK * 32; i += kGThreads) {
            first_k[i] = C;
            last_q[i] = -1;
        }
        if (tid < NV * 32) last_o[tid] = -1;
        if (tid < C) row_k[tid] = row_o[tid] = 0;
        if (tid < 3) ends[tid] = tid < 2 ? -1 : C;
        if (tid == 0) bad = 0;
        __syncthreads();
    };
    Item it;
    find(blockIdx.x * per, &it);
    if (it.u >= last) return;
    request(it, true, true);
    request_states(it, true);
    clear();
    // the decays of an item, beside the one before it
    auto gates_of = [&](const Item &i, int which) {
        gate_scan<C>(dcs[which], Gates::value(gx, a), lane < i.left, a.gate_form, lane, a.scale);
    };
    if (w == 1) gates_of(it, 0);
    f4 acc[NTK];  // dQ or dK of the wavefront's tokens
#pragma unroll
    for (int i = 0; i < NTK; ++i) acc[i] = zf4();

    // dlog g of an item's tokens, by one wavefront: x its gate arguments, reach
    // the tokens an infinity or NaN reaches (from the first, up to the last)
    auto finish = [&](const Item &done, int was, float x, float gall, int up_to, int from) {
        const Sums &q = sums[was];
        // suffix sums run over the tokens backwards, lane i at token C - 1 - i
        float su = 0.f, pb = 0.f, rw[RT];
        const int t = C - 1 - lane;
#pragma unroll
        for (int i = 0; i < RT; ++i) rw[i] = 0.f;
        if (lane < C) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                su += q.a[i][t];
                pb += q.b[i][lane];
            }
#pragma unroll
            for (int i = 0; i + 1 < RT; ++i)
                rw[i] = t >= 16 * i + 16 ? q.row[t][i] : 0.f;  // rows below the tile
        }
        su = scan64(su);
        pb = scan64(pb);
#pragma unroll
        for (int i = 0; i + 1 < RT; ++i) {
            const float r = scan64(rw[i]);
            if (t >= 16 * (i + 1)) su += r;
        }
        float F = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) F += q.f[i];
        F *= gall;
        const float before = __shfl_up(pb, 1);
        su = __shfl(su, C - 1 - lane);
        if (lane < C) su += q.inner[lane];
        if (lane < C && lane < done.left) {
            float r = (su + (lane ? before : 0.f) + F) * log_gate_slope(x, a.gate_form);
            if (lane <= up_to || lane > from) r = __builtin_nanf("");
            const int64_t at = (done.un.tok0 + done.t0 + lane) * a.H + done.h;
            if (a.gate_dtype) reinterpret_cast<uint16_t *>(a.dgate)[at] = to_bf16(r);
            else reinterpret_cast<float *>(a.dgate)[at] = r;
        }
    };
    Item done;
    bool later = false;
    float gdone = 0.f, gall = 0.f;
    int up_to = -1, from = C;
    for (int odd = 0;; odd ^= 1) {
        const Decay<C> &dc = dcs[odd];
        Sums &sm = sums[odd];
        // addresses and comparisons are formed anew, not kept across the loop
        // (there are more of them than registers)
        asm volatile("" : "+v"(tid), "+v"(lane), "+v"(l16), "+v"(g4));
        const int h = it.h;
        const bool mine = 16 * rt + l16 < it.left;  // this lane's token exists
        if (h == it.hk * reps) {
            SK::template store<TK>(rq, qt, tid);
            SK::template store<TK>(rk, kt, tid);
            SK::template scrub<TK>(rq, qt, tid, [&](int row, int c) {
                atomicMax(&last_q[c], row);
                atomicMax(&ends[0], row);
                bad = 1;
            });
            SK::template scrub<TK>(rk, kt, tid, [&](int row, int c) {
                atomicMin(&first_k[c], row);
                atomicMin(&ends[2], row);
                row_k[row] = 1;
                bad = 1;
            });
        }
        SV::template store<TV>(rv, vt, tid);
        SV::template store<TV>(ro, ot, tid);
        SV::template scrub<TV>(ro, ot, tid, [&](int row, int c) {
            atomicMax(&last_o[c], row);
            atomicMax(&ends[1], row);
            row_o[row] = 1;
            bad = 1;
        });
        keep(rs, state, 0);
        if constexpr (both) keep(rd, second, 2 * NK);
        float x = Gates::value(gx, a);
        asm volatile("" : "+v"(x));  // now: gx is about to be loaded again
        {  // F = e^(L_end) <S, dS>
            float f = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const float d = dot16(rs[i], rd[i], T());
                f += sizeof(S) == 2 ? d * (factor(i, 0) * factor(i, 2 * NK)) : d;
            }
            f = scan64(f);
            if (lane == 63) sm.f[w] = f;
        }
        Item next = it;
        const bool same = h + 1 < (it.hk + 1) * reps;  // another head of this chunk
        if (same) ++next.h;
        else advance(&next);
        const bool more = next.u < last;
        __syncthreads();
        const bool nan = bad != 0;
        request(next, more, !same);
        if (w == 0) {
            if (later) finish(done, odd ^ 1, gdone, gall, up_to, from);
            done = it;
            gdone = x;
            gall = dc.g;
            up_to = nan ? (ends[0] > ends[1] ? ends[0] : ends[1]) : -1;
            from = nan ? ends[2] : C;
        }
        later = true;

        Frag pf[KS], df[KS];
        if (!keys) {
            // dQ^T = K^T (dP . D)^T + scale e^L S dO^T
            Frag of[NV];
            f4 p[RT], fac[RT];
            factors<true>(dc, fac, rt, a.scale, l16, g4);
#pragma unroll
            for (int kk = 0; kk < NV; ++kk) of[kk] = lv.row(ot, 16 * rt, kk);
#pragma unroll
            for (int ct = 0; ct < RT; ++ct) p[ct] = zf4();
            mma_group(p, of, [&](int ct, int kk) { return lv.row(vt, 16 * ct, kk); });
            apply<true>(p, fac, rt, l16, g4);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) to_frag(p[2 * kk], p[2 * kk + 1], &df[kk]);
            const float e = a.scale * dc.e[16 * rt + l16];
            float as = 0.f;
#pragma unroll
            for (int i0 = 0; i0 < NTK; i0 += G) {
                f4 y[G];
#pragma unroll
                for (int i = 0; i < G; ++i) y[i] = zf4();
                mma_group(y, of, [&](int i, int kk) { return ST::get(state, (i0 + i) * CH + ch, kk, lane); });
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    y[i] *= e;
                    const f4 qv = lk.quad(qt, 16 * rt, (i0 + i) * CH + ch);
#pragma unroll
                    for (int j = 0; j < 4; ++j) as += y[i][j] * qv[j];
                    y[i] += acc[i0 + i];
                }
                mma_group(y, df, [&](int i, int kk) { return lk.col(kt, 32 * kk, (i0 + i) * CH + ch); });
#pragma unroll
                for (int i = 0; i < G; ++i) acc[i0 + i] = y[i];
            }
            if (nan)
#pragma unroll
                for (int i = 0; i < NTK; ++i)
                    acc[i] = poison<false>(acc[i], &first_k[16 * (i * CH + ch) + g4], 16 * rt + l16,
                                           row_o[16 * rt + l16]);
            as += __shfl_xor(as, 16);
            as += __shfl_xor(as, 32);
            if (lane < 16) sm.a[ch][16 * rt + lane] = as;
        } else {
            Frag kf[NK], vf[NV];
            f4 p[RT], y[RT], fac[RT];
            factors<false>(dc, fac, rt, a.scale, l16, g4);
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) kf[kk] = lk.row(kt, 16 * rt, kk);
#pragma unroll
            for (int kk = 0; kk < NV; ++kk) vf[kk] = lv.row(vt, 16 * rt, kk);
#pragma unroll
            for (int ut = 0; ut < RT; ++ut) p[ut] = y[ut] = zf4();
            mma_group(p, kf, [&](int ut, int kk) { return lk.row(qt, 16 * ut, kk); });
            mma_group(y, vf, [&](int ut, int kk) { return lv.row(ot, 16 * ut, kk); });
            apply<false>(p, fac, rt, l16, g4);
            // W below the diagonal: sums over s < t of the tile's columns, for u >= t
            if (ch == 0) {
                float v[4 * RT], below = 0.f, in = 0.f;
                f4 own = zf4();
#pragma unroll
                for (int ut = 0; ut < RT; ++ut) {
                    f4 x = zf4();
                    if (ut >= rt) x = p[ut] * y[ut];
                    if (ut > rt) below += (x[0] + x[1]) + (x[2] + x[3]);
                    if (ut == rt) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = g4 + j > l16 ? x[j] : 0.f;
                        own = x;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[4 * ut + j] = x[j];
                }
                const float row = sums_to_lanes(v, lane);
                if (l16 < 4 * RT) sm.row[16 * (l16 >> 2) + g4 + (l16 & 3)][rt] = row;
                in = dpp<0x111>(scan16(below));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float before = dpp<0x111>(scan16(own[j]));
                    in += g4 + j >= l16 ? before : 0.f;
                }
                in += __shfl_xor(in, 16);
                in += __shfl_xor(in, 32);
                if (lane < 16) sm.inner[16 * rt + lane] = in;
            }
            apply<false>(y, fac, rt, l16, g4);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                to_frag(p[2 * kk], p[2 * kk + 1], &pf[kk]);
                to_frag(y[2 * kk], y[2 * kk + 1], &df[kk]);
                if (ch == 0) scores[rt][kk][lane] = pf[kk];
            }
        }
        // dV^T = dO^T (P . D) + e^(L_end - L) dS^T K^T, MV column tiles: the states'
        // part, without the scores of the key wavefronts, and the rest.  bf16: the
        // query wavefronts' all, as the key wavefronts have more scores to form.
        constexpr int MV = CH == 1 ? 2 * NV : NV / 2, GV = MV < 4 ? MV : 4;
        const int m0 = CH == 1 ? 0 : (2 * ch + keys) * MV;
        const bool has = CH > 1 || !keys;
        const float ds = dc.d[16 * rt + l16];
        // the states' part before the barrier, where there are registers to hold it
        constexpr bool early = NK * NV < 16;
        f4 val[early ? MV : 1];
        auto value_of_state = [&](int i0, f4 (&y)[GV]) {
            Frag kf[NK];
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) kf[kk] = lk.row(kt, 16 * rt, kk);
#pragma unroll
            for (int i = 0; i < GV; ++i) y[i] = zf4();
            mma_group(y, kf, [&](int i, int kk) { return ST::turned(after, m0 + i0 + i, kk, lane); });
#pragma unroll
            for (int i = 0; i < GV; ++i) y[i] *= ds;
        };
        if constexpr (early) {
            if (has)
#pragma unroll
                for (int i0 = 0; i0 < MV; i0 += GV) value_of_state(i0, reinterpret_cast<f4 (&)[GV]>(val[i0]));
        }
        if constexpr (both) {
            if (more && w == 1) gates_of(next, odd ^ 1);
            request_states(next, more);
            __syncthreads();  // the scores are there
        } else {
            __syncthreads();  // the states have been read
            keep(rd, state, 2 * NK);
            __syncthreads();
            if (more && w == 1) gates_of(next, odd ^ 1);
            request_states(next, more);
        }
        if (keys) {
            // dK^T = Q^T (dP . D) + e^(L_end - L) dS V^T
            Frag vf[NV];
            float bs = 0.f;
#pragma unroll
            for (int kk = 0; kk < NV; ++kk) vf[kk] = lv.row(vt, 16 * rt, kk);
#pragma unroll
            for (int i0 = 0; i0 < NTK; i0 += G) {
                f4 y[G];
#pragma unroll
                for (int i = 0; i < G; ++i) y[i] = zf4();
                mma_group(y, vf, [&](int i, int kk) { return ST::get(after, (i0 + i) * CH + ch, kk, lane); });
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    y[i] *= ds;
                    const f4 kv = lk.quad(kt, 16 * rt, (i0 + i) * CH + ch);
#pragma unroll
                    for (int j = 0; j < 4; ++j) bs += y[i][j] * kv[j];
                    y[i] += acc[i0 + i];
                }
                mma_group(y, df, [&](int i, int kk) { return lk.col(qt, 32 * kk, (i0 + i) * CH + ch); });
#pragma unroll
                for (int i = 0; i < G; ++i) acc[i0 + i] = y[i];
            }
            if (nan)
#pragma unroll
                for (int i = 0; i < NTK; ++i)
                    acc[i] = poison<true>(acc[i], &last_q[16 * (i * CH + ch) + g4], 16 * rt + l16,
                                          16 * rt + l16 <= ends[1]);
            bs += __shfl_xor(bs, 16);
            bs += __shfl_xor(bs, 32);
            if (lane < 16) sm.b[ch][16 * rt + lane] = bs;
        }
        if (has) {
            const __amdgpu_buffer_rsrc_t out = buffer(
                reinterpret_cast<S *>(a.dv) + ((it.un.tok0 + it.t0) * a.H + h) * a.Dv);
            const uint32_t o = (uint32_t)((16 * rt + l16) * a.H * a.Dv + g4) * (uint32_t)sizeof(S);
            if (CH == 1 || !keys)
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) pf[kk] = scores[rt][kk][lane];
#pragma unroll
            for (int i0 = 0; i0 < MV; i0 += GV) {
                f4 y[GV];
                if constexpr (early) {
#pragma unroll
                    for (int i = 0; i < GV; ++i) y[i] = val[i0 + i];
                } else {
                    value_of_state(i0, y);
                }
                mma_group(y, pf, [&](int i, int kk) { return lv.at_col(ot, 32 * kk, lv.col_off(m0 + i0 + i)); });
#pragma unroll
                for (int i = 0; i < GV; ++i) {
                    const int c = 16 * (m0 + i0 + i);
                    store4(out, mine && c + g4 < a.Dv ? o + c * (uint32_t)sizeof(S) : kNowhere, y[i], T());
                }
            }
            if (nan && mine) {
                S *p = reinterpret_cast<S *>(a.dv) + ((it.un.tok0 + it.t0 + 16 * rt + l16) * a.H + h) * a.Dv;
#pragma unroll 1
                for (int i = 0; i < 4 * MV; ++i) {
                    const int c = 16 * (m0 + i / 4) + g4 + i % 4;
                    if (c < a.Dv && (16 * rt + l16 <= last_o[c] || 16 * rt + l16 <= ends[0] ||
                                     row_k[16 * rt + l16]))
                        put1(p + c, __builtin_nanf(""));
                }
            }
        }
        __syncthreads();
        if (!same) {  // the chunk's last head
            const __amdgpu_buffer_rsrc_t out = buffer(reinterpret_cast<S *>(keys ? a.dk : a.dq) +
                                                      ((it.un.tok0 + it.t0) * a.Hk + it.hk) * a.Dk);
            const uint32_t o = (uint32_t)((16 * rt + l16) * a.Hk * a.Dk + g4) * (uint32_t)sizeof(S);
#pragma unroll
            for (int i = 0; i < NTK; ++i) {
                const int c = 16 * (i * CH + ch);
                store4(out, mine && c + g4 < a.Dk ? o + c * (uint32_t)sizeof(S) : kNowhere, acc[i], T());
            }
#pragma unroll
            for (int i = 0; i < NTK; ++i) acc[i] = zf4();
        }
        if (!more) {
            if (w == 0) finish(done, odd, gdone, gall, up_to, from);
            break;
        }
        if (nan) {
            __syncthreads();
            if (!same) {
                clear();
            } else {  // d_out's of this head (q's and k's stay)
                if (tid < NV * 32) last_o[tid] = -1;
                if (tid < C) row_o[tid] = 0;
                if (tid == 0) ends[1] = -1;
                __syncthreads();
            }
        }
        it = next;
    }
}

Parts2 parts_of(const StatePlan &p)
{
    return Parts2{{p.st_part, p.st_part_r}, {p.st_dec, p.st_dec_r}};
}

// 32-wide units of the keys: three where they suffice (widths 72 to 96: 4206
// packed fp32 tokens, 12 heads of 96 x 80: 98 us, with four units 108), in the
// kernels whose states nobody else reads.
template <class T>
hipError_t part_launch(const StatePlan &p, const StateArgs &a, int ways, hipStream_t st)
{
    const int slices = (a.Dv + kSlice - 1) / kSlice;
    auto *k = a.Dk <= 64 ? gscan_state_part_kernel<T, 2>
                         : a.Dk <= 96 ? gscan_state_part_kernel<T, 3> : gscan_state_part_kernel<T, 4>;
    hipLaunchKernelGGL(k, dim3((unsigned)(p.units * a.H * slices * ways)),
                       dim3(2 * kSThreads), 0, st, a, slices, ways, p.per, parts_of(p));
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = (a.Dk * a.Dv / 4 + kSThreads - 1) / kSThreads;
    hipLaunchKernelGGL(gscan_state_join_kernel, dim3((unsigned)(a.B * a.H * blocks * ways)),
                       dim3(kSThreads), 0, st, a, ways, p.per, parts_of(p));
    return hipGetLastError();
}

template <class T>
hipError_t fwd_launch(const StatePlan &p, const StateArgs &a, hipStream_t st)
{
    const int slices = (a.Dv + kSlice - 1) / kSlice;
    if (p.split) {
        const hipError_t e = part_launch<T>(p, a, 1, st);
        if (e != hipSuccess) return e;
    }
    auto *k = a.Dk <= 64 ? gscan_state_fwd_kernel<T, 2>
                         : a.Dk <= 96 ? gscan_state_fwd_kernel<T, 3> : gscan_state_fwd_kernel<T, 4>;
    hipLaunchKernelGGL(k, dim3((unsigned)(p.units * a.H * slices)),
                       dim3(2 * kSThreads), 0, st, a, slices, p.per, p.st_part);
    return hipGetLastError();
}

template <class T, int NK, int NV>
hipError_t bwd_launch(const StatePlan &p, const StateArgs &a, hipStream_t st)
{
    hipError_t e;
    if (p.split) {
        e = part_launch<T>(p, a, 2, st);
        if (e != hipSuccess) return e;
    }
    const PassWs o = {p.st_s, p.st_ds, p.down, parts_of(p)};
    hipLaunchKernelGGL((gscan_state_pass_kernel<T, NK, NV>), dim3((unsigned)(p.units * a.H * NK)),
                       dim3(2 * kSThreads), 0, st, a, p.per, o);
    e = hipGetLastError();
    if (e != hipSuccess || a.T == 0) return e;
    const int64_t units = p.chunks * a.Hk;
    const int64_t each = (units + kCus - 1) / kCus;
    hipLaunchKernelGGL((gscan_state_grad_kernel<T, NK, NV>), dim3((unsigned)((units + each - 1) / each)),
                       dim3(kGThreads), 0, st, a, (uint32_t)units, (uint32_t)each, o);
    return hipGetLastError();
}

template <class T>
hipError_t bwd_widths(const StatePlan &p, const StateArgs &a, hipStream_t st)
{
    if (p.nk == 2) return p.nv == 2 ? bwd_launch<T, 2, 2>(p, a, st) : bwd_launch<T, 2, 4>(p, a, st);
    return p.nv == 2 ? bwd_launch<T, 4, 2>(p, a, st) : bwd_launch<T, 4, 4>(p, a, st);
}

}  // namespace

// Sequences may be split into units of `per` tokens that are walked in
// parallel: then the units' own states are formed first (part) and joined in
// order.  What a division into units of p chunks costs, in times of one chunk:
// the walks, one per CU at a time, 5/4 p a round, the part's included; the join
// 1/4 per unit of a sequence, and one for each 2^20 elements of the units'
// states, which are written and read; all of this once per direction; three for
// the launches.  Unsplit there are only the rounds, a chunk each.  Of a packed
// batch the host does not know the lengths: it counts as one sequence there, and
// its rounds by their sum.  Over the 229 cases it was fitted to (1 to 8 sequences
// of 300 to 32771 tokens, 5 to 32 heads, both types and directions, 17 divisions
// each) the division of least cost was 2 per cent off the fastest on average, 16 at
// most; the walks have become up to a tenth faster since and the rule was kept.
// Many short packed sequences are planned like one long one: then the units' pass
// finds nothing to do (72 sequences of 64 to 192 tokens, 8 heads of 64 x 64: 5 us and
// 4 for the join, beside 29 for the scan).
// 24000 bf16 tokens, 8 heads of 64 x 64: unsplit 555 us, 4 chunks per unit 70,
// 12 (chosen) 49, 48 123; 8 sequences of 2048, 16 heads of 64 x 128: unsplit
// (chosen) 66 us, split 99 and more (all figures of one build).
StatePlan make_state_plan(const StateArgs &a, bool backward)
{
    StatePlan p;
    p.chunk = a.dtype ? BF::C : FP::C;
    p.nk = a.Dk <= 64 ? 2 : 4;
    p.nv = a.Dv <= 64 ? 2 : 4;
    const int64_t nc = a.T > p.chunk ? (a.T + p.chunk - 1) / p.chunk : 1;
    // packed: sum over sequences of max(1, ceil(len / C)) <= T / C + B
    p.chunks = a.off ? a.T / p.chunk + a.B : a.B * nc;
    const int64_t walks = (int64_t)a.H * (backward ? p.nk : (a.Dv + kSlice - 1) / kSlice);
    auto units = [&](int64_t c) {
        const int64_t per = c * p.chunk;
        return a.off ? a.T / per + a.B : a.B * ((a.T + per - 1) / per);
    };
    const int64_t ways = backward ? 2 : 1, state = (int64_t)a.H * a.Dk * a.Dv;
    auto rounds = [&](int64_t n) { return (n * walks + kCus - 1) / kCus; };
    int64_t best = 0, least = 4 * (a.off ? (nc * kCus > p.chunks * walks ? nc : p.chunks * walks / kCus)
                                         : nc * rounds(a.B));  // (all in quarters of a chunk)
    auto consider = [&](int64_t c) {
        if (c < 2 || c >= nc) return;
        const int64_t run = a.off ? c / 2 + p.chunks * walks / kCus : c * rounds(units(c));
        const int64_t cost = ways * (5 * run + nc / c + (units(c) * state >> 18)) + 12;
        if (cost < least) {
            least = cost;
            best = c;
        }
    };
    for (int64_t c = 2; c <= 4096; c = c & (c - 1) ? c / 3 * 4 : c + c / 2) consider(c);  // 2 3 4 6 8 12 ..
    for (int64_t r = 1; r <= 4 && !a.off; ++r)  // whole rounds
        if (const int64_t u = r * kCus / (walks * a.B)) consider((nc + u - 1) / u);
    p.split = best != 0;
    p.per = (p.split ? best : nc) * p.chunk;
    p.units = p.split ? units(best) : a.B;
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
        p.st_s = take(one);
        p.st_ds = take(one);
        if (a.dtype) p.down = take((size_t)p.chunks * (size_t)a.H * (size_t)(4 * p.nk) * 4u);
    }
    p.bytes = at;
    return p;
}

hipError_t launch_state_forward(const StatePlan &p, const StateArgs &args, hipStream_t st)
{
    StateArgs a = args;
    a.chunks = p.chunks;
    return a.dtype ? fwd_launch<BF>(p, a, st) : fwd_launch<FP>(p, a, st);
}

hipError_t launch_state_backward(const StatePlan &p, const StateArgs &args, hipStream_t st)
{
    StateArgs a = args;
    a.chunks = p.chunks;
    return a.dtype ? bwd_widths<BF>(p, a, st) : bwd_widths<FP>(p, a, st);
}

}  // namespace gscan
