// Matrix products of the gated projection and the vocabulary's cross entropy:
//
//   C[m][n] = sum over k of A(m, k) B(n, k),
//
// where m is the index that the output has contiguous and n its row.  An
// operand has k contiguous (its rows are m or n; KC below) or m or n contiguous
// (its rows are k; RC):
//   logits, both projections   A weights  KC   B tokens     KC
//   gradient of the tokens     A weights  RC   B gradients  KC   (k: outputs)
//   gradient of the weights    A tokens   RC   B gradients  RC   (k: tokens)
// What a tile's sums become is the epilogue: the sums of a lane are those of
// one n and of groups of four m that follow each other.
#pragma once

#include <type_traits>

#include "gscan_lm_dev.h"

namespace gscan {
namespace {

typedef float f16v __attribute__((ext_vector_type(16)));

enum Epi {
    EPI_STORE,   // out[n][m]
    EPI_GATE,    // act(a) * b, of the halves a, b of the tile's m
    EPI_DGATE,   // the gradients of a and b from dout
    EPI_LSE,     // maximum and sum of exponentials of the tile's logits, for each n
    EPI_DLOGIT,  // the gradient of the logits
    EPI_ADD      // a sum over several calls: fp32 between them, the last into rows of out
};
enum Limit { LIMIT_NONE, LIMIT_N, LIMIT_K };

struct MmArgs {
    const void *a = nullptr, *a2 = nullptr;  // a2: of the second half (two weights); else null
    const void *b = nullptr;
    int64_t lda = 0, lda2 = 0, ldb = 0;
    int64_t M = 0, N = 0, K = 0;
    int64_t K1 = 0;                 // A RC with a2: the k at which it begins
    // Rows that the device knows the number of: N or K is *count.  Where that
    // is less than what the host knows, the tokens' operand (b, or a where K is
    // limited) is alt, in which they follow each other.
    const int32_t *count = nullptr;
    const void *alt = nullptr;
    int64_t ldalt = 0;
    void *out = nullptr, *out2 = nullptr;
    int64_t ldo = 0, N1 = 0;        // rows from N1 on are out2's
    const void *dout = nullptr;
    int64_t ldd = 0;
    const int32_t *target = nullptr, *row = nullptr;  // by n: target, place in the caller's order
    const void *tokens = nullptr;   // targets as the caller has them (few tokens)
    int tok64 = 0;
    const float *up = nullptr, *lse = nullptr;        // by n (up null: one)
    const float *factor = nullptr;  // EPI_STORE, EPI_ADD: of the whole output (null: one)
    float2 *part = nullptr;         // [tile of m][N]
    float *picked = nullptr;        // by n: the target's logit, in powers of two
    int64_t v0 = 0;                 // the vocabulary's entry of m = 0
    float *sum = nullptr;           // EPI_ADD between calls, [N][M]
    int first = 1, last = 1;
    float scale = 1.f;
    int act = 0;
    int parts = 0;                  // of the tiles that are left, at most (Work)
    float *partial = nullptr;       // their sums
};

// -------------------------------------------------------------- activations

// Hardware exponential and reciprocal (a few 2^-24 times |x|) where the result is
// rounded to bf16.
template <bool BF>
__device__ __forceinline__ float sigmoid_(float x)
{
    return BF ? __builtin_amdgcn_rcpf(1.f + exp2_(-1.44269504f * x)) : 1.f / (1.f + expf(-x));
}

// act(a) and its derivative.  0: a sigmoid(a); 1: a Phi(a), Phi the normal
// distribution's sum; 2: the same with the hyperbolic tangent's approximation
// of Phi, 0.5 (1 + tanh(u)) = sigmoid(2 u).
template <bool BF>
__device__ __forceinline__ void activation(float a, int act, float &f, float &slope)
{
    if (act == 0) {
        const float g = sigmoid_<BF>(a);
        f = a * g;
        slope = fmaf(f, 1.f - g, g);
    } else if (act == 1) {
        const float p = 0.5f * erfcf(-0.70710678118654752f * a);
        f = a * p;
        slope = fmaf(a * 0.39894228040143268f, BF ? exp2_(-0.72134752044448170f * a * a) : expf(-0.5f * a * a), p);
    } else {
        const float c = 0.79788456080286536f;
        const float q = fminf(a * a, 1e6f), g = sigmoid_<BF>(2.f * c * a * fmaf(0.044715f, q, 1.f));
        f = a * g;
        slope = fmaf(2.f * f * (1.f - g), c * fmaf(0.134145f, q, 1.f), g);
    }
}

// (maximum, sum of powers of two relative to it) of two sets joined, logits in
// powers of two.  An empty set is (-inf, 0); relative to an infinite maximum means relative
// to zero, so that the sum is zero, infinite, or NaN if a logit is.
__device__ __forceinline__ float lse_base(float top) { return fabsf(top) == INFINITY ? 0.f : top; }
__device__ __forceinline__ void join_lse(float &m, float &s, float m2, float s2)
{
    const float top = fmaxf(m, m2);
    const float base = lse_base(top);
    s = s * exp2_(m - base) + s2 * exp2_(m2 - base);
    m = top;
}

// ------------------------------------------------------------------ the tiles

// Where tile t lies: eight tiles of n before the next tile of m, so that tiles that
// run at the same time on an XCD share their rows in that XCD's L2.
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t tm, uint32_t tn, int64_t &im, int64_t &in)
{
    const uint32_t g = t / (8 * tm), left = tn - 8 * g, w = left < 8 ? left : 8, u = t - g * 8 * tm;
    const uint32_t q = left < 8 ? u / w : u / 8;
    in = 8 * g + (u - q * w);
    im = q;
}

// Workgroups go to the eight XCDs in turn; each XCD takes consecutive ones of n
// places.  -1: none.
__device__ __forceinline__ int place_of(int id, int n)
{
    const int q = n / 8, r = n % 8, x = id % 8, y = id / 8;
    return y < q + (x < r ? 1 : 0) ? x * q + (x < r ? x : r) + y : -1;
}

// The 16 elements of a lane among 32 m (groups of four at 8 g + 4 (lane / 32)) to or from
// row[m ..]; in(x) says whether the eight m from x on exist.  bf16: the halves of the
// wavefront exchange theirs, so that a lane has eight that follow each other: 16
// bytes instead of 8, half as many accesses.
template <bool BF, class In>
__device__ __forceinline__ void store16(void *out, int64_t row, int m, const f4 (&v)[4], int hi, In in)
{
    if constexpr (BF) {
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const auto s = __builtin_amdgcn_permlane32_swap(pack_bf16(v[g][2 * e], v[g][2 * e + 1]),
                                                                pack_bf16(v[g + 1][2 * e], v[g + 1][2 * e + 1]),
                                                                false, false);
                x[e] = s[0];
                x[2 + e] = s[1];
            }
            const int to = m + 8 * (g + hi);
            if (in(to)) *reinterpret_cast<u4 *>(reinterpret_cast<uint16_t *>(out) + row + to) = u4{x[0], x[1], x[2], x[3]};
        }
    } else {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (in(m + 8 * g)) *reinterpret_cast<f4 *>(reinterpret_cast<float *>(out) + row + m + 8 * g + 4 * hi) = v[g];
    }
}

template <bool BF, class In>
__device__ __forceinline__ void load16(const void *from, int64_t row, int m, f4 (&v)[4], int hi, In in)
{
    if constexpr (BF) {
        u4 x[2];
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
            const int at = m + 8 * (g + hi);
            x[g / 2] = u4{};
            if (in(at)) x[g / 2] = *reinterpret_cast<const u4 *>(reinterpret_cast<const uint16_t *>(from) + row + at);
        }
#pragma unroll
        for (int g = 0; g < 4; g += 2)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const auto s = __builtin_amdgcn_permlane32_swap(x[g / 2][e], x[g / 2][2 + e], false, false);
                v[g][2 * e] = bf_lo(s[0]);
                v[g][2 * e + 1] = bf_hi(s[0]);
                v[g + 1][2 * e] = bf_lo(s[1]);
                v[g + 1][2 * e + 1] = bf_hi(s[1]);
            }
    } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            v[g] = f4{};
            if (in(m + 8 * g))
                v[g] = *reinterpret_cast<const f4 *>(reinterpret_cast<const float *>(from) + row + m + 8 * g + 4 * hi);
        }
    }
}

// What a workgroup's sums become.  acc[i][j]: the 32 x 32 sums of the rows
// m0 + mat(i) .. + 31 and n0 + nat + 32 j .. + 31; element r of a lane is m = 8 (r / 4)
// + 4 (lane / 32) + r % 4, n = lane % 32.  Gated tiles hold the same m of both
// weights in acc[i] and acc[i + MI / 2].  TM, TN: the tile's m and n; red: LDS of WM *
// TN pairs.
template <Epi E, bool BF, int MI, int NI, int WM, class MAt>
__device__ __forceinline__ void epilogue(const MmArgs &a, f16v (&acc)[MI][NI], int64_t im, int64_t m0,
                                         int64_t n0, int64_t N, int wm, int nat, int TM, int TN, MAt mat,
                                         float2 *red)
{
    const int lane = threadIdx.x & 63, hi = lane >> 5, col = lane & 31;
    const bool whole = m0 + TM <= a.M;
    if constexpr (E == EPI_LSE) {
        const int end = (int)(whole ? TM : a.M - m0);
        const float unit = a.scale * 1.4426950408889634f;  // logits in powers of two
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int64_t n = n0 + nat + 32 * j + col;
            const int t = n < N ? (int)(a.target[n] - a.v0 - m0) : -1;
            const int from = mat(0), to = mat(MI - 1) + 32;
            if (__any(t >= from && t < to)) {
                float z = 0.f;
                bool has = false;
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (mat(i) + 8 * (r / 4) + 4 * hi + r % 4 == t) {
                            z = acc[i][j][r];
                            has = true;
                        }
                if (has) a.picked[n] = z * unit;
            }
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] *= unit;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (mat(i) + 8 * (r / 4) + 4 * hi + r % 4 >= end) acc[i][j][r] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, acc[i][j][r]);
            top = fmaxf(top, __shfl_xor(top, 32));
            const float base = lse_base(top);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) s += exp2_(acc[i][j][r] - base);
            s += __shfl_xor(s, 32);
            if (hi == 0) red[wm * TN + nat + 32 * j + col] = float2{top, s};
        }
        __syncthreads();
        for (int n = threadIdx.x; n < TN; n += blockDim.x) {
            float2 x = red[n];
#pragma unroll
            for (int w = 1; w < WM; ++w) {
                const float2 y = red[w * TN + n];
                join_lse(x.x, x.y, y.x, y.y);
            }
            if (n0 + n < N) a.part[im * a.N + n0 + n] = x;
        }
    } else {
        float factor = 1.f;
        if constexpr (E == EPI_STORE || E == EPI_ADD)
            if (a.factor) factor = *a.factor;
        // `all`: every m of the tile exists.  Else M is a multiple of eight (the gradients of the
        // logits are padded to it with zeros).
        auto finish = [&](auto all) __attribute__((always_inline)) {
            constexpr int HI = E == EPI_GATE || E == EPI_DGATE ? MI / 2 : MI;
            auto inside = [&](int m) { return all.value || m0 + m < a.M; };
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int64_t n = n0 + nat + 32 * j + col;
                if (n >= N) continue;  // (the halves of a wavefront have the same n: both are there or neither)
                const int64_t at = n * a.ldo + m0;
                auto sums = [&](int i, f4 (&v)[4]) {
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        v[g] = f4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                };
                if constexpr (E == EPI_DLOGIT) {
                    const int t = (int)(a.target[n] - a.v0 - m0) - 4 * hi;
                    const float up = a.up ? a.up[n] : 1.f, lse = a.lse[n];
                    const float unit = a.scale * 1.4426950408889634f, base = -1.4426950408889634f * lse;
                    const int64_t padded = (a.M + 7) / 8 * 8;
#pragma unroll
                    for (int i = 0; i < HI; ++i) {
                        f4 v[4];
                        sums(i, v);
#pragma unroll
                        for (int g = 0; g < 4; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[g][e] = BF ? exp2_(fmaf(v[g][e], unit, base)) : expf(v[g][e] * a.scale - lse);
                        if (__any(t >= mat(i) - 4 && t < mat(i) + 32)) {  // someone's target is here
#pragma unroll
                            for (int g = 0; g < 4; ++g)
#pragma unroll
                                for (int e = 0; e < 4; ++e) v[g][e] -= mat(i) + 8 * g + e == t ? 1.f : 0.f;
                        }
#pragma unroll
                        for (int g = 0; g < 4; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[g][e] = inside(mat(i) + 8 * g + 4 * hi + e) ? v[g][e] * up : 0.f;
                        store16<BF>(a.out, at, mat(i), v, hi, [&](int m) { return all.value || m0 + m < padded; });
                    }
                } else if constexpr (E == EPI_STORE) {
                    void *out = n < a.N1 ? a.out : a.out2;
                    const int64_t to = n < a.N1 ? at : at - a.N1 * a.ldo;
#pragma unroll
                    for (int i = 0; i < HI; ++i) {
                        f4 v[4];
                        sums(i, v);
#pragma unroll
                        for (int g = 0; g < 4; ++g) v[g] *= factor;
                        store16<BF>(out, to, mat(i), v, hi, inside);
                    }
                } else if constexpr (E == EPI_ADD) {
                    const int64_t between = n * a.M + m0, to = a.last ? a.row[n] * a.ldo + m0 : 0;
#pragma unroll
                    for (int i = 0; i < HI; ++i) {
                        f4 v[4], s[4];
                        sums(i, v);
                        if (!a.first) {
                            load16<false>(a.sum, between, mat(i), s, hi, inside);
#pragma unroll
                            for (int g = 0; g < 4; ++g) v[g] += s[g];
                        }
                        if (a.last) {
#pragma unroll
                            for (int g = 0; g < 4; ++g) v[g] *= factor;
                            store16<BF>(a.out, to, mat(i), v, hi, inside);
                        } else {
                            store16<false>(a.sum, between, mat(i), v, hi, inside);
                        }
                    }
                } else {
                    f4 d[HI][4];
                    if constexpr (E == EPI_DGATE) {
#pragma unroll
                        for (int i = 0; i < HI; ++i)
                            load16<BF>(a.dout, n * a.ldd + m0, mat(i), d[i], hi, inside);
                    }
#pragma unroll
                    for (int i = 0; i < HI; ++i) {
                        f4 o[4], o2[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float f, slope;
                                activation<BF>(acc[i][j][4 * g + e], a.act, f, slope);
                                const float b = acc[HI + i][j][4 * g + e];
                                if constexpr (E == EPI_GATE) {
                                    o[g][e] = f * b;
                                } else {
                                    o[g][e] = d[i][g][e] * b * slope;
                                    o2[g][e] = d[i][g][e] * f;
                                }
                            }
                        store16<BF>(a.out, at, mat(i), o, hi, inside);
                        if constexpr (E == EPI_DGATE) store16<BF>(a.out, at + a.M, mat(i), o2, hi, inside);
                    }
                }
            }
        };
        if (whole) finish(std::true_type{});
        else finish(std::false_type{});
    }
}

// ------------------------------------------------------------------ products

// Tiles of 32 MI WM by 32 NI WN, a wavefront's part 32 MI x 32 NI in registers.
// Steps of 128 bytes of k (64 bf16, 32 fp32) go from memory straight into LDS (16
// bytes per lane, no register in between), into the half that the step before has
// been read from.  The 64 banks of LDS take 16 lanes' pieces of 16 bytes at once, 32 of
// 8 or 64 of 4.  Rows of a KC tile hold eight pieces; piece c of row r lies at c ^ (r / 2 %
// 8), so that no two of 16 rows meet at a bank.  Rows of an RC tile are k; bf16: their
// pieces lie at c ^ 4 (k % 4) (64 columns: 4 (k / 2 % 2)), so that the four rows of a
// transposed read (32 lanes, 64 bytes of each) do not meet either; fp32: at c ^ 8 (k / 4 %
// 2), as half of the wavefront reads four rows on.  No conflicts are counted, and LDS is
// busy for a quarter of the cycles of 8192 tokens' gated products (half of them with the
// banks taken for 32; the time, which power sets, is the same within 1 per cent).
// Memory outside the operands is not touched: what of a tile or of the last step lies
// outside is read from past the end of the buffer, where the hardware finds zeros.
//
// A quarter of a step is read from LDS while the products of the quarter before are
// formed; a step's first quarter is read behind the barrier that ends the step before
// it, but before that step's last products.
//
// bf16 products run at what the card's power allows: 8192 tokens, 2048 x 2 x 5504,
// at 1150 to 1200 TFLOP/s in the steps (zeros instead of random values: 1390; a
// large library product: 1140 to 1320, 2250 on zeros).  Four stages of half a step,
// three on their way, were slower where k is contiguous (64 bytes of a row at a time:
// 403 -> 457 us) and no faster elsewhere.
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));
template <class T>
using lds_t = __attribute__((address_space(3))) T;
template <class T>
__device__ __forceinline__ lds_t<T> *in_lds(uint32_t address)
{
    return (lds_t<T> *)(uintptr_t)address;
}

template <bool BF>
constexpr int kSize = BF ? 2 : 4;
template <bool BF>
constexpr int kBK = 128 / kSize<BF>;  // k of a step
constexpr uint32_t kNowhere = 0x7ffffff0u;  // past the end of every buffer

// 64 lanes' 16 bytes at their offsets (and `more`) of the buffer, one after the other
// from the LDS address on.  The wait for them is load_wait().  (m0 is a reserved register: the
// compiler keeps nothing in it, warns of it among the clobbers, and uses it nowhere else in
// these kernels.)
__device__ __forceinline__ void load_to_lds(const u4 &buffer, uint32_t offset, uint32_t more, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :
                 : "v"(offset), "s"(buffer), "s"(more), "s"(lds)
                 : "memory");
}
__device__ __forceinline__ void load_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A buffer of an operand from `base` on.
__device__ __forceinline__ u4 buffer_at(uint64_t base)
{
    return u4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)base),
              (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32)) & 0xffffu, 0x7fffffe0u,
              0x00020000u};
}

// What a lane gives to the products of a quarter of a step: eight bf16 of a row,
// k = 8 (lane / 32) .. + 7 of 16, or four fp32, k = 4 (lane / 32) .. + 3 of 8.
template <bool BF>
using Piece = typename std::conditional<BF, bf8, f4>::type;

__device__ __forceinline__ void multiply(const bf8 &x, const bf8 &y, f16v &acc)
{
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, acc, 0, 0, 0);
}
__device__ __forceinline__ void multiply(const f4 &x, const f4 &y, f16v &acc)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], acc, 0, 0, 0);
}

// A tile of T rows (KC) or columns (RC): offsets of a lane's loads, and where the
// lane finds its elements.
template <bool BF, bool RC, int T, int W>
struct Tile {
    static constexpr int kSz = kSize<BF>, kIn = 16 / kSz;  // elements of a piece
    static constexpr int kLoads = T / 8 / W;               // of a wavefront
    static constexpr int kPer = 1024 / (kSz * T);          // RC: rows that one load covers
    uint32_t off[kLoads];
    uint32_t at[4];  // RC: of its groups of 32 columns; KC: of the quarters of a step

    // Load i of a lane: row (KC: of the tile, RC: k) and piece (KC: of k, RC: of the
    // tile's columns).
    static __device__ __forceinline__ int row(int i, int wave, int lane)
    {
        const int q = wave + W * i;
        return RC ? q * kPer + lane / (64 / kPer) : 8 * q + (lane >> 3);
    }
    static __device__ __forceinline__ int swizzle(int k)
    {
        return !BF ? 8 * ((k >> 2) & 1) : T == 64 ? 4 * ((k >> 1) & 1) : 4 * (k & 3);
    }
    static __device__ __forceinline__ int piece(int i, int wave, int lane)
    {
        if constexpr (RC) return (lane % (64 / kPer)) ^ swizzle(row(i, wave, lane));
        else return (lane & 7) ^ ((row(i, wave, lane) >> 1) & 7);
    }

    // `mine`: the first of the wavefront's rows (KC) or columns (RC), a multiple of 32
    __device__ __forceinline__ void place(int lane, int mine)
    {
        if constexpr (RC && BF) {
            const int p = lane & 15, g = lane >> 4;
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                const int c = (4 * (mine / 32 + o) + 2 * (g & 1) + ((p & 3) >> 1)) ^ swizzle(p >> 2);
                at[o] = (uint32_t)((8 * (g >> 1) + (p >> 2)) * 2 * T + 16 * c + 8 * (p & 1));
            }
        } else if constexpr (RC) {
#pragma unroll
            for (int o = 0; o < 4; ++o)
                at[o] = (uint32_t)((4 * (lane >> 5)) * 4 * T + 128 * ((mine / 32 + o) ^ (lane >> 5)) + 4 * (lane & 31));
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s)
                at[s] = (uint32_t)((mine + (lane & 31)) * 128 + 16 * ((2 * s + (lane >> 5)) ^ ((lane >> 1) & 7)));
        }
    }

    // The loads i0 .. i1 - 1 of a tile of which `there` rows (KC) or columns (RC) exist.
    // KC: the tile's rows from `from` on are rows of another matrix (two weights).
    __device__ __forceinline__ void aim(int i0, int i1, int wave, int lane, uint32_t ld, int there, int from = 0)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i >= i0 && i < i1) {
                const int r = row(i, wave, lane) - from, c = piece(i, wave, lane);
                off[i] = (RC ? kIn * c : r) < there ? (uint32_t)r * ld * kSz + (uint32_t)c * 16 : kNowhere;
            }
    }

    // Nothing from the `left`-th k of a step on.
    __device__ __forceinline__ void cut(int wave, int lane, int left)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if ((RC ? row(i, wave, lane) : kIn * piece(i, wave, lane)) >= left) off[i] = kNowhere;
    }

    // Load i of a step; `k`: where the step begins (KC), in bytes.
    __device__ __forceinline__ void load(int i, const u4 &buffer, uint32_t k, uint32_t lds, int wave) const
    {
        load_to_lds(buffer, off[i], k, lds + (uint32_t)(wave + W * i) * 1024u);
    }

    // The s-th quarter of a step, of the group `i` of 32 rows or columns from the
    // wavefront's first.
    static constexpr int kReads = !RC ? 1 : BF ? 2 : 4;
    __device__ __forceinline__ Piece<BF> get(uint32_t lds, int i, int s) const
    {
        if constexpr (RC && BF) {
            const uint32_t p = lds + at[i] + (uint32_t)(s * 16 * 2 * T);
            const s4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(in_lds<s4v>(p));
            const s4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(in_lds<s4v>(p + 4 * 2 * T));
            const u4 v = {__builtin_bit_cast(uint2, x).x, __builtin_bit_cast(uint2, x).y,
                          __builtin_bit_cast(uint2, y).x, __builtin_bit_cast(uint2, y).y};
            return __builtin_bit_cast(bf8, v);
        } else if constexpr (RC) {
            const uint32_t p = lds + at[i] + (uint32_t)(s * 8 * 4 * T);
            return f4{*in_lds<float>(p), *in_lds<float>(p + 4 * T), *in_lds<float>(p + 8 * T),
                      *in_lds<float>(p + 12 * T)};
        } else {
            return *in_lds<Piece<BF>>(lds + at[s] + (uint32_t)(i * 4096));
        }
    }
};

// Who does what.  Every workgroup (as many as fit the device at once) does whole
// tiles while there are enough for all.  Where what is left is for half of them or
// fewer, and it saves more than it costs, every one of those tiles is divided along
// k into as many parts as there are workgroups for: the parts are sums in memory,
// which a second kernel adds in order.  All tiles are divided at the same k, so that
// workgroups that run at the same time read the same rows of the operands.  (Divided
// one behind the other, evenly over all workgroups, they read them at different times:
// 84 tiles of 696 steps took 543 us, 7 TB/s.)
struct Work {
    int tiles = 0, whole = 0;   // whole: tiles that one workgroup does alone
    int steps = 0;              // of a tile
    int groups = 0;             // workgroups
    int splits = 0;             // parts of each tile that is left (0: none is)

    __host__ __device__ int left() const { return tiles - whole; }
    __host__ __device__ int parts() const { return left() * splits; }
    __host__ __device__ int first_step(int split) const
    {
        const int share = steps / splits, more = steps % splits;
        return split * share + (split < more ? split : more);
    }
};

// One of the kernels' tiles, and what it takes, in ns: a step with all workgroups at
// work, and at least; a tile besides its steps; a part's sums through memory (3.5
// TB/s); the second kernel.  Measured at 300 to 8192 rows; fewer use the same figures.
struct MmShape {
    int m, n, groups, step, least, tile, part, join;
};
// 0: 256 x 256 (bf16 only), 1: 128 x 128, 2: 128 (of m) x 64.
constexpr MmShape kShapesF32[2] = {{128, 128, 512, 4400, 2200, 3000, 37, 5000}, {128, 64, 768, 3300, 1100, 3000, 19, 5000}};
constexpr MmShape kShapesBf16[3] = {{256, 256, 256, 1650, 1650, 5000, 150, 6000},
                                    {128, 128, 512, 1050, 680, 2500, 37, 5000},
                                    {128, 64, 768, 1170, 600, 2000, 19, 5000}};
constexpr int first_shape(bool bf) { return bf ? 0 : 1; }
constexpr MmShape shape_of(bool bf, int i) { return bf ? kShapesBf16[i] : kShapesF32[i - 1]; }

// ns of a step while n workgroups are at work, at most those that fit at once
__host__ __device__ __forceinline__ int step_ns(const MmShape &c, int n)
{
    const int t = c.step * ((n + 255) / 256) / (c.groups / 256);
    return t > c.least ? t : c.least;
}

constexpr int kPartSteps = 4;   // at least so many steps to a part
// Parts that the device may make where the host sees no reason to, as tokens that do not count
// leave few tiles: a workgroup per CU (fp32, 1141 tokens, half of which count, 1248 x 1134:
// losses 66 -> 49 us, gradients 136 -> 108; where all count, 147 -> 152 by joins that find
// nothing to do).
constexpr int kSpare = 256;

// The work with the tiles that are left divided into `parts` parts at most (tokens that
// the host does not know of leave fewer tiles, or steps).
__host__ __device__ __forceinline__ Work divide_work(int tiles, int steps, const MmShape &c, int parts)
{
    Work w;
    w.tiles = w.whole = tiles;
    w.steps = steps;
    w.groups = c.groups;
    const int left = (int)((uint32_t)tiles % (uint32_t)c.groups);
    if (left && 2 * left <= parts) {
        const int most = steps / kPartSteps, n = (int)((uint32_t)parts / (uint32_t)left);
        w.splits = n < most ? n : most;
        if (w.splits > 1) w.whole = tiles - left;
        else w.splits = 0;
    }
    return w;
}

Work plan_work(int tiles, int steps, const MmShape &c)
{
    Work best = divide_work(tiles, steps, c, 0);
    const int left = tiles % c.groups;
    if (!left) return best;
    int64_t least = (int64_t)steps * step_ns(c, left);
    for (int n = 2; left * n <= c.groups && steps / n >= kPartSteps; ++n) {
        const int64_t ns = (int64_t)(steps / n + 1) * step_ns(c, left * n) + (int64_t)(left * n) * c.part + c.join;
        if (ns >= least) continue;
        least = ns;
        best = divide_work(tiles, steps, c, left * n);
    }
    return best;
}

__host__ __device__ constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Steps of bk of k: of each of the two weights by itself where k runs over both.
__host__ __device__ __forceinline__ int64_t steps_of(int64_t K, int64_t K1, int bk)
{
    return K1 ? 2 * ceil_div(K1, bk) : ceil_div(K, bk);
}

// What every kernel of a product knows of its operands.
template <Limit L>
struct Operands {
    int64_t N, K, lda, ldb;
    const void *pa, *pb;

    __device__ __forceinline__ explicit Operands(const MmArgs &a)
        : N(a.N), K(a.K), lda(a.lda), ldb(a.ldb), pa(a.a), pb(a.b)
    {
        if constexpr (L != LIMIT_NONE) {
            const int64_t c = __builtin_amdgcn_readfirstlane(*a.count);
            if (a.alt && c < (L == LIMIT_N ? N : K)) {
                (L == LIMIT_N ? pb : pa) = a.alt;
                (L == LIMIT_N ? ldb : lda) = a.ldalt;
            }
            (L == LIMIT_N ? N : K) = c;
        }
    }
};

// Workgroups per CU at once: one of 512 threads (128 kB of LDS); of 256 threads, two of
// 128 x 128 (64 kB) or three of 128 x 64 (48 kB).
constexpr int per_cu(int ni, int waves) { return waves == 8 ? 1 : ni == 2 ? 2 : 3; }

// A workgroup's tiles in turn: whole ones, then a part of one.
struct Tiles {
    int id, place, mine;   // workgroup; its place in a full round; its part (-1: none)
    int at = 0;            // the round's first tile
    // the present one: tile, steps s0 .. s1 - 1, slot of its sums (-1: it is whole)
    int t = 0, s0 = 0, s1 = 0, slot = -1;

    __device__ __forceinline__ Tiles(const Work &w, int id_) : id(id_)
    {
        place = place_of(id, w.groups);
        mine = w.splits ? place_of(id, w.parts()) : -1;
    }
    __device__ __forceinline__ bool next(const Work &w)
    {
        t = -1;
        if (at < w.whole) {
            const int last = w.whole - at;
            const int p = last >= w.groups ? place : place_of(id, last);
            if (p >= 0) t = at + p;
            at += w.groups;
        }
        s0 = 0;
        s1 = w.steps;
        slot = -1;
        if (t < 0) {
            if (mine < 0) return false;
            const int left = w.left(), split = (int)((uint32_t)mine / (uint32_t)left);
            t = w.whole + mine - split * left;
            s0 = w.first_step(split);
            s1 = w.first_step(split + 1);
            slot = mine;
            mine = -1;
        }
        return true;
    }
};

template <Epi E, bool BF, bool RCA, bool RCB, Limit L, int MI, int NI, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, per_cu(NI, WM *WN) == 3 ? 3 : 2) gscan_mm_kernel(MmArgs a)
{
    constexpr bool kGated = E == EPI_GATE || E == EPI_DGATE;
    constexpr int kW = WM * WN, kTA = 32 * MI * WM, kTN = 32 * NI * WN, kSz = kSize<BF>, kStep = kBK<BF>;
    constexpr int kTM = kGated ? kTA / 2 : kTA;  // of m
    constexpr uint32_t kStage = (kTA + kTN) * 128, kB = kTA * 128;
    __shared__ __align__(1024) char lds[2 * kStage];
    __shared__ float2 red[E == EPI_LSE ? WM * kTN : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const Operands<L> o(a);
    const int64_t M = a.M, N = o.N, lda = o.lda, ldb = o.ldb, lda2 = a.lda2;
    const uint64_t pa = reinterpret_cast<uint64_t>(o.pa), pb = reinterpret_cast<uint64_t>(o.pb);
    const uint64_t pa2 = reinterpret_cast<uint64_t>(a.a2);
    const int tm = (int)ceil_div(M, kTM), tn = (int)ceil_div(N, kTN);
    constexpr bool kTwo = RCA && !RCB && E == EPI_STORE;
    const bool two = kTwo && a.a2;  // a second weight behind the first along k
    const int64_t part = two ? a.K1 : o.K;
    const int part_steps = (int)ceil_div(part, kStep);
    constexpr MmShape kMine = shape_of(BF, kW == 8 ? 0 : NI == 2 ? 1 : 2);
    const Work work = divide_work(tm * tn, two ? 2 * part_steps : part_steps, kMine, a.parts);

    Tile<BF, RCA, kTA, kW> ta;
    Tile<BF, RCB, kTN, kW> tb;
    ta.place(lane, kGated ? 16 * MI * wm : 32 * MI * wm);
    tb.place(lane, 32 * NI * wn);
    const uint32_t base = (uint32_t)(uintptr_t)(lds_t<char> *)lds;

    // Requests: two steps ahead of the products, so with tiles of their own.
    Tiles ask(work, (int)blockIdx.x);
    bool more = ask.next(work);
    if (!more) return;
    uint64_t ba = 0, ba2 = 0, bb = 0;   // the operands from the tile's first row (KC) or the step's (RC) on
    int asked = ask.s0, k0 = 0;         // the step, and its first k (of one weight)
    auto aim = [&]() __attribute__((always_inline)) {
        int64_t im, in;
        tile_at((uint32_t)ask.t, (uint32_t)tm, (uint32_t)tn, im, in);
        const int64_t m0 = im * kTM, n0 = in * kTN;
        const int rows = (int)(M - m0 < kTM ? M - m0 : kTM), cols = (int)(N - n0 < kTN ? N - n0 : kTN);
        const bool second = kTwo && two && asked >= part_steps;
        k0 = (second ? asked - part_steps : asked) * kStep;
        uint64_t p = pa;
        int64_t ld = lda;
        if (second) {
            p = pa2;
            ld = lda2;
        }
        ta.aim(0, kGated ? ta.kLoads / 2 : ta.kLoads, wave, lane, (uint32_t)ld, rows);
        ba = p + (uint64_t)(RCA ? m0 + k0 * ld : m0 * ld) * (uint64_t)kSz;
        if constexpr (kGated) {
            ta.aim(ta.kLoads / 2, ta.kLoads, wave, lane, (uint32_t)lda2, rows, kTM);
            ba2 = pa2 + (uint64_t)(m0 * lda2) * (uint64_t)kSz;
        }
        tb.aim(0, tb.kLoads, wave, lane, (uint32_t)ldb, cols);
        if constexpr (RCB) bb = pb + (uint64_t)(n0 + k0 * ldb) * (uint64_t)kSz;
        else bb = pb + (uint64_t)(n0 * ldb + (second ? part : 0)) * (uint64_t)kSz;
    };
    u4 da = {}, da2 = {}, db = {};
    uint32_t ka = 0, kb = 0;
    // A step's loads: what they need, one after the other, and on to the next step.
    // Behind the last one loads go nowhere.
    auto begin = [&]() __attribute__((always_inline)) {
        const int64_t left = more ? part - k0 : 0;
        if (left < kStep) {
            ta.cut(wave, lane, (int)left);
            tb.cut(wave, lane, (int)left);
        }
        da = buffer_at(ba);
        if (kGated) da2 = buffer_at(ba2);
        db = buffer_at(bb);
        ka = RCA ? 0u : (uint32_t)__builtin_amdgcn_readfirstlane(kSz * k0);
        kb = RCB ? 0u : (uint32_t)__builtin_amdgcn_readfirstlane(kSz * k0);
    };
    auto load_a = [&](int i, uint32_t stage) __attribute__((always_inline)) {
        ta.load(i, kGated && i >= ta.kLoads / 2 ? da2 : da, ka, stage, wave);
    };
    auto load_b = [&](int i, uint32_t stage) __attribute__((always_inline)) { tb.load(i, db, kb, stage + kB, wave); };
    auto advance = [&]() __attribute__((always_inline)) {
        if (!more) return;
        if (++asked == ask.s1) {
            more = ask.next(work);
            asked = ask.s0;
            if (more) aim();
            return;
        }
        if (kTwo && two && asked == part_steps) {
            aim();
            return;
        }
        k0 += kStep;
        if constexpr (RCA) {
            int64_t ld = lda;
            if (kTwo && two && asked > part_steps) ld = lda2;
            ba += (uint64_t)(ld * 128);
        }
        if constexpr (RCB) bb += (uint64_t)(ldb * 128);
    };
    auto request = [&](uint32_t stage) __attribute__((always_inline)) {
        begin();
#pragma unroll
        for (int i = 0; i < ta.kLoads; ++i) load_a(i, stage);
#pragma unroll
        for (int i = 0; i < tb.kLoads; ++i) load_b(i, stage);
        advance();
    };

    Tiles now(work, (int)blockIdx.x);
    bool busy = now.next(work);
    f16v acc[MI][NI], sum[BF ? 1 : MI][BF ? 1 : NI];  // fp32: sums of 256 k are joined in `sum`
    Piece<BF> x[2][MI], y[2][NI];
    auto group = [&](int i) { return kGated && i >= MI / 2 ? i - MI / 2 + kTM / 32 : i; };
    auto mat = [&](int i) { return (kGated ? 16 : 32) * MI * wm + 32 * i; };
    uint32_t here = base, there = base + kStage;
    if (work.steps > 0) {
        aim();
        request(here);
        load_wait();
        __syncthreads();
        begin();  // the second step's; the loop goes on with them
#pragma unroll
        for (int i = 0; i < ta.kLoads; ++i) load_a(i, there);
#pragma unroll
        for (int i = 0; i < MI; ++i) x[0][i] = ta.get(here, group(i), 0);
#pragma unroll
        for (int j = 0; j < NI; ++j) y[0][j] = tb.get(here + kB, j, 0);
    }
    while (busy) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                acc[i][j] = f16v{};
                if constexpr (!BF) sum[i][j] = f16v{};
            }
        for (int t = now.s0; t < now.s1; ++t) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {  // quarters
                const int u = s & 1, v = u ^ 1;
                uint32_t from = here;
                if (s == 3) {
                    // everything of this step has been read and the next one's is there
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    load_wait();
                    __syncthreads();
                    from = there;
                    begin();
                }
                const int s1 = (s + 1) % 4;
#pragma unroll
                for (int j = 0; j < NI; ++j) y[v][j] = tb.get(from + kB, j, s1);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    x[v][i] = ta.get(from, group(i), s1);
                    // the loads of the step after the next, into what this step leaves, a few at
                    // a time: all at once they hold the wavefront up for as long as the
                    // memory's queue takes to accept those of all eight
#pragma unroll
                    for (int l = i * ta.kLoads / MI; l < (i + 1) * ta.kLoads / MI; ++l)
                        if (s == 3) load_a(l, here);
#pragma unroll
                    for (int l = i * tb.kLoads / MI; l < (i + 1) * tb.kLoads / MI; ++l)
                        if (s == 0) load_b(l, there);
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        multiply(x[u][i], y[u][j], acc[i][j]);
                }
                if (s == 0) advance();
                // reads between the products
                __builtin_amdgcn_sched_group_barrier(0x100, NI * tb.kReads, 0);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x100, ta.kReads, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, BF ? NI : 4 * NI, 0);
                }
            }
            const uint32_t h = here;
            here = there;
            there = h;
            if constexpr (!BF) {
                if ((t - now.s0) % 8 == 7 || t + 1 == now.s1) {
#pragma unroll
                    for (int i = 0; i < MI; ++i)
#pragma unroll
                        for (int j = 0; j < NI; ++j) {
                            sum[i][j] += acc[i][j];
                            acc[i][j] = f16v{};
                        }
                }
            }
        }
        if constexpr (!BF) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[i][j] = sum[i][j];
        }
        int64_t im, in;
        tile_at((uint32_t)now.t, (uint32_t)tm, (uint32_t)tn, im, in);
        if (now.slot >= 0) {
            f4 *p = reinterpret_cast<f4 *>(a.partial) + (int64_t)now.slot * (kTA * kTN / 4) + wave * MI * NI * 256 + lane;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        p[((i * NI + j) * 4 + g) * 64] = f4{acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                                           acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        } else {
            epilogue<E, BF, MI, NI, WM>(a, acc, im, im * kTM, in * kTN, N, wm, 32 * NI * wn, kTM, kTN, mat, red);
        }
        // Loads of the epilogue that some path leaves unused would make the compiler
        // wait at the head of every step, for the requests too: wait for them here.
        if constexpr (E != EPI_GATE) __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        busy = now.next(work);
    }
    load_wait();  // nothing may arrive in LDS that is another workgroup's
}

// The divided tiles: a workgroup adds the parts of a tile in order (all of it for
// EPI_LSE; else those of one of its groups of 32 x 32 per wavefront, or of the same
// group of both weights) and finishes it.
template <Epi E, int MI, int NI>
constexpr int kShares = E == EPI_LSE ? 1 : (E == EPI_GATE || E == EPI_DGATE) ? MI / 2 * NI : MI * NI;

template <Epi E, bool BF, Limit L, int MI, int NI, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, 2) gscan_mm_join_kernel(MmArgs a)
{
    constexpr bool kGated = E == EPI_GATE || E == EPI_DGATE;
    constexpr int kTA = 32 * MI * WM, kTN = 32 * NI * WN, kTM = kGated ? kTA / 2 : kTA;
    constexpr int kN = kShares<E, MI, NI>, kI = E == EPI_LSE ? MI : kGated ? 2 : 1, kJ = E == EPI_LSE ? NI : 1;
    __shared__ float2 red[E == EPI_LSE ? WM * kTN : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int i0 = kN == 1 ? 0 : (int)(blockIdx.x % kN) / NI, j0 = kN == 1 ? 0 : (int)(blockIdx.x % kN) % NI;
    const Operands<L> o(a);
    const int tm = (int)ceil_div(a.M, kTM), tn = (int)ceil_div(o.N, kTN), d = (int)(blockIdx.x / kN);
    constexpr MmShape kMine = shape_of(BF, WM * WN == 8 ? 0 : NI == 2 ? 1 : 2);
    const Work work = divide_work(tm * tn, (int)steps_of(o.K, a.K1, kBK<BF>), kMine, a.parts);
    if (d >= work.left()) return;
    f16v acc[kI][kJ];
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) acc[i][j] = f16v{};
    for (int w = 0; w < work.splits; ++w) {
        const f4 *p = reinterpret_cast<const f4 *>(a.partial) + (int64_t)(w * work.left() + d) * (kTA * kTN / 4) +
                      wave * MI * NI * 256 + lane;
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f4 v = p[(((i0 + i * (MI / kI)) * NI + j0 + j) * 4 + g) * 64];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][4 * g + e] += v[e];
                }
    }
    int64_t im, in;
    tile_at((uint32_t)(work.whole + d), (uint32_t)tm, (uint32_t)tn, im, in);
    auto mat = [&](int i) { return (kGated ? 16 : 32) * MI * wm + 32 * (i + i0); };
    epilogue<E, BF, kI, kJ, WM>(a, acc, im, im * kTM, in * kTN, o.N, wm, 32 * (NI * wn + j0), kTM, kTN, mat, red);
}

// The kernel of a product: the one that the busiest workgroup is done with first.
struct MmPlan {
    int shape = 0;
    Work work;
    size_t bytes = 0;   // of parts of tiles
    int parts = 0, divided = 0;  // parts, and tiles that have any, at most
    int64_t ns = 0;
};
MmPlan plan_mm(int64_t M, int64_t N, int64_t K, int64_t K1, bool gated, bool limited, int dtype)
{
    MmPlan best;
    for (int i = first_shape(dtype); i < 3; ++i) {
        const MmShape c = shape_of(dtype, i);
        MmPlan p;
        p.shape = i;
        p.work = plan_work((int)(ceil_div(M, gated ? c.m / 2 : c.m) * ceil_div(N, c.n)),
                           (int)steps_of(K, K1, dtype ? kBK<true> : kBK<false>), c);
        const Work &w = p.work;
        p.divided = w.left();
        const int full = w.whole / c.groups, last = w.whole % c.groups;
        p.ns = (int64_t)full * ((int64_t)w.steps * c.step + c.tile);
        if (last) p.ns += (int64_t)w.steps * step_ns(c, last) + c.tile;
        if (w.splits)
            p.ns += (int64_t)(w.steps / w.splits + 1) * step_ns(c, w.parts()) + c.tile +
                    (int64_t)w.parts() * c.part + c.join;
        p.parts = w.parts();
        if (limited) {  // fewer tokens may leave other tiles
            if (!w.splits && w.tiles <= kSpare &&
                (int64_t)w.steps * c.least / 2 > c.join + kSpare * (int64_t)c.part)
                p.parts = kSpare;
            if (w.splits && w.splits == c.groups / w.left()) p.parts = c.groups;
            p.divided = w.tiles < p.parts / 2 ? w.tiles : p.parts / 2;
        }
        p.bytes = (size_t)p.parts * (size_t)(c.m * c.n) * sizeof(float);
        if (!best.ns || p.ns < best.ns) best = p;
    }
    return best;
}

size_t mm_bytes(int64_t M, int64_t N, int64_t K, int64_t K1, bool gated, bool limited, int dtype)
{
    return plan_mm(M, N, K, K1, gated, limited, dtype).bytes;
}

template <Epi E, bool BF, bool RCA, bool RCB, Limit L, int MI, int NI, int WM, int WN>
hipError_t launch_shape(const MmArgs &a, const MmPlan &p, hipStream_t st)
{
    const dim3 threads(64 * WM * WN);
    const int most = p.parts > p.work.tiles ? p.parts : p.work.tiles;
    const int n = most < p.work.groups ? most : p.work.groups;
    hipLaunchKernelGGL((gscan_mm_kernel<E, BF, RCA, RCB, L, MI, NI, WM, WN>), dim3((unsigned)n), threads, 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.divided) return e;
    hipLaunchKernelGGL((gscan_mm_join_kernel<E, BF, L, MI, NI, WM, WN>),
                       dim3((unsigned)(p.divided * kShares<E, MI, NI>)), threads, 0, st, a);
    return hipGetLastError();
}

// `partial`: mm_bytes() of memory.
template <Epi E, bool RCA, bool RCB, Limit L>
hipError_t launch_mm(MmArgs a, int dtype, void *partial, hipStream_t st)
{
    constexpr bool kGated = E == EPI_GATE || E == EPI_DGATE;
    if (!a.M || !a.N) return hipSuccess;
    const MmPlan p = plan_mm(a.M, a.N, a.K, a.K1, kGated, L != LIMIT_NONE, dtype);
    a.parts = p.parts;
    a.partial = reinterpret_cast<float *>(partial);
    if (!dtype)
        return p.shape == 1 ? launch_shape<E, false, RCA, RCB, L, 2, 2, 2, 2>(a, p, st)
                            : launch_shape<E, false, RCA, RCB, L, 2, 1, 2, 2>(a, p, st);
    return p.shape == 0   ? launch_shape<E, true, RCA, RCB, L, 4, 2, 2, 4>(a, p, st)
           : p.shape == 1 ? launch_shape<E, true, RCA, RCB, L, 2, 2, 2, 2>(a, p, st)
                          : launch_shape<E, true, RCA, RCB, L, 2, 1, 2, 2>(a, p, st);
}

// Tiles of m: the partial results of EPI_LSE for each n.
int64_t tiles_of_m(int64_t M, int64_t N, int64_t K, int dtype)
{
    return ceil_div(M, shape_of(dtype, plan_mm(M, N, K, 0, false, true, dtype).shape).m);
}

}  // namespace
}  // namespace gscan
