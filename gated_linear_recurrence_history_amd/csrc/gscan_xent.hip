// Cross entropy over a large vocabulary, forward and backward, for gfx950
// (MI355X), without the logits in memory:
//
//   z = scale * h W^T,  lse_n = log sum over v of exp(z_nv),
//   loss_n = lse_n - z_n,target
//   G_nv = scale * u_n * (exp(z_nv - lse_n) - [v is the target]),
//   dh = G W,  dW = G^T h         (u_n: the gradient that reaches loss_n)
//
// Where all u are one (a sum, a mean) they are left out of G and multiply the
// outputs: most of G is the -1 at the targets, which is then exact, where the
// rounding of -u would be the same for every token and move the whole gradient.
//
// Forward: every tile of the product leaves, for each token, the maximum of its
// logits and the sum of their exponentials relative to it; a second kernel joins
// a token's.  Backward: the vocabulary is taken in pieces.  Of a piece, G is
// formed from the product again and rounded to the type of the operands once;
// it adds to dh (fp32 between the pieces) and makes the piece's rows of dW
// whole.
//
// Tokens that do not count (their target is outside the vocabulary) are left
// out: a first kernel lists the others, and where some are missing copies their rows
// so that they follow each other.  What is in the rows left out, NaN
// included, reaches nothing.
//
// The products bound all of it: 8192 tokens, 2048 x 32000, forward 908 us (1183 TFLOP/s), of
// which the list and the joins are 17.
#include "gscan_few.h"

namespace gscan {
namespace {

constexpr int kLThreads = 1024;
// G of a piece (more where 2048 columns, the least, take more: from 131072 bf16 or 65536 fp32
// tokens on).  Gradients of 16384 tokens with 256, 512 and 1023 MiB: 512 x 65000, 3730, 3430
// and 3330 us; 2048 x 65000, 10830, 10580 and 10930; of 6007 tokens, 1024 x 50021, 1600, 1560
// and 1590.
constexpr int64_t kPieceBytes = 512ll << 20;
constexpr int kJoinRows = 16;
constexpr int kListGroups = 256;

// By place among the tokens that count.
struct Listed {
    int32_t *count = nullptr, *row = nullptr, *target = nullptr;
    float *factor = nullptr, *up = nullptr, *lse = nullptr, *picked = nullptr, *loss = nullptr;
    void *h = nullptr;          // their rows, where some do not count
    float2 *part = nullptr;
    void *g = nullptr;
    float *sum = nullptr;
    void *partial = nullptr;    // of tiles
    int64_t piece = 0;
    size_t bytes = 0;
};

Listed lay_out(void *ws, int64_t N, int64_t V, int D, int dtype, bool backward)
{
    const size_t es = dtype ? 2 : 4;
    Listed l;
    size_t at = 0;
    auto take = [&](size_t bytes) -> void * {
        void *p = reinterpret_cast<char *>(ws) + at;
        at = (at + bytes + 255) & ~(size_t)255;
        return p;
    };
    l.count = (int32_t *)take(4);
    l.row = (int32_t *)take((size_t)N * 4);
    l.target = (int32_t *)take((size_t)N * 4);
    l.h = take((size_t)N * D * es);
    if (backward) {
        l.factor = (float *)take(4);
        l.up = (float *)take((size_t)N * 4);
        l.lse = (float *)take((size_t)N * 4);
        // whole tiles, at least 2048 columns
        const int64_t fit = N > 0 ? kPieceBytes / (N * (int64_t)es) / 256 * 256 : V;
        l.piece = fit < 2048 ? 2048 : fit;
        if (l.piece > V) l.piece = V;
        const int64_t ld = (l.piece + 7) / 8 * 8;
        l.g = take((size_t)N * ld * es);
        if (l.piece < V) l.sum = (float *)take((size_t)N * D * 4);
        size_t parts = 0;
        for (const int64_t v : {l.piece, V % l.piece}) {  // a last piece is smaller
            if (!v) continue;
            for (const size_t b : {mm_bytes(v, N, D, 0, false, true, dtype), mm_bytes(D, N, v, 0, false, true, dtype),
                                   mm_bytes(D, v, N, 0, false, true, dtype)})
                if (b > parts) parts = b;
        }
        l.partial = take(parts);
    } else {
        l.picked = (float *)take((size_t)N * 4);
        l.loss = (float *)take((size_t)N * 4);
        size_t parts = (size_t)tiles_of_m(V, N, D, dtype);
        if (N <= kFew && parts < (size_t)kFewGrid) parts = (size_t)kFewGrid;
        l.part = (float2 *)take(parts * N * sizeof(float2));
        l.partial = take(mm_bytes(V, N, D, 0, false, true, dtype));
    }
    l.bytes = at;
    return l;
}

// The workgroup's sum of a number per wavefront, and of the wavefronts before this one.
__device__ __forceinline__ int sum_before(int32_t (&n_of)[kLThreads / 64], int own, int &all)
{
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) n_of[wave] = own;
    __syncthreads();
    int before = 0;
    all = 0;
    for (int w = 0; w < kLThreads / 64; ++w) {
        before += w < wave ? n_of[w] : 0;
        all += n_of[w];
    }
    return before;
}

// Lists the tokens that count, in order, 1024 ITEMS at a time; where some do not, copies
// of the others' rows, one after the other, and zeros for the gradients of those that do
// not.  Every workgroup goes through all targets, chunk after chunk, twice if there are
// more than one; the first one writes the list, each some of the rows.  Up to 8192 tokens
// that costs less than a launch of its own for the rows; it grows with the tokens: 8192,
// 65536 and 2^20 take 6, 43 and 695 us, with rows of 1024 bf16 to copy (an eighth left
// out) 12, 67 and 1320, beside 0.5, 4 and 60 ms of products for the losses of 32000 classes.
template <bool BWD, int ITEMS>
__global__ void __launch_bounds__(kLThreads) gscan_xent_list_kernel(XentArgs a, Listed l)
{
    constexpr int kChunk = kLThreads * ITEMS, kOwn = kChunk / kListGroups;
    __shared__ int32_t n_of[kLThreads / 64];
    __shared__ int32_t place[kOwn];  // of the workgroup's tokens among those that count, or -1
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, o0 = wave * (64 * ITEMS) + lane;
    const bool first_group = blockIdx.x == 0;
    int64_t count = 0, done = 0;
    if (a.N > kChunk) {
        for (int64_t b = 0; b < a.N; b += kChunk) {
            uint32_t key[ITEMS];
            token_keys<ITEMS>(a.target, a.target64, a.V, b + o0, a.N, key);
            int own = 0, all;
#pragma unroll
            for (int j = 0; j < ITEMS; ++j) own += __popcll(__ballot(key[j] < (uint32_t)a.V));
            sum_before(n_of, own, all);
            count += all;
        }
    }
    for (int64_t b = 0; b < a.N; b += kChunk) {
        uint32_t key[ITEMS];
        float lse[ITEMS], up[ITEMS];
        token_keys<ITEMS>(a.target, a.target64, a.V, b + o0, a.N, key);
        int own = 0, all;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const bool in = key[j] < (uint32_t)a.V;
            lse[j] = BWD && in && first_group ? a.lse[b + o0 + 64 * j] : 0.f;
            up[j] = BWD && in && first_group && !a.reduction ? a.dloss[b + o0 + 64 * j] : 0.f;
            own += __popcll(__ballot(in));
        }
        int64_t first = done + sum_before(n_of, own, all);
        done += all;
        if (a.N <= kChunk) count = done;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const int64_t i = b + o0 + 64 * j;
            const uint64_t some = __ballot(key[j] < (uint32_t)a.V);
            const bool in = key[j] < (uint32_t)a.V;
            const int64_t at = first + __popcll(some & ((1ull << lane) - 1));
            first += __popcll(some);
            if ((o0 + 64 * j) / kOwn == (int)blockIdx.x) place[(o0 + 64 * j) % kOwn] = in ? (int32_t)at : -1;
            if (!first_group) continue;
            if (in) {
                l.row[at] = (int32_t)i;
                l.target[at] = (int32_t)key[j];
                if (BWD) l.lse[at] = lse[j];
                if (BWD && !a.reduction) l.up[at] = a.scale * up[j];
            } else if (!BWD && i < a.N) {
                a.lse[i] = 0.f;
                (a.reduction ? l.loss : a.loss)[i] = 0.f;
            }
        }
        if (count == a.N) continue;
        __syncthreads();
        for (int r = wave; r < kOwn; r += kLThreads / 64) {
            const int64_t i = b + (int64_t)blockIdx.x * kOwn + r;
            if (i >= a.N) break;
            const int64_t at = place[r];
            for (int c = 8 * lane; c < a.D; c += 8 * 64) {
                if (at < 0) {
                    if (!BWD || !a.dh) break;
                    if (a.dtype) store_oct<true>(a.dh, i * a.D + c, Oct{});
                    else store_oct<false>(a.dh, i * a.D + c, Oct{});
                } else if (a.dtype) {
                    reinterpret_cast<u4 *>(l.h)[(at * a.D + c) / 8] = load_oct<true>(a.h, i * a.ldh + c).a;
                } else {
                    const OctRaw<false> x = load_oct<false>(a.h, i * a.ldh + c);
                    reinterpret_cast<f4 *>(l.h)[(at * a.D + c) / 4] = x.a;
                    reinterpret_cast<f4 *>(l.h)[(at * a.D + c) / 4 + 1] = x.b;
                }
            }
        }
    }
    if (!first_group || tid) return;
    *l.count = (int32_t)done;
    // (no token: sums of nothing are zero, also times a gradient that is no number)
    if (BWD && a.reduction) *l.factor = done ? a.scale * *a.dloss / (a.reduction == 2 ? (float)done : 1.f) : 0.f;
}

// A token's partial results: 16 tokens, 16 lanes each.
__global__ void __launch_bounds__(256) gscan_xent_join_kernel(XentArgs a, Listed l, int64_t parts)
{
    __shared__ float2 red[16][kJoinRows];
    const int r = threadIdx.x & 15, q = threadIdx.x >> 4;
    const int64_t count = *l.count;
    for (int64_t n0 = (int64_t)blockIdx.x * kJoinRows; n0 < count; n0 += (int64_t)gridDim.x * kJoinRows) {
        const int64_t n = n0 + r;
        float m = -INFINITY, s = 0.f;
        if (n < count)
            for (int64_t p = q; p < parts; p += 16) {
                const float2 x = l.part[p * a.N + n];
                join_lse(m, s, x.x, x.y);
            }
        __syncthreads();
        red[q][r] = float2{m, s};
        __syncthreads();
        if (q == 0 && n < count) {
            for (int i = 1; i < 16; ++i) join_lse(m, s, red[i][r].x, red[i][r].y);
            const float tail = log2f(s), unit = 0.69314718055994531f;
            const int64_t i = l.row[n];
            a.lse[i] = (m + tail) * unit;
            (a.reduction ? l.loss : a.loss)[i] = (m - l.picked[n] + tail) * unit;
        }
    }
}

__global__ void __launch_bounds__(kLThreads) gscan_xent_total_kernel(XentArgs a, Listed l)
{
    __shared__ double red[kLThreads];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < a.N; i += kLThreads) s += (double)l.loss[i];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int h = kLThreads / 2; h > 0; h /= 2) {
        if (threadIdx.x < h) red[threadIdx.x] += red[threadIdx.x + h];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const int32_t n = *l.count;
        *a.loss = (float)(a.reduction == 2 && n ? red[0] / n : red[0]);
    }
}

// Few tokens: a wavefront joins a token's partial results, and the last step of a sum or
// a mean is the workgroup's.
__global__ void __launch_bounds__(kLThreads) gscan_xent_few_join_kernel(XentArgs a, Listed l, int parts)
{
    __shared__ float losses[kFew];
    __shared__ int counted[kFew];
    const int lane = threadIdx.x & 63;
    for (int n = threadIdx.x >> 6; n < a.N; n += kLThreads / 64) {
        float m = -INFINITY, s = 0.f;
        float2 x[kFewGrid / 64];
#pragma unroll
        for (int i = 0; i < kFewGrid / 64; ++i) {
            x[i] = float2{-INFINITY, 0.f};
            if (lane + 64 * i < parts) x[i] = l.part[(int64_t)n * parts + lane + 64 * i];
        }
#pragma unroll
        for (int i = 0; i < kFewGrid / 64; ++i) join_lse(m, s, x[i].x, x[i].y);
        for (int k = 32; k > 0; k /= 2) join_lse(m, s, __shfl_xor(m, k), __shfl_xor(s, k));
        if (lane) continue;
        const bool counts = token_at(a.target, n, a.target64, a.V) >= 0;
        const float tail = log2f(s), unit = 0.69314718055994531f;
        a.lse[n] = counts ? (m + tail) * unit : 0.f;
        counted[n] = counts;
        losses[n] = counts ? (m - l.picked[n] + tail) * unit : 0.f;
        if (!a.reduction) a.loss[n] = losses[n];
    }
    if (!a.reduction) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
        int count = 0;
        for (int n = 0; n < a.N; ++n) {
            all += (double)losses[n];
            count += counted[n];
        }
        *a.loss = (float)(a.reduction == 2 && count ? all / count : all);
    }
}

hipError_t launch_list(const XentArgs &x, const Listed &l, bool backward, hipStream_t st)
{
    auto *list = x.N <= kLThreads ? (backward ? gscan_xent_list_kernel<true, 1> : gscan_xent_list_kernel<false, 1>)
                                  : (backward ? gscan_xent_list_kernel<true, 8> : gscan_xent_list_kernel<false, 8>);
    const int64_t own = (x.N <= kLThreads ? 1 : 8) * kLThreads / kListGroups, n = (x.N + own - 1) / own;
    hipLaunchKernelGGL(list, dim3((unsigned)(n < 1 ? 1 : n < kListGroups ? n : kListGroups)), dim3(kLThreads), 0, st, x,
                       l);
    return hipGetLastError();
}

MmArgs logits_of(const XentArgs &x, const Listed &l, int64_t v0, int64_t v1)
{
    MmArgs a;
    a.a = reinterpret_cast<const char *>(x.w) + v0 * x.ldw * (x.dtype ? 2 : 4);
    a.lda = x.ldw;
    a.b = x.h;
    a.ldb = x.ldh;
    a.M = v1 - v0;
    a.N = x.N;
    a.K = x.D;
    a.count = l.count;
    a.alt = l.h;
    a.ldalt = x.D;
    a.target = l.target;
    a.v0 = v0;
    a.scale = x.scale;
    return a;
}

}  // namespace

size_t xent_forward_workspace_bytes(int64_t N, int64_t V, int D, int dtype)
{
    return lay_out(nullptr, N, V, D, dtype, false).bytes;
}

size_t xent_backward_workspace_bytes(int64_t N, int64_t V, int D, int dtype)
{
    return lay_out(nullptr, N, V, D, dtype, true).bytes;
}

hipError_t launch_xent_forward(const XentArgs &x, hipStream_t st)
{
    const Listed l = lay_out(x.ws, x.N, x.V, x.D, x.dtype, false);
    hipError_t e;
    if (x.N && x.N <= kFew) {
        MmArgs a = logits_of(x, l, 0, x.V);
        a.part = l.part;
        a.picked = l.picked;
        a.tokens = x.target;
        a.tok64 = x.target64;
        if ((e = launch_few<EPI_LSE>(a, x.dtype, st)) != hipSuccess) return e;
        hipLaunchKernelGGL(gscan_xent_few_join_kernel, dim3(1), dim3(kLThreads), 0, st, x, l, few_grid(few_groups<EPI_LSE>(a)));
        return hipGetLastError();
    }
    if ((e = launch_list(x, l, false, st)) != hipSuccess) return e;
    if (x.N) {
        MmArgs a = logits_of(x, l, 0, x.V);
        a.part = l.part;
        a.picked = l.picked;
        if ((e = launch_mm<EPI_LSE, false, false, LIMIT_N>(a, x.dtype, l.partial, st)) != hipSuccess) return e;
        hipLaunchKernelGGL(gscan_xent_join_kernel, groups_of((x.N + kJoinRows - 1) / kJoinRows), dim3(256), 0, st, x, l, tiles_of_m(x.V, x.N, x.D, x.dtype));
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!x.reduction) return hipSuccess;
    hipLaunchKernelGGL(gscan_xent_total_kernel, dim3(1), dim3(kLThreads), 0, st, x, l);
    return hipGetLastError();
}

hipError_t launch_xent_backward(const XentArgs &x, hipStream_t st)
{
    const Listed l = lay_out(x.ws, x.N, x.V, x.D, x.dtype, true);
    const size_t es = x.dtype ? 2 : 4;
    hipError_t e = launch_list(x, l, true, st);
    if (e != hipSuccess) return e;
    for (int64_t v0 = 0; v0 < x.V; v0 += l.piece) {
        const int64_t v1 = v0 + l.piece < x.V ? v0 + l.piece : x.V;
        const int64_t ld = (v1 - v0 + 7) / 8 * 8;
        if (x.N) {
            MmArgs a = logits_of(x, l, v0, v1);
            a.up = x.reduction ? nullptr : l.up;
            a.lse = l.lse;
            a.out = l.g;
            a.ldo = ld;
            if ((e = launch_mm<EPI_DLOGIT, false, false, LIMIT_N>(a, x.dtype, l.partial, st)) != hipSuccess) return e;
        }
        if (x.dh && x.N) {
            MmArgs a;
            a.a = reinterpret_cast<const char *>(x.w) + (size_t)v0 * x.ldw * es;
            a.lda = x.ldw;
            a.b = l.g;
            a.ldb = ld;
            a.M = x.D;
            a.N = x.N;
            a.K = v1 - v0;
            a.count = l.count;
            a.row = l.row;
            a.out = x.dh;
            a.ldo = x.D;
            a.sum = l.sum;
            a.factor = x.reduction ? l.factor : nullptr;
            a.first = v0 == 0;
            a.last = v1 == x.V;
            if ((e = launch_mm<EPI_ADD, true, false, LIMIT_N>(a, x.dtype, l.partial, st)) != hipSuccess) return e;
        }
        if (x.dw) {  // zeros without tokens
            MmArgs a;
            a.a = x.h;
            a.lda = x.ldh;
            a.b = l.g;
            a.ldb = ld;
            a.M = x.D;
            a.N = v1 - v0;
            a.N1 = a.N;
            a.K = x.N;
            a.count = l.count;
            a.alt = l.h;
            a.ldalt = x.D;
            a.out = reinterpret_cast<char *>(x.dw) + (size_t)v0 * x.D * es;
            a.ldo = x.D;
            a.factor = x.reduction ? l.factor : nullptr;
            if ((e = launch_mm<EPI_STORE, true, true, LIMIT_K>(a, x.dtype, l.partial, st)) != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace gscan
