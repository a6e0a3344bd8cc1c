// Token embedding, forward and backward, for gfx950 (MI355X).
//
//   out[n] = scale * table[t_n],   dtable[v] = scale * sum of dout[n], t_n = v
//
// Forward: a gather, bound by memory.  Lanes hold eight elements each, a row
// takes as many lanes as it has pieces (a power of two up to the workgroup),
// and every lane group requests several rows before it stores the first.
//
// Backward.  The positions of the tokens are sorted by token (stable, so that
// every row sums its gradients in the order of the positions: no atomics,
// bitwise reproducible), then cut into chunks of equal length.  A workgroup
// takes a chunk and a slice of the columns, adds up the runs of equal tokens
// in registers and writes a row of the table's gradient where the whole run
// lies in its chunk.  Of a run that crosses chunks every chunk leaves a partial
// sum, which a second kernel adds in order: no token, however frequent, is
// walked by one workgroup alone.  Sums are fp32.
//
// Sort: counting by digits of eight bits, from the lowest.  A wavefront takes
// 64 keys at a time; the lanes with the same digit find each other by one
// ballot per bit, which gives every key its rank among those before it.  Up to
// 16384 tokens one workgroup does all digits with the keys in LDS; beyond, each
// digit takes a launch that counts and one that moves.
#include <type_traits>

#include "gscan_lm_dev.h"

namespace gscan {
namespace {

constexpr int kEThreads = 256;
constexpr int kERows = 4;              // rows of a lane group requested together
constexpr int kSThreads = 1024;        // the sort's workgroup,
constexpr int kSWaves = kSThreads / 64;
constexpr int kSItems = 16;            // keys per lane
constexpr int64_t kSBlock = kSThreads * kSItems;
constexpr int kDigits = 256;
constexpr int kChunk = 32;             // positions per chunk, at least
constexpr int kAhead = 8;              // rows a lane requests together
constexpr int64_t kFewBlocks = 64;     // so many histograms every workgroup adds up by itself

template <bool BFI, bool BFO>
__global__ void __launch_bounds__(kEThreads) gscan_embed_fwd_kernel(EmbedArgs a, int lpr)
{
    const int sub = threadIdx.x & (lpr - 1), rpp = kEThreads / lpr;
    const int64_t r0 = (int64_t)blockIdx.x * rpp * kERows + threadIdx.x / lpr;
    int64_t t[kERows];
#pragma unroll
    for (int i = 0; i < kERows; ++i) {
        const int64_t r = r0 + (int64_t)i * rpp;
        t[i] = r < a.N ? token_at(a.tokens, r, a.tok64, a.V) : -1;
    }
    for (int c = 8 * sub; c < a.D; c += 8 * lpr) {
        OctRaw<BFI> x[kERows];
#pragma unroll
        for (int i = 0; i < kERows; ++i) {
            x[i] = OctRaw<BFI>{};
            if (t[i] >= 0) x[i] = load_oct<BFI>(a.table, t[i] * a.ld + c);
        }
#pragma unroll
        for (int i = 0; i < kERows; ++i) {
            const int64_t r = r0 + (int64_t)i * rpp;
            if (r >= a.N) continue;
            Oct y = widen(x[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) y.v[e] = t[i] >= 0 ? y.v[e] * a.scale : 0.f;
            store_oct<BFO>(a.out, r * a.D + c, y);
        }
    }
}

// ---------------------------------------------------------------- the sort

struct SortLds {
    uint32_t hist[kSWaves][kDigits];
    uint32_t total[kDigits], lead[4];
};

// Lanes (of those in `in`) with the same digit.
__device__ __forceinline__ uint64_t peers_of(uint32_t digit, uint64_t in)
{
    uint64_t m = in;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint64_t s = __ballot((digit >> b) & 1u);
        m &= ((digit >> b) & 1u) ? s : ~s;
    }
    return m;
}

// Ranks of the workgroup's n keys by their digit: item (wave, j, lane) is key
// (wave * steps + j) * 64 + lane.  rank[j] counts the equal digits before it
// in its wavefront; the histograms then become, per wavefront and digit, where
// its first key goes among the workgroup's own.
__device__ void rank_keys(SortLds &s, const uint32_t (&key)[kSItems], uint32_t (&rank)[kSItems], int n,
                          int steps, int shift)
{
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    for (int i = tid; i < kSWaves * kDigits; i += kSThreads) s.hist[i / kDigits][i % kDigits] = 0;
    __syncthreads();
    volatile uint32_t *h = s.hist[wave];  // read by lanes that others of the wavefront write for
#pragma unroll
    for (int j = 0; j < kSItems; ++j) {
        const bool in = j < steps && (wave * steps + j) * 64 + lane < n;
        const uint32_t d = (key[j] >> shift) & (kDigits - 1);
        const uint64_t peers = peers_of(d, __ballot(in));
        const uint64_t before = peers & ((1ull << lane) - 1);
        uint32_t seen = 0;
        if (in) seen = h[d];
        rank[j] = seen + (uint32_t)__popcll(before);
        if (in && before == 0) h[d] = seen + (uint32_t)__popcll(peers);
    }
    __syncthreads();
    uint32_t sum = 0;
    if (tid < kDigits) {
        for (int w = 0; w < kSWaves; ++w) {
            const uint32_t c = s.hist[w][tid];
            s.hist[w][tid] = sum;
            sum += c;
        }
        s.total[tid] = sum;
    }
    __syncthreads();
}

// Exclusive sums of x over the first 256 threads, into s.total.
__device__ void scan_digits(SortLds &s, uint32_t x)
{
    const int tid = threadIdx.x, lane = tid & 63;
    uint32_t y = x;
    for (int k = 1; k < 64; k *= 2) {
        const uint32_t o = __shfl_up(y, k);
        if (lane >= k) y += o;
    }
    if (tid < kDigits && lane == 63) s.lead[tid >> 6] = y;
    __syncthreads();
    if (tid < kDigits) {
        for (int w = 0; w < (tid >> 6); ++w) y += s.lead[w];
        s.total[tid] = y - x;
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t key_of(const EmbedArgs &a, int64_t i)
{
    const int64_t t = token_at(a.tokens, i, a.tok64, a.V);
    return t >= 0 ? (uint32_t)t : (uint32_t)a.V;  // padding after everything
}

// All digits at once, up to kSBlock tokens.
__global__ void __launch_bounds__(kSThreads) gscan_sort_small_kernel(EmbedArgs a, int passes, uint32_t *keys,
                                                                    uint32_t *order)
{
    __shared__ SortLds s;
    __shared__ uint32_t lk[kSBlock];
    __shared__ uint16_t lp[kSBlock];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = (int)a.N;
    const int steps = (n + kSThreads - 1) / kSThreads;
    uint32_t key[kSItems], rank[kSItems];
    uint16_t pos[kSItems];
#pragma unroll
    for (int j = 0; j < kSItems; ++j) {
        const int i = (wave * steps + j) * 64 + lane;
        key[j] = 0;
        pos[j] = (uint16_t)i;
        if (j < steps && i < n) key[j] = key_of(a, i);
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = 8 * p;
        rank_keys(s, key, rank, n, steps, shift);
        scan_digits(s, tid < kDigits ? s.total[tid] : 0u);
#pragma unroll
        for (int j = 0; j < kSItems; ++j) {
            if (j < steps && (wave * steps + j) * 64 + lane < n) {
                const uint32_t d = (key[j] >> shift) & (kDigits - 1);
                const uint32_t at = s.total[d] + s.hist[wave][d] + rank[j];
                lk[at] = key[j];
                lp[at] = pos[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSItems; ++j) {
            const int i = (wave * steps + j) * 64 + lane;
            if (j < steps && i < n) {
                key[j] = lk[i];
                pos[j] = lp[i];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kSItems; ++j) {
        const int i = (wave * steps + j) * 64 + lane;
        if (j < steps && i < n) {
            keys[i] = key[j];
            order[i] = pos[j];
        }
    }
}

// One digit of many tokens.  Keys and positions come from the tokens in the
// first pass.  count[block][digit].
template <bool FIRST>
__device__ __forceinline__ void load_keys(const EmbedArgs &a, const uint32_t *keys, const uint32_t *order,
                                          int64_t base, int n, uint32_t (&key)[kSItems],
                                          uint32_t (&pos)[kSItems])
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < kSItems; ++j) {
        const int i = (wave * kSItems + j) * 64 + lane;
        key[j] = pos[j] = 0;
        if (i < n) {
            key[j] = FIRST ? key_of(a, base + i) : keys[base + i];
            pos[j] = FIRST ? (uint32_t)(base + i) : order[base + i];
        }
    }
}

template <bool FIRST>
__global__ void __launch_bounds__(kSThreads) gscan_sort_count_kernel(EmbedArgs a, const uint32_t *keys, int shift,
                                                                    uint32_t *count)
{
    __shared__ uint32_t h[kDigits];
    const int64_t base = (int64_t)blockIdx.x * kSBlock;
    const int n = (int)(a.N - base < kSBlock ? a.N - base : kSBlock);
    if (threadIdx.x < kDigits) h[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSThreads) {
        const uint32_t k = FIRST ? key_of(a, base + i) : keys[base + i];
        atomicAdd(&h[(k >> shift) & (kDigits - 1)], 1u);  // whole numbers: any order
    }
    __syncthreads();
    if (threadIdx.x < kDigits) count[(int64_t)blockIdx.x * kDigits + threadIdx.x] = h[threadIdx.x];
}

// Many workgroups: one per digit turns its counts into sums over the
// workgroups before, and leaves the digit's total behind them.
__global__ void __launch_bounds__(kSThreads) gscan_sort_prefix_kernel(uint32_t *count, int64_t blocks)
{
    __shared__ uint32_t part[kSWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t carry = 0;
    for (int64_t b0 = 0; b0 < blocks; b0 += kSThreads) {
        const int64_t b = b0 + tid;
        const uint32_t x = b < blocks ? count[b * kDigits + blockIdx.x] : 0u;
        uint32_t y = x;
        for (int k = 1; k < 64; k *= 2) {
            const uint32_t o = __shfl_up(y, k);
            if (lane >= k) y += o;
        }
        __syncthreads();
        if (lane == 63) part[wave] = y;
        __syncthreads();
        uint32_t all = 0;
        for (int w = 0; w < kSWaves; ++w) {
            y += w < wave ? part[w] : 0u;
            all += part[w];
        }
        if (b < blocks) count[b * kDigits + blockIdx.x] = carry + y - x;
        carry += all;
    }
    if (tid == 0) count[blocks * kDigits + blockIdx.x] = carry;
}

template <bool FIRST>
__global__ void __launch_bounds__(kSThreads) gscan_sort_move_kernel(EmbedArgs a, const uint32_t *keys,
                                                                   const uint32_t *order, int shift,
                                                                   const uint32_t *count, int64_t blocks,
                                                                   uint32_t *keys_out, uint32_t *order_out)
{
    __shared__ SortLds s;
    __shared__ uint32_t first[kDigits];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t base = (int64_t)blockIdx.x * kSBlock;
    const int n = (int)(a.N - base < kSBlock ? a.N - base : kSBlock);
    uint32_t key[kSItems], pos[kSItems], rank[kSItems];
    load_keys<FIRST>(a, keys, order, base, n, key, pos);
    rank_keys(s, key, rank, n, kSItems, shift);
    uint32_t mine = 0, all = 0;  // of this digit: in workgroups before, in all
    if (tid < kDigits) {
        if (blocks > kFewBlocks) {
            mine = count[(int64_t)blockIdx.x * kDigits + tid];
            all = count[blocks * kDigits + tid];
        } else {
            for (int64_t b = 0; b < blocks; ++b) {
                const uint32_t c = count[b * kDigits + tid];
                mine += b < blockIdx.x ? c : 0u;
                all += c;
            }
        }
    }
    scan_digits(s, all);
    if (tid < kDigits) first[tid] = s.total[tid] + mine;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSItems; ++j) {
        if ((wave * kSItems + j) * 64 + lane < n) {
            const uint32_t d = (key[j] >> shift) & (kDigits - 1);
            const uint32_t at = first[d] + s.hist[wave][d] + rank[j];
            keys_out[at] = key[j];
            order_out[at] = pos[j];
        }
    }
}

// ---------------------------------------------------------------- the sums

template <bool BF>
__global__ void __launch_bounds__(kEThreads) gscan_embed_zero_kernel(void *dtable, int64_t octs)
{
    const int64_t i = (int64_t)blockIdx.x * kEThreads + threadIdx.x;
    if (i < octs) store_oct<BF>(dtable, 8 * i, Oct{});
}

// A chunk's runs over 8 * 64 columns.  part[2 c]: the chunk's first run, which
// began before it; part[2 c + 1]: its last, which goes on.
template <bool BF, bool BFT>
__global__ void __launch_bounds__(64) gscan_embed_sum_kernel(EmbedArgs a, const uint32_t *keys,
                                                            const uint32_t *order, int chunk, float *part)
{
    const int c = (blockIdx.y * 64 + threadIdx.x) * 8;
    const int64_t p0 = (int64_t)blockIdx.x * chunk;
    const int64_t p1 = p0 + chunk < a.N ? p0 + chunk : a.N;
    const bool in = c < a.D;
    bool begun = p0 == 0 || keys[p0 - 1] != keys[p0];  // the run began in this chunk
    Oct sum = {};
    for (int64_t b = p0; b < p1; b += kAhead) {
        OctRaw<BF> x[kAhead];
        uint32_t k[kAhead + 1];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            k[i] = b + i < p1 ? keys[b + i] : (uint32_t)a.V;
            x[i] = OctRaw<BF>{};
            if (in && k[i] < a.V) x[i] = load_oct<BF>(a.dout, (int64_t)order[b + i] * a.ld + c);
        }
        k[kAhead] = b + kAhead < a.N ? keys[b + kAhead] : (uint32_t)a.V;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (k[i] >= a.V) break;
            const Oct v = widen(x[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum.v[e] += v.v[e];
            const bool last = b + i == p1 - 1;
            const uint32_t next = last ? (p1 < a.N ? keys[p1] : (uint32_t)a.V) : k[i + 1];
            const bool ends = next != k[i];
            if (!ends && !last) continue;
            if (in) {
                if (begun && ends) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum.v[e] *= a.scale;
                    store_oct<BFT>(a.dtable, (int64_t)k[i] * a.D + c, sum);
                } else {
                    store_oct<false>(part, (2 * (int64_t)blockIdx.x + (begun ? 1 : 0)) * a.D + c, sum);
                }
            }
            sum = Oct{};
            begun = true;
        }
    }
}

// Runs that began in a chunk and go on: its partial and those of the chunks
// behind, in order.
template <bool BFT>
__global__ void __launch_bounds__(64) gscan_embed_join_kernel(EmbedArgs a, const uint32_t *keys, int chunk,
                                                             const float *part)
{
    const int c = (blockIdx.y * 64 + threadIdx.x) * 8;
    const int64_t chunks = (a.N + chunk - 1) / chunk;
    const int64_t p0 = (int64_t)blockIdx.x * chunk, p1 = p0 + chunk;
    if (p1 >= a.N) return;
    const uint32_t k = keys[p1 - 1];
    if (k >= a.V || keys[p1] != k) return;           // nothing goes on
    if (p0 > 0 && keys[p0 - 1] == k) return;         // nor did it begin here
    if (c >= a.D) return;
    Oct sum = widen(load_oct<false>(part, (2 * (int64_t)blockIdx.x + 1) * a.D + c));
    for (int64_t b = blockIdx.x + 1; b < chunks; b += kAhead) {
        OctRaw<false> x[kAhead];
        bool on[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            on[i] = b + i < chunks && keys[(b + i) * chunk] == k;
            x[i] = OctRaw<false>{};
            if (on[i]) x[i] = load_oct<false>(part, 2 * (b + i) * a.D + c);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const Oct v = widen(x[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum.v[e] += on[i] ? v.v[e] : 0.f;
        }
        if (!on[kAhead - 1]) break;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum.v[e] *= a.scale;
    store_oct<BFT>(a.dtable, (int64_t)k * a.D + c, sum);
}

int lanes_per_row(int D)
{
    int lpr = 1;
    while (lpr < kEThreads && lpr * 8 < D) lpr *= 2;
    return lpr;
}

struct EmbedPlan {
    int passes = 1, chunk = kChunk;
    int64_t blocks = 0, chunks = 0;
    size_t keys[2], order[2], count = 0, part = 0, bytes = 0;
};

size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

// Chunks grow with the tokens, so that a run of all of them has a few thousand
// partials at most.
EmbedPlan plan_embed(int64_t N, int64_t V, int D)
{
    EmbedPlan p;
    while (p.passes < 4 && (V >> (8 * p.passes)) != 0) ++p.passes;  // keys are 0 .. V
    while ((int64_t)p.chunk * p.chunk * 64 < N) p.chunk *= 2;
    p.blocks = (N + kSBlock - 1) / kSBlock;
    p.chunks = (N + p.chunk - 1) / p.chunk;
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        p.keys[i] = at;
        at = round_up(at + (size_t)N * 4);
        p.order[i] = at;
        at = round_up(at + (size_t)N * 4);
        if (p.blocks <= 1) {  // one workgroup: no second copy
            p.keys[1] = p.keys[0];
            p.order[1] = p.order[0];
            break;
        }
    }
    p.count = at;
    if (p.blocks > 1) at = round_up(at + (size_t)(p.blocks + 1) * kDigits * 4);
    p.part = at;
    p.bytes = at + (size_t)p.chunks * 2 * (size_t)D * sizeof(float);
    return p;
}

}  // namespace

size_t embed_workspace_bytes(int64_t N, int64_t V, int D)
{
    return N > 0 ? plan_embed(N, V, D).bytes : 0;
}

hipError_t launch_embed_forward(const EmbedArgs &a, hipStream_t st)
{
    if (!a.N) return hipSuccess;
    const int lpr = lanes_per_row(a.D), rows = kEThreads / lpr * kERows;
    auto *k = a.table_dtype ? (a.dtype ? gscan_embed_fwd_kernel<true, true> : gscan_embed_fwd_kernel<true, false>)
                            : (a.dtype ? gscan_embed_fwd_kernel<false, true> : gscan_embed_fwd_kernel<false, false>);
    hipLaunchKernelGGL(k, dim3((unsigned)((a.N + rows - 1) / rows)), dim3(kEThreads), 0, st, a, lpr);
    return hipGetLastError();
}

hipError_t launch_embed_backward(const EmbedArgs &a, hipStream_t st)
{
    hipError_t e;
    const int64_t octs = a.V * a.D / 8;
    {
        auto *k = a.table_dtype ? gscan_embed_zero_kernel<true> : gscan_embed_zero_kernel<false>;
        hipLaunchKernelGGL(k, dim3((unsigned)((octs + kEThreads - 1) / kEThreads)), dim3(kEThreads), 0, st,
                           a.dtable, octs);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!a.N) return hipSuccess;
    const EmbedPlan p = plan_embed(a.N, a.V, a.D);
    char *ws = reinterpret_cast<char *>(a.ws);
    uint32_t *keys[2], *order[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = reinterpret_cast<uint32_t *>(ws + p.keys[i]);
        order[i] = reinterpret_cast<uint32_t *>(ws + p.order[i]);
    }
    int at = 0;
    if (p.blocks == 1) {
        hipLaunchKernelGGL(gscan_sort_small_kernel, dim3(1), dim3(kSThreads), 0, st, a, p.passes, keys[0],
                           order[0]);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    } else {
        uint32_t *count = reinterpret_cast<uint32_t *>(ws + p.count);
        const dim3 grid((unsigned)p.blocks), blk(kSThreads);
        for (int i = 0; i < p.passes; ++i, at ^= 1) {
            const int shift = 8 * i;
            if (i == 0)
                hipLaunchKernelGGL(gscan_sort_count_kernel<true>, grid, blk, 0, st, a, keys[at ^ 1], shift, count);
            else
                hipLaunchKernelGGL(gscan_sort_count_kernel<false>, grid, blk, 0, st, a, keys[at ^ 1], shift, count);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            if (p.blocks > kFewBlocks) {
                hipLaunchKernelGGL(gscan_sort_prefix_kernel, dim3(kDigits), blk, 0, st, count, p.blocks);
                if ((e = hipGetLastError()) != hipSuccess) return e;
            }
            if (i == 0)
                hipLaunchKernelGGL(gscan_sort_move_kernel<true>, grid, blk, 0, st, a, keys[at ^ 1], order[at ^ 1],
                                   shift, count, p.blocks, keys[at], order[at]);
            else
                hipLaunchKernelGGL(gscan_sort_move_kernel<false>, grid, blk, 0, st, a, keys[at ^ 1],
                                   order[at ^ 1], shift, count, p.blocks, keys[at], order[at]);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        at ^= 1;
    }
    float *part = reinterpret_cast<float *>(ws + p.part);
    const dim3 grid((unsigned)p.chunks, (unsigned)((a.D + 511) / 512)), blk(64);
    auto *sum = a.dtype ? (a.table_dtype ? gscan_embed_sum_kernel<true, true> : gscan_embed_sum_kernel<true, false>)
                        : (a.table_dtype ? gscan_embed_sum_kernel<false, true> : gscan_embed_sum_kernel<false, false>);
    hipLaunchKernelGGL(sum, grid, blk, 0, st, a, keys[at], order[at], p.chunk, part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (p.chunks == 1) return hipSuccess;
    auto *join = a.table_dtype ? gscan_embed_join_kernel<true> : gscan_embed_join_kernel<false>;
    hipLaunchKernelGGL(join, grid, blk, 0, st, a, keys[at], p.chunk, part);
    return hipGetLastError();
}

}  // namespace gscan
