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
// bitwise reproducible), then cut into chunks of equal length.  A wavefront takes a
// chunk and 512 of the columns, adds up the runs of equal tokens in registers and
// writes a row of the table's gradient where the whole run lies in its chunk.  Of a
// run that crosses chunks every chunk leaves a partial sum, which a second kernel
// adds in order: no token, however frequent, is walked by one wavefront alone.
// Sums are fp32.  Rows without a token are zeros, which other workgroups write
// meanwhile: beside the one that sorts few tokens, whose tokens they mark in a bit per
// row of theirs, or beside the sums of many, looking their rows up among the sorted
// tokens.  Every row is written once.
//
// Sort: counting by digits of eight bits, from the lowest.  A wavefront takes
// 64 keys at a time; the lanes with the same digit find each other by one
// ballot per bit, which gives every key its rank among those before it.  Up to
// 16384 tokens (of a vocabulary below 2^18: token and position share a word) one
// workgroup does all digits with the keys in LDS; else each digit takes a launch that
// counts and one that moves.
#include <type_traits>

#include "gscan_lm_dev.h"

namespace gscan {
namespace {

constexpr int kEThreads = 256;
constexpr int kERows = 4;              // rows of a lane group requested together
constexpr int kSThreads = 1024;        // the sort's workgroup,
constexpr int kSWaves = kSThreads / 64;
constexpr int kSItems = 8;             // keys per lane of many workgroups
constexpr int64_t kSBlock = kSThreads * kSItems;
constexpr int64_t kSSmall = 16384;     // tokens that one workgroup sorts
constexpr int kPosBits = 14;           // of their positions
constexpr int kDigits = 256;
constexpr int kAhead = 16;             // rows a lane requests together
constexpr int64_t kFewBlocks = 64;     // so many histograms every workgroup adds up by itself
constexpr int kZeroRows = 64;          // rows of the table that a workgroup looks up,
constexpr int kMarkRows = 1024;        // or marks, at most

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
// (wave * ITEMS + j) * 64 + lane.  rank[j] counts the equal digits before it
// in its wavefront; the histograms then become, per wavefront and digit, where
// its first key goes among the workgroup's own.
template <int ITEMS>
__device__ __forceinline__ void rank_keys(SortLds &s, const uint32_t (&key)[ITEMS], uint32_t (&rank)[ITEMS], int n,
                                          int shift)
{
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    for (int i = tid; i < kSWaves * kDigits; i += kSThreads) s.hist[i / kDigits][i % kDigits] = 0;
    __syncthreads();
    volatile uint32_t *h = s.hist[wave];  // read by lanes that others of the wavefront write for
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const bool in = (wave * ITEMS + j) * 64 + lane < n;
        const uint32_t d = (key[j] >> shift) & (kDigits - 1);
        const uint64_t peers = peers_of(d, __ballot(in));
        const uint32_t before = __builtin_amdgcn_mbcnt_hi((uint32_t)(peers >> 32),
                                                          __builtin_amdgcn_mbcnt_lo((uint32_t)peers, 0u));
        uint32_t seen = 0;
        if (in) seen = h[d];
        rank[j] = seen + before;
        if (in && before == 0) h[d] = seen + (uint32_t)__popcll(peers);
    }
    __syncthreads();
    if (tid < kDigits) {
        uint32_t c[kSWaves], sum = 0;
#pragma unroll
        for (int w = 0; w < kSWaves; ++w) c[w] = s.hist[w][tid];
#pragma unroll
        for (int w = 0; w < kSWaves; ++w) {
            s.hist[w][tid] = sum;
            sum += c[w];
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

// Zeros for the rows first .. first + rows - 1 that no token has.
template <bool BFT>
__device__ __forceinline__ void zero_unmarked(const EmbedArgs &a, int64_t first, int rows)
{
    __shared__ uint32_t marks[kMarkRows / 32];
    if (threadIdx.x < kMarkRows / 32) marks[threadIdx.x] = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < a.N; i += kSThreads) {
        const int64_t r = token_at(a.tokens, i, a.tok64, a.V) - first;
        if (r >= 0 && r < rows) atomicOr(&marks[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    const int octs = a.D / 8;
    for (int r = threadIdx.x >> 6; r < rows; r += kSWaves) {
        if (marks[r >> 5] >> (r & 31) & 1u) continue;
        for (int c = threadIdx.x & 63; c < octs; c += 64) store_oct<BFT>(a.dtable, (first + r) * a.D + 8 * c, Oct{});
    }
}

// All digits at once, up to 1024 ITEMS tokens, by the first workgroup; the others
// take `rows` rows of the table each and write zeros.
template <int ITEMS>
__global__ void __launch_bounds__(kSThreads) gscan_sort_small_kernel(EmbedArgs a, int passes, int rows, uint32_t *keys,
                                                                    uint32_t *order)
{
    if (blockIdx.x > 0) {
        const int64_t first = (int64_t)(blockIdx.x - 1) * rows;
        const int n = (int)(a.V - first < rows ? a.V - first : rows);
        if (a.table_dtype) zero_unmarked<true>(a, first, n);
        else zero_unmarked<false>(a, first, n);
        return;
    }
    __shared__ SortLds s;
    __shared__ uint32_t moved[kSThreads * ITEMS];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = (int)a.N;
    uint32_t item[ITEMS], rank[ITEMS];  // token and position
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const int i = (wave * ITEMS + j) * 64 + lane;
        item[j] = i < n ? key_of(a, i) << kPosBits | (uint32_t)i : 0u;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = kPosBits + 8 * p;
        rank_keys<ITEMS>(s, item, rank, n, shift);
        scan_digits(s, tid < kDigits ? s.total[tid] : 0u);
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            if ((wave * ITEMS + j) * 64 + lane < n) {
                const uint32_t d = (item[j] >> shift) & (kDigits - 1);
                moved[s.total[d] + s.hist[wave][d] + rank[j]] = item[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
            const int i = (wave * ITEMS + j) * 64 + lane;
            if (i < n) item[j] = moved[i];
        }
    }
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const int i = (wave * ITEMS + j) * 64 + lane;
        if (i < n) {
            keys[i] = item[j] >> kPosBits;
            order[i] = item[j] & ((1u << kPosBits) - 1);
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
    rank_keys<kSItems>(s, key, rank, n, shift);
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

// Zeros for the rows first .. first + kZeroRows - 1 that no token has.
template <bool BFT>
__device__ __forceinline__ void zero_rows(const EmbedArgs &a, const uint32_t *keys, int64_t first)
{
    __shared__ uint32_t absent[kZeroRows], count;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    const int64_t row = first + threadIdx.x;
    if (threadIdx.x < kZeroRows && row < a.V) {
        int64_t lo = 0, hi = a.N;  // the first key that is not below the row
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (keys[mid] < (uint32_t)row) lo = mid + 1;
            else hi = mid;
        }
        if (lo == a.N || keys[lo] != (uint32_t)row) absent[atomicAdd(&count, 1u)] = threadIdx.x;
    }
    __syncthreads();
    const int octs = a.D / 8;
    for (uint32_t r = 0; r < count; ++r)
        for (int c = threadIdx.x; c < octs; c += kEThreads)
            store_oct<BFT>(a.dtable, (first + absent[r]) * a.D + 8 * c, Oct{});
}

// A chunk's runs over 8 * 64 columns for each wavefront; behind the chunks'
// workgroups, those that write zeros.  part[2 c]: the chunk's first run, which
// began before it; part[2 c + 1]: its last, which goes on.
template <bool BF, bool BFT>
__global__ void __launch_bounds__(kEThreads) gscan_embed_sum_kernel(EmbedArgs a, const uint32_t *keys,
                                                                   const uint32_t *order, int chunk, int64_t waves,
                                                                   int slices, float *part)
{
    const int64_t groups = (waves + 3) / 4;
    // every second workgroup writes zeros while there are such: their stores run
    // beside the others' loads
    const int64_t zeros = gridDim.x - groups, both = 2 * (zeros < groups ? zeros : groups);
    int64_t id = blockIdx.x;
    const bool zero = id < both ? id % 2 == 1 : zeros > groups;
    id = id < both ? id / 2 : id - both / 2;
    if (zero) {
        zero_rows<BFT>(a, keys, id * kZeroRows);
        return;
    }
    const int64_t w = id * 4 + (threadIdx.x >> 6);
    if (w >= waves) return;
    const int lane = threadIdx.x & 63, c = (int)(w % slices) * 512 + lane * 8;
    const int64_t at = w / slices, p0 = at * chunk;
    const int n = (int)(a.N - p0 < chunk ? a.N - p0 : chunk);
    const bool in = c < a.D;
    Oct sum = {};
    bool begun = true;  // the run began in this chunk
    for (int b = 0; b < n; b += 32) {
        // the next 32 keys, the one behind them (lane 32) and the one before (63), 32 positions
        const int64_t i = lane == 63 ? p0 + b - 1 : p0 + b + lane;
        const uint32_t mine = (lane <= 32 || lane == 63) && i >= 0 && i < a.N ? keys[i] : (uint32_t)a.V;
        const uint32_t from = lane < 32 && i < a.N ? order[i] : 0u;
        const int m = n - b < 32 ? n - b : 32;
        if (b == 0) begun = __builtin_amdgcn_readlane(mine, 63) != __builtin_amdgcn_readlane(mine, 0);
        for (int g = 0; g < m; g += kAhead) {
            OctRaw<BF> x[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t row = (int64_t)__builtin_amdgcn_readlane(from, g + k);
                x[k] = OctRaw<BF>{};
                if (in && g + k < m && (uint32_t)__builtin_amdgcn_readlane(mine, g + k) < a.V)
                    x[k] = load_oct<BF>(a.dout, row * a.ld + c);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t key = __builtin_amdgcn_readlane(mine, g + k);
                if (g + k >= m || key >= a.V) break;
                const Oct v = widen(x[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum.v[e] += v.v[e];
                const bool last = b + g + k == n - 1;
                const bool ends = (uint32_t)__builtin_amdgcn_readlane(mine, g + k + 1) != key;
                if (!ends && !last) continue;
                if (in) {
                    if (begun && ends) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum.v[e] *= a.scale;
                        store_oct<BFT>(a.dtable, (int64_t)key * a.D + c, sum);
                    } else {
                        store_oct<false>(part, (2 * at + (begun ? 1 : 0)) * a.D + c, sum);
                    }
                }
                sum = Oct{};
                begun = true;
            }
        }
    }
}

// Runs that began in a chunk and go on: its partial and those of the chunks
// behind, in order.
template <bool BFT>
__global__ void __launch_bounds__(kEThreads) gscan_embed_join_kernel(EmbedArgs a, const uint32_t *keys, int chunk,
                                                                    int64_t waves, int slices, const float *part)
{
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (w >= waves) return;
    const int lane = threadIdx.x & 63, c = (int)(w % slices) * 512 + lane * 8;
    const int64_t at = w / slices, chunks = (a.N + chunk - 1) / chunk;
    const int64_t p0 = at * chunk, p1 = p0 + chunk;
    if (p1 >= a.N) return;
    const uint32_t k = keys[p1 - 1], after = keys[p1], before = p0 > 0 ? keys[p0 - 1] : (uint32_t)a.V;
    if (k >= a.V || after != k || before == k) return;  // nothing goes on, nor did it begin here
    const bool in = c < a.D;
    Oct sum = {};
    if (in) sum = widen(load_oct<false>(part, (2 * at + 1) * a.D + c));
    for (int64_t b = at + 1; b < chunks; b += 64) {
        const uint64_t on = __ballot(b + lane < chunks && keys[(b + lane < chunks ? b + lane : b) * chunk] == k);
        const int m = __builtin_popcountll(on);  // they follow each other
        for (int g = 0; g < m; g += kAhead / 2) {
            OctRaw<false> x[kAhead / 2];
#pragma unroll
            for (int i = 0; i < kAhead / 2; ++i) {
                x[i] = OctRaw<false>{};
                if (in && g + i < m) x[i] = load_oct<false>(part, 2 * (b + g + i) * a.D + c);
            }
#pragma unroll
            for (int i = 0; i < kAhead / 2; ++i) {
                const Oct v = widen(x[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum.v[e] += g + i < m ? v.v[e] : 0.f;
            }
        }
        if (m < 64) break;
    }
    if (!in) return;
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
    int passes = 1, chunk = 8;
    bool small = false;         // one workgroup sorts
    int64_t blocks = 0, chunks = 0;
    size_t keys[2], order[2], count = 0, part = 0, bytes = 0;
};

size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

// Chunks grow with the tokens, for a few thousand wavefronts at widths that fill them, and so
// that a run of all tokens has a few thousand partials at most.
EmbedPlan plan_embed(int64_t N, int64_t V, int D)
{
    EmbedPlan p;
    while (p.passes < 4 && (V >> (8 * p.passes)) != 0) ++p.passes;  // keys are 0 .. V
    while (p.chunk < 32 ? (int64_t)p.chunk * 512 < N : (int64_t)p.chunk * p.chunk * 64 < N) p.chunk *= 2;
    p.small = N <= kSSmall && V < int64_t(1) << (32 - kPosBits);
    p.blocks = (N + kSBlock - 1) / kSBlock;
    p.chunks = (N + p.chunk - 1) / p.chunk;
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        p.keys[i] = at;
        at = round_up(at + (size_t)N * 4);
        p.order[i] = at;
        at = round_up(at + (size_t)N * 4);
        if (p.small) {  // no second copy
            p.keys[1] = p.keys[0];
            p.order[1] = p.order[0];
            break;
        }
    }
    p.count = at;
    if (!p.small) at = round_up(at + (size_t)(p.blocks + 1) * kDigits * 4);
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
    const EmbedPlan p = plan_embed(a.N, a.V, a.D);
    char *ws = reinterpret_cast<char *>(a.ws);
    uint32_t *keys[2], *order[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = reinterpret_cast<uint32_t *>(ws + p.keys[i]);
        order[i] = reinterpret_cast<uint32_t *>(ws + p.order[i]);
    }
    int at = 0;
    if (!a.N) {
        // only zeros
    } else if (p.small) {
        const int items = (int)((a.N + kSThreads - 1) / kSThreads);
        auto *k = items <= 1   ? gscan_sort_small_kernel<1>
                  : items <= 2 ? gscan_sort_small_kernel<2>
                  : items <= 4 ? gscan_sort_small_kernel<4>
                  : items <= 8 ? gscan_sort_small_kernel<8>
                               : gscan_sort_small_kernel<16>;
        int64_t rows = (a.V + 254) / 255;  // a workgroup per CU, of which one sorts
        if (rows > kMarkRows) rows = kMarkRows;
        hipLaunchKernelGGL(k, dim3((unsigned)(1 + (a.V + rows - 1) / rows)), dim3(kSThreads), 0, st, a, p.passes,
                           (int)rows, keys[0], order[0]);
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
    const int slices = (a.D + 511) / 512;
    const int64_t waves = p.chunks * slices, groups = (waves + 3) / 4;
    const int64_t zeros = p.small && a.N ? 0 : (a.V + kZeroRows - 1) / kZeroRows;
    const dim3 blk(kEThreads);
    auto *sum = a.dtype ? (a.table_dtype ? gscan_embed_sum_kernel<true, true> : gscan_embed_sum_kernel<true, false>)
                        : (a.table_dtype ? gscan_embed_sum_kernel<false, true> : gscan_embed_sum_kernel<false, false>);
    hipLaunchKernelGGL(sum, dim3((unsigned)(groups + zeros)), blk, 0, st, a, keys[at], order[at], p.chunk, waves,
                       slices, part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (p.chunks <= 1) return hipSuccess;
    auto *join = a.table_dtype ? gscan_embed_join_kernel<true> : gscan_embed_join_kernel<false>;
    hipLaunchKernelGGL(join, dim3((unsigned)groups), blk, 0, st, a, keys[at], p.chunk, waves, slices, part);
    return hipGetLastError();
}

}  // namespace gscan
