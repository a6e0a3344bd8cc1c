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
// Sums are fp32.  Rows without a token are zeros.  Every row is written once.
//
// Sort, up to 32768 tokens (and 2^20 rows): every workgroup has up to 256 rows of the
// table, goes through all tokens, counts those of the rows before its own and sorts its
// own by their row; it also writes its rows' zeros.  One launch for any number of
// rows, and hardly any work for most wavefronts: they skip 64 tokens of which none is
// theirs after a comparison (16384 tokens of 32000 rows: 16 us; one workgroup that sorts
// them all by two digits took 30).  Up to 2048 tokens (rows of more than 512: 64) the
// workgroup adds them up as well, and nothing else is launched: 777 tokens, 1003 rows
// of 200 fp32, 7.5 us, with the sums and their join in launches of their own 15; rows
// of 2048 are the other way round from there on (777 tokens, 32000 rows: 58 to 70 us
// against 56), as the workgroups with frequent tokens add up slice after slice.
// More tokens are sorted by digits of eight bits, from the lowest, with a launch that
// counts and one that moves for each; zeros are then written beside the sums, by
// workgroups that look their rows up among the sorted tokens.
// Ranks: a wavefront takes 64 keys at a time; the lanes with the same digit find each
// other by one ballot per bit, which gives every key its rank among those before it.
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
constexpr int64_t kSFew = 2048;        // tokens that are sorted and added up at once,
constexpr int64_t kSWide = 64;         // of wide rows these,
constexpr int kFewItems = (int)kSFew / kSThreads;
// and that are sorted by one launch, of a table of fewer rows, and tokens times rows.  The whole
// gradient of 64 columns, fp32 of bf16: 65536 of 32000 rows took 86 us (77 by digits), 32768 of
// 2^19 146 (139), 32768 of 2^18 95 (100), 16384 of 2^20 144 (163).
constexpr int64_t kSSome = 32768, kSRows = int64_t(1) << 20, kSProduct = int64_t(1) << 34;
constexpr int kLoadItems = 16;         // tokens that a lane requests together
constexpr int kAlone = 32;             // few tokens: so many of a row are one wavefront's,
constexpr int kFewAhead = 8;           // which requests so many of them together
constexpr int kDigits = 256;
constexpr int kAhead = 16;             // rows a lane requests together
constexpr int64_t kFewBlocks = 64;     // so many histograms every workgroup adds up by itself
constexpr int kZeroRows = 64;          // rows of the table that a workgroup looks up

template <bool BFI, bool BFO>
__global__ void __launch_bounds__(kEThreads) gscan_embed_fwd_kernel(EmbedArgs a, int lpr)
{
    const int sub = threadIdx.x & (lpr - 1), rpp = kEThreads / lpr;
    const int64_t step = (int64_t)rpp * kERows;
    for (int64_t r0 = blockIdx.x * step + threadIdx.x / lpr; r0 < a.N; r0 += gridDim.x * step) {
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
}

// ---------------------------------------------------------------- the sort

struct SortLds {
    uint32_t hist[kSWaves][kDigits];
    uint32_t total[kDigits + 1], lead[4];
};

// Lanes (of those in `in`) with the same digit, of so many bits.
__device__ __forceinline__ uint64_t peers_of(uint32_t digit, uint64_t in, int bits)
{
    uint64_t m = in;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        if (b >= bits) break;
        const uint64_t s = __ballot((digit >> b) & 1u);
        m &= ((digit >> b) & 1u) ? s : ~s;
    }
    return m;
}

// Ranks of the workgroup's items by their digit (kDigits: not one of them): item
// (wave, j, lane) comes before (wave, j, lane + 1), (wave, j + 1, ..) and (wave + 1, ..).
// item[j] becomes digit << 16 | the equal digits before it in its wavefront; the
// histograms then become, per wavefront and digit, those of the wavefronts before.
template <int ITEMS>
__device__ __forceinline__ void rank_items(SortLds &s, uint32_t (&item)[ITEMS], int bits)
{
    const int tid = threadIdx.x, wave = tid >> 6;
    for (int i = tid; i < kSWaves * kDigits; i += kSThreads) s.hist[i / kDigits][i % kDigits] = 0;
    __syncthreads();
    volatile uint32_t *h = s.hist[wave];  // read by lanes that others of the wavefront write for
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t d = item[j];
        const bool in = d < (uint32_t)kDigits;
        const uint64_t some = __ballot(in);
        item[j] = d << 16;
        if (!some) continue;
        // often all of them are one frequent token (32768 tokens of 32000 rows 54 -> 48 us)
        const uint32_t d0 = __builtin_amdgcn_readlane(d, __builtin_ctzll(some));
        const uint64_t peers = __ballot(in && d == d0) == some ? some : peers_of(d, some, bits);
        const uint32_t before = __builtin_amdgcn_mbcnt_hi((uint32_t)(peers >> 32),
                                                          __builtin_amdgcn_mbcnt_lo((uint32_t)peers, 0u));
        uint32_t seen = 0;
        if (in) seen = h[d];
        item[j] |= seen + before;
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

// Of a ranked item: its digit, and where it goes among the equal ones.
__device__ __forceinline__ uint32_t digit_of(uint32_t item) { return item >> 16; }
__device__ __forceinline__ uint32_t rank_of(const SortLds &s, uint32_t item)
{
    return s.hist[threadIdx.x >> 6][item >> 16] + (item & 0xffffu);
}

// Exclusive sums of x over the first 256 threads, into s.total; all of it behind them.
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
        if (tid == kDigits - 1) s.total[kDigits] = y;
    }
    __syncthreads();
}

// The tokens of the rows first .. first + rows - 1 (row V: padding), ranked by their row:
// their digit is the row's number here.  Returns how many there are of the rows before.
template <int ITEMS>
__device__ __forceinline__ uint32_t rank_rows(const EmbedArgs &a, uint32_t first, uint32_t rows, SortLds &s,
                                              uint32_t (&item)[ITEMS])
{
    __shared__ uint32_t below;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0) below = 0;
    __syncthreads();
    uint32_t before = 0;
    constexpr int kBatch = ITEMS < kLoadItems ? ITEMS : kLoadItems;
#pragma unroll
    for (int b = 0; b < ITEMS; b += kBatch) {
        uint32_t key[kBatch];
        token_keys<kBatch>(a.tokens, a.tok64, a.V, (int64_t)(wave * ITEMS + b) * 64 + lane, a.N, key);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            before += (uint32_t)__popcll(__ballot(key[j] < first));
            item[b + j] = key[j] - first < rows ? key[j] - first : (uint32_t)kDigits;
        }
    }
    if (lane == 0) atomicAdd(&below, before);  // whole numbers: any order
    rank_items<ITEMS>(s, item, 32 - __builtin_clz(rows | 1u));
    scan_digits(s, threadIdx.x < kDigits ? s.total[threadIdx.x] : 0u);
    return below;
}

// Up to 1024 ITEMS tokens: sorted, and zeros for the rows without one.
template <int ITEMS>
__global__ void __launch_bounds__(kSThreads) gscan_sort_rows_kernel(EmbedArgs a, int rows, uint32_t *keys,
                                                                   uint32_t *order)
{
    __shared__ SortLds s;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t first = (int64_t)blockIdx.x * rows;
    uint32_t item[ITEMS];
    const uint32_t below = rank_rows<ITEMS>(a, (uint32_t)first, (uint32_t)rows, s, item);
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
        const uint32_t d = digit_of(item[j]);
        if (d < (uint32_t)kDigits) {
            const uint32_t at = below + s.total[d] + rank_of(s, item[j]);
            keys[at] = (uint32_t)first + d;
            order[at] = (uint32_t)((wave * ITEMS + j) * 64 + lane);
        }
    }
    const int octs = a.D / 8;
    for (int r = wave; r < rows && first + r < a.V; r += kSWaves) {
        if (s.total[r] != s.total[r + 1]) continue;
        for (int c = lane; c < octs; c += 64) {
            if (a.table_dtype) store_oct<true>(a.dtable, (first + r) * a.D + 8 * c, Oct{});
            else store_oct<false>(a.dtable, (first + r) * a.D + 8 * c, Oct{});
        }
    }
}

// The rows of dout at list[b .. e - 1], eight columns from c on, in order.
template <bool BF>
__device__ __forceinline__ Oct add_rows(const EmbedArgs &a, const uint32_t *list, uint32_t b, uint32_t e, int c)
{
    Oct sum = {};
    const bool in = c < a.D;
    for (; b < e; b += kFewAhead) {
        OctRaw<BF> x[kFewAhead];
#pragma unroll
        for (int k = 0; k < kFewAhead; ++k) {
            x[k] = OctRaw<BF>{};
            if (in && b + k < e) x[k] = load_oct<BF>(a.dout, (int64_t)list[b + k] * a.ld + c);
        }
#pragma unroll
        for (int k = 0; k < kFewAhead; ++k) {
            if (b + k >= e) break;
            const Oct v = widen(x[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum.v[i] += v.v[i];
        }
    }
    return sum;
}

// Few tokens: sorted and added up, `rows` rows of the table for a workgroup.  A row
// of up to 32 tokens is one wavefront's; of more every wavefront takes its share, and
// the shares are added in order.
template <bool BF, bool BFT>
__global__ void __launch_bounds__(kSThreads) gscan_embed_few_kernel(EmbedArgs a, int rows)
{
    __shared__ SortLds s;
    __shared__ uint32_t list[kSFew], many[kSFew / kAlone], count;
    __shared__ __align__(16) float share[kSWaves][512];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t first = (int64_t)blockIdx.x * rows;
    uint32_t item[kFewItems];
    if (threadIdx.x == 0) count = 0;
    rank_rows<kFewItems>(a, (uint32_t)first, (uint32_t)rows, s, item);
#pragma unroll
    for (int j = 0; j < kFewItems; ++j) {
        const uint32_t d = digit_of(item[j]);
        if (d < (uint32_t)kDigits)
            list[s.total[d] + rank_of(s, item[j])] = (uint32_t)((wave * kFewItems + j) * 64 + lane);
    }
    if (threadIdx.x < rows && first + threadIdx.x < a.V && s.total[threadIdx.x + 1] - s.total[threadIdx.x] > kAlone)
        many[atomicAdd(&count, 1u)] = threadIdx.x;  // each by itself: any order
    __syncthreads();
    auto put = [&](Oct sum, int64_t r, int c) {
        if (c >= a.D) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum.v[i] *= a.scale;
        store_oct<BFT>(a.dtable, (first + r) * a.D + c, sum);
    };
    for (int c0 = 512 * (int)blockIdx.y; c0 < a.D; c0 += 512 * (int)gridDim.y) {
        const int c = c0 + 8 * lane;
        for (int r = wave; r < rows && first + r < a.V; r += kSWaves) {
            const uint32_t b = __builtin_amdgcn_readfirstlane(s.total[r]),
                           e = __builtin_amdgcn_readfirstlane(s.total[r + 1]);
            if (b == e) {
                if (c < a.D) store_oct<BFT>(a.dtable, (first + r) * a.D + c, Oct{});
            } else if (e - b <= kAlone) {
                put(add_rows<BF>(a, list, b, e, c), r, c);
            }
        }
        for (uint32_t m = 0; m < count; ++m) {
            const uint32_t r = many[m], b = s.total[r], e = s.total[r + 1], each = (e - b + kSWaves - 1) / kSWaves;
            const uint32_t b1 = b + wave * each, e1 = b1 + each < e ? b1 + each : e;
            const Oct x = add_rows<BF>(a, list, b1, e1, c);
            store_oct<false>(share[wave], 8 * lane, x);
            __syncthreads();
            if (wave == 0) {
                Oct sum = x;
                for (int w = 1; w < kSWaves; ++w) {
                    const Oct y = widen(load_oct<false>(share[w], 8 * lane));
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum.v[i] += y.v[i];
                }
                put(sum, r, c);
            }
            __syncthreads();
        }
    }
}

// One digit of many tokens.  Keys and positions come from the tokens in the
// first pass.  count[block][digit].
template <bool FIRST>
__device__ __forceinline__ void load_keys(const EmbedArgs &a, const uint32_t *keys, const uint32_t *order,
                                          int64_t base, int64_t end, uint32_t (&key)[kSItems],
                                          uint32_t (&pos)[kSItems])
{
    const int64_t i0 = base + (threadIdx.x >> 6) * kSItems * 64 + (threadIdx.x & 63);
    if constexpr (FIRST) {
        token_keys<kSItems>(a.tokens, a.tok64, a.V, i0, end, key);
#pragma unroll
        for (int j = 0; j < kSItems; ++j) pos[j] = (uint32_t)(i0 + 64 * j);
    } else {
#pragma unroll
        for (int j = 0; j < kSItems; ++j) {
            key[j] = ~0u;
            pos[j] = 0;
            if (i0 + 64 * j < end) {
                key[j] = keys[i0 + 64 * j];
                pos[j] = order[i0 + 64 * j];
            }
        }
    }
}

template <bool FIRST>
__global__ void __launch_bounds__(kSThreads) gscan_sort_count_kernel(EmbedArgs a, const uint32_t *keys, int shift,
                                                                    uint32_t *count)
{
    __shared__ uint32_t h[kDigits];
    const int64_t base = (int64_t)blockIdx.x * kSBlock;
    const int64_t end = a.N - base < kSBlock ? a.N : base + kSBlock;
    if (threadIdx.x < kDigits) h[threadIdx.x] = 0;
    __syncthreads();
    uint32_t key[kSItems], pos[kSItems];
    load_keys<FIRST>(a, keys, keys, base, end, key, pos);
#pragma unroll
    for (int j = 0; j < kSItems; ++j)
        if (key[j] != ~0u) atomicAdd(&h[(key[j] >> shift) & (kDigits - 1)], 1u);  // whole numbers: any order
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
    const int tid = threadIdx.x;
    const int64_t base = (int64_t)blockIdx.x * kSBlock, end = a.N - base < kSBlock ? a.N : base + kSBlock;
    uint32_t key[kSItems], pos[kSItems], item[kSItems];
    load_keys<FIRST>(a, keys, order, base, end, key, pos);
#pragma unroll
    for (int j = 0; j < kSItems; ++j) item[j] = key[j] != ~0u ? (key[j] >> shift) & (kDigits - 1) : (uint32_t)kDigits;
    rank_items<kSItems>(s, item, 8);
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
        if (key[j] != ~0u) {
            const uint32_t at = first[digit_of(item[j])] + rank_of(s, item[j]);
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
    __syncthreads();
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
        for (; id * kZeroRows < a.V; id += zeros) zero_rows<BFT>(a, keys, id * kZeroRows);
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
    bool few = false, some = false;  // one launch does it all, sorts
    int rows = 0;               // of a workgroup of that
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
    p.some = N <= kSSome && V < kSRows && N * V < kSProduct;
    p.few = p.some && (D <= 512 ? N <= kSFew : D <= 4096 && N <= kSWide);
    // a workgroup per CU (two: 16384 tokens 38 -> 43 us); padding is row V
    const int64_t rows = (V + 256) / 256;
    p.rows = (int)(rows < kDigits ? rows : kDigits);
    if (p.few) return p;
    p.blocks = (N + kSBlock - 1) / kSBlock;
    p.chunks = (N + p.chunk - 1) / p.chunk;
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        p.keys[i] = at;
        at = round_up(at + (size_t)N * 4);
        p.order[i] = at;
        at = round_up(at + (size_t)N * 4);
        if (p.some) {  // no second copy
            p.keys[1] = p.keys[0];
            p.order[1] = p.order[0];
            break;
        }
    }
    p.count = at;
    if (!p.some) at = round_up(at + (size_t)(p.blocks + 1) * kDigits * 4);
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
    hipLaunchKernelGGL(k, groups_of((a.N + rows - 1) / rows), dim3(kEThreads), 0, st, a, lpr);
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
    } else if (p.few) {
        auto *k = a.dtype ? (a.table_dtype ? gscan_embed_few_kernel<true, true> : gscan_embed_few_kernel<true, false>)
                          : (a.table_dtype ? gscan_embed_few_kernel<false, true> : gscan_embed_few_kernel<false, false>);
        const int64_t groups = (a.V + p.rows) / p.rows, slices = (a.D + 511) / 512;
        int64_t apart = 256 / groups;  // few rows: their columns are divided too
        apart = apart < 1 ? 1 : apart > slices ? slices : apart;
        hipLaunchKernelGGL(k, dim3((unsigned)groups, (unsigned)apart), dim3(kSThreads), 0, st, a, p.rows);
        return hipGetLastError();
    } else if (p.some) {
        const int items = (int)((a.N + kSThreads - 1) / kSThreads);
        auto *k = items <= 4    ? gscan_sort_rows_kernel<4>
                  : items <= 8  ? gscan_sort_rows_kernel<8>
                  : items <= 16 ? gscan_sort_rows_kernel<16>
                                : gscan_sort_rows_kernel<32>;
        hipLaunchKernelGGL(k, dim3((unsigned)((a.V + p.rows) / p.rows)), dim3(kSThreads), 0, st, a, p.rows, keys[0],
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
    const int slices = (a.D + 511) / 512;
    const int64_t waves = p.chunks * slices, groups = (waves + 3) / 4;
    const int64_t zeros = p.some && a.N ? 0 : groups_of((a.V + kZeroRows - 1) / kZeroRows).x;
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
