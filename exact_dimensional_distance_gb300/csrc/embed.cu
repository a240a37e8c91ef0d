// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward    out[i] = scale * table[token[i]]
//   backward   grad[v] = scale * sum of dy[i] over the positions i that hold token v
//
// Both are bound by memory.  The forward pass reads the rows its tokens touch
// and writes n rows.  The backward pass must read n rows of dy and
// write the whole gradient, mostly zeros for a large vocabulary:
//
//   1. the positions are sorted by token (stable LSD radix sort, up to 9 bits
//      per pass; tokens of a vocabulary below 2^18 take two), while the SMs that the sort
//      leaves idle write the zeros of the rows without positions;
//   2. k_sum cuts the sorted positions into units of kUnit and sums runs of equal
//      tokens: a run belongs to the unit it begins in, which follows it
//      into the next unit.  A run that goes on past that one leaves a float32 partial
//      sum per unit, so the work of a unit is bounded however often a token occurs;
//   3. k_join adds the partial sums of each long run in unit order.
//
// Sums are float32 in an order that depends on the positions alone: no
// floating-point atomics.  Few positions take one kernel instead (k_grad_few).
#include <algorithm>
#include <atomic>

#include "hiss_internal.cuh"
#include "numeric.cuh"
#include "ptx.cuh"

namespace hiss {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 16;  // columns per lane of the sums

// The table row of position i; kPadRow for padding and kBadRow for a token
// outside the table, both rows of zeros.  The caller raises *a.bad once it has
// issued its loads (a store between them would make each wait for the last).
constexpr int64_t kPadRow = -1, kBadRow = -2;
__device__ __forceinline__ int64_t row_of(const EmbedArgs &a, int64_t i)
{
    const int64_t t =
        a.token_bits == 64 ? static_cast<const int64_t *>(a.tokens)[i] : static_cast<const int32_t *>(a.tokens)[i];
    return t == a.pad ? kPadRow : t < 0 || t >= a.vocab ? kBadRow : t;
}

// ---- forward --------------------------------------------------------------------

// lanes (a power of two up to 32) take one tile of lanes * E * NV columns of
// one position.
template <typename TI, typename TO, int E, int NV>
__global__ void __launch_bounds__(kThreads) k_embed(EmbedArgs a, int lanes, int tiles)
{
    const int per_block = kThreads / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t items = a.n * tiles, step = (int64_t)gridDim.x * per_block;
    for (int64_t it = (int64_t)blockIdx.x * per_block + threadIdx.x / lanes; it < items; it += step) {
        const int64_t i = tiles == 1 ? it : it / tiles;
        const int c0 = ((int)(it - i * tiles) * lanes * NV + lane) * E;
        const int64_t r = row_of(a, i);
        const TI *p = static_cast<const TI *>(a.rows) + r * a.rows_stride;
        TO *q = static_cast<TO *>(a.out) + i * a.out_stride;
        Pack<TI, E> v[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * lanes * E;
            if (r >= 0 && c < a.width) v[k] = load_pack<TI, E>(p + c);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * lanes * E;
            if (c >= a.width) continue;
            Pack<TO, E> o;
#pragma unroll
            for (int e = 0; e < E; ++e) o.v[e] = from_f32<TO>(r >= 0 ? a.scale * to_f32(v[k].v[e]) : 0.0f);
            store_pack<TO, E>(q + c, o);
        }
        if (r == kBadRow) *a.bad = 1;
    }
}

// ---- the sort ---------------------------------------------------------------------

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxItems = 8;  // positions per thread
constexpr int kMaxBits = 9;  // one bin per thread
constexpr int kMaxBins = 1 << kMaxBits;
// The sort is a chain of latencies.  Tiles are as small as kManyTiles
// allows: few large ones leave it on few SMs.  Up to kSumTiles each block of the
// scatter adds up the tiles' counts itself; above, their prefix sums are a kernel of
// their own.
constexpr int kManyTiles = 128;
constexpr int kSumTiles = 32;
constexpr int kBitmapWords = 8192;  // of a block's bitmap of tokens (32 KB: a vocabulary of 262,144)

struct SortArgs {
    const uint2 *in;     // (key, position); NULL: the tokens and their positions
    uint2 *out;
    uint32_t *counts;    // digit counts of the input's tiles: [tiles][bins], exclusive over the
                         // tiles once scanned; then [bins] totals
    uint32_t *counts_out;  // the next digit's counts of the output's tiles (NULL: last pass)
    uint32_t *present;   // [ceil(vocab / 32)] bit: the token occurs (NULL: not wanted); 0 between calls
    uint32_t *runs;      // number of long runs (SumArgs), set to 0 by the first kernel
    uint32_t *clear;     // the later passes' counts, set to 0 by the first kernel
    int64_t clear_n;
    int tiles, shift, bits, scanned;
};

// Entry i: the token (vocab for a position without a row) and its position.
__device__ __forceinline__ uint2 entry(const EmbedArgs &a, const SortArgs &s, int64_t i, bool *bad)
{
    if (s.in) return s.in[i];
    const int64_t r = row_of(a, i);
    *bad = *bad || r == kBadRow;
    return make_uint2((uint32_t)(r < 0 ? a.vocab : r), (uint32_t)i);
}

template <typename T>
__device__ __forceinline__ void zero_row(char *p, int64_t bytes, int lane)
{
    for (int64_t i = lane * sizeof(T); i < bytes; i += 32 * sizeof(T)) *reinterpret_cast<T *>(p + i) = T{};
}

// Zeros (all bits 0 in every type) for the rows that no position holds, in
// this kernel's share [f0, f1) of kShares of the vocabulary.  warp of warps.
constexpr int kShares = 8, kScatterShare = 2;
struct Fill {
    const uint32_t *present;
    int f0, f1;
    int store;           // bytes per store that the gradient's rows allow
    int blocks;          // blocks of the kernel that do this, behind the others
};
__device__ void fill_empty(const EmbedArgs &a, const Fill &f, int64_t warp, int64_t warps)
{
    const int lane = threadIdx.x & 31;
    const int64_t words = (a.vocab + 31) / 32;
    const int64_t v0 = words * f.f0 / kShares * 32, v1 = min(words * f.f1 / kShares * 32, a.vocab);
    const int size = a.out_dtype == HISS_F32 ? 4 : 2;
    const int64_t bytes = (int64_t)a.width * size, stride = a.out_stride * size;
    int rows = 32;  // per warp and turn: a power of two, so that they share a word
    while (rows > 1 && (v1 - v0) < warps * rows) rows >>= 1;
    for (int64_t v = v0 + warp * rows; v < v1; v += warps * rows) {
        uint32_t empty = ~(f.present[v >> 5] >> (v & 31));
        if (rows < 32) empty &= (1u << rows) - 1u;
        while (empty) {
            const int64_t r = v + __ffs(empty) - 1;
            empty &= empty - 1;
            if (r >= v1) break;
            char *p = static_cast<char *>(a.out) + r * stride;
            if (f.store == 16) zero_row<uint4>(p, bytes, lane);
            else if (f.store == 4) zero_row<uint32_t>(p, bytes, lane);
            else zero_row<uint16_t>(p, bytes, lane);
        }
    }
}

// First digit's counts of each tile, and which tokens occur.
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) k_sort_count(EmbedArgs a, SortArgs s)
{
    __shared__ uint32_t hist[kMaxBins];
    extern __shared__ uint32_t bitmap[];  // the tile's tokens, up to kBitmapWords
    const int words = s.present ? (int)((a.vocab + 31) / 32) : 0;
    const bool merge = words <= kBitmapWords;
    wait_for_previous();
    hist[threadIdx.x] = 0;
    if (merge)
        for (int i = threadIdx.x; i < words; i += kSortThreads) bitmap[i] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *s.runs = 0;
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < s.clear_n; i += (int64_t)gridDim.x * kSortThreads)
        s.clear[i] = 0;
    __syncthreads();
    const uint32_t mask = (1u << s.bits) - 1u;
    const int64_t base = (int64_t)blockIdx.x * (kSortThreads * ITEMS);
    uint32_t key[ITEMS];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int64_t i = base + k * kSortThreads + threadIdx.x;
        key[k] = i < a.n ? entry(a, s, i, &bad).x : ~0u;
    }
    if (bad) *a.bad = 1;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        if (base + k * kSortThreads + threadIdx.x >= a.n) continue;
        // the tile's tokens are collected first: frequent ones share a few
        // sectors, and one access per position to those is served in turn
        if (words && key[k] < (uint32_t)a.vocab)
            atomicOr(merge ? &bitmap[key[k] >> 5] : &s.present[key[k] >> 5], 1u << (key[k] & 31));
        atomicAdd(&hist[(key[k] >> s.shift) & mask], 1u);
    }
    __syncthreads();
    if (merge)
        for (int i = threadIdx.x; i < words; i += kSortThreads)
            if (bitmap[i]) atomicOr(&s.present[i], bitmap[i]);
    const int bins = 1 << s.bits;
    if ((int)threadIdx.x < bins) s.counts[(int64_t)blockIdx.x * bins + threadIdx.x] = hist[threadIdx.x];
    let_next_start();
}

// counts[t][bin] := sum over the tiles before t; totals behind them.  32 bins
// per block, the tiles in 32 consecutive parts.
__global__ void __launch_bounds__(1024) k_sort_scan(SortArgs s)
{
    __shared__ uint32_t sum[32][33];
    wait_for_previous();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int bins = 1 << s.bits, bin = blockIdx.x * 32 + lane;
    const int t0 = (int)((int64_t)s.tiles * w / 32), t1 = (int)((int64_t)s.tiles * (w + 1) / 32);
    uint32_t v = 0;
    if (bin < bins)
        for (int t = t0; t < t1; ++t) v += s.counts[(int64_t)t * bins + bin];
    sum[w][lane] = v;
    __syncthreads();
    uint32_t run = 0;
    for (int i = 0; i < w; ++i) run += sum[i][lane];
    if (bin >= bins) return;
    for (int t = t0; t < t1; ++t) {
        const uint32_t c = s.counts[(int64_t)t * bins + bin];
        s.counts[(int64_t)t * bins + bin] = run;
        run += c;
    }
    if (w == 31) s.counts[(int64_t)s.tiles * bins + bin] = run;
    let_next_start();
}

// One stable pass: each tile's positions go behind those of the tiles before
// it, digit by digit.  Counts the next digit of the tiles it writes to on the way.
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) k_sort_scatter(EmbedArgs a, SortArgs s, Fill f)
{
    __shared__ uint32_t whist[kSortWarps][kMaxBins];
    __shared__ uint32_t base_of[kMaxBins];
    __shared__ uint32_t warp_total[kSortWarps];
    wait_for_previous();
    if ((int)blockIdx.x >= s.tiles) {
        fill_empty(a, f, (int64_t)(blockIdx.x - s.tiles) * kSortWarps + (threadIdx.x >> 5), (int64_t)f.blocks * kSortWarps);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int bins = 1 << s.bits, bin = threadIdx.x;
    const uint32_t mask = (uint32_t)bins - 1u;
    for (int i = threadIdx.x; i < kSortWarps * kMaxBins; i += kSortThreads) (&whist[0][0])[i] = 0;
    // warp-contiguous items, in order
    const int64_t base = (int64_t)blockIdx.x * (kSortThreads * ITEMS) + warp * (32 * ITEMS);
    uint2 item[ITEMS];
    uint32_t rank[ITEMS];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (base + k * 32 + lane < a.n) item[k] = entry(a, s, base + k * 32 + lane, &bad);
    // this thread's bin: positions in the tiles before this one, and in all
    uint32_t before = 0, total = 0;
    if (bin < bins) {
        if (s.scanned) {
            before = s.counts[(int64_t)blockIdx.x * bins + bin];
            total = s.counts[(int64_t)s.tiles * bins + bin];
        } else {
#pragma unroll 32
            for (int t = 0; t < s.tiles; ++t) {
                const uint32_t c = s.counts[(int64_t)t * bins + bin];
                total += c;
                if (t < (int)blockIdx.x) before += c;
            }
        }
    }
    uint32_t incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    uint32_t first = incl - total;
    for (int i = 0; i < warp; ++i) first += warp_total[i];
    base_of[bin] = first + before;
    // lanes with the same digit, one ballot per bit (a match instruction takes
    // as long as the warp has distinct digits)
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const bool valid = base + k * 32 + lane < a.n;
        const uint32_t d = valid ? (item[k].x >> s.shift) & mask : 0u;
        uint32_t peers = __ballot_sync(0xffffffffu, valid);
#pragma unroll
        for (int b = 0; b < kMaxBits; ++b) {
            const uint32_t set = __ballot_sync(0xffffffffu, (d >> b) & 1u);
            peers &= (d >> b) & 1u ? set : ~set;
        }
        const uint32_t below = __popc(peers & ((1u << lane) - 1u));
        rank[k] = 0;
        if (valid) rank[k] = whist[warp][d] + below;
        __syncwarp();
        if (valid && below == 0) whist[warp][d] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    uint32_t run = base_of[bin];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = whist[w][bin];
        whist[w][bin] = run;
        run += c;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
        if (base + k * 32 + lane < a.n) {
            const uint32_t at = whist[warp][(item[k].x >> s.shift) & mask] + rank[k];
            s.out[at] = item[k];
            if (s.counts_out)
                atomicAdd(&s.counts_out[(int64_t)(at / (kSortThreads * ITEMS)) * bins + ((item[k].x >> (s.shift + s.bits)) & mask)], 1u);
        }
    let_next_start();
}

// ---- the sums ---------------------------------------------------------------------

constexpr int kUnit = 32;  // sorted positions per unit

struct SumArgs {
    const uint2 *items;           // sorted (token, position)
    float *part;                  // [units][2][width]: sum of the long run that comes in from the unit
                                  // before, and of the long run that begins here
    uint32_t *runs;               // [0]: number of long runs; then (key, first unit) of each
    uint32_t *last;               // [vocab]: last unit of a long run
    uint32_t *present;            // cleared at the end
    int64_t units;
    int lanes, tiles;             // lanes * kCols columns per tile
    int blocks;                   // of k_sum that sum (the others write empty rows)
};

// Write (or add) a finished row's columns.
template <typename TO, int E, int NV>
__device__ __forceinline__ void write_row(const EmbedArgs &a, uint32_t v, int c0, int lanes, const float (&s)[kCols])
{
    TO *p = static_cast<TO *>(a.out) + (int64_t)v * a.out_stride;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = c0 + k * lanes * E;
        if (c >= a.width) continue;
        Pack<TO, E> o;
        if (a.accumulate) o = load_pack<TO, E>(p + c);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float x = a.scale * s[k * E + e];
            if (a.accumulate) x += to_f32(o.v[e]);
            o.v[e] = from_f32<TO>(x);
        }
        store_pack<TO, E>(p + c, o);
    }
}

template <int E, int NV>
__device__ __forceinline__ void write_part(const EmbedArgs &a, float *p, int c0, int lanes, const float (&s)[kCols])
{
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = c0 + k * lanes * E;
        if (c >= a.width) continue;
        Pack<float, E> o;
#pragma unroll
        for (int e = 0; e < E; ++e) o.v[e] = s[k * E + e];
        store_pack<float, E>(p + c, o);
    }
}

constexpr int kAhead = 4;  // rows in flight per lane

template <typename TI, int E>
constexpr size_t sum_bytes() { return (size_t)kThreads * kAhead * kCols * sizeof(TI); }

// FULL: 32 lanes, so that a lane's packs are a constant distance apart.
template <typename TI, typename TO, int E, bool FULL>
__global__ void __launch_bounds__(kThreads) k_sum(EmbedArgs a, SumArgs s, Fill f)
{
    constexpr int NV = kCols / E;
    using P = Pack<TI, E>;
    constexpr bool kAsync = sizeof(TI) * E >= 4;  // single 16-bit elements cannot be copied asynchronously
    extern __shared__ __align__(16) char ring[];
    wait_for_previous();
    if ((int)blockIdx.x >= s.blocks) {
        fill_empty(a, f, (int64_t)(blockIdx.x - s.blocks) * (kThreads / 32) + (threadIdx.x >> 5),
                   (int64_t)f.blocks * (kThreads / 32));
        return;
    }
    const int lanes = FULL ? 32 : s.lanes;
    const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    if (item >= s.units * s.tiles) return;
    // tiles of a unit are neighbours: they read the same rows of dy
    const int64_t unit = item / s.tiles;
    const int tile = (int)(item - unit * s.tiles);
    const int c0 = (tile * lanes * NV + lane) * E;
    const int packs = min(NV, (a.width - tile * lanes * kCols + lanes * E - 1) / (lanes * E));  // of a row in this tile
    const int n = (int)a.n, i0 = (int)unit * kUnit, i1 = min(i0 + kUnit, n);
    const uint32_t vocab = (uint32_t)a.vocab, none = ~0u;
    auto key_of = [&](int i) { return i >= 0 && i < n ? s.items[i].x : none; };
    const uint32_t k0 = key_of(i0), k1 = key_of(i1 - 1);
    const uint32_t prev = key_of(i0 - 1), prev_unit = key_of(i0 - kUnit), prev_unit2 = key_of(i0 - kUnit - 1);
    const uint32_t next = key_of(i1), next_unit = key_of(i1 + kUnit);
    if (k0 >= vocab) return;  // only positions without a row from here on
    // the run that comes in: summed by the unit before when it began there and
    // ends here, a part of a long run otherwise
    const bool comes_in = prev == k0;
    const bool long_in = comes_in && !((prev_unit != k0 || prev_unit2 != k0) && (next != k0 || k1 != k0));
    // the run that goes out: followed into the next unit when it ends there
    const bool goes_out = next == k1 && k1 < vocab;
    const bool begins = goes_out && !(k0 == k1 && comes_in);
    const bool long_out = goes_out && (!begins || next_unit == k1);
    int i = i0, end = i1;
    if (comes_in && !long_in)
        while (i < i1 && s.items[i].x == k0) ++i;
    if (goes_out && !long_out)
        while (end < n && s.items[end].x == k1) ++end;
    while (end > i && s.items[end - 1].x >= vocab) --end;
    if (long_out && begins && tile == 0 && lane == 0) {
        const uint32_t at = atomicAdd(s.runs, 1u);
        s.runs[1 + 2 * at] = k1;
        s.runs[2 + 2 * at] = (uint32_t)unit;
    }
    if (long_in && (next != k0 || k1 != k0) && tile == 0 && lane == 0) s.last[k0] = (uint32_t)unit;
    if (i >= end) return;

    P *slot = reinterpret_cast<P *>(ring) + threadIdx.x;
    const TI *rows = static_cast<const TI *>(a.rows) + c0;
    auto fetch = [&](int j) {
        if (j < end) {
            const TI *p = rows + (int64_t)s.items[j].y * a.rows_stride;
            P *d = slot + (j & (kAhead - 1)) * (NV * kThreads);
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                if (q >= packs) break;
                if (q == packs - 1 && c0 + q * lanes * E >= a.width) break;
                if constexpr (kAsync) copy_pack_async<TI, E>(d + q * kThreads, p + q * lanes * E);
                else d[q * kThreads] = load_pack<TI, E>(p + q * lanes * E);
            }
        }
        cp_async_commit();
    };
    for (int k = 0; k < kAhead - 1; ++k) fetch(i + k);
    float acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = 0.0f;
    float *part = s.part + unit * 2 * a.width;
    bool head = long_in;  // the current run is the long one that came in
    uint32_t key = s.items[i].x;
    while (i < end) {
        fetch(i + kAhead - 1);
        cp_async_wait<kAhead - 1>();
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            if (q >= packs) break;
            const P v = slot[((i & (kAhead - 1)) * NV + q) * kThreads];
            if constexpr (E == 1) {
                acc[q] += to_f32(v.v[0]);
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 p = __fadd2_rn(make_float2(acc[q * E + e], acc[q * E + e + 1]), pair_of(v.v + e));
                    acc[q * E + e] = p.x;
                    acc[q * E + e + 1] = p.y;
                }
            }
        }
        ++i;
        const uint32_t k = i < end ? s.items[i].x : none;
        if (k == key) continue;
        const bool tail = i >= end && long_out;
        if (head || tail) write_part<E, NV>(a, head ? part : part + a.width, c0, lanes, acc);
        else write_row<TO, E, NV>(a, key, c0, lanes, acc);
        key = k;
        head = false;
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] = 0.0f;
    }
    let_next_start();
}

constexpr int kJoinThreads = 512;
constexpr int kJoinBlocks = 2 * kSMs;

// The row of each long run: the second part of the unit it begins in and the
// first parts of the units up to its last.  One block per run and tile at a
// time; its groups of lanes each take a stretch of the units, and a thread per
// column adds the groups up in order.
template <typename TO, int E>
__global__ void __launch_bounds__(kJoinThreads) k_join(EmbedArgs a, SumArgs s)
{
    constexpr int NV = kCols / E;
    __shared__ float sh[kJoinThreads * kCols];  // [group][column of the tile]
    wait_for_previous();
    const int lanes = s.lanes, groups = kJoinThreads / lanes, cols = lanes * kCols;
    const int group = threadIdx.x / lanes, lane = threadIdx.x & (lanes - 1);
    if (s.present)
        for (int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; i < (a.vocab + 31) / 32; i += (int64_t)gridDim.x * kJoinThreads)
            s.present[i] = 0;
    const int64_t items = (int64_t)s.runs[0] * s.tiles;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t run = it / s.tiles;
        const int tile0 = (int)(it - run * s.tiles) * cols;
        const uint32_t key = s.runs[1 + 2 * run];
        const int64_t first = s.runs[2 + 2 * run], count = (int64_t)s.last[key] - first + 1;
        float acc[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] = 0.0f;
        const int64_t to = first + count * (group + 1) / groups;
#pragma unroll 4
        for (int64_t u = first + count * group / groups; u < to; ++u) {
            const float *p = s.part + (u * 2 + (u == first)) * a.width + tile0;
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int c = (q * lanes + lane) * E;
                if (tile0 + c >= a.width) continue;
                const auto v = load_pack<float, E>(p + c);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[q * E + e] += v.v[e];
            }
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            Pack<float, E> v;
#pragma unroll
            for (int e = 0; e < E; ++e) v.v[e] = acc[q * E + e];
            store_pack<float, E>(sh + group * cols + (q * lanes + lane) * E, v);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < cols && tile0 + c < a.width; c += kJoinThreads) {
            float x = 0.0f;
            for (int g = 0; g < groups; ++g) x += sh[g * cols + c];
            x *= a.scale;
            TO *p = static_cast<TO *>(a.out) + (int64_t)key * a.out_stride + tile0 + c;
            if (a.accumulate) x += to_f32(*p);
            *p = from_f32<TO>(x);
        }
        __syncthreads();
    }
}

// ---- few positions -------------------------------------------------------------------

constexpr int64_t kFew = 1024;
constexpr int kFewThreads = 256;
constexpr int kFewFloats = 8192;  // accumulators of a block

// One kernel without a sort: a block owns some rows and a range of columns (its
// accumulators in shared memory), picks the positions whose token is one of
// its rows, in order, and adds them up; every one of its rows is written.
template <typename TI, typename TO, int E>
__global__ void __launch_bounds__(kFewThreads) k_grad_few(EmbedArgs a, int rows, int lanes)
{
    __shared__ float acc[kFewFloats];
    __shared__ uint32_t found[kFew];     // (row in the range) << 10 | position
    __shared__ uint32_t warp_count[kFewThreads / 32];
    __shared__ uint8_t touched[kFewFloats];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // row i of the block is row i * blocks + block of the table: frequent
    // tokens, which a vocabulary often has next to one another, go to different blocks
    const uint32_t blocks = gridDim.x, block = blockIdx.x;
    const int nrows = (int)((a.vocab - block + blocks - 1) / blocks);
    const int cols = lanes * E;              // columns of the tile
    const int c0 = blockIdx.y * cols;
    for (int i = threadIdx.x; i < rows; i += kFewThreads) touched[i] = 0;
    constexpr int R = kFew / kFewThreads;
    int r[R];  // row in the block, -1: another block's or none
    bool bad = false;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int64_t i = k * kFewThreads + threadIdx.x;
        const int64_t v = i < a.n ? row_of(a, i) : kPadRow;
        bad = bad || v == kBadRow;
        r[k] = v >= 0 && (uint32_t)v % blocks == block ? (int)((uint32_t)v / blocks) : -1;
    }
    if (bad) *a.bad = 1;
    __syncthreads();
    uint32_t count = 0;
    for (int k = 0; k < R; ++k) {
        const bool hit = r[k] >= 0;
        const uint32_t m = __ballot_sync(0xffffffffu, hit);
        if (lane == 0) warp_count[warp] = __popc(m);
        __syncthreads();
        uint32_t at = count;
        for (int w = 0; w < kFewThreads / 32; ++w) {
            if (w < warp) at += warp_count[w];
            count += warp_count[w];
        }
        if (hit) {
            found[at + __popc(m & ((1u << lane) - 1u))] = (uint32_t)r[k] << 10 | (uint32_t)(k * kFewThreads + threadIdx.x);
            touched[r[k]] = 1;
        }
        __syncthreads();
    }
    // a group of lanes takes the rows of its residue: rows of other groups are not its concern
    const int group = threadIdx.x / lanes, groups = kFewThreads / lanes, gl = threadIdx.x - group * lanes;
    const int c = c0 + gl * E;
    if (group >= groups || c >= a.width) return;
    for (int i = group; i < nrows; i += groups)
        if (touched[i])
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i * cols + gl * E + e] = 0.0f;
    constexpr int U = 8;  // rows in flight
    for (uint32_t j = 0; j < count; j += U) {
        Pack<TI, E> v[U];
        int at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t f = j + u < count ? found[j + u] : 0u;
            at[u] = j + u < count && (int)((f >> 10) % groups) == group ? (int)(f >> 10) * cols + gl * E : -1;
            if (at[u] >= 0)
                v[u] = load_pack<TI, E>(static_cast<const TI *>(a.rows) + (int64_t)(f & 1023u) * a.rows_stride + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at[u] >= 0)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[at[u] + e] += to_f32(v[u].v[e]);
    }
    for (int i = group; i < nrows; i += groups) {
        if (a.accumulate && !touched[i]) continue;
        TO *p = static_cast<TO *>(a.out) + ((int64_t)i * blocks + block) * a.out_stride + c;
        Pack<TO, E> o;
        if (a.accumulate) o = load_pack<TO, E>(p);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float x = touched[i] ? a.scale * acc[i * cols + gl * E + e] : 0.0f;
            if (a.accumulate) x += to_f32(o.v[e]);
            o.v[e] = from_f32<TO>(x);
        }
        store_pack<TO, E>(p, o);
    }
}

// ---- dispatch ---------------------------------------------------------------------

int bits_of(int64_t v)
{
    int b = 0;
    while (v >> b) ++b;
    return b;
}

size_t up(size_t b) { return (b + 255) & ~(size_t)255; }

// Elements per access that both matrices allow.
int pack_of(const EmbedArgs &a, int wide)
{
    for (int e : {wide, 2})
        if (a.width % e == 0 && rows_aligned(a.rows, a.rows_stride, a.rows_dtype, e) &&
            rows_aligned(a.out, a.out_stride, a.out_dtype, e))
            return e;
    return 1;
}

template <int V>
using Int = std::integral_constant<int, V>;

// f(TI{}, TO{}, E) for the accesses of a.
template <typename F>
cudaError_t with_types(const EmbedArgs &a, F &&f)
{
    return with_dtype(a.rows_dtype, [&](auto ti) {
        return with_dtype(a.out_dtype, [&](auto to) {
            // 16 bytes of the narrower type
            constexpr int W = sizeof(ti) == 4 && sizeof(to) == 4 ? 4 : 8;
            const int e = pack_of(a, W);
            if (e == W) return f(ti, to, Int<W>{});
            if (e == 2) return f(ti, to, Int<2>{});
            return f(ti, to, Int<1>{});
        });
    });
}

// Lanes (a power of two up to 32) for a row at kCols columns per lane, and the
// tiles a wider row takes.
void lanes_of(int width, int *lanes, int *tiles)
{
    *lanes = 1;
    while (*lanes < 32 && *lanes * kCols < width) *lanes <<= 1;
    *tiles = (width + *lanes * kCols - 1) / (*lanes * kCols);
}

struct GradLayout {
    int passes = 0, items = 1, tiles = 0, bins = 0;
    int64_t units = 0;
    size_t sorted[2] = {}, counts = 0, counts_later = 0, later_n = 0, part = 0, runs = 0, last = 0, bytes = 0;
};

GradLayout layout(const EmbedArgs &a)
{
    GradLayout l;
    if (a.n <= kFew) return l;
    const int bits = bits_of(a.vocab);  // keys 0 .. vocab
    l.passes = (bits + kMaxBits - 1) / kMaxBits;
    l.bins = 1 << ((bits + l.passes - 1) / l.passes);
    while (l.items < kMaxItems && a.n > (int64_t)kManyTiles * kSortThreads * l.items) l.items <<= 1;
    l.tiles = (int)((a.n + kSortThreads * l.items - 1) / (kSortThreads * l.items));
    l.units = (a.n + kUnit - 1) / kUnit;
    size_t at = 0;
    auto take = [&](size_t b) { const size_t p = at; at += up(b); return p; };
    for (size_t &p : l.sorted) p = take(8 * (size_t)a.n);
    const size_t counts_n = (size_t)l.bins * (l.tiles + 1);
    l.counts = take(4 * counts_n);
    l.later_n = counts_n * (l.passes - 1);
    l.counts_later = take(4 * l.later_n);
    l.part = take(8 * (size_t)l.units * a.width);
    l.runs = take(8 * (size_t)l.units + 4);  // a long run begins in a unit of its own
    l.last = take(4 * (size_t)a.vocab);
    l.bytes = at;
    return l;
}

}  // namespace

cudaError_t embed(const EmbedArgs &a, cudaStream_t s, int64_t *launches)
{
    return with_types(a, [&](auto ti, auto to, auto e) {
        constexpr int E = decltype(e)::value, NV = E >= 8 ? 4 : 16 / E;
        int lanes = 1;
        while (lanes < 32 && lanes * E * NV < a.width) lanes <<= 1;
        const int tiles = (a.width + lanes * E * NV - 1) / (lanes * E * NV);
        const int64_t want = (a.n * tiles * lanes + kThreads - 1) / kThreads;
        const unsigned grid = (unsigned)std::min<int64_t>(want, 16 * kSMs);
        k_embed<decltype(ti), decltype(to), E, NV><<<grid, kThreads, 0, s>>>(a, lanes, tiles);
        ++*launches;
        return cudaGetLastError();
    });
}

size_t embed_grad_tmp_bytes(const EmbedArgs &a) { return layout(a).bytes; }

size_t embed_grad_present_bytes(const EmbedArgs &a) { return a.accumulate || a.n <= kFew ? 0 : 4 * (size_t)((a.vocab + 31) / 32); }

cudaError_t embed_grad(const EmbedArgs &a, void *tmp, uint32_t *present, cudaStream_t st, int64_t *launches)
{
    const GradLayout l = layout(a);
    if (!l.passes) {
        return with_types(a, [&](auto ti, auto to, auto e) {
            constexpr int E = decltype(e)::value;
            // up to 32 lanes of columns; as many rows as the accumulators
            // hold, fewer when that leaves SMs without a block
            const int lanes = std::min((a.width + E - 1) / E, 64);
            const int tiles = (a.width + lanes * E - 1) / (lanes * E);
            int64_t rows = std::min<int64_t>(kFewFloats / (lanes * E), a.vocab);
            while (rows > 8 && (a.vocab + rows - 1) / rows * tiles < 4 * kSMs) rows >>= 1;
            const dim3 grid((unsigned)((a.vocab + rows - 1) / rows), tiles);
            k_grad_few<decltype(ti), decltype(to), E><<<grid, kFewThreads, 0, st>>>(a, (int)rows, lanes);
            ++*launches;
            return cudaGetLastError();
        });
    }
    char *p = static_cast<char *>(tmp);
    SortArgs s{};
    s.counts = (uint32_t *)(p + l.counts);
    s.runs = (uint32_t *)(p + l.runs);
    s.tiles = l.tiles;
    s.bits = bits_of(l.bins) - 1;
    s.scanned = l.tiles > kSumTiles;
    uint2 *items[2] = {(uint2 *)(p + l.sorted[0]), (uint2 *)(p + l.sorted[1])};
    s.present = a.accumulate ? nullptr : present;
    s.clear = (uint32_t *)(p + l.counts_later);
    s.clear_n = (int64_t)l.later_n;
    // the empty rows: an eighth with each scatter, whose latencies leave the
    // memory idle, and the rest beside the sums
    Fill f{};
    f.present = s.present;
    for (f.store = 16; f.store > 2; f.store = f.store == 4 ? 2 : 4) {
        const int e = f.store / (int)dtype_bytes(a.out_dtype);
        if (a.width % e == 0 && rows_aligned(a.out, a.out_stride, a.out_dtype, e)) break;
    }
    auto fill_blocks = [&](int warps) {  // for the share f0 .. f1
        return (int)std::min<int64_t>(2 * kSMs, (a.vocab * (f.f1 - f.f0) / kShares + warps - 1) / warps);
    };
    auto sort = [&](auto per_thread) {
        constexpr int ITEMS = decltype(per_thread)::value;
        const size_t words = s.present ? (size_t)((a.vocab + 31) / 32) : 0;
        HISS_TRY(launch_after(k_sort_count<ITEMS>, l.tiles, kSortThreads, words <= kBitmapWords ? 4 * words : 0, st, a, s));
        ++*launches;
        for (int i = 0; i < l.passes; ++i) {
            s.shift = i * s.bits;
            s.in = i ? items[(i - 1) & 1] : nullptr;
            s.out = items[i & 1];
            if (i) s.counts = s.counts_out;
            s.counts_out = i + 1 < l.passes ? s.clear + (size_t)l.bins * (l.tiles + 1) * i : nullptr;
            if (s.scanned) {
                HISS_TRY(launch_after(k_sort_scan, (l.bins + 31) / 32, 1024, 0, st, s));
                ++*launches;
            }
            f.f0 = f.f1;
            f.f1 = f.f0 + kScatterShare;
            f.blocks = s.present ? fill_blocks(kSortWarps) : 0;
            HISS_TRY(launch_after(k_sort_scatter<ITEMS>, l.tiles + f.blocks, kSortThreads, 0, st, a, s, f));
            ++*launches;
        }
        return cudaSuccess;
    };
    HISS_TRY(l.items == 1 ? sort(Int<1>{}) : l.items == 2 ? sort(Int<2>{}) : l.items == 4 ? sort(Int<4>{}) : sort(Int<8>{}));
    return with_types(a, [&](auto ti, auto to, auto e) {
        using TO = decltype(to);
        constexpr int E = decltype(e)::value;
        SumArgs m{};
        m.items = s.out;
        m.part = (float *)(p + l.part);
        m.runs = s.runs;
        m.last = (uint32_t *)(p + l.last);
        m.units = l.units;
        lanes_of(a.width, &m.lanes, &m.tiles);
        m.present = s.present;
        m.blocks = (int)((l.units * m.tiles * m.lanes + kThreads - 1) / kThreads);
        f.f0 = f.f1;
        f.f1 = kShares;
        f.blocks = s.present && f.f0 < f.f1 ? fill_blocks(kThreads / 32) : 0;
        using TI = decltype(ti);
        auto sum = [&](auto full) {
            auto kernel = k_sum<TI, TO, E, decltype(full)::value>;
            constexpr size_t smem = sum_bytes<TI, E>();
            static std::atomic<bool> allowed{false};  // of this kernel
            if (smem > 48 * 1024 && !allowed.load(std::memory_order_acquire)) {
                HISS_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
                allowed.store(true, std::memory_order_release);
            }
            return launch_after(kernel, m.blocks + f.blocks, kThreads, smem, st, a, m, f);
        };
        HISS_TRY(m.lanes == 32 ? sum(std::true_type{}) : sum(std::false_type{}));
        HISS_TRY(launch_after(k_join<TO, E>, kJoinBlocks, kJoinThreads, 0, st, a, m));
        *launches += 2;
        return cudaSuccess;
    });
}

}  // namespace hiss
