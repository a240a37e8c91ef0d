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
//   2. k_sum cuts the sorted positions into units of 8 to 32 and sums runs of equal
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
constexpr int kRawThreads = 128;  // of k_embed_raw

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
// one position.  Bound by writes, which this memory takes at 4.0 TB/s alone: 131,072
// positions x 1024, float32 to bfloat16, 72 us (3.7 TB/s written, 1.8 read).
// Four blocks per SM (64 registers) against three: 60,000 x 768 bfloat16 31 -> 27 us;
// two packs per lane instead of four: 38.  The limit of 64 spills 8 to 24 bytes per thread
// in five of the aligned builds (float32 or bfloat16 to bfloat16 among them).
template <typename TI, typename TO, int E, int NV>
__global__ void __launch_bounds__(kThreads, 4) k_embed(EmbedArgs a, int lanes, int tiles)
{
    const int per_block = kThreads / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t items = a.n * tiles, step = (int64_t)gridDim.x * per_block;
    int64_t it = (int64_t)blockIdx.x * per_block + threadIdx.x / lanes;
    auto position = [&](int64_t item) { return tiles == 1 ? item : item / tiles; };
    int64_t next = it < items ? row_of(a, position(it)) : kPadRow;
    bool bad = false;
    for (; it < items; it += step) {
        const int64_t i = position(it);
        const int c0 = ((int)(it - i * tiles) * lanes * NV + lane) * E;
        const int64_t r = next;
        const TI *p = static_cast<const TI *>(a.rows) + r * a.rows_stride;
        TO *q = static_cast<TO *>(a.out) + i * a.out_stride;
        Pack<TI, E> v[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * lanes * E;
            if (r >= 0 && c < a.width) v[k] = load_pack<TI, E>(p + c);
        }
        // the next position's token is on its way while this row is
        if (it + step < items) next = row_of(a, position(it + step));
        bad = bad || r == kBadRow;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = c0 + k * lanes * E;
            if (c >= a.width) continue;
            Pack<TO, E> o;
#pragma unroll
            for (int e = 0; e < E; ++e) o.v[e] = from_f32<TO>(r >= 0 ? a.scale * to_f32(v[k].v[e]) : 0.0f);
            store_pack<TO, E>(q + c, o);
        }
    }
    if (bad) *a.bad = 1;
}

// The 16-byte lines that hold E elements of any address, and those elements shifted
// into place.  Lanes of two rows sit in one warp, so nothing here branches.
template <typename T, int E>
struct Lines {
    static constexpr int W = E * sizeof(T) / 4, L = E * sizeof(T) / 16 + 1;  // words; lines they can lie in
    uint4 q[L];

    __device__ __forceinline__ void load(const T *p, bool wanted)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        const uint4 *line = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            q[i] = make_uint4(0, 0, 0, 0);
            if (wanted && (i + 1 < L || (at & 15))) q[i] = line[i];
        }
    }
    __device__ __forceinline__ void shifted(const T *p, Pack<T, E> &v) const
    {
        const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15;
        uint32_t w[4 * L];
#pragma unroll
        for (int i = 0; i < L; ++i) w[4 * i] = q[i].x, w[4 * i + 1] = q[i].y, w[4 * i + 2] = q[i].z, w[4 * i + 3] = q[i].w;
#pragma unroll
        for (int i = 0; i < W + 2; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < W + 1; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
        uint32_t *o = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] = sizeof(T) == 2 ? __funnelshift_r(w[i], w[i + 1], 8 * (off & 2)) : w[i];
    }
};

template <typename T, int E>
__device__ __forceinline__ void store_sector(T *p, const Pack<T, E> &v)
{
    static_assert(sizeof(v) == 32, "one sector, one store");
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Rows that are not aligned to 16 bytes, in or out: a thread writes the E elements
// of one 32-byte sector of the output, at column E k - s for sector k of a row that
// begins s elements into its first.  The sectors of all rows are dealt out in
// turn (sectors per row; magic divides by it), so that a row's length need not fit a
// warp; a row's first and last sector go word by word, and packs whose
// input lines reach outside the table are loaded element by element.
//
// Bound by instructions (3.1 per cycle) and, almost as much, by writes: 214,863 x 526
// float16 60 us (3.8 TB/s written); 92 with 16 bytes per thread, whose
// indexing costs the same, and 171 with a warp per 512 columns of one row.
// Two sectors per thread 75, blocks of 256 threads 64.  44,985 x 1853 bfloat16 44 us.
template <typename TI, typename TO, int E>
__global__ void __launch_bounds__(kRawThreads) k_embed_raw(EmbedArgs a, int sectors, uint32_t magic)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(a.rows), hi = lo + ((a.vocab - 1) * a.rows_stride + a.width) * sizeof(TI);
    const int64_t first = (int64_t)blockIdx.x * kRawThreads;
    const int64_t i0 = first <= 0xffffffffll ? (int64_t)((uint32_t)first / (uint32_t)sectors) : first / sectors;
    const uint32_t x = (uint32_t)(first - i0 * sectors) + threadIdx.x, d = sectors > 1 ? __umulhi(x, magic) : x;
    const int64_t i = i0 + d;
    if (i >= a.n) return;
    const int64_t r = row_of(a, i);
    TO *q = static_cast<TO *>(a.out) + i * a.out_stride;
    const int c = (int)(x - d * sectors) * E - (int)((reinterpret_cast<uintptr_t>(q) & 31) / sizeof(TO));
    q += c;
    const TI *p = static_cast<const TI *>(a.rows) + r * a.rows_stride + c;
    const uintptr_t from = reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15;
    const uintptr_t to = (reinterpret_cast<uintptr_t>(p + E) + 15) & ~(uintptr_t)15;
    const bool inside = from >= lo && to <= hi;
    Lines<TI, E> in;
    in.load(p, r >= 0 && inside);
    if (r == kBadRow) *a.bad = 1;
    Pack<TI, E> v;
    in.shifted(p, v);
    const int e0 = max(-c, 0), e1 = min(a.width - c, E);  // its elements e0 .. e1 are the row's
    if (r >= 0 && !inside)
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e >= e0 && e < e1) v.v[e] = p[e];
    // a row that is not there: +0 times the zeros that were not loaded
    const float2 scale = both(r >= 0 ? a.scale : 0.0f);
    Pack<TO, E> o;
#pragma unroll
    for (int e = 0; e < E; e += 2) set_pair(o.v + e, __fmul2_rn(scale, pair_of(v.v + e)));
    if (e1 - e0 == E) {
        store_sector(q, o);
        return;
    }
    // its whole 4-byte words, and the elements of 2 bytes beside them
    constexpr int PER = 4 / sizeof(TO);
    const int w0 = (e0 + PER - 1) / PER, w1 = e1 / PER;
    const uint32_t here = w1 > w0 ? (1u << w1) - (1u << w0) : 0;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&o);
#pragma unroll
    for (int j = 0; j < E / PER; ++j)
        if (here >> j & 1) reinterpret_cast<uint32_t *>(q)[j] = w[j];
    if constexpr (PER == 2) {
        if (e0 < e1 && (e0 & 1)) q[e0] = from_f32<TO>(r >= 0 ? a.scale * to_f32(p[e0]) : 0.0f);
        if (e0 < e1 && (e1 & 1)) q[e1 - 1] = from_f32<TO>(r >= 0 ? a.scale * to_f32(p[e1 - 1]) : 0.0f);
    }
}

// ---- the sort ---------------------------------------------------------------------

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxItems = 8;  // positions per thread
constexpr int kMaxBits = 9;  // one bin per thread
constexpr int kMaxBins = 1 << kMaxBits;
// The sort is a chain of latencies.  Up to kSumTiles tiles each block of the
// scatter adds up the tiles' counts itself; above, their prefix sums are a kernel of
// their own, and tiles are as small as kManyTiles allows (few large ones leave
// the sort on few SMs: 262,144 positions in 64 tiles 6 us more than in 128).
constexpr int kSumTiles = 32, kSumItems = 4;
constexpr int kManyTiles = 128;
constexpr int kBitmapWords = 8192;  // of a block's bitmap of tokens (32 KB: a vocabulary of 262,144)

struct SortArgs {
    const uint2 *in;     // (key, position); NULL: the tokens and their positions
    uint2 *out;
    uint32_t *counts;    // digit counts of the input's tiles: [tiles][bins], exclusive over the
                         // tiles once scanned; then [bins] totals
    uint32_t *counts_out;  // the next digit's counts of the output's tiles (NULL: last pass)
    uint32_t *present;   // [ceil(vocab / 32)] bit: the token occurs (NULL: not wanted); 0 between calls
    uint32_t *runs;      // numbers of long runs (SumArgs), set to 0 by the first kernel
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

// Zeros (all bits 0 in every type) for bytes at p, a multiple of 2, by a warp.
__device__ __forceinline__ void zero_bytes(char *p, int64_t bytes, int lane)
{
    const int head = (int)min((int64_t)(-reinterpret_cast<uintptr_t>(p) & 15), bytes);
    const int64_t lines = (bytes - head) / 16;
    const int tail = (int)(bytes - head) & 15;
    if (2 * lane < head) reinterpret_cast<uint16_t *>(p)[lane] = 0;
    p += head;
    for (int64_t i = lane; i < lines; i += 32) reinterpret_cast<uint4 *>(p)[i] = uint4{};
    if (2 * lane < tail) reinterpret_cast<uint16_t *>(p + 16 * lines)[lane] = 0;
}

// Zeros for the rows base + i, i < count, of the gradient whose bit i is not
// set; warp of warps.  A run of such rows without gaps between them is one stretch of
// bytes, so that narrow and unaligned rows are written in whole lines too: 1,000
// positions over 131,072 x 16 bfloat16 24 -> 17 us, 5,000 over 58,391 x 1333 73 -> 56.
__device__ void fill_rows(const EmbedArgs &a, const uint32_t *held, int64_t base, int64_t count, int64_t warp, int64_t warps)
{
    const int lane = threadIdx.x & 31;
    const int size = a.out_dtype == HISS_F32 ? 4 : 2;
    const int64_t bytes = (int64_t)a.width * size, stride = a.out_stride * size;
    int rows = 32;  // per warp and turn: a power of two, so that they share a word
    while (rows > 1 && count < warps * rows) rows >>= 1;
    for (int64_t v = warp * rows; v < count; v += warps * rows) {
        uint32_t empty = ~(held[v >> 5] >> (v & 31));
        const int n = (int)min((int64_t)rows, count - v);
        if (n < 32) empty &= (1u << n) - 1u;
        while (empty) {
            const int first = __ffs(empty) - 1;
            const uint32_t rest = ~(empty >> first);  // its lowest bit: the run's end
            const int run = stride != bytes ? 1 : rest ? __ffs(rest) - 1 : 32;
            empty &= ~((run < 32 ? (1u << run) - 1u : ~0u) << first);
            zero_bytes(static_cast<char *>(a.out) + (base + v + first) * stride, run * bytes, lane);
        }
    }
}

// The rows that no position holds, in this kernel's share [f0, f1) of kShares of the vocabulary.
constexpr int kShares = 8, kScatterShare = 2;
struct Fill {
    const uint32_t *present;
    int f0, f1;
    int blocks;          // blocks of the kernel that do this, behind the others
};
// The share in words of the bitmap, and the rows of the vocabulary that those hold.
struct Share {
    int64_t word, rows;
};
__host__ __device__ __forceinline__ Share share_of(int64_t vocab, const Fill &f)
{
    const int64_t words = (vocab + 31) / 32, w0 = words * f.f0 / kShares, end = 32 * (words * f.f1 / kShares);
    return {w0, (end < vocab ? end : vocab) - 32 * w0};
}
__device__ void fill_empty(const EmbedArgs &a, const Fill &f, int64_t warp, int64_t warps)
{
    const Share s = share_of(a.vocab, f);
    fill_rows(a, f.present + s.word, 32 * s.word, s.rows, warp, warps);
}

// First digit's counts of each tile, and which tokens occur.  Latency: 65,536
// positions 6 us, most of it one round trip to memory.
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
    if (blockIdx.x == 0 && threadIdx.x < 2) s.runs[threadIdx.x] = 0;
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
    constexpr int B = 4;  // counts held per thread: up to 128 tiles in one batch
    uint32_t c[B], v = 0;
    if (bin < bins)
        for (int t = t0; t < t1; t += B) {
#pragma unroll
            for (int u = 0; u < B; ++u) c[u] = t + u < t1 ? s.counts[(int64_t)(t + u) * bins + bin] : 0u;
#pragma unroll
            for (int u = 0; u < B; ++u) v += c[u];
        }
    sum[w][lane] = v;
    __syncthreads();
    uint32_t run = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) run += i < w ? sum[i][lane] : 0u;
    if (bin >= bins) return;
    for (int t = t0; t < t1; t += B) {
        if (t1 - t0 > B) {
#pragma unroll
            for (int u = 0; u < B; ++u) c[u] = t + u < t1 ? s.counts[(int64_t)(t + u) * bins + bin] : 0u;
        }
#pragma unroll
        for (int u = 0; u < B; ++u)
            if (t + u < t1) {
                s.counts[(int64_t)(t + u) * bins + bin] = run;
                run += c[u];
            }
    }
    if (w == 31) s.counts[(int64_t)s.tiles * bins + bin] = run;
    let_next_start();
}

// One stable pass: each tile's positions go behind those of the tiles before
// it, digit by digit.  Counts the next digit of the tiles it writes to on the way
// (one launch less per pass).  Latency again: 65,536 positions about 9 us,
// 12 beside the zeros of a quarter of 50,001 x 1024 float32.
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
            // in batches: the loads of a loop of unknown length wait for one another
            constexpr int B = 16;
            for (int t0 = 0; t0 < s.tiles; t0 += B) {
                uint32_t c[B];
#pragma unroll
                for (int u = 0; u < B; ++u) c[u] = t0 + u < s.tiles ? s.counts[(int64_t)(t0 + u) * bins + bin] : 0u;
#pragma unroll
                for (int u = 0; u < B; ++u) {
                    total += c[u];
                    if (t0 + u < (int)blockIdx.x) before += c[u];
                }
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

struct SumArgs {
    const uint2 *items;           // sorted (token, position)
    float *part;                  // [units][2][width]: sum of the long run that comes in from the unit
                                  // before, and of the long run that begins here
    uint32_t *runs;               // [0]: number of long runs; then (key, last unit) of each, those of many
                                  // units from the end of the list backwards, counted in [1]
    uint32_t *first;              // [vocab]: first unit of a long run
    uint32_t *present;            // cleared at the end
    int64_t units;
    int unit;                     // positions per unit
    int lanes, tiles;             // lanes per unit and tile; tiles of a row
    int blocks;                   // of k_sum that sum (the others write empty rows)
};

// How a group of lanes takes a tile of lanes * C columns of a row.
//   packed: packs of E elements, pack k of lane l at column (k lanes + l) E of the tile;
//           each lane copies its own packs to shared memory, ahead of their sum;
//   raw (E <= 2): rows that are not aligned to 16 bytes.  The group copies the 16-byte
//           lines that hold the tile and each lane reads its single elements or pairs.
// BIG tiles (32 lanes of 16 columns) cost the fewest instructions per element (262,144
// positions x 322 float16: 91 us, 130 with small ones), small ones spread a narrow
// row, or few positions, over more lanes.
template <typename TI, int E, bool BIG>
struct SumShape {
    static constexpr bool RAW = E <= 2;
    static constexpr int C = BIG ? 16 : RAW ? 2 * E : E;   // columns per lane
    static constexpr int kAhead = BIG ? 4 : 8;             // rows in the ring
    // bytes of a row of the ring: a raw tile begins at its offset in a line
    __host__ __device__ static constexpr int row_bytes(int lanes)
    {
        return RAW ? (lanes * C * (int)sizeof(TI) + 16 + 15) / 16 * 16 : lanes * C * (int)sizeof(TI);
    }
    static constexpr size_t smem(int lanes) { return (size_t)(kThreads / lanes) * kAhead * row_bytes(lanes); }
};

// Write (or add) a finished row's columns.
template <typename TO, int E, int C>
__device__ __forceinline__ void write_row(const EmbedArgs &a, uint32_t v, int c0, int lanes, const float (&s)[C])
{
    TO *p = static_cast<TO *>(a.out) + (int64_t)v * a.out_stride;
#pragma unroll
    for (int k = 0; k < C / E; ++k) {
        const int c = c0 + k * lanes * E;
        if (c >= a.width) break;
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

template <int E, int C>
__device__ __forceinline__ void write_part(const EmbedArgs &a, float *p, int c0, int lanes, const float (&s)[C])
{
#pragma unroll
    for (int k = 0; k < C / E; ++k) {
        const int c = c0 + k * lanes * E;
        if (c >= a.width) break;
        Pack<float, E> o;
#pragma unroll
        for (int e = 0; e < E; ++e) o.v[e] = s[k * E + e];
        store_pack<float, E>(p + c, o);
    }
}

constexpr int kManyUnits = 64;  // a run over more units is summed by a whole block

// The sums of the runs.  65,536 positions x 1024 bfloat16 over 50,001 float32 rows,
// with half of the empty rows' zeros: 49 us at 4.7 TB/s, bound by memory.  262,144 x
// 322 float16, rows aligned to 4 bytes, bound by instructions: the call 66 us; 74
// with every row's address computed by the whole warp when it comes up, not by one lane each
// beforehand.  Rows wait in a shared-memory ring, and there is one copy of the code that writes a
// finished row: inside a loop unrolled over the rows it made the kernel take 93 us.
template <typename TI, typename TO, int E, bool BIG>
__global__ void __launch_bounds__(kThreads) k_sum(EmbedArgs a, SumArgs s, Fill f)
{
    using S = SumShape<TI, E, BIG>;
    constexpr bool RAW = S::RAW;
    constexpr int C = S::C, A = S::kAhead, NV = C / E;
    using P = Pack<TI, E>;
    extern __shared__ __align__(16) char ring[];
    wait_for_previous();
    if ((int)blockIdx.x >= s.blocks) {
        fill_empty(a, f, (int64_t)(blockIdx.x - s.blocks) * (kThreads / 32) + (threadIdx.x >> 5),
                   (int64_t)f.blocks * (kThreads / 32));
        return;
    }
    const int lanes = BIG ? 32 : s.lanes;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    const int lane = threadIdx.x & (lanes - 1);
    if (item >= s.units * s.tiles) return;
    // tiles of a unit are neighbours: they read the same rows of dy
    const int64_t unit = item / s.tiles;
    const int tile = (int)(item - unit * s.tiles);
    const int t0 = tile * lanes * C, cols = min(lanes * C, a.width - t0);  // the tile's columns
    const int c0 = t0 + lane * E;
    const int n = (int)a.n, i0 = (int)unit * s.unit, i1 = min(i0 + s.unit, n);
    const uint32_t vocab = (uint32_t)a.vocab, none = ~0u;
    auto key_of = [&](int i) { return i >= 0 && i < n ? s.items[i].x : none; };
    const uint32_t k0 = key_of(i0), k1 = key_of(i1 - 1);
    const uint32_t prev = key_of(i0 - 1), prev_unit = key_of(i0 - s.unit), prev_unit2 = key_of(i0 - s.unit - 1);
    const uint32_t next = key_of(i1), next_unit = key_of(i1 + s.unit);
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
    if (long_out && begins && tile == 0 && lane == 0) s.first[k1] = (uint32_t)unit;
    if (long_in && (next != k0 || k1 != k0) && tile == 0 && lane == 0) {
        const bool many = key_of(i0 - kManyUnits * s.unit) == k0;
        const uint32_t at = atomicAdd(s.runs + many, 1u);
        *reinterpret_cast<uint2 *>(s.runs + 2 * (many ? s.units - at : 1 + at)) = make_uint2(k0, (uint32_t)unit);
    }
    if (i >= end) return;

    const int row_bytes = S::row_bytes(lanes);
    char *group_ring = ring + (threadIdx.x / lanes) * (A * row_bytes);
    const TI *rows = static_cast<const TI *>(a.rows) + t0;
    // raw: lines that reach outside the matrix are copied by element: they belong
    // to the first and last rows
    const uint32_t edge = a.rows_stride > 0 ? (uint32_t)((15 + a.rows_stride) / a.rows_stride) : 0x7fffffffu;
    // the address of row y, with bit 0 (raw) set for those
    auto place = [&](uint32_t y) {
        const uint64_t p = reinterpret_cast<uint64_t>(rows + (int64_t)y * a.rows_stride);
        return RAW && !(y >= edge && y + edge < (uint32_t)n) ? p | 1 : p;
    };
    // start copying the row at a place into slot st of the ring
    auto copy = [&](uint64_t at, int st) {
        char *d = group_ring + st * row_bytes;
        if constexpr (RAW) {
            const int off = (int)at & 14, bytes = off + cols * (int)sizeof(TI);
            const char *q = reinterpret_cast<const char *>(at & ~(uint64_t)15);
            if (!(at & 1)) {
                if constexpr (BIG) {
#pragma unroll
                    for (int k = 0; k < (512 * (int)sizeof(TI) + 15 + 511) / 512; ++k) {
                        if (512 * k >= bytes) break;
                        if (512 * k + 16 * lane < bytes) cp_async16(d + 512 * k + 16 * lane, q + 512 * k + 16 * lane);
                    }
                } else {
                    for (int b = 16 * lane; b < bytes; b += 16 * lanes) cp_async16(d + b, q + b);
                }
            } else {
                const uintptr_t lo = reinterpret_cast<uintptr_t>(a.rows), hi = lo + ((a.n - 1) * a.rows_stride + a.width) * sizeof(TI);
                const uintptr_t line0 = at & ~(uint64_t)15, b0 = line0 + off, b1 = b0 + cols * sizeof(TI);
                for (int b = 16 * lane; b < bytes; b += 16 * lanes) {
                    if (line0 + b >= lo && line0 + b + 16 <= hi) {
                        cp_async16(d + b, q + b);
                    } else {
                        for (uintptr_t e = max(line0 + b, b0); e < min(line0 + b + 16, b1); e += sizeof(TI))
                            *reinterpret_cast<TI *>(d + (e - line0)) = *reinterpret_cast<const TI *>(e);
                    }
                }
            }
        } else {
            const TI *p = reinterpret_cast<const TI *>(at);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * lanes + lane) * E;
                if (c >= cols) break;
                copy_pack_async<TI, E>(reinterpret_cast<P *>(d) + k * lanes + lane, p + c);
            }
        }
    };
    float acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.0f;
    // add the row in slot st; at: the low bits of its place
    auto add = [&](uint32_t at, int st) {
        const char *d = group_ring + st * row_bytes;
        if constexpr (RAW) d += at & 14;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k * lanes * E >= cols) break;
            // what lies beyond the tile's columns is not written
            const P v = reinterpret_cast<const P *>(d)[k * lanes + lane];
            if constexpr (E == 1) {
                acc[k] += to_f32(v.v[0]);
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 p = __fadd2_rn(make_float2(acc[k * E + e], acc[k * E + e + 1]), pair_of(v.v + e));
                    acc[k * E + e] = p.x;
                    acc[k * E + e + 1] = p.y;
                }
            }
        }
    };
    float *part = s.part + unit * 2 * a.width;
    bool head = long_in;  // the current run is the long one that came in
    // a run is complete, with its last position before the end or not
    auto flush = [&](uint32_t key, bool at_end) {
        if (head || (at_end && long_out)) write_part<E, C>(a, head ? part : part + a.width, c0, lanes, acc);
        else write_row<TO, E, C>(a, key, c0, lanes, acc);
        head = false;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = 0.0f;
    };
    const int m = end - i;  // positions, at most two units
    if constexpr (BIG) {
        // the rows' places (at most 64) wait in shared memory, the tokens in the
        // warp's lanes, and where a run ends in a mask
        __shared__ uint64_t where[kThreads / 32][64];
        uint64_t *const place_of = where[threadIdx.x / 32];
        uint32_t it[2];
        uint64_t ends = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = i + 32 * h + lane;
            const uint2 item = j < end ? s.items[j] : make_uint2(none, 0);
            it[h] = item.x;
            if (j < end) place_of[32 * h + lane] = place(item.y);
            const uint32_t after = j + 1 < end ? s.items[j + 1].x : none;
            ends |= (uint64_t)__ballot_sync(0xffffffffu, item.x != after) << (32 * h);
        }
        __syncwarp();
        for (int k = 0; k < A - 1; ++k) {
            if (k < m) copy(place_of[k], k);
            cp_async_commit();
        }
        for (int j = 0; j < m; ++j) {
            cp_async_wait<A - 2>();
            // raw: the row was copied by the whole warp, and the row before it has been
            // read by the whole warp before its place in the ring is filled again
            if (RAW) __syncwarp();
            if (j + A - 1 < m) copy(place_of[j + A - 1], (j + A - 1) & (A - 1));
            cp_async_commit();
            add(RAW ? (uint32_t)place_of[j] : 0u, j & (A - 1));
            if (ends >> j & 1) {
                const uint32_t x0 = __shfl_sync(0xffffffffu, it[0], j & 31), x1 = __shfl_sync(0xffffffffu, it[1], j & 31);
                flush(j < 32 ? x0 : x1, j + 1 == m);
            }
        }
    } else {
        const uint32_t mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
        for (int k = 0; k < A - 1; ++k) {
            if (k < m) copy(place(s.items[i + k].y), k);
            cp_async_commit();
        }
        uint2 it = s.items[i];
        for (int j = 0; j < m; ++j) {
            cp_async_wait<A - 2>();
            if (RAW) __syncwarp(mask);
            if (j + A - 1 < m) copy(place(s.items[i + j + A - 1].y), (j + A - 1) & (A - 1));
            cp_async_commit();
            add(RAW ? (uint32_t)place(it.y) : 0u, j & (A - 1));
            const uint32_t key = it.x;
            it = j + 1 < m ? s.items[i + j + 1] : make_uint2(none, 0);
            if (it.x != key) flush(key, j + 1 == m);
        }
    }
    let_next_start();
}

constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinCols = 64;      // columns per tile of a run of many units
constexpr int kJoinBlocks = 2 * kSMs;

// The row of each long run: the second part of the unit it begins in and the
// first parts of the units up to its last.  The first half of the blocks takes the
// runs of many units, a run and tile at a time: a thread per column and stretch of
// units, the stretches added up in order.  In the other half each warp
// takes a run and 128 columns.  Latency: 7 to 9 us for 95 to 300 runs (41 us
// for 268 runs of five units x 2749 columns when every run took a block).
template <typename TO>
__global__ void __launch_bounds__(kJoinThreads) k_join(EmbedArgs a, SumArgs s)
{
    constexpr int G = kJoinThreads / kJoinCols;
    __shared__ float sh[G][kJoinCols];
    wait_for_previous();
    if (s.present)
        for (int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; i < (a.vocab + 31) / 32; i += (int64_t)gridDim.x * kJoinThreads)
            s.present[i] = 0;
    const bool many = blockIdx.x < gridDim.x / 2;
    const int64_t runs = s.runs[many];
    auto record = [&](int64_t run) { return *reinterpret_cast<const uint2 *>(s.runs + 2 * (many ? s.units - run : 1 + run)); };
    auto finish = [&](uint32_t key, int c, float x) {
        x *= a.scale;
        TO *p = static_cast<TO *>(a.out) + (int64_t)key * a.out_stride + c;
        if (a.accumulate) x += to_f32(*p);
        *p = from_f32<TO>(x);
    };
    constexpr int U = 8;  // parts in flight
    if (many) {
        const int group = threadIdx.x / kJoinCols, lane = threadIdx.x % kJoinCols;
        const int tiles = (a.width + kJoinCols - 1) / kJoinCols;
        for (int64_t it = blockIdx.x; it < runs * tiles; it += gridDim.x / 2) {
            const int64_t run = it / tiles;
            const int c = (int)(it - run * tiles) * kJoinCols + lane;
            const uint2 r = record(run);
            const int64_t first = s.first[r.x], count = (int64_t)r.y - first + 1;
            const int64_t to = first + count * (group + 1) / G;
            float x = 0.0f;
            for (int64_t u = first + count * group / G; u < to; u += U) {
                float v[U];
#pragma unroll
                for (int k = 0; k < U; ++k)
                    v[k] = u + k < to && c < a.width ? s.part[((u + k) * 2 + (u + k == first)) * a.width + c] : 0.0f;
#pragma unroll
                for (int k = 0; k < U; ++k) x += v[k];
            }
            sh[group][lane] = x;
            __syncthreads();
            if (group == 0 && c < a.width) {
#pragma unroll
                for (int g = 1; g < G; ++g) x += sh[g][lane];
                finish(r.x, c, x);
            }
            __syncthreads();
        }
    } else {
        constexpr int N = 4;
        const int lane = threadIdx.x & 31;
        const int tiles = (a.width + 32 * N - 1) / (32 * N);
        const int64_t warp = (int64_t)(blockIdx.x - gridDim.x / 2) * kJoinWarps + (threadIdx.x >> 5);
        for (int64_t it = warp; it < runs * tiles; it += (int64_t)(gridDim.x - gridDim.x / 2) * kJoinWarps) {
            const int64_t run = it / tiles;
            const int c = (int)(it - run * tiles) * 32 * N + lane;
            const uint2 r = record(run);
            const int64_t first = s.first[r.x], to = (int64_t)r.y + 1;
            float x[N] = {};
            for (int64_t u = first; u < to; u += U) {
                float v[U][N];
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int q = 0; q < N; ++q)
                        v[k][q] = u + k < to && c + 32 * q < a.width ? s.part[((u + k) * 2 + (u + k == first)) * a.width + c + 32 * q] : 0.0f;
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int q = 0; q < N; ++q) x[q] += v[k][q];
            }
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (c + 32 * q < a.width) finish(r.x, c + 32 * q, x[q]);
        }
    }
}

// ---- few positions -------------------------------------------------------------------

// Up to here one kernel replaces the sort: about where the two meet (1,500 positions over
// 5,000 x 1024 rows 15 us against 26, 2,000 over 32,000 x 1024 38 against 34, where the
// zeros count for more than the positions).
constexpr int kFew = 2048;
constexpr int kFewRound = kFew / kThreads;  // tokens per thread
constexpr int kFewPacks = 4;                // packs per lane
constexpr int kFewRows = 8192;              // most rows of a fill block

struct FewArgs {
    int lanes, tiles;    // lanes (a power of two) per row and tile; tiles of a row
    int sums;            // blocks that sum: one per position and tile
    int rows;            // rows of a fill block (the blocks behind those)
};

// One kernel without a sort.  A block per position (and tile of columns): the
// first position of a token collects the token's other positions, in order,
// and writes the row; the others leave.  Further blocks write zeros to the rows of
// their range that no position holds.  384 positions x 256 over 5,003 rows: 5 us, a
// token load, a dy load and a store one after the other; with a large vocabulary the
// zeros bound it (94 x 2968 over 27,183 rows: 48 us, 3.4 TB/s written).  Four blocks per SM
// cost the build of four float32 columns 16 bytes of spills.
template <typename TI, typename TO, int E>
__global__ void __launch_bounds__(kThreads, 4) k_grad_few(EmbedArgs a, FewArgs f)
{
    constexpr int U = E == 8 ? 4 : 8;  // rows in flight
    __shared__ uint16_t found[kFew];
    __shared__ uint32_t warp_count[kThreads / 32];
    __shared__ union {
        float part[kThreads * E];
        uint32_t held[kFewRows / 32];
    } sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int r[kFewRound];  // a row is below 2^31
#pragma unroll
    for (int k = 0; k < kFewRound; ++k) {
        const int i = k * kThreads + threadIdx.x;
        r[k] = i < a.n ? (int)row_of(a, i) : (int)kPadRow;
    }
    if ((int)blockIdx.x >= f.sums) {
        const int64_t v0 = (int64_t)(blockIdx.x - f.sums) * f.rows, v1 = min(v0 + f.rows, a.vocab);
        for (int i = threadIdx.x; i < (f.rows + 31) / 32; i += kThreads) sh.held[i] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kFewRound; ++k)
            if (r[k] >= v0 && r[k] < v1) atomicOr(&sh.held[(r[k] - v0) >> 5], 1u << ((r[k] - v0) & 31));
        __syncthreads();
        fill_rows(a, sh.held, v0, v1 - v0, warp, kThreads / 32);
        return;
    }
    const int pos = blockIdx.x / f.tiles, tile = blockIdx.x - pos * f.tiles;
    const int row = (int)row_of(a, pos);
    if (row < 0) {
        if (row == kBadRow && threadIdx.x == 0) *a.bad = 1;
        return;
    }
    bool earlier = false;
#pragma unroll
    for (int k = 0; k < kFewRound; ++k) earlier = earlier || (r[k] == row && k * kThreads + (int)threadIdx.x < pos);
    if (__syncthreads_or(earlier)) return;
    int count = 0;
    for (int k = 0; k * kThreads < a.n; ++k) {
        bool hit = false;
#pragma unroll
        for (int q = 0; q < kFewRound; ++q) hit = hit || (q == k && r[q] == row);
        const uint32_t m = __ballot_sync(0xffffffffu, hit);
        if (lane == 0) warp_count[warp] = __popc(m);
        __syncthreads();
        int at = count;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) at += warp_count[w];
            count += warp_count[w];
        }
        if (hit) found[at + __popc(m & ((1u << lane) - 1u))] = (uint16_t)(k * kThreads + threadIdx.x);
        __syncthreads();
    }
    // each group of lanes takes a stretch of the positions
    const int group = threadIdx.x / f.lanes, groups = kThreads / f.lanes, l = threadIdx.x & (f.lanes - 1);
    const int c0 = (tile * f.lanes * kFewPacks + l) * E;
    const int from = count * group / groups, to = count * (group + 1) / groups;
    TO *out = static_cast<TO *>(a.out) + row * a.out_stride;
    auto add = [&](int c, float(&acc)[E]) {
        const TI *p = static_cast<const TI *>(a.rows) + c;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        for (int j = from; j < to; j += U) {
            Pack<TI, E> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j + u < to) v[u] = load_pack<TI, E>(p + (int64_t)found[j + u] * a.rows_stride);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j + u < to)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += to_f32(v[u].v[e]);
        }
    };
    auto write = [&](int c, const float(&acc)[E]) {
        Pack<TO, E> o;
        if (a.accumulate) o = load_pack<TO, E>(out + c);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float x = a.scale * acc[e];
            if (a.accumulate) x += to_f32(o.v[e]);
            o.v[e] = from_f32<TO>(x);
        }
        store_pack<TO, E>(out + c, o);
    };
    float acc[E];
    if (groups > 1) {  // a row is one pack per lane; the groups' sums are added up in order
        if (c0 < a.width) {
            add(c0, acc);
#pragma unroll
            for (int e = 0; e < E; ++e) sh.part[(group * E + e) * f.lanes + l] = acc[e];
        }
        __syncthreads();
        if (group > 0 || c0 >= a.width) return;
        for (int g = 1; g < groups; ++g)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += sh.part[(g * E + e) * f.lanes + l];
        write(c0, acc);
        return;
    }
#pragma unroll 1
    for (int c = c0; c < min(c0 + f.lanes * kFewPacks * E, a.width); c += f.lanes * E) {
        add(c, acc);
        write(c, acc);
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

// Elements per access where rows are aligned: 16 bytes of the narrower type.
template <typename TI, typename TO>
constexpr int kWide = sizeof(TI) == 4 && sizeof(TO) == 4 ? 4 : 8;

// f(TI{}, TO{}, E) for the accesses of a.
template <typename F>
cudaError_t with_types(const EmbedArgs &a, F &&f)
{
    return with_dtype(a.rows_dtype, [&](auto ti) {
        return with_dtype(a.out_dtype, [&](auto to) {
            constexpr int W = kWide<decltype(ti), decltype(to)>;
            const int e = pack_of(a, W);
            if (e == W) return f(ti, to, Int<W>{});
            if (e == 2) return f(ti, to, Int<2>{});
            return f(ti, to, Int<1>{});
        });
    });
}

struct GradLayout {
    int passes = 0, items = 1, tiles = 0, bins = 0;
    int unit = 0;
    int64_t units = 0;
    size_t sorted[2] = {}, counts = 0, counts_later = 0, later_n = 0, part = 0, runs = 0, first = 0, bytes = 0;
};

GradLayout layout(const EmbedArgs &a)
{
    GradLayout l;
    if (a.n <= kFew) return l;
    const int bits = bits_of(a.vocab);  // keys 0 .. vocab
    l.passes = (bits + kMaxBits - 1) / kMaxBits;
    l.bins = 1 << ((bits + l.passes - 1) / l.passes);
    const int64_t tiles = a.n <= (int64_t)kSumTiles * kSortThreads * kSumItems ? kSumTiles : kManyTiles;
    while (l.items < kMaxItems && a.n > tiles * kSortThreads * l.items) l.items <<= 1;
    l.tiles = (int)((a.n + kSortThreads * l.items - 1) / (kSortThreads * l.items));
    // positions per unit: 32, fewer where that gives less than 16 warps per SM
    // (a narrow row takes only some of a warp's lanes)
    const int64_t per = std::max<int64_t>(1, (int64_t)a.width / 256 * 32 + (a.width % 256 + 7) / 8);  // lanes of a row
    l.unit = 32;
    while (l.unit > 8 && a.n / l.unit * per < 32 * 16 * kSMs) l.unit /= 2;
    l.units = (a.n + l.unit - 1) / l.unit;
    size_t at = 0;
    auto take = [&](size_t b) { const size_t p = at; at += up(b); return p; };
    for (size_t &p : l.sorted) p = take(8 * (size_t)a.n);
    const size_t counts_n = (size_t)l.bins * (l.tiles + 1);
    l.counts = take(4 * counts_n);
    l.later_n = counts_n * (l.passes - 1);
    l.counts_later = take(4 * l.later_n);
    l.part = take(8 * (size_t)l.units * a.width);
    l.runs = take(8 * (size_t)(l.units + 1));  // a long run ends in a unit of its own
    l.first = take(4 * (size_t)a.vocab);
    l.bytes = at;
    return l;
}

}  // namespace

cudaError_t embed(const EmbedArgs &a, cudaStream_t s, int64_t *launches)
{
    ++*launches;
    return with_dtype(a.rows_dtype, [&](auto ti) {
        return with_dtype(a.out_dtype, [&](auto to) {
            using TI = decltype(ti);
            using TO = decltype(to);
            constexpr int E = kWide<TI, TO>;
            if (pack_of(a, E) != E) {
                constexpr int E = 32 / sizeof(TO);
                const int sectors = (a.width + E - 1 + E - 1) / E;  // a row begins anywhere inside its first one
                const int64_t blocks = (a.n * sectors + kRawThreads - 1) / kRawThreads;
                if (blocks > 0x7fffffff) return cudaErrorInvalidValue;  // an output of 8 TB
                // exact for the numbers below sectors + kRawThreads that it divides
                const uint32_t magic = sectors > 1 ? 0xffffffffu / sectors + 1 : 0;
                k_embed_raw<TI, TO, E><<<(unsigned)blocks, kRawThreads, 0, s>>>(a, sectors, magic);
            } else {
                constexpr int NV = 4;  // packs per lane
                int lanes = 1;
                while (lanes < 32 && lanes * E * NV < a.width) lanes <<= 1;
                const int tiles = (a.width + lanes * E * NV - 1) / (lanes * E * NV);
                const int64_t want = (a.n * tiles * lanes + kThreads - 1) / kThreads;
                k_embed<TI, TO, E, NV><<<(unsigned)std::min<int64_t>(want, 16 * kSMs), kThreads, 0, s>>>(a, lanes, tiles);
            }
            return cudaGetLastError();
        });
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
            FewArgs f{};
            for (f.lanes = 1; f.lanes < kThreads && f.lanes * E < a.width;) f.lanes <<= 1;
            const int packs = f.lanes < kThreads ? 1 : kFewPacks;
            f.tiles = (a.width + f.lanes * E * packs - 1) / (f.lanes * E * packs);
            f.sums = (int)a.n * f.tiles;
            // at least 4 fill blocks per SM
            f.rows = (int)std::min<int64_t>(kFewRows, std::max<int64_t>(1, a.vocab / (4 * kSMs)));
            const int64_t fills = a.accumulate ? 0 : (a.vocab + f.rows - 1) / f.rows;
            if (f.sums + fills == 0) return cudaSuccess;
            k_grad_few<decltype(ti), decltype(to), E><<<(unsigned)(f.sums + fills), kThreads, 0, st>>>(a, f);
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
    // the empty rows: a quarter with each scatter, whose latencies leave the
    // memory idle, and the rest beside the sums
    Fill f{};
    f.present = s.present;
    auto fill_blocks = [&](int warps) {  // for the share f0 .. f1
        return (int)std::min<int64_t>(2 * kSMs, (share_of(a.vocab, f).rows + warps - 1) / warps);
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
    SumArgs m{};
    m.items = s.out;
    m.part = (float *)(p + l.part);
    m.runs = s.runs;
    m.first = (uint32_t *)(p + l.first);
    m.present = s.present;
    m.units = l.units;
    m.unit = l.unit;
    f.f0 = f.f1;
    f.f1 = kShares;
    f.blocks = s.present && f.f0 < f.f1 ? fill_blocks(kThreads / 32) : 0;
    HISS_TRY(with_types(a, [&](auto ti, auto to, auto e) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int E = decltype(e)::value;
        auto sum = [&](auto shape) {
            constexpr bool BIG = decltype(shape)::value;
            using S = SumShape<TI, E, BIG>;
            auto kernel = k_sum<TI, TO, E, BIG>;
            for (m.lanes = BIG ? 32 : 1; m.lanes < 32 && m.lanes * S::C < a.width;) m.lanes <<= 1;
            // shorter tiles where fewer lanes of the last one are idle: 115,404 x 132 bfloat16
            // 56 -> 49 us, 166,078 x 141 float32 97 -> 86 (91 with at least 16 lanes)
            auto tiles = [&](int lanes) { return (a.width + lanes * S::C - 1) / (lanes * S::C); };
            if (!BIG)
                for (int l = m.lanes / 2; l >= 8; l /= 2)
                    if (tiles(l) * l < tiles(m.lanes) * m.lanes) m.lanes = l;
            m.tiles = tiles(m.lanes);
            m.blocks = (int)((l.units * m.tiles + kThreads / m.lanes - 1) / (kThreads / m.lanes));
            static std::atomic<uint64_t> allowed{0};
            HISS_TRY(allow_shared(kernel, 128 * 1024, allowed));
            ++*launches;
            return launch_after(kernel, m.blocks + f.blocks, kThreads, S::smem(m.lanes), st, a, m, f);
        };
        // big tiles where they still give 16 warps per SM
        if (a.width > 256 && l.units * ((a.width + 511) / 512) >= 16 * kSMs) return sum(std::true_type{});
        return sum(std::false_type{});
    }));
    ++*launches;
    return with_dtype(a.out_dtype, [&](auto to) {
        return launch_after(k_join<decltype(to)>, kJoinBlocks, kJoinThreads, 0, st, a, m);
    });
}

}  // namespace hiss
