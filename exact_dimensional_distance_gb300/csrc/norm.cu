// Layer norm, forward and backward.
//
//   forward    m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), y = (x - m) r w + b
//   backward   h = (x - m) r, g = dy w:  dx = r (g - mean(g) - h mean(g h)),
//              dw = sum over rows of dy h,  db = sum over rows of dy
//
// Both are bound by memory: 2 (forward) and 3 (backward) elements moved per
// element, a dozen float32 operations.  A group of lanes owns a row, NV packs of
// E elements per lane, so that everything is read from memory once.  A group is
// a power of two of lanes inside a warp (narrow rows, several per warp), or
// whole warps that meet at a named barrier once per row.  Blocks are persistent:
// the weights (and in the backward pass each lane's column sums of dw and
// db) stay in registers from row to row.  The rows to come are copied
// into a shared-memory ring (cp.async), so the loads in flight cost no
// registers: each thread copies its own packs where rows are aligned to 16
// bytes, and no barrier guards the ring; a group copies the 16-byte lines that
// hold a row of any other alignment.  Rows too wide for a group of kMaxLanes are
// shared by two blocks, and those above 16,384 elements go through the looping kernels at
// the end of the file.
#include <algorithm>
#include <cfloat>

#include "hiss_internal.cuh"
#include "numeric.cuh"
#include "ptx.cuh"

namespace hiss {
namespace {

constexpr int kMaxLanes = 512;  // of a group, and threads of a block
constexpr int kMaxWarps = kMaxLanes / 32;
constexpr size_t kSharedBytes = 216 * 1024;  // dynamic shared memory of a block

// ---- groups ---------------------------------------------------------------------

struct Group {
    int lanes, id, lane;   // lanes per group; this thread's group in the block and lane in the group
    int warps, warp;       // warps per group and this thread's warp in the group (NARROW: 1 and 0)
    int span;              // half the power of two that covers the warps
};

template <bool NARROW>
__device__ __forceinline__ Group group_of(int lanes)
{
    Group g;
    g.lanes = lanes;
    g.id = threadIdx.x / lanes;
    g.lane = threadIdx.x - g.id * lanes;
    g.warps = NARROW ? 1 : lanes >> 5;
    g.warp = NARROW ? 0 : g.lane >> 5;
    g.span = 0;
    while (g.warps > (g.span ? 2 * g.span : 1)) g.span = g.span ? 2 * g.span : 1;
    return g;
}

// First column of a lane; its pack v is E * (NARROW ? lanes : 32) * v further on,
// so that a warp of a wide group owns consecutive columns.
template <bool NARROW, int E, int NV>
__device__ __forceinline__ int column_of(const Group &g)
{
    return NARROW ? g.lane * E : (g.warp * 32 * NV + (g.lane & 31)) * E;
}

__device__ __forceinline__ void group_barrier(const Group &g)
{
    asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.lanes) : "memory");
}

// Sum over the group's lanes of this warp.
template <bool NARROW>
__device__ __forceinline__ float warp_sum(const Group &g, float v)
{
    if (NARROW) {
        for (int o = g.lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// Sum over the first lanes of a warp that hold a value per warp of the group
// (the others hold 0), in every lane.
__device__ __forceinline__ float group_sum(const Group &g, float v)
{
    for (int o = g.span; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
}

// 1 / sqrt(v): the hardware's approximation and one Newton step.
__device__ __forceinline__ float inv_sqrt(float v)
{
    const float r = rsqrtf(v);
    const float n = fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
    return r > 0.0f && r < INFINITY ? n : r;  // v = 0, infinite, negative or NaN: as it is
}

// Whether n values with sum of squared differences q lie so close to their mean that
// the mean's own rounding (of a sum of about 20 steps, and of a product with
// a rounded 1 / n) is not far below their spread: a spread of up to 2^-10 of the mean.  Such a mean is
// corrected by the mean of the differences, which are nearly exact, and the
// differences are taken again, so that a constant row has its value for a mean and
// differences of zero.  Above that the mean is off by less than 2^-9 of the spread.
// Rows of zeros need no correction, and squares that overflow are left alone.  The test
// costs other rows little (131,072 x 768 bfloat16 79 -> 83 us, 65,536 x 4096 175 on both sides);
// 65,536 x 4096 constant ones take 294.
__device__ __forceinline__ bool small_spread(float q, float n, float mean)
{
    return q <= fminf(__fmul_rn(__fmul_rn(mean, mean), n * 0x1p-20f), FLT_MAX) && mean != 0.0f;
}

// One float2 per warp of a group, double-buffered by parity so that one
// barrier per row is enough: a warp that writes a buffer again has passed the
// barrier of the row between, which every reader of the buffer's old contents
// had reached.
struct Exchange {
    float2 slot[2][kMaxWarps];
};

// ---- rows shared by two blocks -----------------------------------------------------
// Rows too wide for a group of kMaxLanes are cut in two, a half for each block
// of a cluster: the block's view of the operands is its half's columns, and
// the warps' exchange of a row's sums reaches both blocks.  Backward, 3,825 x 12,032
// float32: 128 us, against 262 in the looping kernels; 4,000 x 16,384 bfloat16 with
// float32 dy 144 against 324; forward, 4,000 x 11,111 float32 126 against 128.  Bound
// by the latency of a row, 2 us from one to the next: the sums, the barrier of the cluster,
// and the sums over the warps.

constexpr int kPair = 2;

struct PairExchange {
    float2 slot[2][kPair * kMaxWarps];
};

// The columns of the first half of a row, the longer one: every pack stays whole and aligned.
__host__ __device__ __forceinline__ int first_half(int width) { return ((width + 1) / 2 + 15) & ~15; }

template <typename T>
__device__ __forceinline__ void advance(T *&p, int dtype, int64_t n)
{
    using C = std::conditional_t<std::is_const_v<T>, const char, char>;
    if (p) p = static_cast<C *>(p) + n * (dtype == HISS_F32 ? 4 : 2);
}

// a's view of the columns of this block's half; returns its first column.
__device__ __forceinline__ int take_half(NormArgs &a)
{
    const int half = first_half(a.width);
    if (blockIdx.x % kPair == 0) {
        a.width = half;
        return 0;
    }
    a.width -= half;
    advance(a.x, a.x_dtype, half);
    advance(a.y, a.y_dtype, half);
    advance(a.dy, a.y_dtype, half);
    advance(a.dx, a.x_dtype, half);
    advance(a.weight, a.p_dtype, half);
    advance(a.bias, a.p_dtype, half);
    advance(a.dweight, a.p_dtype, half);
    advance(a.dbias, a.p_dtype, half);
    return half;
}

// Barrier of the pair's threads; orders shared memory of both blocks.  Both
// take the same rows, so that they meet equally often.
__device__ __forceinline__ void pair_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// v into *p of block `rank` of the pair (p: the same variable in this block).
__device__ __forceinline__ void store_in_block(float2 *p, int rank, float2 v)
{
    asm volatile("{\n\t.reg .b32 q;\n\tmapa.shared::cluster.u32 q, %0, %1;\n\tst.shared::cluster.v2.f32 [q], {%2, %3};\n\t}" ::"r"(
                     smem_u32(p)),
                 "r"(rank), "f"(v.x), "f"(v.y)
                 : "memory");
}

// Give every warp of the pair this warp's value; lane 16 r + w of a warp returns that
// of warp w of block r (0 where there is none).
__device__ __forceinline__ float2 pair_exchange(PairExchange &ex, const Group &g, int parity, float2 v)
{
    static_assert(kPair * kMaxWarps == 32, "a lane for every warp");
    const int lane = threadIdx.x & 31;
    float2 *slot = ex.slot[parity];
    if (lane < kPair) store_in_block(slot + blockIdx.x % kPair * kMaxWarps + g.warp, lane, v);
    pair_barrier();
    return lane % kMaxWarps < g.warps ? slot[lane] : make_float2(0.0f, 0.0f);
}

// A lane's elements are handled as float32 pairs, in chunks: the pairs of a
// pack, or two packs of one element.
template <int E>
constexpr int kPairs = E == 1 ? 1 : E / 2;
template <int E, int NV>
constexpr int kChunks = E == 1 ? NV / 2 : NV;

// ---- the rows to come -------------------------------------------------------------

// Whether rows are copied by lines (they are not aligned to 16 bytes).
template <int E>
constexpr bool kRaw = E <= 2;

// Rows of one operand, S of them in shared memory.
//   packed: pack v of this thread at slot v of the thread;
//   raw:    the group's copy of the lines that hold the row, which begins at
//           the row's offset in its first line.
template <typename T, int E, int NV, int S, bool NARROW>
struct Ring {
    using P = Pack<T, E>;
    char *base;
    int stage;           // bytes from one row to the next
    uintptr_t lo, hi;    // the matrix: lines that reach outside are copied by element

    static __host__ __device__ int line_bytes(int width) { return (width * (int)sizeof(T) + 15 + 15) / 16 * 16; }
    static size_t bytes(int threads, int lanes, int width)
    {
        return kRaw<E> ? (size_t)(threads / lanes) * S * line_bytes(width) : (size_t)threads * S * NV * sizeof(P);
    }
    // at: the block's part of shared memory for this operand
    __device__ __forceinline__ void open(char *at, const Group &g, const void *p, int64_t n, int64_t stride, int width)
    {
        if constexpr (kRaw<E>) {
            stage = line_bytes(width);
            base = at + g.id * (S * stage);
            lo = reinterpret_cast<uintptr_t>(p);
            hi = lo + ((n - 1) * stride + width) * sizeof(T);
        } else {
            stage = blockDim.x * NV * (int)sizeof(P);
            base = at + threadIdx.x * sizeof(P);
        }
    }
    // Start copying a row into stage st.
    __device__ __forceinline__ void fetch(int st, const T *row, const Group &g, int col, int vs, int width)
    {
        char *d = base + st * stage;
        if constexpr (kRaw<E>) {
            const uintptr_t b0 = reinterpret_cast<uintptr_t>(row), b1 = b0 + width * sizeof(T), line0 = b0 & ~(uintptr_t)15;
            const int bytes = (int)(b1 - line0);
            const char *q = reinterpret_cast<const char *>(line0);
            if (line0 >= lo && line0 + (bytes + 15) / 16 * 16 <= hi) {
#pragma unroll 2
                for (int b = 16 * g.lane; b < bytes; b += 16 * g.lanes) cp_async16(d + b, q + b);
            } else {  // the first and last rows
                for (int b = 16 * g.lane; b < bytes; b += 16 * g.lanes) {
                    if (line0 + b >= lo && line0 + b + 16 <= hi) {
                        cp_async16(d + b, q + b);
                    } else {
                        for (uintptr_t e = max(line0 + b, b0); e < min(line0 + b + 16, b1); e += sizeof(T))
                            *reinterpret_cast<T *>(d + (e - line0)) = *reinterpret_cast<const T *>(e);
                    }
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (col + v * vs < width)
                    copy_pack_async<T, E>(reinterpret_cast<P *>(d + v * blockDim.x * sizeof(P)), row + col + v * vs);
        }
    }
    // Chunk c of the row in stage st: a pack as float32 pairs, or two packs of
    // one element as a pair, the second 0 unless the row reaches it.
    __device__ __forceinline__ void get(int st, const T *row, int col, int vs, int c, bool second, float2 (&x)[kPairs<E>]) const
    {
        const char *d = base + st * stage;
        if constexpr (E == 1) {
            const T *v = reinterpret_cast<const T *>(d + (reinterpret_cast<uintptr_t>(row) & 15)) + col;
            x[0] = make_float2(to_f32(v[2 * c * vs]), second ? to_f32(v[(2 * c + 1) * vs]) : 0.0f);
        } else {
            P p;
            if constexpr (kRaw<E>) p = load_pack<T, E>(reinterpret_cast<const T *>(d + (reinterpret_cast<uintptr_t>(row) & 15)) + col + c * vs);
            else p = *reinterpret_cast<const P *>(d + c * blockDim.x * sizeof(P));
#pragma unroll
            for (int h = 0; h < E / 2; ++h) x[h] = pair_of(p.v + 2 * h);
        }
    }
};

// Before a raw row is read, and before the place of the row before it is
// filled again.
template <bool NARROW>
__device__ __forceinline__ void group_sync(const Group &g)
{
    if (NARROW || g.warps == 1) __syncwarp();
    else group_barrier(g);
}

// Rows in the ring: at most 4, so many that a block of kMaxLanes threads fits
// with other bytes per lane beside the ring.
constexpr int stages(size_t row_bytes, size_t other)
{
    const int s = (int)(((kSharedBytes - 1024) / kMaxLanes - other) / row_bytes);  // lines: up to 30 bytes more per row
    return s > 4 ? 4 : s;
}

// ---- geometry -----------------------------------------------------------------

struct Rows {
    int e = 0, nv = 0;     // elements per pack, packs per lane; e = 0: looping kernels
    int lanes = 0, groups = 0;
    bool narrow = false;
    bool pair = false;     // a row per two blocks, lanes of each
    bool one_block = false;
};

// The widest pack that the width and every row's alignment allow; 16 elements
// per lane, or 32 where that is too few and the caller has such a kernel for
// the pack, or else two blocks per row; as many groups per block as reach the given threads without leaving
// SMs idle.
Rows plan_rows(const NormArgs &a, bool has32, bool has32_wide, int threads, bool one_block)
{
    const bool half = a.x_dtype != HISS_F32;
    auto fits = [&](int e) {
        if (a.width % e) return false;
        bool ok = rows_aligned(a.x, a.x_stride, a.x_dtype, e) && rows_aligned(a.weight, 0, a.p_dtype, e) &&
                  rows_aligned(a.bias, 0, a.p_dtype, e);
        if (a.y) ok = ok && rows_aligned(a.y, a.y_stride, a.y_dtype, e);
        if (a.dy) ok = ok && rows_aligned(a.dy, a.y_stride, a.y_dtype, e);
        if (a.dx) ok = ok && rows_aligned(a.dx, a.dx_stride, a.x_dtype, e);
        return ok;
    };
    const int wide = half ? 8 : 4;
    Rows r;
    const int e = fits(wide) ? wide : half && fits(2) ? 2 : 1;
    int per = 16;
    const bool can = e == wide ? has32_wide : has32;
    if (can && (a.width > per * kMaxLanes || (half && a.width > 512))) per = 32;
    int lanes = (a.width + per - 1) / per;
    if (lanes > kMaxLanes && !can) {
        r.pair = true;
        lanes = (first_half(a.width) + per - 1) / per;
    }
    if (lanes > kMaxLanes) return Rows{};
    r.e = e;
    r.nv = per / e;
    r.narrow = lanes <= 16;
    if (r.narrow) {
        r.lanes = 1;
        while (r.lanes < lanes) r.lanes <<= 1;
        r.groups = 32 / r.lanes;
    } else {
        r.lanes = (lanes + 31) & ~31;
        r.groups = 1;
    }
    // a raw row takes up to 30 bytes more than its elements, which counts for very narrow ones
    const size_t row = 4 * (a.width * (dtype_bytes(a.x_dtype) + (a.dy ? dtype_bytes(a.y_dtype) : 0)) + 60);
    const auto fits_block = [&](int groups) {
        return groups * r.lanes <= threads && (!r.narrow || groups * row <= kSharedBytes);
    };
    // the backward pass of at most two rows per group of one block: a second
    // launch to add up the blocks' sums takes longer than the second row
    if (one_block) {
        int groups = r.groups;
        while (groups < a.n && fits_block(2 * groups)) groups <<= 1;
        if (a.n <= 2 * groups) {
            r.groups = groups;
            r.one_block = true;
            return r;
        }
    }
    while ((int64_t)r.groups * kSMs < a.n && fits_block(2 * r.groups)) r.groups <<= 1;
    return r;
}

// Resident blocks per SM of a kernel: those that its registers allow at a block
// size, asked for once, and those that its shared memory leaves.
struct Residency {
    std::atomic<uint64_t> allowed{0};  // devices on which it may use kSharedBytes
    std::atomic<int> blocks[kMaxWarps + 1] = {};
};
template <typename K>
cudaError_t resident(K kernel, int threads, size_t smem, Residency &cache, int *blocks)
{
    HISS_TRY(allow_shared(kernel, kSharedBytes, cache.allowed));
    std::atomic<int> &c = cache.blocks[threads / 32];
    int v = c.load(std::memory_order_relaxed);
    if (v == 0) {
        HISS_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kernel, threads, 0));
        c.store(v, std::memory_order_relaxed);
    }
    const int fit = (int)(227 * 1024 / (smem + sizeof(Exchange) * kMaxWarps + 1024));  // 1 KB per block is the system's
    *blocks = std::max(1, std::min(v, fit));
    return cudaSuccess;
}

// ---- parameters -----------------------------------------------------------------

// The weights (or biases) of a lane's columns, as float32 pairs, for every row
// the block takes: in registers, or with 32 16-bit elements per lane in shared
// memory (one copy per block, accesses without bank conflicts): 64 registers of
// them would halve the warps per SM.
template <bool NARROW, int E, int NV>
struct Params {
    static constexpr bool kShared = E * NV == 32 && E != 4;
    static constexpr size_t kLaneBytes = kShared ? 4 * E * NV : 0;  // of shared memory
    float2 held[kShared ? 1 : kChunks<E, NV>][kPairs<E>];
    char *sh;
    int lanes;

    // Called by every thread; the block synchronises before the first get.
    __device__ __forceinline__ void open(const Group &g, const void *p, int dtype, float none, int col, int vs, int width,
                                         char *base)
    {
        sh = base + g.lane * (E == 8 ? 16 : 8);
        lanes = g.lanes;
        float first = none;  // E = 1: of a chunk's two elements
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float t[E];
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = none;
            if (p && col + v * vs < width) load_params<E>(p, dtype, col + v * vs, t);
            if constexpr (kShared && E == 8) {
                if (g.id == 0)
#pragma unroll
                    for (int e = 0; e < E; e += 4)
                        *reinterpret_cast<float4 *>(sh + 16 * (v * 2 + e / 4) * lanes) = make_float4(t[e], t[e + 1], t[e + 2], t[e + 3]);
            } else if constexpr (kShared) {
                if (E == 2 && g.id == 0) *reinterpret_cast<float2 *>(sh + 8 * v * lanes) = make_float2(t[0], t[E - 1]);
                if (E == 1 && (v & 1) && g.id == 0) *reinterpret_cast<float2 *>(sh + 8 * (v / 2) * lanes) = make_float2(first, t[0]);
                first = t[0];
            } else if constexpr (E == 1) {
                if (v & 1) held[v / 2][0].y = t[0];
                else held[v / 2][0].x = t[0];
            } else {
#pragma unroll
                for (int h = 0; h < E / 2; ++h) held[v][h] = make_float2(t[2 * h], t[2 * h + 1]);
            }
        }
    }
    __device__ __forceinline__ void get(int c, float2 (&t)[kPairs<E>]) const
    {
        if constexpr (kShared && E == 8) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 f = *reinterpret_cast<const float4 *>(sh + 16 * (c * 2 + q) * lanes);
                t[2 * q] = make_float2(f.x, f.y);
                t[2 * q + 1] = make_float2(f.z, f.w);
            }
        } else if constexpr (kShared) {
            t[0] = *reinterpret_cast<const float2 *>(sh + 8 * c * lanes);
        } else {
#pragma unroll
            for (int h = 0; h < kPairs<E>; ++h) t[h] = held[c][h];
        }
    }
};

// Store chunk c of a row at p (the lane's first column).
template <typename T, int E>
__device__ __forceinline__ void store_chunk(T *p, int c, int vs, bool second, const float2 (&r)[kPairs<E>])
{
    if constexpr (E == 1) {
        p[2 * c * vs] = from_f32<T>(r[0].x);
        if (second) p[(2 * c + 1) * vs] = from_f32<T>(r[0].y);
    } else {
        Pack<T, E> o;
#pragma unroll
        for (int h = 0; h < E / 2; ++h) set_pair(o.v + 2 * h, r[h]);
        store_pack<T, E>(p + c * vs, o);
    }
}

// ---- forward --------------------------------------------------------------------

template <typename TX, int E, int NV, bool NARROW>
struct Forward {
    static constexpr size_t kParamBytes = 2 * Params<NARROW, E, NV>::kLaneBytes;
    static constexpr int kStages = stages(sizeof(TX) * E * NV, kParamBytes);
    static_assert(kStages >= 2, "a row ahead");
    using X = Ring<TX, E, NV, kStages, NARROW>;
    static size_t smem(int threads, int lanes, int width) { return X::bytes(threads, lanes, width) + kParamBytes * lanes; }
};

// 65,536 x 4096 bfloat16: 176 us, 6.1 TB/s (0.91 of the copy rate), 13.7
// instructions per 32 elements; bound by memory, with the weights' shared-memory
// reads next.  Before float32 pairs, 32 elements per lane and products for divisions
// it took 294 us and 25 instructions.  20,011 x 1021 float16 to float32: 31 us
// (3.9 TB/s), bound by instructions, since the elements of odd 16-bit rows are read one by one.
//
// PAIR: two blocks per row.
template <typename TX, typename TY, int E, int NV, bool NARROW, bool PAIR>
__global__ void __launch_bounds__(kMaxLanes) k_norm(NormArgs a, int lanes, int groups)
{
    using F = Forward<TX, E, NV, NARROW>;
    using PA = Params<NARROW, E, NV>;
    constexpr int S = F::kStages, C = NV * E, H = kPairs<E>, NC = kChunks<E, NV>;
    extern __shared__ __align__(16) char ring[];
    __shared__ std::conditional_t<PAIR, PairExchange, Exchange> ex[PAIR ? 1 : kMaxWarps];
    const int row_width = a.width;
    if constexpr (PAIR) {
        take_half(a);
        pair_barrier();  // both blocks are there
    }
    const Group g = group_of<NARROW>(lanes);
    const int col = column_of<NARROW, E, NV>(g);
    const int vs = E * (NARROW ? lanes : 32);
    // the row reaches chunk c of this lane, (packs of one element) its second
    // half, and chunk c of any lane of the warp; full: every chunk of every lane
    auto has = [&](int c) { return col + (E == 1 ? 2 * c : c) * vs < a.width; };
    auto has_second = [&](int c) { return E > 1 || col + (2 * c + 1) * vs < a.width; };
    const int warp_col = NARROW ? 0 : g.warp * 32 * NV * E;
    auto any = [&](int c) { return warp_col + (E == 1 ? 2 * c : c) * vs < a.width; };
    const bool full = warp_col + NV * vs <= a.width;
    const int64_t step = (int64_t)(gridDim.x / (PAIR ? kPair : 1)) * groups;
    int64_t row = (int64_t)(blockIdx.x / (PAIR ? kPair : 1)) * groups + g.id;
    // the loop runs for whole warps: as long as the warp's first row exists
    int64_t first = row - (NARROW ? (threadIdx.x & 31) / lanes : 0);
    typename F::X xs;
    char *params = ring;  // first: their accesses need the alignment
    xs.open(ring + F::kParamBytes * lanes, g, a.x, a.n, a.x_stride, a.width);
    const TX *x0 = static_cast<const TX *>(a.x);
    auto fetch = [&](int st, int64_t r) {
        if (r < a.n) xs.fetch(st, x0 + r * a.x_stride, g, col, vs, a.width);
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i, row + i * step);
    PA w, b;
    w.open(g, a.weight, a.p_dtype, 1.0f, col, vs, a.width, params);
    b.open(g, a.bias, a.p_dtype, 0.0f, col, vs, a.width, params + PA::kLaneBytes * lanes);
    if constexpr (PA::kShared) __syncthreads();
    const float inv_width = 1.0f / (float)row_width;
    // columns of this thread's warp, and of warp (lane id) of the group
    auto columns = [&](int width, int i) { return (float)min(max(width - i * 32 * C, 0), 32 * C); };
    const float my_n = NARROW ? (float)a.width : columns(a.width, g.warp), inv_my_n = my_n > 0.0f ? 1.0f / my_n : 0.0f;
    float lane_n = 0.0f;
    if constexpr (PAIR) {
        const int half = first_half(row_width), l = threadIdx.x & 31;
        lane_n = columns(l < kMaxWarps ? half : row_width - half, l % kMaxWarps);
    } else if (!NARROW) {
        lane_n = columns(a.width, threadIdx.x & 31);
    }
    int st = 0;
    int parity = 0;
    // one row; FULL: no column to be left out
    auto body = [&](auto is_full) {
        constexpr bool FULL = decltype(is_full)::value;
        const int before = st == 0 ? S - 1 : st - 1;
        const TX *x_row = x0 + row * a.x_stride;
        if constexpr (kRaw<E>) {
            cp_async_wait<S - 2>();
            group_sync<NARROW>(g);
            fetch(before, row + (S - 1) * step);
        } else {
            fetch(before, row + (S - 1) * step);
            cp_async_wait<S - 1>();
        }
        float2 x[NC][H];
        float2 s2 = both(0.0f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (!FULL && !any(c)) break;
            if (FULL || has(c)) {
                xs.get(st, x_row, col, vs, c, FULL || has_second(c), x[c]);
#pragma unroll
                for (int h = 0; h < H; ++h) s2 = __fadd2_rn(s2, x[c][h]);
            }
        }
        // mean and sum of squared differences of the warp's columns, then of the
        // row from those of its warps: M2 = sum of (M2_w + n_w (m_w - m)^2)
        float mean = warp_sum<NARROW>(g, s2.x + s2.y) * inv_my_n;
        float2 q2 = both(0.0f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (!FULL && !any(c)) break;
            if (FULL || has(c))
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float2 d = __fadd2_rn(x[c][h], both(-mean));
                    if (!FULL && !has_second(c)) d.y = 0.0f;
                    q2 = __ffma2_rn(d, d, q2);
                }
        }
        float q = warp_sum<NARROW>(g, q2.x + q2.y);
        // sum over the warp's columns of the differences from m, or of their squares, for
        // rows of small spread.  The row is read from the ring again: another use of x
        // costs the usual path 43 registers with four packs of 8
        auto about = [&](float m, bool squares) {
            float2 s = both(0.0f);
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
                if (!any(c)) break;
                if (!has(c)) continue;
                float2 v[H];
                xs.get(st, x_row, col, vs, c, has_second(c), v);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float2 d = __fadd2_rn(v[h], both(-m));
                    if (!has_second(c)) d.y = 0.0f;
                    s = squares ? __ffma2_rn(d, d, s) : __fadd2_rn(s, d);
                }
            }
            return warp_sum<NARROW>(g, s.x + s.y);
        };
        if (PAIR || (!NARROW && g.warps > 1)) {
            const int l = threadIdx.x & 31;
            auto exchange = [&](float2 v) {
                if constexpr (PAIR) {
                    return pair_exchange(ex[0], g, parity, v);
                } else {
                    float2 *slot = ex[g.id].slot[parity];
                    if (l == 0) slot[g.warp] = v;
                    group_barrier(g);
                    return l < g.warps ? slot[l] : make_float2(0.0f, 0.0f);
                }
            };
            auto sum = [&](float v) {
                if constexpr (PAIR) return warp_sum<false>(g, v);
                else return group_sum(g, v);
            };
            const float2 mine = exchange(make_float2(mean, q));
            // the decision below holds barriers, so it has to be the same in every warp of the
            // row: both bodies round every step alike (the _rn functions are never fused)
            mean = __fmul_rn(sum(__fmul_rn(lane_n, mine.x)), inv_width);
            const float d = __fsub_rn(mine.x, mean);
            q = sum(lane_n > 0.0f ? __fmaf_rn(__fmul_rn(lane_n, d), d, mine.y) : 0.0f);
            if (small_spread(q, (float)row_width, mean)) {
                auto total = [&](float v) {
                    if constexpr (PAIR) pair_barrier();  // the slots have been read
                    else group_barrier(g);
                    return sum(exchange(make_float2(v, 0.0f)).x);
                };
                mean = __fmaf_rn(total(about(mean, false)), inv_width, mean);
                q = total(about(mean, true));
            }
        } else {
            const bool correct = small_spread(q, (float)row_width, mean);
            if (NARROW ? __any_sync(0xffffffffu, correct) : correct) {  // a narrow warp's rows: each keeps to its own
                const float d = about(mean, false);
                if (correct) mean = __fmaf_rn(d, inv_my_n, mean);
                const float again = about(mean, true);
                if (correct) q = again;
            }
        }
        const float rstd = inv_sqrt(q * inv_width + a.eps);
        if (row < a.n) {
            TY *y = static_cast<TY *>(a.y) + row * a.y_stride + col;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (!FULL && !any(c)) break;
                if (!FULL && !has(c)) continue;
                float2 tw[H], tb[H], r[H];
                w.get(c, tw);
                b.get(c, tb);
#pragma unroll
                for (int h = 0; h < H; ++h)
                    r[h] = __ffma2_rn(__fmul2_rn(__fadd2_rn(x[c][h], both(-mean)), both(rstd)), tw[h], tb[h]);
                store_chunk<TY, E>(y, c, vs, FULL || has_second(c), r);
            }
            if (g.lane == 0 && (!PAIR || blockIdx.x % kPair == 0)) {
                if (a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
        }
        st = st == S - 1 ? 0 : st + 1;
        parity ^= 1;
    };
    // a body of its own for full warps where the checks cost most: one per
    // element, or 32 elements (65,536 x 4096 bfloat16 204 -> 176 us, 47,397 x 2569
    // float16 249 -> 177); with four packs of four float32 it costs 7%
    constexpr bool kTwo = kRaw<E> || C == 32;
    if (kTwo && full)
        for (; first < a.n; first += step, row += step) body(std::integral_constant<bool, kTwo>{});
    else
        for (; first < a.n; first += step, row += step) body(std::false_type{});
}

// ---- backward -------------------------------------------------------------------

template <typename TX, typename TY, int E, int NV, bool NARROW>
struct Backward {
    static constexpr size_t kParamBytes = Params<NARROW, E, NV>::kLaneBytes;
    static constexpr int kStages = stages((sizeof(TX) + sizeof(TY)) * E * NV, kParamBytes);
    static_assert(kStages >= 2, "a row ahead");
    using X = Ring<TX, E, NV, kStages, NARROW>;
    using Y = Ring<TY, E, NV, kStages, NARROW>;
    // the rings and the weights; their memory holds the column sums of half of
    // the block's threads at the end
    static size_t smem(int threads, int lanes, int width, bool many)
    {
        return std::max(X::bytes(threads, lanes, width) + Y::bytes(threads, lanes, width) + kParamBytes * lanes,
                        many ? 4 * (size_t)threads * E * NV : 0);
    }
};

// 32,768 x 2048 bfloat16: 66 us (5.6 TB/s), with k_norm_param 70; bound by memory
// and issue alike.  20,000 x 128 float32: 11 us, the latency of two rows per group and
// of the sums' tree.
//
// Each block leaves its column sums in part[block][0 .. width) (dw) and
// [width .. 2 width) (db): k_norm_param adds the blocks up.  direct: the only block
// writes dweight and dbias itself.  x_bytes: of x's ring.  PAIR: two blocks per row.
template <typename TX, typename TY, int E, int NV, bool NARROW, bool PAIR>
__global__ void __launch_bounds__(kMaxLanes) k_norm_grad(NormArgs a, int lanes, int groups, int x_bytes, float *part, bool direct)
{
    using B = Backward<TX, TY, E, NV, NARROW>;
    using PA = Params<NARROW, E, NV>;
    constexpr int S = B::kStages, H = kPairs<E>, NC = kChunks<E, NV>;
    extern __shared__ __align__(16) char ring[];
    __shared__ std::conditional_t<PAIR, PairExchange, Exchange> ex[PAIR ? 1 : kMaxWarps];
    const int row_width = a.width;
    const int block = blockIdx.x / (PAIR ? kPair : 1), blocks = gridDim.x / (PAIR ? kPair : 1);
    if constexpr (PAIR) {
        const int first_col = take_half(a);
        if (part) part += first_col;
        pair_barrier();  // both blocks are there
    }
    const Group g = group_of<NARROW>(lanes);
    const int col = column_of<NARROW, E, NV>(g);
    const int vs = E * (NARROW ? lanes : 32);
    // the row reaches chunk c of this lane, (packs of one element) its second
    // half, and chunk c of any lane of the warp; full: every chunk of every lane
    auto has = [&](int c) { return col + (E == 1 ? 2 * c : c) * vs < a.width; };
    auto has_second = [&](int c) { return E > 1 || col + (2 * c + 1) * vs < a.width; };
    const int warp_col = NARROW ? 0 : g.warp * 32 * NV * E;
    auto any = [&](int c) { return warp_col + (E == 1 ? 2 * c : c) * vs < a.width; };
    const bool full = warp_col + NV * vs <= a.width;
    const int64_t step = (int64_t)blocks * groups;
    int64_t row = (int64_t)block * groups + g.id;
    int64_t first = row - (NARROW ? (threadIdx.x & 31) / lanes : 0);
    typename B::X xs;
    typename B::Y ys;
    xs.open(ring + B::kParamBytes * lanes, g, a.x, a.n, a.x_stride, a.width);
    ys.open(ring + B::kParamBytes * lanes + x_bytes, g, a.dy, a.n, a.y_stride, a.width);
    const TX *x0 = static_cast<const TX *>(a.x);
    const TY *y0 = static_cast<const TY *>(a.dy);
    auto fetch = [&](int st, int64_t r) {
        if (r < a.n) {
            xs.fetch(st, x0 + r * a.x_stride, g, col, vs, a.width);
            ys.fetch(st, y0 + r * a.y_stride, g, col, vs, a.width);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i, row + i * step);
    PA w;
    w.open(g, a.weight, a.p_dtype, 1.0f, col, vs, a.width, ring);
    if constexpr (PA::kShared) __syncthreads();
    float2 dw[NC][H], db[NC][H];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int h = 0; h < H; ++h) dw[c][h] = db[c][h] = both(0.0f);
    const float inv_width = 1.0f / (float)row_width;
    float mean_n = row < a.n ? a.mean[row] : 0.0f, rstd_n = row < a.n ? a.rstd[row] : 0.0f;
    int st = 0;
    int parity = 0;
    auto body = [&](auto is_full) {
        constexpr bool FULL = decltype(is_full)::value;
        const int before = st == 0 ? S - 1 : st - 1;
        const TX *x_row = x0 + row * a.x_stride;
        const TY *y_row = y0 + row * a.y_stride;
        if constexpr (kRaw<E>) {
            cp_async_wait<S - 2>();
            group_sync<NARROW>(g);
            fetch(before, row + (S - 1) * step);
        } else {
            fetch(before, row + (S - 1) * step);
            cp_async_wait<S - 1>();
        }
        const float mean = mean_n, rstd = rstd_n;
        if (row + step < a.n) {
            mean_n = a.mean[row + step];
            rstd_n = a.rstd[row + step];
        }
        float2 sg2 = both(0.0f), sgh2 = both(0.0f);
        if (row < a.n) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (!FULL && !any(c)) break;
                if (!FULL && !has(c)) continue;
                float2 x[H], d[H], t[H];
                xs.get(st, x_row, col, vs, c, FULL || has_second(c), x);
                ys.get(st, y_row, col, vs, c, FULL || has_second(c), d);
                w.get(c, t);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    float2 n = __fmul2_rn(__fadd2_rn(x[h], both(-mean)), both(rstd));
                    if (!FULL && !has_second(c)) n.y = 0.0f;  // dy is 0 there
                    const float2 gr = __fmul2_rn(d[h], t[h]);
                    db[c][h] = __fadd2_rn(db[c][h], d[h]);
                    dw[c][h] = __ffma2_rn(d[h], n, dw[c][h]);
                    sg2 = __fadd2_rn(sg2, gr);
                    sgh2 = __ffma2_rn(gr, n, sgh2);
                }
            }
        }
        if (a.dx) {
            float sg = warp_sum<NARROW>(g, sg2.x + sg2.y), sgh = warp_sum<NARROW>(g, sgh2.x + sgh2.y);
            if constexpr (PAIR) {
                const float2 mine = pair_exchange(ex[0], g, parity, make_float2(sg, sgh));
                sg = warp_sum<false>(g, mine.x);
                sgh = warp_sum<false>(g, mine.y);
            } else if (!NARROW && g.warps > 1) {
                float2 *slot = ex[g.id].slot[parity];
                if ((threadIdx.x & 31) == 0) slot[g.warp] = make_float2(sg, sgh);
                group_barrier(g);
                const float2 mine = (threadIdx.x & 31) < g.warps ? slot[threadIdx.x & 31] : make_float2(0.0f, 0.0f);
                sg = group_sum(g, mine.x);
                sgh = group_sum(g, mine.y);
            }
            // dx = g r - (h (r mean(g h)) + r mean(g))
            const float2 mg = both(-rstd * (sg * inv_width)), mgh = both(-rstd * (sgh * inv_width));
            if (row < a.n) {
                TX *dx = static_cast<TX *>(a.dx) + row * a.dx_stride + col;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (!FULL && !any(c)) break;
                    if (!FULL && !has(c)) continue;
                    // read and computed again: holding h and g from above would
                    // take 2 registers per element
                    float2 x[H], d[H], t[H], r[H];
                    xs.get(st, x_row, col, vs, c, FULL || has_second(c), x);
                    ys.get(st, y_row, col, vs, c, FULL || has_second(c), d);
                    w.get(c, t);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const float2 n = __fmul2_rn(__fadd2_rn(x[h], both(-mean)), both(rstd));
                        r[h] = __ffma2_rn(__fmul2_rn(d[h], t[h]), both(rstd), __ffma2_rn(n, mgh, mg));
                    }
                    store_chunk<TX, E>(dx, c, vs, FULL || has_second(c), r);
                }
            }
        }
        st = st == S - 1 ? 0 : st + 1;
        parity ^= 1;
    };
    // with packs the checks cost less than the registers of a second body
    if (kRaw<E> && full)
        for (; first < a.n; first += step, row += step) body(std::integral_constant<bool, kRaw<E>>{});
    else
        for (; first < a.n; first += step, row += step) body(std::false_type{});
    if (!part && !direct) return;
    // the block's column sums: over the groups of a warp, then over the warps (or
    // groups of warps) in a fixed tree, through the ring's memory
    cp_async_wait<0>();
    float2 *sh = reinterpret_cast<float2 *>(ring);  // (dw, db) of an element
    auto sums = [&](auto f) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                f(2 * (c * H + h), dw[c][h].x, db[c][h].x);
                f(2 * (c * H + h) + 1, dw[c][h].y, db[c][h].y);
            }
    };
    if (NARROW)
        for (int o = lanes; o < 32; o <<= 1)
            sums([&](int, float &p, float &q) {
                p += __shfl_xor_sync(0xffffffffu, p, o);
                q += __shfl_xor_sync(0xffffffffu, q, o);
            });
    const int unit_lanes = NARROW ? 32 : lanes;
    const int unit = threadIdx.x / unit_lanes, lane = threadIdx.x - unit * unit_lanes;
    for (int half = blockDim.x / unit_lanes / 2; half > 0; half >>= 1) {
        __syncthreads();
        const int stride = half * unit_lanes;
        if (unit >= half && unit < 2 * half)
            sums([&](int k, float &p, float &q) { sh[k * stride + (unit - half) * unit_lanes + lane] = make_float2(p, q); });
        __syncthreads();
        if (unit < half)
            sums([&](int k, float &p, float &q) {
                const float2 o = sh[k * stride + unit * unit_lanes + lane];
                p += o.x;
                q += o.y;
            });
    }
    if (unit == 0 && lane < lanes && direct) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int c0 = col + (E == 1 ? 2 * c : c) * vs + 2 * h, c1 = E == 1 ? c0 + vs : c0 + 1;
                if (c0 < a.width && a.dweight) store_any(a.dweight, a.p_dtype, c0, dw[c][h].x);
                if (c0 < a.width && a.dbias) store_any(a.dbias, a.p_dtype, c0, db[c][h].x);
                if (c1 < a.width && a.dweight) store_any(a.dweight, a.p_dtype, c1, dw[c][h].y);
                if (c1 < a.width && a.dbias) store_any(a.dbias, a.p_dtype, c1, db[c][h].y);
            }
    } else if (unit == 0 && lane < lanes) {
        float *p = part + (int64_t)block * 2 * row_width + col;
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (has(c)) {
                store_chunk<float, E>(p, c, vs, has_second(c), dw[c]);
                store_chunk<float, E>(p + row_width, c, vs, has_second(c), db[c]);
            }
    }
    let_next_start();
}

// dweight and dbias from the parts: 32 of the 2 width columns per block, 32
// parts at a time.  4 us at 152 parts, of which 2 hide behind the kernel before.
__global__ void __launch_bounds__(1024) k_norm_param(NormArgs a, const float *part, int parts)
{
    __shared__ float sh[32][33];
    wait_for_previous();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < 2 * a.width)
        for (int i = w; i < parts; i += 32) s += part[(int64_t)i * 2 * a.width + c];
    sh[w][lane] = s;
    __syncthreads();
    s = sh[lane][w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int k = blockIdx.x * 32 + w;  // this warp's column
    if (lane == 0 && k < 2 * a.width) {
        if (k < a.width) {
            if (a.dweight) store_any(a.dweight, a.p_dtype, k, s);
        } else if (a.dbias) {
            store_any(a.dbias, a.p_dtype, k - a.width, s);
        }
    }
}

// ---- rows of any width and alignment, read again for each pass ---------------------
// For rows above 16,384 elements.  A block per row, the second and third reading
// from L2; 5,437 x 9594 bfloat16 took 98 us here and takes 72 in k_norm.  Bound by the latency of
// loads of single elements: 2,000 x 32,768 bfloat16 forward 212 us, backward 369, 1,000 x
// 65,536 float32 351 and 496, a fifth of what the copy rate would give.

constexpr int kLoopThreads = 512;
constexpr int kLoopSplits = 64;  // row ranges of the column sums

__device__ __forceinline__ float loop_sum(float v)
{
    __shared__ float part[kLoopThreads / 32];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kLoopThreads / 32; ++w) s += part[w];
    return s;
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(kLoopThreads) k_norm_loop(NormArgs a)
{
    const int64_t r = blockIdx.x;
    const TX *x = static_cast<const TX *>(a.x) + r * a.x_stride;
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kLoopThreads) s += to_f32(x[c]);
    float mean = loop_sum(s) / a.width;
    auto squares = [&] {
        float v = 0.0f;
        for (int c = threadIdx.x; c < a.width; c += kLoopThreads) {
            const float e = to_f32(x[c]) - mean;
            v += e * e;
        }
        return loop_sum(v);
    };
    float q = squares();
    if (small_spread(q, (float)a.width, mean)) {  // the same for every thread
        s = 0.0f;
        for (int c = threadIdx.x; c < a.width; c += kLoopThreads) s += to_f32(x[c]) - mean;
        mean += loop_sum(s) / a.width;
        q = squares();
    }
    const float rstd = 1.0f / sqrtf(q / a.width + a.eps);
    TY *y = static_cast<TY *>(a.y) + r * a.y_stride;
    for (int c = threadIdx.x; c < a.width; c += kLoopThreads) {
        float v = (to_f32(x[c]) - mean) * rstd;
        if (a.weight) v *= load_any(a.weight, a.p_dtype, c);
        if (a.bias) v += load_any(a.bias, a.p_dtype, c);
        y[c] = from_f32<TY>(v);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(kLoopThreads) k_norm_dx_loop(NormArgs a)
{
    const int64_t r = blockIdx.x;
    const TX *x = static_cast<const TX *>(a.x) + r * a.x_stride;
    const TY *dy = static_cast<const TY *>(a.dy) + r * a.y_stride;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float sg = 0.0f, sgh = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kLoopThreads) {
        const float g = to_f32(dy[c]) * (a.weight ? load_any(a.weight, a.p_dtype, c) : 1.0f);
        sg += g;
        sgh += g * ((to_f32(x[c]) - mean) * rstd);
    }
    const float mg = loop_sum(sg) / a.width, mgh = loop_sum(sgh) / a.width;
    TX *dx = static_cast<TX *>(a.dx) + r * a.dx_stride;
    for (int c = threadIdx.x; c < a.width; c += kLoopThreads) {
        const float g = to_f32(dy[c]) * (a.weight ? load_any(a.weight, a.p_dtype, c) : 1.0f);
        dx[c] = from_f32<TX>(rstd * (g - mg - (to_f32(x[c]) - mean) * rstd * mgh));
    }
}

// Column sums of one range of rows (blockIdx.y of gridDim.y), one column per thread.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kLoopThreads) k_norm_param_loop(NormArgs a, float *part)
{
    const int c = blockIdx.x * kLoopThreads + threadIdx.x;
    if (c < a.width) {
        const int64_t r0 = a.n * blockIdx.y / gridDim.y, r1 = a.n * (blockIdx.y + 1) / gridDim.y;
        float dw = 0.0f, db = 0.0f;
        for (int64_t r = r0; r < r1; ++r) {
            const float dy = to_f32(static_cast<const TY *>(a.dy)[r * a.y_stride + c]);
            db += dy;
            dw += dy * ((to_f32(static_cast<const TX *>(a.x)[r * a.x_stride + c]) - a.mean[r]) * a.rstd[r]);
        }
        float *p = part + (int64_t)blockIdx.y * 2 * a.width;
        p[c] = dw;
        p[a.width + c] = db;
    }
    let_next_start();
}

// ---- dispatch ------------------------------------------------------------------------

// f(TX{}, TY{}): y has x's type or float32.
template <typename F>
cudaError_t with_xy(const NormArgs &a, F &&f)
{
    return with_dtype(a.x_dtype, [&](auto tx) {
        if (a.y_dtype == HISS_F32) return f(tx, float{});
        return f(tx, tx);
    });
}

template <int V>
using Int = std::integral_constant<int, V>;

// f(E, NV, NARROW, PAIR) for the packs of r.
template <typename TX, bool HAS32, bool HAS32_WIDE, typename F>
cudaError_t with_packs(const Rows &r, F &&f)
{
    constexpr int W = 16 / (int)sizeof(TX);
    auto with_width = [&](auto e) {
        constexpr int E = decltype(e)::value;
        if constexpr (E == W ? HAS32_WIDE : HAS32) {
            if (r.e * r.nv == 32) return f(e, Int<32 / E>{}, std::false_type{}, std::false_type{});
        } else {
            if (r.pair) return f(e, Int<16 / E>{}, std::false_type{}, std::true_type{});
        }
        if (r.narrow) return f(e, Int<16 / E>{}, std::true_type{}, std::false_type{});
        return f(e, Int<16 / E>{}, std::false_type{}, std::false_type{});
    };
    if (r.e == W) return with_width(Int<W>{});
    if constexpr (W == 8)
        if (r.e == 2) return with_width(Int<2>{});
    return with_width(Int<1>{});
}

// Blocks, or pairs of blocks (an even number of SMs share a cluster's place,
// so that all of them find room).
unsigned grid_for(const NormArgs &a, const Rows &r, int per_sm)
{
    const int64_t want = (a.n + r.groups - 1) / r.groups, room = (int64_t)kSMs * per_sm / (r.pair ? kPair : 1);
    return (unsigned)(want < room ? want : room);
}

template <typename... P, typename... A>
cudaError_t launch_rows(void (*kernel)(P...), const Rows &r, unsigned grid, size_t smem, cudaStream_t s, const A &...args)
{
    const unsigned threads = r.lanes * r.groups;
    if (!r.pair) {
        kernel<<<grid, threads, smem, s>>>(static_cast<P>(args)...);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kPair * grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kPair;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

Rows plan_forward(const NormArgs &a) { return plan_rows(a, a.x_dtype != HISS_F32, true, 256, false); }

// 32 elements per lane with a float32 operand would not leave room for two
// rows in the ring.
Rows plan_backward(const NormArgs &a)
{
    const bool both16 = a.y_dtype != HISS_F32;
    return plan_rows(a, both16, both16, kMaxLanes, a.dweight || a.dbias);
}

// Blocks (and parts) of the backward pass: one per SM, so that there are few
// parts to add up.
unsigned grad_grid(const NormArgs &a, const Rows &r) { return r.one_block ? 1 : grid_for(a, r, 1); }

}  // namespace

cudaError_t layer_norm(const NormArgs &a, cudaStream_t s, int64_t *launches)
{
    const Rows r = plan_forward(a);
    ++*launches;
    return with_xy(a, [&](auto tx, auto ty) {
        using TX = decltype(tx);
        using TY = decltype(ty);
        if (!r.e) {
            k_norm_loop<TX, TY><<<(unsigned)a.n, kLoopThreads, 0, s>>>(a);
            return cudaGetLastError();
        }
        return with_packs<TX, sizeof(TX) == 2, true>(r, [&](auto e, auto nv, auto narrow, auto pair) {
            constexpr int E = decltype(e)::value, NV = decltype(nv)::value;
            constexpr bool NARROW = decltype(narrow)::value;
            static Residency cache;
            auto kernel = k_norm<TX, TY, E, NV, NARROW, decltype(pair)::value>;
            const int threads = r.lanes * r.groups;
            const size_t smem = Forward<TX, E, NV, NARROW>::smem(threads, r.lanes, r.pair ? first_half(a.width) : a.width);
            int per_sm = 1;
            HISS_TRY(resident(kernel, threads, smem, cache, &per_sm));
            return launch_rows(kernel, r, grid_for(a, r, per_sm), smem, s, a, r.lanes, r.groups);
        });
    });
}

size_t layer_norm_grad_tmp_bytes(const NormArgs &a)
{
    const Rows r = plan_backward(a);
    return 8 * (size_t)a.width * (r.e ? grad_grid(a, r) : kLoopSplits);
}

cudaError_t layer_norm_grad(const NormArgs &a, void *tmp, cudaStream_t s, int64_t *launches)
{
    const bool params = a.dweight || a.dbias;
    float *part = params ? static_cast<float *>(tmp) : nullptr;
    unsigned parts = 0;
    bool direct = false;
    if (a.n > 0) {
        const Rows r = plan_backward(a);
        HISS_TRY(with_xy(a, [&](auto tx, auto ty) {
            using TX = decltype(tx);
            using TY = decltype(ty);
            if (!r.e) {
                if (a.dx) {
                    k_norm_dx_loop<TX, TY><<<(unsigned)a.n, kLoopThreads, 0, s>>>(a);
                    ++*launches;
                }
                if (params) {
                    parts = (unsigned)(a.n < kLoopSplits ? a.n : kLoopSplits);
                    k_norm_param_loop<TX, TY><<<dim3((a.width + kLoopThreads - 1) / kLoopThreads, parts), kLoopThreads, 0, s>>>(
                        a, part);
                    ++*launches;
                }
                return cudaGetLastError();
            }
            return with_packs<TX, sizeof(TY) == 2, sizeof(TY) == 2>(r, [&](auto e, auto nv, auto narrow, auto pair) {
                constexpr int E = decltype(e)::value, NV = decltype(nv)::value;
                static std::atomic<uint64_t> allowed{0};
                auto kernel = k_norm_grad<TX, TY, E, NV, decltype(narrow)::value, decltype(pair)::value>;
                const int threads = r.lanes * r.groups;
                const bool many = threads > (r.narrow ? 32 : r.lanes);  // sums of several warps or groups to add up
                using B = Backward<TX, TY, E, NV, decltype(narrow)::value>;
                const int width = r.pair ? first_half(a.width) : a.width;  // of a block
                const size_t smem = B::smem(threads, r.lanes, width, many);
                HISS_TRY(allow_shared(kernel, kSharedBytes, allowed));
                parts = grad_grid(a, r);
                direct = r.one_block;
                ++*launches;
                return launch_rows(kernel, r, parts, smem, s, a, r.lanes, r.groups, (int)B::X::bytes(threads, r.lanes, width),
                                   r.one_block ? nullptr : part, r.one_block);
            });
        }));
    }
    if (!params || direct) return cudaSuccess;
    ++*launches;
    return launch_after(k_norm_param, (unsigned)((2 * a.width + 31) / 32), 1024, 0, s, a, part, (int)parts);
}

}  // namespace hiss
