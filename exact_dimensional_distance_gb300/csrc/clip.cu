// Clipping by the global gradient norm over many tensors.
//
//   N = sqrt(sum g^2),  g <- g * max_norm / N  if N is finite and > max_norm.
//
// Two launches whatever the number of tensors (up to kMaxTensors; further
// tensors go to further launches): k_sum_squares leaves one float64 partial sum per
// block, its last block to finish adds them up in the blocks' order and
// leaves the factor, and k_clip scales.  float64 runs at a sixty-fourth of
// float32's rate, so it is kept to one thread or one block at a time.  The list
// of tensors travels in the kernels' parameters: no copy to the device, nothing
// to keep alive after the call, and a captured graph holds its own.
//
// The work is cut into chunks of one tensor each, dealt out to the blocks in
// turn.  The norm needs every element before the first write, so a set larger
// than L2 is read twice: 2 reads and 1 write per element bound it, not 1 and
// 1.  k_clip takes the chunks in reverse order, so that it starts with what
// the first pass left in L2.
#include <algorithm>

#include "hiss_internal.cuh"
#include "numeric.cuh"

namespace hiss {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSM = 4;    // 2^30 elements: 1,003 us; five 1,052, six 1,098
constexpr int kMaxBlocks = kSMs * kBlocksPerSM;
constexpr int kUnroll = 4;         // accesses in flight per thread
constexpr int kMaxTensors = 1000;  // 29 KB of parameters per launch (the limit is 32,764 bytes)
// Shorter lists for fewer: a launch copies its parameters (356 short tensors: 22.2 us
// a call with the middle list, 24.6 with the longest).
constexpr int kFewTensors = 64, kSomeTensors = 384;

template <int CAP>
struct TensorList {
    const void *in[CAP];
    void *out[CAP];
    int64_t n[CAP];
    int32_t first[CAP + 1];  // first chunk of each tensor; first[count] = number of chunks
    uint8_t dtype[CAP];
    int32_t count;
    int32_t chunk;           // elements per chunk, a multiple of 2048
};

// Whether a sum of squares lost nothing that matters: no square overflowed, and what
// float32 loses of small squares, half of 2^-149 each, is below 2^-37 of the sum.
__device__ __forceinline__ bool in_range(float s) { return s >= 0x1p-110f && s <= 0x1p100f; }

// Adds the squares of U packs to *narrow in float32; a pack whose sum is not in
// range is computed again in float64 and added to *wide instead, unless it is all
// zeros (the gradient of a table is mostly those, and float64 is slow: values
// around 1e-20 take 12 times as long).  One branch for all U packs:
// with one per pack the compiler waits for each load in turn (1.7 TB/s against 4.5).
template <typename T, int E, int U>
__device__ __forceinline__ void add_squares(const Pack<T, E> (&p)[U], float *narrow, double *wide)
{
    float s[U];
    bool odd = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (E == 1) {
            const float v = to_f32(p[u].v[0]);
            s[u] = v * v;
        } else {
            float2 q = both(0.0f);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = pair_of(p[u].v + e);
                q = __ffma2_rn(v, v, q);
            }
            s[u] = q.x + q.y;
        }
        // s = 0: in order only if every element is zero
        uint32_t bits = 0;
        if constexpr (sizeof(Pack<T, E>) == 16) {
            const uint4 w = *reinterpret_cast<const uint4 *>(&p[u]);
            bits = (w.x | w.y | w.z | w.w) & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu);
        } else {
            bits = to_f32(p[u].v[0]) != 0.0f;
        }
        odd = odd || !(in_range(s[u]) || bits == 0);
    }
    if (odd) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (in_range(s[u])) continue;
            s[u] = 0.0f;
#pragma unroll  // an index known only at run time would put every pack in local memory
            for (int e = 0; e < E; ++e) {
                const double v = to_f32(p[u].v[e]);
                *wide += v * v;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) *narrow += s[u];
}

// Adds this thread's share of the sum of squares of x[0 .. n).
template <typename T>
__device__ void chunk_squares(const T *x, int64_t n, float &narrow, double &wide)
{
    constexpr int E = 16 / sizeof(T);
    const int head = (int)min((int64_t)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T), n);
    const T *v = x + head;
    const int packs = (int)((n - head) / E);
    // the few elements before the first and behind the last pack
    const int tail = (int)(n - head) - packs * E, t = (int)threadIdx.x;
    if (t < head + tail) {
        const Pack<T, 1> p[1] = {load_pack<T, 1>(t < head ? x + t : v + (int64_t)packs * E + (t - head))};
        add_squares<T, 1, 1>(p, &narrow, &wide);
    }
    int i = threadIdx.x;
    for (; i + (kUnroll - 1) * kThreads < packs; i += kUnroll * kThreads) {
        Pack<T, E> p[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) p[u] = load_pack<T, E>(v + (int64_t)(i + u * kThreads) * E);
        add_squares<T, E, kUnroll>(p, &narrow, &wide);
    }
    for (; i < packs; i += kThreads) {
        const Pack<T, E> p[1] = {load_pack<T, E>(v + (int64_t)i * E)};
        add_squares<T, E, 1>(p, &narrow, &wide);
    }
}

// The tensor that holds a chunk.
template <int CAP>
__device__ __forceinline__ int tensor_of(const TensorList<CAP> &l, int chunk)
{
    int lo = 0, hi = l.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (l.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The sums over the lists so far, and what k_clip reads.
struct ClipState {
    unsigned done;   // blocks of the last list's kernel that have finished (0 between calls)
    float factor;    // 0 also where float32 cannot hold it as a normal number:
    double fine;     // then this is it (0 otherwise)
};

// Sum over the block of a float64 per thread, in thread 0.
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double warp_part[kWarps];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kWarps; ++w) v += warp_part[w];
    return v;
}

// 2^30 elements (2.15 GB) in 290 tensors: 307 us, 7.0 TB/s, bound by memory.
// 3.0 million float32 in 60 tensors: 4 to 5 us warm, the latency of finding the tensor, one
// round of loads and the float64 end in the last block.
//
// part: where this list's blocks leave their sums; all, parts: the sums of
// every list; last: this is the last list.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSM)
    k_sum_squares(const __grid_constant__ TensorList<CAP> l, double *part, const double *all, int parts, bool last,
                  float max_norm, float *norm, ClipState *state)
{
    __shared__ double warp_part[kWarps];
    __shared__ bool finish;
    wait_for_previous();
    // float32 over the thread's share of one chunk (at most 128 elements of
    // the usual chunk sizes) and then over a warp, float64 above that
    float narrow = 0.0f;
    double wide = 0.0;
    const int chunks = l.first[l.count];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        if (c != (int)blockIdx.x) {
            wide += (double)narrow;
            narrow = 0.0f;
        }
        const int t = tensor_of(l, c);
        const int64_t at = (int64_t)(c - l.first[t]) * l.chunk, n = min((int64_t)l.chunk, l.n[t] - at);
        if (l.dtype[t] == HISS_F32) chunk_squares(static_cast<const float *>(l.in[t]) + at, n, narrow, wide);
        else if (l.dtype[t] == HISS_F16) chunk_squares(static_cast<const __half *>(l.in[t]) + at, n, narrow, wide);
        else chunk_squares(static_cast<const __nv_bfloat16 *>(l.in[t]) + at, n, narrow, wide);
    }
    for (int o = 16; o > 0; o >>= 1) narrow += __shfl_xor_sync(0xffffffffu, narrow, o);
    if (__any_sync(0xffffffffu, __double_as_longlong(wide) != 0))
        for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xffffffffu, wide, o);
    if ((threadIdx.x & 31) == 0) warp_part[threadIdx.x >> 5] = wide + (double)narrow;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = warp_part[0];
        for (int w = 1; w < kWarps; ++w) s += warp_part[w];
        part[blockIdx.x] = s;
        __threadfence();
        finish = last && atomicAdd(&state->done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (finish) {
        __threadfence();
        double s = 0.0;
        for (int i = threadIdx.x; i < parts; i += kThreads) s += *(volatile const double *)(all + i);
        s = block_sum(s);
        if (threadIdx.x == 0) {
            const double total = sqrt(s);
            *norm = (float)total;
            const double factor = isfinite(total) && total > (double)max_norm ? (double)max_norm / total : 1.0;
            state->factor = factor < 0x1p-126 ? 0.0f : (float)factor;
            state->fine = factor < 0x1p-126 ? factor : 0.0;
            state->done = 0;
        }
    }
    let_next_start();
}

template <typename T>
__device__ void chunk_scale(const T *x, T *y, int64_t n, float f)
{
    constexpr int E = 16 / sizeof(T);
    const int off = (int)(reinterpret_cast<uintptr_t>(x) & 15);
    if (off != (int)(reinterpret_cast<uintptr_t>(y) & 15)) {  // no common 16-byte alignment
        for (int64_t i = threadIdx.x; i < n; i += kThreads) y[i] = f == 1.0f ? x[i] : from_f32<T>(to_f32(x[i]) * f);
        return;
    }
    const int head = (int)min((int64_t)((16 - off) & 15) / (int)sizeof(T), n);
    if ((int)threadIdx.x < head)
        y[threadIdx.x] = f == 1.0f ? x[threadIdx.x] : from_f32<T>(to_f32(x[threadIdx.x]) * f);
    const T *v = x + head;
    T *w = y + head;
    const int packs = (int)((n - head) / E);
    int i = threadIdx.x;
    auto scaled = [f](Pack<T, E> p) {
        if (f != 1.0f)  // a factor of 1 copies the bits, NaN and infinities included
#pragma unroll
            for (int e = 0; e < E; ++e) p.v[e] = from_f32<T>(to_f32(p.v[e]) * f);
        return p;
    };
    for (; i + (kUnroll - 1) * kThreads < packs; i += kUnroll * kThreads) {
        Pack<T, E> p[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) p[u] = load_pack<T, E>(v + (int64_t)(i + u * kThreads) * E);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) store_pack<T, E>(w + (int64_t)(i + u * kThreads) * E, scaled(p[u]));
    }
    for (; i < packs; i += kThreads) store_pack<T, E>(w + (int64_t)i * E, scaled(load_pack<T, E>(v + (int64_t)i * E)));
    const int tail = (int)(n - head) - packs * E;
    if ((int)threadIdx.x < tail) {
        const int64_t at = (int64_t)packs * E + threadIdx.x;
        w[at] = f == 1.0f ? v[at] : from_f32<T>(to_f32(v[at]) * f);
    }
}

// A factor that float32 holds as a subnormal number or as zero (a norm around 1e38 and
// above, clipped to 1 or less): products in float64, rounded to float32 and to the
// type as the others are.
template <typename T>
__device__ __noinline__ void chunk_scale_fine(const T *x, T *y, int64_t n, double f)
{
    for (int64_t i = threadIdx.x; i < n; i += kThreads) y[i] = from_f32<T>((float)((double)to_f32(x[i]) * f));
}

// 2^30 elements: 683 us, 6.3 TB/s read and written, bound by memory.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSM)
    k_clip(const __grid_constant__ TensorList<CAP> l, const ClipState *state)
{
    wait_for_previous();
    const float f = state->factor;
    const double fine = state->fine;
    const int chunks = l.first[l.count];
    for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
        const int c = chunks - 1 - i;
        const int t = tensor_of(l, c);
        if (f == 1.0f && l.in[t] == l.out[t]) continue;
        const int64_t at = (int64_t)(c - l.first[t]) * l.chunk, n = min((int64_t)l.chunk, l.n[t] - at);
        auto scale = [&](auto type) {
            using T = decltype(type);
            const T *x = static_cast<const T *>(l.in[t]) + at;
            T *y = static_cast<T *>(l.out[t]) + at;
            if (fine != 0.0) chunk_scale_fine(x, y, n, fine);
            else chunk_scale(x, y, n, f);
        };
        if (l.dtype[t] == HISS_F32) scale(float{});
        else if (l.dtype[t] == HISS_F16) scale(__half{});
        else scale(__nv_bfloat16{});
    }
}

// The next up to CAP tensors of t from *i on; tensors without elements are
// skipped, those behind the last one taken too.
template <int CAP>
void fill(TensorList<CAP> &l, const hiss_tensor *t, int64_t count, int64_t *i, int64_t chunk)
{
    l.chunk = (int32_t)chunk;
    l.count = 0;
    l.first[0] = 0;
    int64_t chunks = 0;
    for (; *i < count && l.count < CAP; ++*i) {
        const hiss_tensor &e = t[*i];
        if (e.n == 0) continue;
        const int k = l.count++;
        l.in[k] = e.in;
        l.out[k] = e.out ? e.out : const_cast<void *>(e.in);
        l.n[k] = e.n;
        l.dtype[k] = (uint8_t)e.dtype;
        chunks += (e.n + chunk - 1) / chunk;
        l.first[k + 1] = (int32_t)chunks;
    }
    while (*i < count && t[*i].n == 0) ++*i;
}

struct Plan {
    int64_t used = 0;    // tensors with elements
    int64_t lists = 0;   // launches of each kernel
    int64_t chunk = 0;
};

// Chunks are 2^11 to 2^15 elements (above that only so that a tensor's chunk
// count fits 32 bits): small enough that a small set reaches every block,
// large enough that finding the chunk's tensor costs nothing.
Plan plan(const hiss_tensor *t, int64_t count)
{
    Plan p;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        total += t[i].n;
        p.used += t[i].n > 0;
    }
    p.lists = (p.used + kMaxTensors - 1) / kMaxTensors;
    p.chunk = 1 << 11;
    while (p.chunk < (1 << 15) && total > p.chunk * kMaxBlocks) p.chunk <<= 1;
    while (total / p.chunk > (1 << 28)) p.chunk <<= 1;
    return p;
}

template <int CAP>
cudaError_t run(const hiss_tensor *t, int64_t count, const Plan &p, float max_norm, float *norm, ClipState *state,
                double *part, cudaStream_t s, int64_t *launches)
{
    TensorList<CAP> l;
    int parts = 0;
    int64_t i = 0;
    do {
        fill(l, t, count, &i, p.chunk);
        const int blocks = std::max(1, std::min(kMaxBlocks, l.first[l.count]));
        HISS_TRY(launch_after(k_sum_squares<CAP>, blocks, kThreads, 0, s, l, part + parts, part, parts + blocks, i >= count,
                              max_norm, norm, state));
        parts += blocks;
        ++*launches;
    } while (i < count);
    i = 0;
    do {
        if (p.lists > 1) fill(l, t, count, &i, p.chunk);
        else i = count;
        const int blocks = std::max(1, std::min(kMaxBlocks, l.first[l.count]));
        HISS_TRY(launch_after(k_clip<CAP>, blocks, kThreads, 0, s, l, state));
        ++*launches;
    } while (i < count);
    return cudaSuccess;
}

}  // namespace

size_t clip_state_bytes() { return sizeof(ClipState); }

size_t clip_tmp_bytes(const hiss_tensor *t, int64_t count)
{
    return 8 * (size_t)kMaxBlocks * (size_t)std::max<int64_t>(1, plan(t, count).lists);
}

cudaError_t clip_grads(const hiss_tensor *t, int64_t count, float max_norm, float *norm, void *state, void *tmp,
                       cudaStream_t s, int64_t *launches)
{
    const Plan p = plan(t, count);
    double *part = static_cast<double *>(tmp);
    ClipState *c = static_cast<ClipState *>(state);
    if (p.used <= kFewTensors) return run<kFewTensors>(t, count, p, max_norm, norm, c, part, s, launches);
    if (p.used <= kSomeTensors) return run<kSomeTensors>(t, count, p, max_norm, norm, c, part, s, launches);
    return run<kMaxTensors>(t, count, p, max_norm, norm, c, part, s, launches);
}

}  // namespace hiss
