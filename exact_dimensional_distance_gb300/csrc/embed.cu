// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: out[i] = scale * table[token[i]].  Backward: grad[v] = scale * sum
// of dy[i] over the positions i that hold token v.  The positions are sorted
// by token (stable radix sort), so each row of the gradient is the sum of one
// contiguous run in position order: no floating-point atomics, and the same
// bits every time.
#include "hiss_internal.cuh"
#include "numeric.cuh"

namespace hiss {
namespace {

constexpr int kThreads = 256;

// The table row of position i, or -1 for a row of zeros (padding, or a token
// outside the table, which sets *bad).
__device__ __forceinline__ int64_t row_of(const void *tokens, int bits, int64_t i, int64_t pad, int64_t vocab, int *bad)
{
    const int64_t t = bits == 64 ? static_cast<const int64_t *>(tokens)[i] : static_cast<const int32_t *>(tokens)[i];
    if (t == pad) return -1;
    if (t < 0 || t >= vocab) {
        *bad = 1;
        return -1;
    }
    return t;
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) k_embed(EmbedArgs a)
{
    const int64_t total = a.n * a.width;
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < total; e += (int64_t)gridDim.x * kThreads) {
        const int64_t i = e / a.width, c = e - i * a.width;
        const int64_t r = row_of(a.tokens, a.token_bits, i, a.pad, a.vocab, a.bad);
        const float v = r < 0 ? 0.0f : a.scale * to_f32(static_cast<const TI *>(a.rows)[r * a.rows_stride + c]);
        static_cast<TO *>(a.out)[i * a.out_stride + c] = from_f32<TO>(v);
    }
}

// Sort keys: the token, or vocab for a position that contributes nothing.
__global__ void __launch_bounds__(kThreads) k_token_keys(EmbedArgs a, uint64_t *keys, uint32_t *vals)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.n) return;
    const int64_t r = row_of(a.tokens, a.token_bits, i, a.pad, a.vocab, a.bad);
    keys[i] = (uint64_t)(r < 0 ? a.vocab : r);
    vals[i] = (uint32_t)i;
}

// First and one past the last sorted position of each token present.
__global__ void __launch_bounds__(kThreads) k_token_runs(const uint64_t *keys, int64_t n, int64_t vocab, int32_t *first,
                                                         int32_t *last)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const int64_t k = (int64_t)keys[i];
    if (k >= vocab) return;
    if (i == 0 || (int64_t)keys[i - 1] != k) first[k] = (int32_t)i;
    if (i == n - 1 || (int64_t)keys[i + 1] != k) last[k] = (int32_t)(i + 1);
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) k_embed_grad(EmbedArgs a, const uint32_t *order, const int32_t *first,
                                                         const int32_t *last)
{
    const int64_t v = blockIdx.x;
    const int32_t i0 = first[v], i1 = last[v];
    if (a.accumulate && i1 <= i0) return;
    TO *out = static_cast<TO *>(a.out) + v * a.out_stride;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
        float s = 0.0f;
        for (int32_t i = i0; i < i1; ++i)
            s += to_f32(static_cast<const TI *>(a.rows)[(int64_t)order[i] * a.rows_stride + c]);
        s *= a.scale;
        if (a.accumulate) s += to_f32(out[c]);
        out[c] = from_f32<TO>(s);
    }
}

int bits_of(int64_t v)
{
    int b = 0;
    while (v >> b) ++b;
    return b;
}

size_t up(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace

cudaError_t embed(const EmbedArgs &a, cudaStream_t s, int64_t *launches)
{
    const int64_t blocks = (a.n * a.width + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)(blocks < 152 * 64 ? blocks : 152 * 64);
    return with_dtype(a.rows_dtype, [&](auto ti) {
        return with_dtype(a.out_dtype, [&](auto to) {
            k_embed<decltype(ti), decltype(to)><<<grid, kThreads, 0, s>>>(a);
            ++*launches;
            return cudaGetLastError();
        });
    });
}

size_t embed_grad_tmp_bytes(const EmbedArgs &a)
{
    return 2 * up(8 * (size_t)a.n) + 2 * up(4 * (size_t)a.n) + up(sort_tmp_bytes(a.n)) + 2 * up(4 * (size_t)a.vocab);
}

cudaError_t embed_grad(const EmbedArgs &a, void *tmp, int *flags, cudaStream_t s, int64_t *launches)
{
    char *p = static_cast<char *>(tmp);
    auto take = [&](size_t b) { char *q = p; p += up(b); return q; };
    uint64_t *keys = (uint64_t *)take(8 * (size_t)a.n), *keys_alt = (uint64_t *)take(8 * (size_t)a.n);
    uint32_t *vals = (uint32_t *)take(4 * (size_t)a.n), *vals_alt = (uint32_t *)take(4 * (size_t)a.n);
    void *sort_tmp = take(sort_tmp_bytes(a.n));
    int32_t *first = (int32_t *)take(4 * (size_t)a.vocab), *last = (int32_t *)take(4 * (size_t)a.vocab);
    HISS_TRY(cudaMemsetAsync(first, 0, 4 * (size_t)a.vocab, s));
    HISS_TRY(cudaMemsetAsync(last, 0, 4 * (size_t)a.vocab, s));
    int in_alt = 0;
    if (a.n > 0) {
        const unsigned blocks = (unsigned)((a.n + kThreads - 1) / kThreads);
        k_token_keys<<<blocks, kThreads, 0, s>>>(a, keys, vals);
        HISS_TRY(sort_pairs(keys, vals, keys_alt, vals_alt, a.n, bits_of(a.vocab), sort_tmp, flags, s, launches, &in_alt));
        k_token_runs<<<blocks, kThreads, 0, s>>>(in_alt ? keys_alt : keys, a.n, a.vocab, first, last);
        *launches += 2;
    }
    return with_dtype(a.rows_dtype, [&](auto ti) {
        return with_dtype(a.out_dtype, [&](auto to) {
            k_embed_grad<decltype(ti), decltype(to)><<<(unsigned)a.vocab, kThreads, 0, s>>>(a, in_alt ? vals_alt : vals,
                                                                                           first, last);
            ++*launches;
            return cudaGetLastError();
        });
    });
}

}  // namespace hiss
