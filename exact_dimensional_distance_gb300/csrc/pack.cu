// Rows in 8 bits: int8 codes with a power-of-two scale for each block of 32
// columns, and back.  The scale's power of two makes x / s and code * s exact, so
// that the codes follow from the definition alone, and lets a bfloat16 or float16 operand
// of a matrix product take the value that was kept without a second rounding.
#include <algorithm>
#include <climits>

#include "hiss_internal.cuh"
#include "packed.cuh"

namespace hiss {
namespace {

constexpr int kThreads = 256;
// Pieces that a thread loads before it uses the first: 4 are 8 us faster than 2 or 8 for packing 65,536 x 4096
// bfloat16, 8 are 7 us faster than 4 for unpacking it.
constexpr int kPackAhead = 4, kUnpackAhead = 8;

// A thread handles 8 columns, four neighbouring lanes a block: its columns are one
// access of 16 bytes (two of float32), its codes one of 8 bytes.  65,536 x 4096 bfloat16: 137 us
// (5.9 TB/s; 148 with the magnitudes one by one, 195 with codes clamped and converted in separate
// operations); bound by memory and issue alike.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_pack(const T *x, int64_t stride, int64_t n, int width, Divider per_row, int8_t *codes,
                                                   uint8_t *scales)
{
    const int64_t total = n * per_row.d, step = (int64_t)gridDim.x * kThreads;
    // whole blocks of threads go round the loop together: a block of columns is four lanes
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 - threadIdx.x < total; i0 += kPackAhead * step) {
        Eight<T, VEC> in[kPackAhead];
        const T *row[kPackAhead];
        int col[kPackAhead];
#pragma unroll
        for (int k = 0; k < kPackAhead; ++k) {
            const int64_t i = i0 + k * step, r = per_row.quotient(i < total ? i : 0);
            row[k] = x + r * stride;
            col[k] = i < total ? (int)(i - r * per_row.d) * 8 : INT_MAX / 2;
            in[k].load(row[k], col[k], width);
        }
#pragma unroll
        for (int k = 0; k < kPackAhead; ++k) {
            const int64_t i = i0 + k * step;
            uint32_t bits[Eight<T, VEC>::W];
            in[k].words(row[k], col[k], width, bits);
            uint32_t m = Eight<T, VEC>::magnitude(bits);
            float v[8];
            Eight<T, VEC>::floats(bits, v);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            if (i >= total) continue;
            const uint32_t byte = scale_byte(m);
            uint32_t w[2];
            codes_of(v, byte, top_byte<T>(), w);
            *reinterpret_cast<uint2 *>(codes + i * 8) = make_uint2(w[0], w[1]);
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
        }
    }
}

// 65,536 x 4096 bfloat16: 124 us (6.6 TB/s), bound by memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_unpack(const int8_t *codes, const uint8_t *scales, int64_t n, int width, Divider per_row,
                                                     T *x, int64_t stride)
{
    const int64_t total = n * per_row.d, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += kUnpackAhead * step) {
        uint2 q[kUnpackAhead];
        uint32_t byte[kUnpackAhead];
#pragma unroll
        for (int k = 0; k < kUnpackAhead; ++k) {
            const int64_t i = i0 + k * step;
            q[k] = i < total ? *reinterpret_cast<const uint2 *>(codes + i * 8) : make_uint2(0, 0);
            byte[k] = i < total ? scales[i >> 2] : 0;
        }
#pragma unroll
        for (int k = 0; k < kUnpackAhead; ++k) {
            const int64_t i = i0 + k * step;
            if (i >= total) break;
            const int64_t r = per_row.quotient(i);
            float v[8];
            values8(q[k], scale_of(byte[k]), v);
            store8<T, true>(x + r * stride, (int)(i - r * per_row.d) * 8, width, v);
        }
    }
}

// The same where rows of x are not aligned to 16 bytes: a thread takes a 16-byte line of x
// instead, E elements whose codes lie across two aligned pairs of words and up to two blocks.
// 20,011 x 1021 float16: 18 us (63 with single elements), bound by issue.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_unpack_lines(const int8_t *codes, const uint8_t *scales, int64_t n, int width, int blocks,
                                                           Divider per_row, T *x, int64_t stride)
{
    constexpr int E = 16 / sizeof(T);
    const int64_t total = n * per_row.d, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += step) {
        const int64_t r = per_row.quotient(i);
        T *row = x + r * stride;
        // the line's first column: -E + 1 .. and, in the last lines, behind the row
        const int c = (int)(i - r * per_row.d) * E - (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        if (c >= width) continue;
        const int8_t *q = codes + r * blocks * kPackBlock;
        const int at = c & ~7, first = max(c, 0) / kPackBlock, last = min(c + E, width) - 1;
        const uint2 a = at >= 0 ? *reinterpret_cast<const uint2 *>(q + at) : make_uint2(0, 0);
        const uint2 b = at + 8 < blocks * kPackBlock ? *reinterpret_cast<const uint2 *>(q + at + 8) : make_uint2(0, 0);
        const uint8_t *s = scales + r * blocks + first;
        const float f0 = scale_of(s[0]), f1 = last / kPackBlock > first ? scale_of(s[1]) : f0;
        const int sh = (c & 7) * 8, edge = (first + 1) * kPackBlock;
        const uint64_t lo = a.x | (uint64_t)a.y << 32, hi = b.x | (uint64_t)b.y << 32;
        const uint64_t w = sh ? lo >> sh | hi << (64 - sh) : lo;
        float v[8];
        values8(make_uint2((uint32_t)w, (uint32_t)(w >> 32)), 1.0f, v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = __fmul_rn(v[e], c + e < edge ? f0 : f1);
        if (c >= 0 && c <= width - E) {
            Pack<T, E> p;
#pragma unroll
            for (int e = 0; e < E; e += 2) set_pair(p.v + e, make_float2(v[e], v[e + 1]));
            store_pack<T, E>(row + c, p);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (c + e >= 0 && c + e < width) row[c + e] = from_f32<T>(v[e]);
        }
    }
}

// A block for every kThreads * each items.
unsigned grid_for(int64_t total, int each)
{
    const int64_t want = (total + each * kThreads - 1) / (each * kThreads), most = 1 << 30;
    return (unsigned)(want < most ? want : most);
}

}  // namespace

cudaError_t pack(const void *x, int dtype, int64_t stride, int64_t n, int width, const hiss_packed &p, cudaStream_t s,
                 int64_t *launches)
{
    if (n == 0) return cudaSuccess;
    const Divider per_row(4 * packed_blocks(width));
    const unsigned grid = grid_for(n * per_row.d, kPackAhead);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        auto *k = rows_aligned(x, stride, dtype, 8) ? k_pack<T, true> : k_pack<T, false>;
        k<<<grid, kThreads, 0, s>>>(static_cast<const T *>(x), stride, n, width, per_row, p.codes, p.scales);
        ++*launches;
        return cudaGetLastError();
    });
}

cudaError_t unpack(const hiss_packed &p, int64_t n, int width, void *x, int dtype, int64_t stride, cudaStream_t s,
                   int64_t *launches)
{
    if (n == 0) return cudaSuccess;
    const int blocks = packed_blocks(width);
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        if (rows_aligned(x, stride, dtype, 8)) {
            const Divider per_row(4 * blocks);
            k_unpack<T><<<grid_for(n * per_row.d, kUnpackAhead), kThreads, 0, s>>>(p.codes, p.scales, n, width, per_row,
                                                                               static_cast<T *>(x), stride);
        } else {
            const Divider per_row((width * (int)sizeof(T) + 14) / 16 + 1);
            const unsigned grid = std::min(grid_for(n * per_row.d, 1), 16u * kSMs);
            k_unpack_lines<T><<<grid, kThreads, 0, s>>>(p.codes, p.scales, n, width, blocks, per_row,
                                                                                static_cast<T *>(x), stride);
        }
        ++*launches;
        return cudaGetLastError();
    });
}

}  // namespace hiss
