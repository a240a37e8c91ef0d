// The arithmetic of rows in 8 bits (see hiss_packed in hiss.h), shared by the
// kernels that write and read them.
#pragma once

#include <cstring>

#include "numeric.cuh"

namespace hiss {

constexpr int kPackBlock = 32;
constexpr float kFloatMax = 3.402823466e38f;

inline int packed_blocks(int width) { return (width + kPackBlock - 1) / kPackBlock; }

// The scale byte of a block whose largest magnitude has these bits (not a finite number's: a
// block that reads back as NaN).  m = f * 2^(E - 127) with 1 <= f < 2 is at most 127 * 2^e from
// e + 127 = E - 6 on, or E - 5 when f > 127 / 64, whose fraction is 0x7E0000: the sum's carry.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits)
{
    if (bits >= 0x7F800000u) return 255;
    const int e = (int)((bits + 0x1FFFFu) >> 23) - 6;
    return e < 1 ? 1 : (uint32_t)e;
}

// 2^(byte - 127); bytes from 1 to 254.  Byte 0 gives 0, byte 255 NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte == 255 ? 0x7FC00000u : byte << 23); }

// The smallest scale byte whose 64 * 2^(byte - 127) is beyond the type.
template <typename T>
__device__ constexpr uint32_t top_byte() { return std::is_same_v<T, __half> ? 137 : 249; }

// Four codes in a word.  x / s is exact and at most 127, so one fused operation rounds it to a
// whole number: 1.5 * 2^23 + x / s, whose float32 neighbours are 1 apart, has the code in its low byte.
constexpr float kRoundUnits = 12582912.0f;
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d)
{
    const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
    return __byte_perm(lo, __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t codes4(const float *v, float inverse)
{
    auto code = [&](float x) { return __fmaf_rn(x, inverse, kRoundUnits); };
    return low_bytes(code(v[0]), code(v[1]), code(v[2]), code(v[3]));
}
// The same where codes stop at 63, and of blocks that read back as NaN: codes of 0.
__device__ __forceinline__ uint32_t codes4_edge(const float *v, uint32_t byte)
{
    if (byte == 255) return 0;
    auto code = [&](float x) {
        return __fadd_rn(fminf(fmaxf(__fmul_rn(x, __uint_as_float((254u - byte) << 23)), -63.0f), 63.0f), kRoundUnits);
    };
    return low_bytes(code(v[0]), code(v[1]), code(v[2]), code(v[3]));
}

// W words of codes of a row's part in one block with this scale byte; top: top_byte of the rows' type.
template <int W>
__device__ __forceinline__ void codes_of(const float *v, uint32_t byte, uint32_t top, uint32_t (&w)[W])
{
    if (byte < top) {
        const float inverse = __uint_as_float((254u - byte) << 23);
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = codes4(v + 4 * j, inverse);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = codes4_edge(v + 4 * j, byte);
    }
}

// The bits of a magnitude: ordered as the magnitudes are, infinity and NaN above all.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The values of four codes.  A code plus 128 is put into the low byte of 2^23, whose
// neighbours are 1 apart: the float32 2^23 + 128 + code, without a conversion.
__device__ __forceinline__ float2 code_pair(uint32_t flipped, int j)
{
    return __fadd2_rn(make_float2(__uint_as_float(__byte_perm(flipped, 0x4B000000u, 0x7540 + j)),
                                  __uint_as_float(__byte_perm(flipped, 0x4B000000u, 0x7541 + j))),
                      both(-8388736.0f));
}
__device__ __forceinline__ void values4(uint32_t codes, float scale, float *v)
{
#pragma unroll
    for (int j = 0; j < 4; j += 2) set_pair(v + j, __fmul2_rn(code_pair(codes ^ 0x80808080u, j), both(scale)));
}
__device__ __forceinline__ void values8(uint2 codes, float scale, float (&v)[8])
{
    values4(codes.x, scale, v);
    values4(codes.y, scale, v + 4);
}

// i / d for i < 2^64 / d, as a product with a rounded-up 2^64 / d.
struct Divider {
    uint64_t magic = 0;
    uint32_t d = 1;
    Divider() = default;
    explicit Divider(uint32_t by) : magic(by > 1 ? ~uint64_t(0) / by + 1 : 0), d(by) {}
    __device__ __forceinline__ int64_t quotient(int64_t i) const { return d > 1 ? (int64_t)__umul64hi((uint64_t)i, magic) : i; }
};

// Columns col .. col + 7 of a row of the given width, as they lie in memory (zeros behind the
// width): 16-byte loads of the lines that hold them, shifted into place where VEC does not
// say that rows are aligned to 16 bytes.  Bytes beside the row are read where they share
// 16 aligned bytes with one of its elements, and not used.
template <typename T, bool VEC>
struct Eight {
    static constexpr int W = 2 * sizeof(T);            // words of eight elements
    static constexpr int LINES = VEC ? W / 4 : W / 4 + 1;
    uint4 line[LINES];

    __device__ __forceinline__ void load(const T *row, int col, int width)
    {
        const uintptr_t p = reinterpret_cast<uintptr_t>(row + col), base = p & ~(uintptr_t)15;
        const int n = width - col < 8 ? width - col : 8, end = (int)(p - base) + n * (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < LINES; ++i)
            line[i] = n > 0 && 16 * i < end ? *reinterpret_cast<const uint4 *>(base + 16 * i) : make_uint4(0, 0, 0, 0);
    }
    // The elements' own bits.
    __device__ __forceinline__ void words(const T *row, int col, int width, uint32_t (&out)[W]) const
    {
        uint32_t w[4 * LINES];
#pragma unroll
        for (int i = 0; i < LINES; ++i) w[4 * i] = line[i].x, w[4 * i + 1] = line[i].y, w[4 * i + 2] = line[i].z, w[4 * i + 3] = line[i].w;
        if constexpr (!VEC) {
            const uint32_t s = (uint32_t)reinterpret_cast<uintptr_t>(row + col);
#pragma unroll
            for (int i = 0; i < W + 2; ++i) w[i] = s & 8 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < W + 1; ++i) w[i] = s & 4 ? w[i + 1] : w[i];
            if (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < W; ++i) w[i] = s & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
            }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) out[i] = w[i];
        if (col > width - 8) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                constexpr int E = 8 / W;  // elements of a word
                const int left = width - col - i * E;
                out[i] = left >= E ? out[i] : left == 1 && E == 2 ? out[i] & 0xFFFFu : 0u;
            }
        }
    }
    static __device__ __forceinline__ void floats(const uint32_t (&w)[W], float (&v)[8])
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                T pair[2];
                memcpy(pair, &w[j], 4);
                set_pair(v + 2 * j, pair_of(pair));
            }
        }
    }
    // The largest magnitude's bits, as of a float32.
    static __device__ __forceinline__ uint32_t magnitude(const uint32_t (&w)[W])
    {
        uint32_t m = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, w[j] & 0x7FFFFFFFu);
            return m;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
            m = max(m & 0xFFFFu, m >> 16);
            const uint16_t h = (uint16_t)m;
            T e;
            memcpy(&e, &h, 2);
            return __float_as_uint(to_f32(e));
        }
    }
    __device__ __forceinline__ void get(const T *row, int col, int width, float (&v)[8]) const
    {
        uint32_t w[W];
        words(row, col, width, w);
        floats(w, v);
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *row, int col, int width, const float (&v)[8])
{
    if (VEC && col <= width - 8) {
        Pack<T, 8> k;
#pragma unroll
        for (int j = 0; j < 8; j += 2) set_pair(k.v + j, make_float2(v[j], v[j + 1]));
        store_pack<T, 8>(row + col, k);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < width) row[col + j] = from_f32<T>(v[j]);
    }
}

}  // namespace hiss
