// Gated feed-forward block and its gradient: matrix products on the tensor cores
// (tcgen05, pairs of CTAs) whose epilogues do everything between them.
//
// Forward: one product of x with gate and up side by side, whose epilogue makes
// h = act(a) * b (and a and b in 8 bits, or in float32); y = h down^T.
// Backward: dh = dy down, whose epilogue reads a and b and makes da, db and h;
// dx = [da db] [gate; up]; the three weights' gradients in one launch.
//
// Operands are 16-bit.  A float32 operand goes through as three bfloat16 planes
// p1 + p2 + p3 = x (8 bits each, exact), and a product of two as the six products of
// planes above 2^-22 of it: p1 q1 in one accumulator, p1 q2 + p2 q1 + p2 q2 + p1 q3 + p3 q1 in
// another, which the epilogue adds to float32 registers every 128 K elements.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <initializer_list>

#include "hiss_internal.cuh"
#include "packed.cuh"

namespace hiss {
namespace {

// ---- the product kernel ------------------------------------------------------------------

constexpr int kBlockM = 256;       // rows of a tile: 128 in each CTA of the pair
constexpr int kBlockK = 64;        // K elements of a stage: rows of 128 bytes
constexpr int kEpilogueWarps = 8;
// Warps 8 and 9: copies, matrix instructions; 10 and 11 are there for the split of the registers alone,
// which goes by groups of four warps.
constexpr int kThreads = (kEpilogueWarps + 4) * 32;
constexpr int kPairs = kSMs / 2;
constexpr int kMaxProblems = 3;
constexpr int kBarrierBytes = 1024;
constexpr int kGroupM = 8;         // tiles run down a group of this many tile rows before the next column

// What an epilogue does with a tile; kGradLong: kGrad over a long K.
enum { kOut = 0, kGated = 1, kGrad = 2, kGradLong = 3 };
template <int EP>
constexpr bool kMiddle = EP == kGrad || EP == kGradLong;

// K blocks that a tile's accumulator i takes in before it is added to float32 registers.  The tensor cores
// cut a sum towards zero at every step of 16 columns, up to 2^-23 of it: one accumulator for all of K is
// off by 9e-10 per column in a and b, always to the same side of a sum that grows, so that codes that are
// kept and signs that relu's derivative takes come out wrong.
//   Three planes: 2.  8192 x 256 through 1024 is 8.7e-7 off the exact value with 4 (61 us), 5.2e-7 with 2 (62),
//   3.6e-7 with 1 (63); float32 sums of plain products are 7.2e-7 off.
//   a and b: 4, but 8 in the two accumulators that the next tile fills beside this tile's epilogue.  4096 columns:
//   bfloat16 are 3.3e-7 of the terms' 2-norm off so, 3.5e-6 with one accumulator (4.0e-7 in a library's float32
//   product).  8192 x 2048 by 2 x 5632, kept in 8 bits: 253 us, 246 with one accumulator, 306 with 4 from the
//   start, 248 with 8 throughout.
//   Others round what they add up, or their terms, to 16 bits: 16 blocks lose up to 2^-18 of a sum of one sign, a
//   128th of float16's half step.  dh up to 4096 columns: all, 2^-16, since sums in registers cost its
//   epilogue (4104 columns of 8192 x 2048: 145 us, 129 in one accumulator).
template <int EP, int P>
__host__ __device__ constexpr int fold_blocks(int i)
{
    return P == 3 ? 2 : EP == kGated ? (i < 2 ? 8 : 4) : EP == kGrad ? 64 : 16;
}

// Registers: an epilogue thread has 128 sums, the issuing warps need few (more with three problems).  Of
// 3 x 168 the last group of warps leaves the rest to the other two.
constexpr int kLaunchRegs = 168;  // of each kernel as it is launched
template <int EP>
constexpr int kIssueRegs = EP == kOut ? 88 : 56;
template <int EP>
constexpr int kEpilogueRegs = (3 * kLaunchRegs - kIssueRegs<EP>) / 2;
static_assert(kEpilogueRegs<kOut> % 8 == 0 && kEpilogueRegs<kGated> % 8 == 0, "whole units");

template <int P>
__host__ __device__ constexpr int stage_bytes(int bn) { return P * (128 + bn / 2) * 2 * kBlockK; }
// Room of an epilogue warp for elements on their way out, in slots of 32 rows: of 32 columns (16-bit),
// three where a result has three planes, else two; where da, db and h leave together, two times
// three of 32 columns, or nine of 16 columns.
constexpr int kSlotBytes = 2048;
template <int P>
constexpr int kGradCols = P == 3 ? 16 : 32;
template <int EP, int P>
constexpr int kSlots = P == 3 ? 3 : 2;
template <int EP, int P>
constexpr int kRoomBytes = kMiddle<EP> ? (P == 3 ? 9 * 1024 : 6 * kSlotBytes) : kSlots<EP, P> * kSlotBytes;
template <int EP, int P>
__host__ __device__ constexpr int stages(int bn)
{
    return (227 * 1024 - kBarrierBytes - 1024 - kEpilogueWarps * kRoomBytes<EP, P>) / stage_bytes<P>(bn);
}
static_assert(stages<kOut, 1>(256) == 6 && stages<kGated, 1>(256) == 6 && stages<kGrad, 1>(256) == 4, "16-bit");
static_assert(stages<kOut, 3>(128) == 2 && stages<kGated, 3>(128) == 2 && stages<kGrad, 3>(128) == 2, "three planes");

// One product D[m][n] = sum over its segments of A B^T, cut into tiles.
struct Problem {
    CUtensorMap a[2], b[2];  // by segment; b by CTA where dual
    CUtensorMap to;          // out, or its partial sums [splits][m][n], where copies can store to it
    int64_t m, n;
    void *out;
    int64_t out_stride;
    int tiles_m, tiles_n;
    int first;               // its first tile
    int by_copy;             // `to` is there
};

struct Args {
    Problem p[kMaxProblems];
    int problems, tiles;
    int blocks[2];           // K blocks of the segments
    int splits, per_split;   // K blocks are cut into `splits` ranges of per_split
    int bn;                  // columns of a tile
    int a_m_major, b_n_major;
    int dual;                // columns bn / 2 .. of a tile are those of the second b at the same place
    int bf16;                // operands: bfloat16, else float16
    // epilogues of the hidden columns
    int act;
    CUtensorMap h, da, db;   // planes [P][m][n]
    float *raw;              // a and b in float32 (see raw_block): written by kGated, read by kGrad
    hiss_packed kept[2];     // written by kGated, read by kGrad
    int keeps;
    int *bad;                // set to 1 when a wait ran out
};

// 2^x and 1 / x as the hardware approximates them (2^-22 and 2^-23), subnormal results as 0.
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float inverse_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float2 exp2_fast(float2 x) { return make_float2(exp2_fast(x.x), exp2_fast(x.y)); }
__device__ __forceinline__ float2 inverse_fast(float2 x) { return make_float2(inverse_fast(x.x), inverse_fast(x.y)); }

constexpr float kLog2E = 1.44269504f;

// The normal distribution's function at -u, u >= 0, over exp(-u^2 / 2): a polynomial in
// t = 1 / (1 + 0.3 u), fitted for the smallest largest relative error over [0, 14.5] by least squares whose
// weights grow with the error (4e-7 in float32 arithmetic; FAST, of two degrees less, 2.2e-6).
template <bool FAST>
__device__ __forceinline__ float2 normal_tail(float2 u)
{
    const float2 t = inverse_fast(__ffma2_rn(both(0.3f), u, both(1.0f)));
    float2 r;
    auto next = [&](float c) { r = __ffma2_rn(r, t, both(c)); };
    if (FAST) {
        r = both(-8.460762352e-02f);
        next(2.406236082e-01f);
        next(-4.871572927e-02f);
        next(1.648150384e-01f);
        next(1.066855714e-01f);
        next(1.212782413e-01f);
        next(-8.004470146e-05f);
    } else {
        r = both(3.840760142e-02f);
        next(-1.693084240e-01f);
        next(2.289536446e-01f);
        next(-7.684164494e-02f);
        next(1.427665353e-01f);
        next(9.458538145e-02f);
        next(1.219453737e-01f);
        next(1.194841936e-01f);
        next(7.373073458e-06f);
    }
    return r;
}

// The activation and its derivative, of two at a time.  FAST, where the result goes into 16 bits: the
// fast exponential (relative error (|x| + 2) 2^-23) and inverse are far below its rounding.  The
// normal density takes them everywhere: where the error counts, the density does not.
struct Activated {
    float2 value, slope;
};
template <bool FAST, int ACT>
__device__ __forceinline__ Activated activate(float2 a)
{
    if (ACT == HISS_RELU)
        return {make_float2(a.x <= 0.0f ? 0.0f : a.x, a.y <= 0.0f ? 0.0f : a.y), make_float2(a.x > 0.0f ? 1.0f : 0.0f, a.y > 0.0f ? 1.0f : 0.0f)};
    if (ACT == HISS_GELU) {
        const float2 e = exp2_fast(__fmul2_rn(__fmul2_rn(a, both(-0.5f * kLog2E)), a));
        const float2 q = __fmul2_rn(e, normal_tail<FAST>(make_float2(fabsf(a.x), fabsf(a.y))));
        const float2 o = __ffma2_rn(q, both(-1.0f), both(1.0f)), p = make_float2(a.x > 0.0f ? o.x : q.x, a.y > 0.0f ? o.y : q.y);
        return {__fmul2_rn(a, p), __ffma2_rn(__fmul2_rn(a, both(0.39894228f)), e, p)};
    }
    const float2 e = FAST ? exp2_fast(__fmul2_rn(a, both(-kLog2E))) : make_float2(expf(-a.x), expf(-a.y));
    const float2 s = FAST ? inverse_fast(__fadd2_rn(e, both(1.0f))) : make_float2(1.0f / (1.0f + e.x), 1.0f / (1.0f + e.y));
    // 1 - s: above 0 the difference cancels (6% off at 16), e s does not
    const float2 left = __ffma2_rn(s, both(-1.0f), both(1.0f)), es = __fmul2_rn(e, s);
    const float2 o = make_float2(a.x > 0.0f ? es.x : left.x, a.y > 0.0f ? es.y : left.y);
    if (ACT == HISS_SIGMOID) return {s, __fmul2_rn(s, o)};
    return {__fmul2_rn(a, s), __fmul2_rn(s, __ffma2_rn(a, o, both(1.0f)))};
}
// f with the activation as a constant: one branch for a row's piece.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F &&f)
{
    if (act == HISS_SILU) f(std::integral_constant<int, HISS_SILU>{});
    else if (act == HISS_GELU) f(std::integral_constant<int, HISS_GELU>{});
    else if (act == HISS_RELU) f(std::integral_constant<int, HISS_RELU>{});
    else f(std::integral_constant<int, HISS_SIGMOID>{});
}

// The three parts of two float32, as pairs of bfloat16: each part is the leading 8 bits
// of what the ones before it left, so the three add up to the number exactly.  (An
// infinity leaves a NaN.)
__device__ __forceinline__ void split3(float x, float y, uint32_t (&w)[3])
{
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        const uint32_t i = __float_as_uint(x), j = __float_as_uint(y);
        w[q] = __byte_perm(i, j, 0x7632);
        if (q < 2) {
            const float2 left = __fadd2_rn(make_float2(x, y), make_float2(__uint_as_float((i & 0xFFFF0000u) ^ 0x80000000u),
                                                                          __uint_as_float((j & 0xFFFF0000u) ^ 0x80000000u)));
            x = left.x;
            y = left.y;
        }
    }
}

// Where a warp's 32 x 32 values leave the chip: each lane has a row of 32 columns, puts it
// into the warp's slots (swizzled as the tensor maps are, so that eight lanes' 16-byte
// pieces lie in different banks), and one lane starts the copy, which runs beside what follows.
struct Slots {
    uint32_t base;
    int lane;
    int next = 0;

    // N slots that no copy reads any more
    template <int N, int ALL>
    __device__ uint32_t take()
    {
        static_assert(N <= ALL && (N == 1 || N == ALL || N == 2), "slots");
        // one group per take: the groups behind the first ALL / N are still reading other slots
        if (lane == 0) store_wait_read<ALL / N - 1>();
        __syncwarp();
        const uint32_t at = base + next * kSlotBytes;
        next = next + N + N > ALL ? 0 : next + N;
        return at;
    }
    __device__ void ready() const
    {
        fence_proxy_async_smem();
        __syncwarp();
    }
};

// Piece j (16 bytes) of lane r's row of 32, 64 or 128 bytes.
__device__ __forceinline__ uint32_t piece32(uint32_t slot, int r, int j) { return slot + r * 32 + ((j ^ (r >> 2)) & 1) * 16; }
__device__ __forceinline__ uint32_t piece64(uint32_t slot, int r, int j) { return slot + r * 64 + ((j ^ (r >> 1)) & 3) * 16; }
__device__ __forceinline__ uint32_t piece128(uint32_t slot, int r, int j) { return slot + r * 128 + ((j ^ r) & 7) * 16; }

__device__ __forceinline__ uint32_t pack2(float x, float y, bool bf16)
{
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void put16(uint32_t slot, int lane, const float (&v)[32], bool bf16)
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sts16(piece64(slot, lane, j), pack2(v[8 * j], v[8 * j + 1], bf16), pack2(v[8 * j + 2], v[8 * j + 3], bf16),
              pack2(v[8 * j + 4], v[8 * j + 5], bf16), pack2(v[8 * j + 6], v[8 * j + 7], bf16));
}
__device__ __forceinline__ void put32(uint32_t slot, int lane, const float (&v)[32])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sts16(piece128(slot, lane, j), __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
              __float_as_uint(v[4 * j + 3]));
}

// Into the operand of a later product; row and col are the warp's first.
template <int EP, int P>
__device__ __forceinline__ void store_planes(Slots &s, const Args &a, const CUtensorMap &to, int64_t row, int64_t col,
                                             const float (&v)[32])
{
    const uint32_t at = s.take<P, kSlots<EP, P>>();
    if constexpr (P == 1) {
        put16(at, s.lane, v, a.bf16);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4][3];
#pragma unroll
            for (int e = 0; e < 4; ++e) split3(v[8 * j + 2 * e], v[8 * j + 2 * e + 1], w[e]);
#pragma unroll
            for (int q = 0; q < 3; ++q) sts16(piece64(at + q * kSlotBytes, s.lane, j), w[0][q], w[1][q], w[2][q], w[3][q]);
        }
    }
    s.ready();
    if (s.lane == 0) {
        tma_store(&to, at, (int)col, (int)row, 0);  // every plane
        store_commit();
    }
}

// To a product's result: `split` is that of its partial sums, or 0.
template <int EP, int P>
__device__ __forceinline__ void store_out(Slots &s, const Args &a, const Problem &p, int64_t row, int64_t col, int split,
                                          const float (&v)[32])
{
    const bool wide = a.splits > 1 || P == 3;
    uint32_t at;
    if (wide) {
        at = s.take<2, 2>();
        put32(at, s.lane, v);
    } else {
        at = s.take<1, 2>();
        put16(at, s.lane, v, a.bf16);
    }
    if (p.by_copy) {
        s.ready();
        if (s.lane == 0) {
            tma_store(&p.to, at, (int)col, (int)row, split);
            store_commit();
        }
        return;
    }
    // rows that copies cannot store to: row by row, a lane per column
    __syncwarp();
    const int rows = (int)min((int64_t)32, p.m - row);
    if (col + s.lane < p.n) {
        if (wide) {
            float *to = static_cast<float *>(p.out) + row * p.out_stride + col + s.lane;
            for (int r = 0; r < rows; ++r, to += p.out_stride)
                *to = __uint_as_float(lds32(piece128(at, r, s.lane >> 2) + (s.lane & 3) * 4));
        } else {
            uint16_t *to = static_cast<uint16_t *>(p.out) + row * p.out_stride + col + s.lane;
            for (int r = 0; r < rows; ++r, to += p.out_stride) *to = (uint16_t)lds16(piece64(at, r, s.lane >> 3) + (s.lane & 7) * 2);
        }
    }
    __syncwarp();
}

// a and b in float32 between kGated and kGrad: blocks of 32 rows and 32 columns in the
// order in which a warp has them, a 16-byte piece of every lane's row after the other.
__device__ __forceinline__ float4 *raw_block(const Args &a, const Problem &p, int64_t row, int64_t col, int which, int lane)
{
    const int64_t blocks = (p.n + 31) / 32;
    return reinterpret_cast<float4 *>(a.raw) + (((row >> 5) * blocks + (col >> 5)) * 2 + which) * 256 + lane;
}

// One row's block of 32 columns in 8 bits (columns beyond the width are zeros).
__device__ __forceinline__ void keep32(const hiss_packed &p, int64_t row, int64_t col, int64_t width, float (&v)[32])
{
    const int64_t blocks = (width + 31) / 32, at = row * blocks + col / 32;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) m = max(m, magnitude(v[j]));  // zeros behind the width, as the weights' rows are there
    const uint32_t byte = scale_byte(m);
    uint32_t w[8];
    codes_of(v, byte, top_byte<float>(), w);
    auto *q = reinterpret_cast<uint4 *>(p.codes + at * 32);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    p.scales[at] = (uint8_t)byte;
}
// The same of a and b, loaded ahead.
struct Kept {
    uint4 a[2], b[2];
    uint32_t sa, sb;
    __device__ __forceinline__ void load(const Args &args, const Problem &p, int64_t row, int64_t col)
    {
        if (row >= p.m || col >= p.n) return;
        const int64_t at = row * ((p.n + 31) / 32) + col / 32;
        const auto *qa = reinterpret_cast<const uint4 *>(args.kept[0].codes + at * 32), *qb = reinterpret_cast<const uint4 *>(args.kept[1].codes + at * 32);
        a[0] = qa[0], a[1] = qa[1], b[0] = qb[0], b[1] = qb[1];
        sa = args.kept[0].scales[at];
        sb = args.kept[1].scales[at];
    }
    static __device__ __forceinline__ void get(const uint4 (&q)[2], uint32_t byte, float (&v)[32])
    {
        const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
        const float s = scale_of(byte);
#pragma unroll
        for (int j = 0; j < 8; ++j) values4(w[j], s, v + 4 * j);
    }
};

// Keeps the compiler from mixing the arithmetic of a row's pieces, which would take more
// registers than there are.
__device__ __forceinline__ void pieces_apart() { asm volatile("" ::: "memory"); }

// Epilogue of 32 columns of a warp's 32 rows; row and col are the first, within the result.
// v: the sums (a where gated), u: b where gated.
template <int EP, int P>
__device__ __forceinline__ void emit(Slots &s, const Args &a, const Problem &p, int split, int64_t row, int64_t col, float (&v)[32],
                                     float (&u)[32])
{
    if constexpr (EP == kOut) {
        store_out<EP, P>(s, a, p, row, col, split, v);
    } else {
        if (a.raw) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float4 *to = raw_block(a, p, row, col, w, s.lane);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    to[32 * j] = w ? make_float4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3])
                                   : make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
            return;
        }
        if (a.keeps && row + s.lane < p.m) {
            keep32(a.kept[0], row + s.lane, col, p.n, v);
            keep32(a.kept[1], row + s.lane, col, p.n, u);
        }
        with_activation(a.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                set_pair(u + j, __fmul2_rn(activate<P == 1, decltype(act)::value>(pair_of(v + j)).value, pair_of(u + j)));
                if (j % 8 == 6) pieces_apart();
            }
        });
        store_planes<EP, P>(s, a, a.h, row, col, u);
    }
}

// da, db and h from dh (v) and a and b (from `kept`, or as float32): COLS columns at a time leave
// in one group of copies.  (Coalesced 16-byte stores of the slots instead took 317 us for 309 on
// 16,384 x 5632 bfloat16, and 105 for 88 on 8192 x 1024 float32.)
template <int P>
__device__ __forceinline__ void emit_grad(Slots &s, const Args &a, const Problem &p, int64_t row, int64_t col, const float (&v)[32],
                                          const Kept &kept)
{
    constexpr int COLS = kGradCols<P>;
    float x[32], b[32];
    if (a.keeps) {
        Kept::get(kept.a, kept.sa, x);
        Kept::get(kept.b, kept.sb, b);
    } else {
        const float4 *fa = raw_block(a, p, row, col, 0, s.lane), *fb = raw_block(a, p, row, col, 1, s.lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 q = fa[32 * j], r = fb[32 * j];
            x[4 * j] = q.x, x[4 * j + 1] = q.y, x[4 * j + 2] = q.z, x[4 * j + 3] = q.w;
            b[4 * j] = r.x, b[4 * j + 1] = r.y, b[4 * j + 2] = r.z, b[4 * j + 3] = r.w;
        }
    }
    with_activation(a.act, [&](auto act) {
#pragma unroll
        for (int c = 0; c < 32; c += COLS) {
            if (s.lane == 0) store_wait_read<P == 1 ? 1 : 0>();
            __syncwarp();
            const uint32_t at = s.base + s.next * 3 * kSlotBytes;
            if (P == 1) s.next ^= 1;
#pragma unroll
            for (int j = 0; j < COLS / 8; ++j) {
                float da[8], db[8], h[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const int k = c + 8 * j + e;
                    const Activated f = activate<P == 1, decltype(act)::value>(pair_of(x + k));
                    const float2 d = pair_of(v + k), u = pair_of(b + k);
                    set_pair(h + e, __fmul2_rn(f.value, u));
                    set_pair(da + e, __fmul2_rn(__fmul2_rn(d, u), f.slope));
                    set_pair(db + e, __fmul2_rn(d, f.value));
                }
                auto put = [&](int which, const float(&r)[8]) {
                    if constexpr (P == 1) {
                        sts16(piece64(at + which * kSlotBytes, s.lane, j), pack2(r[0], r[1], a.bf16), pack2(r[2], r[3], a.bf16),
                              pack2(r[4], r[5], a.bf16), pack2(r[6], r[7], a.bf16));
                    } else {
                        uint32_t w[4][3];
#pragma unroll
                        for (int e = 0; e < 4; ++e) split3(r[2 * e], r[2 * e + 1], w[e]);
#pragma unroll
                        for (int q = 0; q < 3; ++q)
                            sts16(piece32(at + (which * 3 + q) * 1024, s.lane, j), w[0][q], w[1][q], w[2][q], w[3][q]);
                    }
                };
                put(0, da);
                put(1, db);
                put(2, h);
            }
            s.ready();
            if (s.lane == 0 && col + c < p.n) {
                constexpr uint32_t kMatrix = P * (P == 1 ? kSlotBytes : 1024);
                tma_store(&a.da, at, (int)col + c, (int)row, 0);
                tma_store(&a.db, at + kMatrix, (int)col + c, (int)row, 0);
                tma_store(&a.h, at + 2 * kMatrix, (int)col + c, (int)row, 0);
                store_commit();
            }
        }
    });
}

// A unit of work: one tile of one problem and one range of K blocks.
struct Unit {
    int problem, k0, k1, split;
    int64_t tm, tn;
    __device__ Unit(const Args &a, int u)
    {
        const int tile = u / a.splits;
        split = u - tile * a.splits;
        problem = 0;
        while (problem + 1 < a.problems && tile >= a.p[problem + 1].first) ++problem;
        const Problem &p = a.p[problem];
        const int t = tile - p.first, group = t / (kGroupM * p.tiles_n), in = t - group * kGroupM * p.tiles_n;
        const int rows = min(kGroupM, p.tiles_m - group * kGroupM);
        tm = group * kGroupM + in % rows;
        tn = in / rows;
        k0 = split * a.per_split;
        k1 = min(k0 + a.per_split, a.blocks[0] + a.blocks[1]);
    }
};

// Products on 256 x 256 tiles (256 x 128 of float32's planes) by pairs of CTAs, which share B: each
// copies 128 rows of A and half of B's, so a stage of 64 columns is 32 KB a CTA for 512 cycles of
// matrix instructions.  One CTA per SM and 128 x 256 would copy 48 KB for them, above the 64 bytes a
// cycle that L2 gives an SM.  A CTA's warps: eight of the epilogue, one that copies (6 stages; 4 where
// da, db and h leave; 2 of three planes), one that issues.  Two accumulators of
// 256 columns fill tensor memory, so a tile's epilogue runs beside the next one's products.
// Persistent: 76 pairs take the tiles in groups of 8 tile rows (4, 16 and 32: within 1%).
//
// 32,768 x 2048 bfloat16 through 5632: gate and up 0.94 ms (1.61 PFLOP/s), down 0.46 ms (1.64);
// tensor pipe 68 and 72% busy, and the library's best on this GPU is 1.9.  What bounds it: matrix
// instructions and, next to them, the copies (45 bytes a cycle and SM).  Float32, 8192 x 256 by 2 x
// 1024: 41 us, 27 of them the six products' at the library's rate; its backward middle (three results of three planes
// for each sum) 66 to 70 us, bound by the epilogue.
template <int EP, int P>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_product(const __grid_constant__ Args a)
{
    extern __shared__ __align__(1024) unsigned char raw_smem[];
    // barriers, then the stages on a 1024-byte boundary
    uint64_t *full = reinterpret_cast<uint64_t *>(raw_smem), *empty = full + 16, *acc_full = empty + 16, *acc_empty = acc_full + 2;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(acc_empty + 2);
    volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
    const uint32_t stage0 = (smem_u32(raw_smem) + kBarrierBytes + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int ns = stages<EP, P>(a.bn);
    constexpr uint32_t kRowBytes = 2 * kBlockK, kBoxBytes = kBlockK * 128;  // of K-major rows; of 64 M-major columns
    const uint32_t a_bytes = P * 128 * kRowBytes, per_stage = stage_bytes<P>(a.bn);
    const int units = a.tiles * a.splits, first = blockIdx.x / 2, step = gridDim.x / 2;
    if (tid == 0) {
        for (int i = 0; i < ns; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kEpilogueWarps);
        }
        *s_abort = 0;
        fence_mbar_init();
    }
    let_next_start();
    if (warp == kEpilogueWarps) tmem_alloc_pair(s_tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem = *s_tmem;
    wait_for_previous();
    auto give_up = [&]() {
        *s_abort = 1;
        atomicExch(a.bad, 1);
    };

    if (warp >= kEpilogueWarps) {
        fewer_registers<kIssueRegs<EP>>();
        if (warp == kEpilogueWarps) {
            // ---- copies: this CTA's rows of A and of B, into barriers of the first CTA ----
            if (lane == 0) {
                int s = 0;
                uint32_t phase = 1;
                for (int u = first; u < units && !*s_abort; u += step) {
                    const Unit w(a, u);
                    const Problem &p = a.p[w.problem];
                    const int row = (int)(w.tm * kBlockM + rank * 128);
                    const int col = (int)(a.dual ? w.tn * (a.bn / 2) : w.tn * a.bn + rank * (a.bn / 2));
                    for (int k = w.k0; k < w.k1; ++k) {
                        if (!mbar_wait(&empty[s], phase, s_abort)) {
                            give_up();
                            break;
                        }
                        if (rank == 0) mbar_expect_tx(&full[s], 2 * per_stage);
                        const int seg = k >= a.blocks[0], kk = (k - (seg ? a.blocks[0] : 0)) * kBlockK;
                        const CUtensorMap *ma = &p.a[seg], *mb = &p.b[a.dual ? rank : seg];
                        const uint32_t bar = smem_in_cta(&full[s], 0);
                        uint32_t at = stage0 + s * per_stage;
                        // every plane in one copy: a copy's start takes the thread over 100 cycles
                        if (a.a_m_major) {
                            tma_load_pair(at, ma, bar, row, kk, 0);
                            tma_load_pair(at + P * kBoxBytes, ma, bar, row + 64, kk, 0);
                        } else {
                            tma_load_pair(at, ma, bar, kk, row, 0);
                        }
                        at += a_bytes;
                        if (a.b_n_major)
                            for (int j = 0; j < a.bn / 2; j += 64, at += P * kBoxBytes) tma_load_pair(at, mb, bar, col + j, kk, 0);
                        else
                            tma_load_pair(at, mb, bar, kk, col, 0);
                        if (++s == ns) s = 0, phase ^= 1;
                    }
                }
                // the first CTA's last signals to this CTA's barriers have to arrive before it ends
                for (int i = 0; i < ns && !*s_abort; ++i) {
                    if (!mbar_wait(&empty[s], phase, s_abort)) give_up();
                    if (++s == ns) s = 0, phase ^= 1;
                }
            }
        } else if (warp == kEpilogueWarps + 1) {
            // ---- matrix instructions, by one thread of the first CTA for both ----
            if (lane == 0 && rank == 0) {
                const uint32_t idesc = idesc_f16(a.bf16, a.a_m_major, a.b_n_major, kBlockM, a.bn);
                // 16 K elements: 32 bytes within the rows, or 16 rows
                const uint32_t a_step = a.a_m_major ? 16 * 128 / 16 : 2, b_step = a.b_n_major ? 16 * 128 / 16 : 2;
                const uint32_t a_plane = (a.a_m_major ? kBoxBytes : 128 * kRowBytes) / 16;
                const uint32_t b_plane = (a.b_n_major ? kBoxBytes : a.bn / 2 * kRowBytes) / 16;
                int s = 0, acc = 0;
                uint32_t phase = 0, acc_phase = 1;
                for (int u = first; u < units && !*s_abort; u += step) {
                    const Unit w(a, u);
                    int in_fold = 0, folds = 0;  // blocks in this accumulator, accumulators before it
                    for (int k = w.k0; k < w.k1; ++k) {
                        if (in_fold == 0) {
                            if (!mbar_wait(&acc_empty[acc], acc_phase, s_abort)) {
                                give_up();
                                break;
                            }
                            tc_fence_after_sync();
                        }
                        if (!mbar_wait(&full[s], phase, s_abort)) {
                            give_up();
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t base = stage0 + s * per_stage;
                        const uint64_t ad = smem_desc_sw128(base, P * kBoxBytes), bd = smem_desc_sw128(base + a_bytes, P * kBoxBytes);
                        const uint32_t d = tmem + acc * 256;
#pragma unroll
                        for (int j = 0; j < kBlockK / 16; ++j) {
                            if constexpr (P == 1) {
                                mma_f16_pair(d, ad + j * a_step, bd + j * b_step, idesc, in_fold + j > 0);
                            } else {
                                const uint32_t cross = d + 128;
                                auto product = [&](uint32_t to, int pa, int pb, bool add) {
                                    mma_f16_pair(to, ad + j * a_step + pa * a_plane, bd + j * b_step + pb * b_plane, idesc, add);
                                };
                                const bool more = in_fold + j > 0;
                                product(d, 0, 0, more);
                                product(cross, 0, 1, more);
                                product(cross, 0, 2, true);
                                product(cross, 1, 0, true);
                                product(cross, 1, 1, true);
                                product(cross, 2, 0, true);
                            }
                        }
                        mma_commit_pair(&empty[s]);
                        if (++s == ns) s = 0, phase ^= 1;
                        if (++in_fold == fold_blocks<EP, P>(folds) || k == w.k1 - 1) {
                            mma_commit_pair(&acc_full[acc]);
                            acc ^= 1;
                            if (acc == 0) acc_phase ^= 1;
                            in_fold = 0;
                            ++folds;
                        }
                    }
                }
            }
        }
    } else {
        more_registers<kEpilogueRegs<EP>>();
        // ---- epilogue: warp w reads lanes 32 (w % 4) .. of this CTA's rows, columns by halves ----
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        Slots slots{stage0 + ns * per_stage + warp * kRoomBytes<EP, P>, lane};
        int acc = 0;
        uint32_t phase = 0;
        auto release = [&](int i) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(smem_in_cta(&acc_empty[i], 0));
        };
        auto arrived = [&](int i, uint32_t ph) {
            const bool ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[i], ph, s_abort));
            tc_fence_after_sync();
            return ok;
        };
        for (int u = first; u < units && !*s_abort; u += step) {
            const Unit w(a, u);
            const Problem &p = a.p[w.problem];
            const int64_t row = w.tm * kBlockM + rank * 128 + quarter * 32;
            const int cols = EP == kGated ? a.bn / 2 : a.bn;  // of the output
            const int64_t col0 = w.tn * cols + half * (cols / 2);
            Kept kept;
            if (kMiddle<EP> && a.keeps) kept.load(a, p, row + lane, col0);
            // 128 columns of an accumulator, in groups of 32: of a and of b where gated, main and cross products
            // of either group with three planes
            constexpr int G = P == 3 ? 2 : 4, kGroups = EP == kGated ? G / 2 : G;  // of the output
            auto load = [&](int g, float(&v)[32]) {
                const int at = P == 3 ? (g & 1) * 128 + (EP == kGated ? (g >> 1) * 64 + half * 32 : half * 64 + (g >> 1) * 32)
                                      : (EP == kGated ? (g >> 1) * 128 + half * 64 + (g & 1) * 32 : half * 128 + g * 32);
                tmem_ld32(lanes + acc * 256 + at, reinterpret_cast<uint32_t(&)[32]>(v));
                tmem_ld_wait();
            };
            auto add = [](float(&to)[32], const float(&v)[32]) {
#pragma unroll
                for (int j = 0; j < 32; j += 2) set_pair(to + j, __fadd2_rn(pair_of(to + j), pair_of(v + j)));
            };
            auto done = [&]() {
                release(acc);
                acc ^= 1;
                if (acc == 0) phase ^= 1;
            };
            // The last sums leave as they come from tensor memory (kDirect).  The gated ones, whose accumulators are
            // short, are taken first: the products go on in both accumulators then.
            constexpr bool kDirect = P == 1 && EP != kGated, kSums = P == 3 || EP != kGrad;
            float sum[G][32];
            if constexpr (kSums) {
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[g][j] = 0.0f;
            }
            bool ok = true;
            int k = w.k0;
            for (int i = 0; kSums && k + (kDirect ? fold_blocks<EP, P>(i) : 0) < w.k1; k += fold_blocks<EP, P>(i++)) {
                ok = arrived(acc, phase);
                if (!ok) break;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float v[32];
                    load(g, v);
                    add(sum[P == 3 ? g >> 1 : g], v);
                }
                done();
            }
            if (kDirect && ok) ok = arrived(acc, phase);
            if (!ok) {
                give_up();
                break;
            }
            // kGrad's long code once: for four groups, with sums, it took 70 us for 54 on 16,384 x 1024
#pragma unroll(P == 1 && kMiddle<EP> ? 1 : kGroups)
            for (int g = 0; g < kGroups; ++g) {
                const int64_t col = col0 + 32 * g;
                const bool there = row < p.m && col < p.n;
                if constexpr (!kDirect) {
                    if (!there) break;
                    if constexpr (kMiddle<EP>) {
                        if (g && a.keeps) kept.load(a, p, row + lane, col);
                        emit_grad<P>(slots, a, p, row, col, sum[g], kept);
                    } else {
                        emit<EP, P>(slots, a, p, w.split, row, col, sum[g], sum[EP == kGated ? kGroups + g : g]);
                    }
                } else {
                    float v[32];
                    load(g, v);
                    if (g + 1 == kGroups) done();
                    if constexpr (kSums) add(v, sum[EP == kOut ? g : 0]);
                    if constexpr (EP == kOut) {
                        if (there) emit<EP, P>(slots, a, p, w.split, row, col, v, v);
                    } else {
                        if constexpr (kSums) {  // the groups that are left, from the first place on
#pragma unroll
                            for (int i = 0; i + 1 < G; ++i)
#pragma unroll
                                for (int j = 0; j < 32; ++j) sum[i][j] = sum[i + 1][j];
                        }
                        Kept next;
                        if (a.keeps && g + 1 < kGroups) next.load(a, p, row + lane, col + 32);
                        if (there) emit_grad<P>(slots, a, p, row, col, v, kept);
                        kept = next;
                    }
                }
            }
        }
        if (lane == 0) store_wait();
    }
    __syncwarp();
    if (*s_abort) __nanosleep(1000000);  // copies still in flight end long before that
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc_fence_after_sync();
    if (warp == kEpilogueWarps) tmem_dealloc_pair(tmem, 512);
}

// ---- operands -------------------------------------------------------------------------

// A matrix that tensor copies cannot take as it is, and its copy as planes [rows][ld] of 16-bit
// elements: three of float32, else one.
enum { kLines = 0, kShifted = 1, kCodes = 2 };  // rows aligned to 16 bytes, of any alignment, in 8 bits
struct Stage {
    const void *x;
    int64_t stride;
    hiss_packed packed;
    int64_t rows;
    int width, kind;
    Divider per_row;
    uint16_t *out;
    int64_t ld, plane;
    unsigned first, blocks;  // thread blocks that it has
};
constexpr int kMaxStages = 5;
struct Stages {
    Stage s[kMaxStages];
    int count;
};

// All of a call's in one launch, 8 columns a thread at a time.  Bound by memory where it is large
// (16,384 x 2048 from 8 bits 17 us), else by its launch: five launches took 17 us where one takes 7.
template <typename T>
__global__ void __launch_bounds__(256) k_stage(const __grid_constant__ Stages all)
{
    constexpr bool THREE = sizeof(T) == 4;
    let_next_start();
    int m = 0;
    while (m + 1 < all.count && blockIdx.x >= all.s[m + 1].first) ++m;
    const Stage &a = all.s[m];
    const int64_t total = a.rows * a.per_row.d, blocks = (a.width + 31) / 32;
    for (int64_t i = (int64_t)(blockIdx.x - a.first) * 256 + threadIdx.x; i < total; i += (int64_t)a.blocks * 256) {
        const int64_t row = a.per_row.quotient(i);
        const int col = (int)(i - row * a.per_row.d) * 8;
        float v[8];
        if (a.kind == kCodes) {
            values8(*reinterpret_cast<const uint2 *>(a.packed.codes + row * blocks * 32 + col),
                    scale_of(a.packed.scales[row * blocks + col / 32]), v);
        } else {
            const T *x = static_cast<const T *>(a.x) + row * a.stride;
            if (a.kind == kLines) {
                Eight<T, true> in;
                in.load(x, col, a.width);
                in.get(x, col, a.width, v);
            } else {
                Eight<T, false> in;
                in.load(x, col, a.width);
                in.get(x, col, a.width, v);
            }
        }
        uint16_t *to = a.out + row * a.ld + col;
        if constexpr (THREE) {
            uint32_t w[4][3];
#pragma unroll
            for (int e = 0; e < 4; ++e) split3(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
            for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4 *>(to + q * a.plane) = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
        } else {
            store8<T, true>(reinterpret_cast<T *>(to), 0, 8, v);
        }
    }
}

// out[i][j] = the sum of the ranges' partial sums [splits][m][ld], in order: four columns a thread.
// 8192 x 128 of two ranges: 4 us (element by element with a 64-bit division each, 9).
__global__ void __launch_bounds__(256) k_join(const float *part, int splits, int64_t m, int n, int64_t ld, void *out, int dtype,
                                              int64_t stride, bool vec)
{
    let_next_start();
    wait_for_previous();
    const int quads = (n + 3) / 4;
    const int64_t total = m * quads;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = total < (int64_t(1) << 31) ? (uint32_t)i / (uint32_t)quads : i / quads;
        const int col = (int)(i - row * quads) * 4;
        const float *from = part + row * ld + col;
        auto v = load_pack<float, 4>(from);
        for (int s = 1; s < splits; ++s) {
            const auto k = load_pack<float, 4>(from + s * m * ld);
#pragma unroll
            for (int e = 0; e < 4; ++e) v.v[e] += k.v[e];
        }
        const int64_t at = row * stride + col;
        if (vec && col + 4 <= n) {
            if (dtype == HISS_F32) store_pack<float, 4>(static_cast<float *>(out) + at, v);
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) =
                    make_uint2(pack2(v.v[0], v.v[1], dtype == HISS_BF16), pack2(v.v[2], v.v[3], dtype == HISS_BF16));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < n) store_any(out, dtype, at + e, v.v[e]);
        }
    }
}

int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

unsigned grid_for(int64_t items) { return (unsigned)std::min<int64_t>((items + 255) / 256, kSMs * 8); }

// An operand that tensor copies can take.
struct Operand {
    const void *p;
    int64_t rows, cols, ld, plane;
};

using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                            const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder()
{
    static const Encode fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    return fn;
}

cudaError_t encode(CUtensorMap *map, CUtensorMapDataType type, size_t size, const Operand &o, int64_t planes, int wide, int high,
                   int deep, CUtensorMapSwizzle swizzle)
{
    const Encode f = encoder();
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dim[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)planes};
    const cuuint64_t stride[2] = {(cuuint64_t)o.ld * size, (cuuint64_t)(planes > 1 ? o.plane : o.ld) * size};
    const cuuint32_t box[3] = {(cuuint32_t)wide, (cuuint32_t)high, (cuuint32_t)deep}, one[3] = {1, 1, 1};
    const CUresult r = f(map, type, 3, const_cast<void *>(o.p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

CUtensorMapDataType half_type(bool bf16) { return bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16; }

// For loads into operands, all planes at once: K-major, `rows` rows of a stage's K elements; M-major, 64 elements of as
// many rows as a stage has K elements.
cudaError_t load_map(CUtensorMap *map, const Operand &o, int planes, bool m_major, int rows, bool bf16)
{
    return m_major ? encode(map, half_type(bf16), 2, o, planes, 64, kBlockK, planes, CU_TENSOR_MAP_SWIZZLE_128B)
                   : encode(map, half_type(bf16), 2, o, planes, kBlockK, rows, planes, CU_TENSOR_MAP_SWIZZLE_128B);
}
// For stores of an epilogue warp's 32 x 32 values (deep: planes at once), or 32 rows of 16 columns.
cudaError_t store_map(CUtensorMap *map, const Operand &o, int64_t planes, bool wide, bool bf16, int deep = 1, int cols = 32)
{
    if (cols == 16) return encode(map, half_type(bf16), 2, o, planes, 16, 32, deep, CU_TENSOR_MAP_SWIZZLE_32B);
    return wide ? encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, o, planes, 32, 32, 1, CU_TENSOR_MAP_SWIZZLE_128B)
                : encode(map, half_type(bf16), 2, o, planes, 32, 32, deep, CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int EP, int P>
cudaError_t launch(const Args &a, bool after, cudaStream_t s, int64_t *launches)
{
    static std::atomic<uint64_t> done{0};
    constexpr size_t smem = 227 * 1024;
    HISS_TRY(allow_shared(k_product<EP, P>, smem, done));
    // a block of fewer would wait for registers that it does not have
    static std::atomic<int> registers{0};
    if (registers.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes at{};
        HISS_TRY(cudaFuncGetAttributes(&at, k_product<EP, P>));
        registers.store(at.numRegs, std::memory_order_relaxed);
    }
    if (registers.load(std::memory_order_relaxed) != kLaunchRegs) return cudaErrorLaunchOutOfResources;
    const int units = a.tiles * a.splits;
    const unsigned grid = 2 * std::min(units, kPairs);
    ++*launches;
    if (after) return launch_after(k_product<EP, P>, grid, kThreads, smem, s, a);
    k_product<EP, P><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

// ---- few rows ----------------------------------------------------------------------------

// Blocks of columns that a lane copies ahead into its ring of shared memory.
constexpr int kRing = 4;

// Up to kFewRows rows of x (or h): a product is a pass over its weights.  A
// warp takes R rows of the weights (of both where gated), 16 bytes a lane and row at a time,
// which each lane copies for itself into a ring of shared memory; `ks` warps share a row's
// columns where there are not enough rows to fill the GPU.  Sums and h are float32.
template <typename T>
constexpr int kFewRows = sizeof(T) == 4 ? 8 : 4;
constexpr int kRowsAtOnce = 2;
constexpr int kRowsThreads = 256;

struct FewArgs {
    const void *w[2];
    int64_t w_stride[2];
    const void *x;
    int64_t x_stride;
    int n, k, m, ks, act, w_vec;
    void *out;
    int64_t out_stride;
    float *sums[2];  // where not NULL: a and b, [n][out_stride]
    int64_t x_part, h_part;  // of x and h in parts, the distance from one to the next
};

// Bound by memory where the weights are large: one row through 4096 x 11008 bfloat16 49 us (5.5 TB/s),
// float32 90 us (6.0); through 1024 x 4096 10 us, of which the two launches are half.  With the loads
// in registers instead of the ring it took 63 to 76 us.
template <typename T, typename X, typename Y, int NR, bool GATED>
__global__ void __launch_bounds__(kRowsThreads) k_few_rows(FewArgs a)
{
    constexpr int R = kRowsAtOnce, G = GATED ? 2 : 1, S = R * G * NR;
    __shared__ float part[kRowsThreads / 32][S];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int share = warp % a.ks, row0 = (blockIdx.x * (kRowsThreads / 32 / a.ks) + warp / a.ks) * R;
    constexpr int E = 16 / sizeof(T);
    extern __shared__ uint4 ring[];  // [kRing][warp][row][lane]
    const T *w[G * R];
#pragma unroll
    for (int p = 0; p < G * R; ++p)
        w[p] = static_cast<const T *>(a.w[p / R]) + (int64_t)min(row0 + p % R, a.m - 1) * a.w_stride[p / R];
    const X *x = static_cast<const X *>(a.x);
    const int step = 32 * E * a.ks, k0 = (share * 32 + lane) * E;
    auto slot = [&](int b, int p) { return &ring[((b % kRing * (kRowsThreads / 32) + warp) * (G * R) + p) * 32 + lane]; };
    auto fetch = [&](int b) {
        const int k = k0 + b * step;
#pragma unroll
        for (int p = 0; p < G * R; ++p) {
            if (a.w_vec) {
                if (k < a.k) cp_async16(slot(b, p), w[p] + k);
            } else {
                Pack<T, E> v;
#pragma unroll
                for (int e = 0; e < E; ++e) v.v[e] = k + e < a.k ? w[p][k + e] : from_f32<T>(0.0f);
                *reinterpret_cast<Pack<T, E> *>(slot(b, p)) = v;
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int b = 0; b < kRing - 1; ++b) fetch(b);
    float acc[G][R][NR] = {};
    if (!GATED) wait_for_previous();
    for (int b = 0, k = k0; k < a.k; ++b, k += step) {
        float u[NR][E];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const X *row = x + (NR == 1 ? 0 : min(i, a.n - 1)) * a.x_stride + k;
            if (a.w_vec) {
                const auto v = load_pack<X, E>(row);
#pragma unroll
                for (int e = 0; e < E; ++e) u[i][e] = to_f32(v.v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) u[i][e] = k + e < a.k ? to_f32(row[e]) : 0.0f;
            }
        }
        fetch(b + kRing - 1);
        cp_async_wait<kRing - 1>();
#pragma unroll
        for (int p = 0; p < G * R; ++p) {
            const auto v = *reinterpret_cast<const Pack<T, E> *>(slot(b, p));
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[p / R][p % R][i] = fmaf(to_f32(v.v[e]), u[i][e], acc[p / R][p % R][i]);
        }
    }
    cp_async_wait<0>();
    if (GATED) let_next_start();
    // lane s of a warp that has the whole sum s
    float mine = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float v = acc[s / (R * NR)][s / NR % R][s % NR];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == s) mine = v;
    }
    static_assert(S <= 32, "a sum a lane");
    if (a.ks > 1) {
        if (lane < S) part[warp][lane] = mine;
        __syncthreads();
        if (share != 0) return;
        if (lane < S)
            for (int s = 1; s < a.ks; ++s) mine += part[warp + s][lane];
    }
    const float b = GATED ? __shfl_sync(0xffffffffu, mine, (lane + R * NR) & 31) : 0.0f;
    const int row = row0 + lane / NR, i = lane % NR;
    if (lane >= R * NR || row >= a.m || i >= a.n) return;
    float v = mine;
    if (GATED && a.sums[0]) {
        a.sums[0][i * a.out_stride + row] = mine;
        a.sums[1][i * a.out_stride + row] = b;
    }
    if (GATED)
        with_activation(a.act, [&](auto act) { v = activate<false, decltype(act)::value>(both(mine)).value.x * b; });
    static_cast<Y *>(a.out)[i * a.out_stride + row] = from_f32<Y>(v);
}

template <typename T, typename X, typename Y, int NR, bool GATED>
cudaError_t few_rows_of(FewArgs a, bool after, cudaStream_t s, int64_t *launches)
{
    static std::atomic<uint64_t> done{0};
    constexpr int R = kRowsAtOnce;
    constexpr size_t smem = 16 * kRing * (size_t)kRowsThreads * R * (GATED ? 2 : 1);
    HISS_TRY(allow_shared(k_few_rows<T, X, Y, NR, GATED>, smem, done));
    // 16 warps a multiprocessor, as long as each has two blocks of columns
    a.ks = 1;
    while (a.ks < 8 && (int64_t)a.ks * a.m / R < 16 * kSMs && a.k > a.ks * 64 * (16 / (int)sizeof(T))) a.ks *= 2;
    const int rows = kRowsThreads / 32 / a.ks * R;
    const unsigned grid = (unsigned)((a.m + rows - 1) / rows);
    ++*launches;
    if (after) return launch_after(k_few_rows<T, X, Y, NR, GATED>, grid, kRowsThreads, smem, s, a);
    k_few_rows<T, X, Y, NR, GATED><<<grid, kRowsThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, typename X, typename Y, bool GATED>
cudaError_t few_rows(const FewArgs &a, bool after, cudaStream_t s, int64_t *launches)
{
    if (a.n == 1) return few_rows_of<T, X, Y, 1, GATED>(a, after, s, launches);
    if (a.n == 2) return few_rows_of<T, X, Y, 2, GATED>(a, after, s, launches);
    if (a.n <= 4) return few_rows_of<T, X, Y, 4, GATED>(a, after, s, launches);
    if constexpr (kFewRows<T> > 4) return few_rows_of<T, X, Y, 8, GATED>(a, after, s, launches);
    return cudaErrorInvalidValue;
}

// The same for up to 64 rows (see forward() for where) with the warps' matrix instructions, which
// these passes over the weights do not come near the rate of: the rows of x are 16-row
// tiles of A, 8 rows of the weights a tile of B.  A lane has 8 consecutive K elements of a
// row of either, which the two steps of 16 take in one order: K is summed in an order of its own.
// The lane copies them for itself into a ring of shared memory, three blocks of 32 columns
// ahead (x through L1: read past it by every warp, the same few lines of L2 cost more than the
// weights).  Of 16-bit types, up to 32 rows h goes on as two parts, h = p + q within 2^-17 (float16:
// 2^-23), so that nothing is lost to it; above, as in the large products, rounded once.  Float32
// goes through as three bfloat16 parts of everything: x and h come as planes, a lane splits
// its weights itself; up to 32 rows.
constexpr int kTileRows = 64;
constexpr int kWarps = 8;

// Parts of x or h; pieces of 16 bytes that a lane has of a block of 32 columns; blocks of the ring.
template <typename T, int MT, bool GATED>
constexpr int kParts = sizeof(T) == 4 ? 3 : GATED || MT > 2 ? 1 : 2;
template <typename T, int MT, bool GATED>
constexpr int kPieces = (GATED ? 2 : 1) * (int)sizeof(T) / 2 + kParts<T, MT, GATED> * MT * 2;
template <typename T, int MT>
constexpr int kDepth = sizeof(T) == 4 && MT > 1 ? 3 : 4;

// Blocks of 32 columns between two additions to the sums: these instructions cut as the large products' do.
// 16 float32 rows through 4096 x 11008 are 6.5e-6 off with one accumulator a warp (295 us), 5e-7 so (299;
// 32 rows 441 and 463).
template <typename T>
constexpr int kFoldBlocks = sizeof(T) == 4 ? 4 : 8;

// MT: 16-row tiles of x.
// 16 rows of bfloat16 through 512 x 2048 9 us, 48 rows 17 (20 in the large products); bound by the
// latency of a ring's blocks.
template <typename T, int MT, bool GATED>
__global__ void __launch_bounds__(kWarps * 32) k_tile_rows(FewArgs a)
{
    constexpr bool WIDE = sizeof(T) == 4, BF16 = !std::is_same_v<T, __half>;
    constexpr int G = GATED ? 2 : 1, PARTS = kParts<T, MT, GATED>, S = G * MT * 4, L = kPieces<T, MT, GATED>;
    constexpr int WP = sizeof(T) / 2, X0 = G * WP, D = kDepth<T, MT>;  // pieces of a row of the weights; the first of x's
    extern __shared__ uint4 ring[];  // [D][warp][piece][lane]; at the end, the shares' sums [warp][S][lane]
    static_assert(S * 4 <= D * L * 16, "room for the sums");
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
    const int share = warp % a.ks, row0 = (blockIdx.x * (kWarps / a.ks) + warp / a.ks) * 8;
    // rows behind the last repeat it: their sums go nowhere
    const T *w_row[G];
#pragma unroll
    for (int g = 0; g < G; ++g) w_row[g] = static_cast<const T *>(a.w[g]) + (int64_t)min(row0 + g8, a.m - 1) * a.w_stride[g];
    const uint16_t *x_row[PARTS * 2 * MT];
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m)
            x_row[q * 2 * MT + m] = static_cast<const uint16_t *>(a.x) + q * a.x_part + min(8 * m + g8, a.n - 1) * a.x_stride;
    const int blocks = a.k > share * 32 ? (a.k - share * 32 + a.ks * 32 - 1) / (a.ks * 32) : 0;  // of this share
    auto slot = [&](int b, int p) { return &ring[((b % D * kWarps + warp) * L + p) * 32 + lane]; };
    // 16 bytes of a row from element k on, one by one
    auto by_element = [&](const auto *row, int k) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(row)>>;
        Pack<E, 16 / sizeof(E)> v;
#pragma unroll
        for (int e = 0; e < (int)(16 / sizeof(E)); ++e) v.v[e] = k + e < a.k ? row[k + e] : E(0.0f);
        uint4 r;
        memcpy(&r, &v, 16);
        return r;
    };
    // the weights' pieces, or x's, of the share's block b
    auto fetch_weights = [&](int b) {
        const int k = (share + b * a.ks) * 32 + t * 8;
#pragma unroll
        for (int p = 0; p < X0; ++p) {
            const T *row = w_row[p / WP];
            const int at = k + p % WP * 4;
            if (a.w_vec && k + 8 <= a.k) cp_async16(slot(b, p), row + at);
            else *slot(b, p) = by_element(row, at);
        }
    };
    auto fetch_x = [&](int b) {
        const int k = (share + b * a.ks) * 32 + t * 8;
#pragma unroll
        for (int p = 0; p < PARTS * 2 * MT; ++p) {
            if (a.w_vec && k + 8 <= a.k) cp_async16_cached(slot(b, X0 + p), x_row[p] + k, p % (2 * MT) * 8 + g8 < a.n);
            else *slot(b, X0 + p) = by_element(x_row[p], k);
        }
    };
    // the weights' first blocks need not wait for the kernel that makes h
#pragma unroll
    for (int b = 0; b < D - 1; ++b)
        if (b < blocks) fetch_weights(b);
    if (!GATED) wait_for_previous();
#pragma unroll
    for (int b = 0; b < D - 1; ++b) {
        if (b < blocks) fetch_x(b);
        cp_async_commit();
    }
    float sum[G][MT][4] = {}, acc[G][MT][4] = {}, cross[WIDE ? G : 1][WIDE ? MT : 1][4] = {};
    auto fold = [&]() {
#pragma unroll
        for (int e = 0; e < S; ++e) {
            float &to = sum[e / (MT * 4)][e / 4 % MT][e % 4], &from = acc[e / (MT * 4)][e / 4 % MT][e % 4];
            to += from;
            from = 0.0f;
            if constexpr (WIDE) {
                float &rest = cross[e / (MT * 4)][e / 4 % MT][e % 4];
                to += rest;
                rest = 0.0f;
            }
        }
    };
    for (int b = 0; b < blocks; ++b) {
        if (b + D - 1 < blocks) {
            fetch_weights(b + D - 1);
            fetch_x(b + D - 1);
        }
        cp_async_commit();
        cp_async_wait<D - 1>();
        uint4 w[G][WIDE ? 3 : 1];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if constexpr (WIDE) {
                const uint4 p = *slot(b, 2 * g), q = *slot(b, 2 * g + 1);
                const uint32_t f[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                uint32_t part[4][3];
#pragma unroll
                for (int j = 0; j < 4; ++j) split3(__uint_as_float(f[2 * j]), __uint_as_float(f[2 * j + 1]), part[j]);
#pragma unroll
                for (int q3 = 0; q3 < 3; ++q3) w[g][q3] = make_uint4(part[0][q3], part[1][q3], part[2][q3], part[3][q3]);
            } else {
                w[g][0] = *slot(b, g);
            }
        }
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint4 lo = *slot(b, X0 + q * 2 * MT + 2 * m), hi = *slot(b, X0 + q * 2 * MT + 2 * m + 1);
                auto product = [&](float(&to)[4], const uint4 &v) {
                    mma_warp<BF16>(to, lo.x, hi.x, lo.y, hi.y, v.x, v.y);
                    mma_warp<BF16>(to, lo.z, hi.z, lo.w, hi.w, v.z, v.w);
                };
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    if constexpr (WIDE) {  // the six products of parts, as in the large products
                        product(q == 0 ? acc[g][m] : cross[g][m], w[g][0]);
                        if (q < 2) product(cross[g][m], w[g][1]);
                        if (q < 1) product(cross[g][m], w[g][2]);
                    } else {
                        product(acc[g][m], w[g][0]);
                    }
                }
            }
        if (b % kFoldBlocks<T> == kFoldBlocks<T> - 1) fold();
    }
    fold();
    if (GATED) let_next_start();
    if (a.ks > 1) {
        float *sums = reinterpret_cast<float *>(ring);
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int e = 0; e < S; ++e) sums[(warp * S + e) * 32 + lane] = sum[e / (MT * 4)][e / 4 % MT][e % 4];
        __syncthreads();
        // each of the row's warps joins its part of the sums
        const int per = (S + a.ks - 1) / a.ks;
        float *mine = sums + (warp - share) * S * 32 + lane;
        for (int e = share * per; e < share * per + per && e < S; ++e) {
            float v = mine[e * 32];
            for (int s = 1; s < a.ks; ++s) v += mine[(s * S + e) * 32];
            mine[e * 32] = v;
        }
        __syncthreads();
        if (share != 0) return;
#pragma unroll
        for (int e = 0; e < S; ++e) sum[e / (MT * 4)][e / 4 % MT][e % 4] = mine[e * 32];
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * m + g8 + (e & 2) * 4, row = row0 + 2 * t + (e & 1);
            if (i >= a.n || row >= a.m) continue;
            const int64_t at = i * a.out_stride + row;
            float v = sum[0][m][e];
            if constexpr (GATED) {
                const float u = sum[1][m][e];
                if (a.sums[0]) a.sums[0][at] = v, a.sums[1][at] = u;
                float h = 0.0f;
                with_activation(a.act, [&](auto act) { h = activate<!WIDE, decltype(act)::value>(both(v)).value.x * u; });
                if constexpr (WIDE) {
                    uint32_t part[3];
                    split3(h, 0.0f, part);
#pragma unroll
                    for (int q = 0; q < 3; ++q) static_cast<uint16_t *>(a.out)[q * a.h_part + at] = (uint16_t)part[q];
                } else {
                    const T p = from_f32<T>(h);
                    const float left = h - to_f32(p);
                    static_cast<T *>(a.out)[at] = p;
                    if (kParts<T, MT, false> == 2)
                        static_cast<T *>(a.out)[a.h_part + at] = from_f32<T>(fabsf(to_f32(p)) <= kFloatMax ? left : 0.0f);
                }
            } else {
                static_cast<T *>(a.out)[at] = from_f32<T>(v);
            }
        }
}

template <typename T, int MT, bool GATED>
cudaError_t tile_rows_of(FewArgs a, bool after, cudaStream_t s, int64_t *launches)
{
    static std::atomic<uint64_t> done{0};
    constexpr size_t smem = 16 * 32 * kDepth<T, MT> * kWarps * (size_t)kPieces<T, MT, GATED>;
    HISS_TRY(allow_shared(k_tile_rows<T, MT, GATED>, smem, done));
    // 12 warps a multiprocessor, as long as each has four blocks of columns
    a.ks = 1;
    while (a.ks < kWarps && (int64_t)a.ks * ((a.m + 7) / 8) < 12 * kSMs && a.k > a.ks * 128) a.ks *= 2;
    const int rows = kWarps / a.ks * 8;
    const unsigned grid = (unsigned)((a.m + rows - 1) / rows);
    ++*launches;
    if (after) return launch_after(k_tile_rows<T, MT, GATED>, grid, kWarps * 32, smem, s, a);
    k_tile_rows<T, MT, GATED><<<grid, kWarps * 32, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, bool GATED>
cudaError_t tile_rows(const FewArgs &a, bool after, cudaStream_t s, int64_t *launches)
{
    if (a.n <= 16) return tile_rows_of<T, 1, GATED>(a, after, s, launches);
    if (a.n <= 32) return tile_rows_of<T, 2, GATED>(a, after, s, launches);
    if constexpr (sizeof(T) == 2) {
        if (a.n <= 48) return tile_rows_of<T, 3, GATED>(a, after, s, launches);
        return tile_rows_of<T, 4, GATED>(a, after, s, launches);
    }
    return cudaErrorInvalidValue;
}

// Everything of one call: workspace, operands and products.
struct Plan {
    const FfnArgs &q;
    const int dtype;
    const bool bf16;
    const int planes;
    char *ws;           // NULL: sizes only
    size_t used = 0;
    cudaStream_t s;
    int64_t *launches;
    int *bad;

    Plan(const FfnArgs &args, void *tmp, int *flag, cudaStream_t stream, int64_t *count)
        : q(args), dtype(args.w.dtype), bf16(dtype != HISS_F16), planes(dtype == HISS_F32 ? 3 : 1), ws(static_cast<char *>(tmp)),
          s(stream), launches(count), bad(flag)
    {
    }

    void *take(size_t bytes)
    {
        void *p = ws ? ws + used : nullptr;
        used += (bytes + 1023) & ~(size_t)1023;
        return p;
    }
    // room for an operand [rows][cols]
    Operand room(int64_t rows, int64_t cols)
    {
        Operand o{nullptr, rows, cols, pad64(cols), rows * pad64(cols)};
        o.p = take(2 * (size_t)planes * o.plane);
        return o;
    }

    // A caller's matrix: as it is where tensor copies can take it, else a copy.
    Operand matrix(const void *p, int64_t stride, int64_t rows, int64_t cols)
    {
        if (planes == 1 && (uintptr_t)p % 16 == 0 && stride % 8 == 0 && stride >= cols) return {p, rows, cols, stride, 0};
        const Operand o = room(rows, cols);
        stage(p, stride, {}, rows_aligned(p, stride, dtype, 8) ? kLines : kShifted, o);
        return o;
    }
    Operand unpacked(const hiss_packed &p, int64_t rows, int64_t cols)
    {
        const Operand o = room(rows, cols);
        stage(nullptr, 0, p, kCodes, o);
        return o;
    }
    Stages staged{};
    unsigned stage_blocks = 0;
    void stage(const void *p, int64_t stride, const hiss_packed &packed, int kind, const Operand &o)
    {
        const Divider per_row((uint32_t)((o.cols + 7) / 8));
        const unsigned blocks = grid_for(o.rows * per_row.d);
        staged.s[staged.count++] = {p, stride, packed, o.rows, (int)o.cols, kind, per_row, static_cast<uint16_t *>(const_cast<void *>(o.p)),
                                    o.ld, o.plane, stage_blocks, blocks};
        stage_blocks += blocks;
    }
    cudaError_t run_stages()
    {
        if (!ws || staged.count == 0) return cudaSuccess;
        ++*launches;
        if (planes == 3) k_stage<float><<<stage_blocks, 256, 0, s>>>(staged);
        else if (bf16) k_stage<__nv_bfloat16><<<stage_blocks, 256, 0, s>>>(staged);
        else k_stage<__half><<<stage_blocks, 256, 0, s>>>(staged);
        after = true;
        return cudaGetLastError();
    }
    bool after = false;  // a kernel of this call came before

    struct Product {
        std::initializer_list<Operand> a, b;  // by segment; two b of one segment where dual
        int64_t m, n;
        void *out;
        int64_t out_stride;
    };

    // The products of one launch: all of one K (per segment) and one order.
    template <int EP>
    cudaError_t run(Args &a, std::initializer_list<Product> products, std::initializer_list<int64_t> k, bool a_m_major, bool b_n_major)
    {
        a.bf16 = bf16;
        a.a_m_major = a_m_major;
        a.b_n_major = b_n_major;
        a.dual = EP == kGated;
        a.bn = planes == 3 ? 128 : 256;
        a.bad = bad;
        a.blocks[0] = (int)((k.begin()[0] + kBlockK - 1) / kBlockK);
        a.blocks[1] = k.size() > 1 ? (int)((k.begin()[1] + kBlockK - 1) / kBlockK) : 0;
        const int cols = EP == kGated ? a.bn / 2 : a.bn;
        a.problems = 0;
        a.tiles = 0;
        for (const Product &r : products) {
            if (r.m == 0 || r.n == 0 || (EP == kOut && !r.out)) continue;
            Problem &p = a.p[a.problems++];
            p.m = r.m;
            p.n = r.n;
            p.out = r.out;
            p.out_stride = r.out_stride;
            p.tiles_m = (int)((r.m + kBlockM - 1) / kBlockM);
            p.tiles_n = (int)((r.n + cols - 1) / cols);
            p.first = a.tiles;
            a.tiles += p.tiles_m * p.tiles_n;
            for (size_t i = 0; ws && i < r.a.size(); ++i) HISS_TRY(load_map(&p.a[i], r.a.begin()[i], planes, a_m_major, 128, bf16));
            for (size_t i = 0; ws && i < r.b.size(); ++i) HISS_TRY(load_map(&p.b[i], r.b.begin()[i], planes, b_n_major, a.bn / 2, bf16));
        }
        if (a.problems == 0) return cudaSuccess;
        const int blocks = a.blocks[0] + a.blocks[1];
        a.splits = 1;
        // few tiles over a long K: ranges of at least 8 blocks that fill the pairs
        if (EP == kOut && 2 * a.tiles <= kPairs) a.splits = std::max(1, std::min(kPairs / a.tiles, blocks / 8));
        a.per_split = (blocks + a.splits - 1) / a.splits;
        a.splits = (blocks + a.per_split - 1) / a.per_split;
        const float *part[kMaxProblems] = {};
        for (int i = 0; EP == kOut && i < a.problems; ++i) {
            Problem &p = a.p[i];
            if (a.splits > 1) {
                const int64_t ld = pad64(p.n);
                part[i] = static_cast<float *>(take(4 * (size_t)p.m * ld * a.splits));
                p.by_copy = 1;
                if (ws) HISS_TRY(store_map(&p.to, {part[i], p.m, p.n, ld, p.m * ld}, a.splits, true, bf16));
            } else {
                p.by_copy = rows_aligned(p.out, p.out_stride, dtype, 8);
                if (ws && p.by_copy) HISS_TRY(store_map(&p.to, {p.out, p.m, p.n, p.out_stride, 0}, 1, planes == 3, bf16));
            }
        }
        if (!ws) return cudaSuccess;
        if (planes == 1) HISS_TRY((launch<EP, 1>(a, after, s, launches)));
        else if constexpr (EP != kGradLong) HISS_TRY((launch<EP, 3>(a, after, s, launches)));
        after = true;
        for (int i = 0; a.splits > 1 && i < a.problems; ++i) {
            const Problem &p = a.p[i];
            HISS_TRY(launch_after(k_join, grid_for(p.m * ((p.n + 3) / 4)), 256, 0, s, part[i], a.splits, p.m, (int)p.n, pad64(p.n), p.out,
                                  dtype, p.out_stride, rows_aligned(p.out, p.out_stride, dtype, 4)));
            ++*launches;
        }
        return cudaSuccess;
    }

    template <typename T>
    cudaError_t few()
    {
        const hiss_ffn &w = q.w;
        const int64_t n = q.n, ld = pad64(w.hidden);
        const bool tiles = n > kFewRows<T>;
        // x and h as they go into the products: float32, or 16-bit parts
        const Operand planes_of_x = tiles && planes == 3 ? matrix(q.g.x, q.g.x_stride, n, w.width) : Operand{q.g.x, n, w.width, q.g.x_stride, 0};
        float *sums[2] = {};
        void *h = take(6 * (size_t)n * ld);
        for (int i = 0; i < 2 && q.keeps; ++i) sums[i] = static_cast<float *>(take(4 * (size_t)n * ld));
        if (!ws) return cudaSuccess;
        HISS_TRY(run_stages());
        // 16-byte loads of whole rows; the tiles take the columns behind the last 8 one by one
        auto vec = [&](const void *p, int64_t stride, int width) { return (tiles || width % 8 == 0) && rows_aligned(p, stride, dtype, 8); };
        FewArgs a{};
        a.w[0] = w.gate, a.w[1] = w.up;
        a.w_stride[0] = w.gate_stride, a.w_stride[1] = w.up_stride;
        a.x = planes_of_x.p, a.x_stride = planes_of_x.ld, a.x_part = planes_of_x.plane;
        a.n = (int)n, a.k = w.width, a.m = w.hidden, a.act = w.activation;
        a.w_vec = vec(w.gate, w.gate_stride, w.width) && vec(w.up, w.up_stride, w.width) &&
                  (planes_of_x.p != q.g.x || vec(q.g.x, q.g.x_stride, w.width));
        a.out = h, a.out_stride = ld, a.h_part = n * ld;
        a.sums[0] = sums[0], a.sums[1] = sums[1];
        FewArgs b{};
        b.w[0] = w.down;
        b.w_stride[0] = w.down_stride;
        b.x = h, b.x_stride = ld, b.x_part = n * ld;
        b.n = (int)n, b.k = w.hidden, b.m = w.out_width;
        b.w_vec = vec(w.down, w.down_stride, w.hidden);
        b.out = q.y, b.out_stride = q.y_stride;
        if (tiles) {
            HISS_TRY((tile_rows<T, true>(a, false, s, launches)));
            HISS_TRY((tile_rows<T, false>(b, true, s, launches)));
        } else {
            HISS_TRY((few_rows<T, T, float, true>(a, false, s, launches)));
            HISS_TRY((few_rows<T, float, T, false>(b, true, s, launches)));
        }
        for (int i = 0; i < 2 && q.keeps; ++i) HISS_TRY(pack(sums[i], HISS_F32, ld, n, w.hidden, q.kept[i], s, launches));
        return cudaSuccess;
    }

    cudaError_t forward()
    {
        const hiss_ffn &w = q.w;
        const int64_t n = q.n, f = w.hidden, d = w.width, o = w.out_width;
        // the tiles' time grows with rows and weights, that of the large products (20 us and up) hardly
        // with the rows: 16 rows of bfloat16 through 1024 x 4096 take 19 and 23 us, 64 rows 37 and 23,
        // 16 through 4096 x 11008 105 and 81
        // (float32: 16 rows through 1024 x 4096 39 and 56, 32 rows 56 and 56, through 4096 x 11008 455 and 523)
        const bool tiles = planes == 3 ? n <= 32 : n <= kTileRows && n * f * (2 * d + o) <= int64_t(3) << 27;
        if (tiles || n <= kFewRows<__half>) return with_dtype(dtype, [&](auto t) { return few<decltype(t)>(); });
        const Operand x = matrix(q.g.x, q.g.x_stride, n, d), gate = matrix(w.gate, w.gate_stride, f, d);
        const Operand up = matrix(w.up, w.up_stride, f, d), down = matrix(w.down, w.down_stride, o, f);
        HISS_TRY(run_stages());
        const Operand h = room(n, f);
        Args a{};
        a.act = w.activation;
        if (ws) HISS_TRY(store_map(&a.h, h, planes, false, bf16, planes));
        a.keeps = q.keeps;
        a.kept[0] = q.kept[0];
        a.kept[1] = q.kept[1];
        HISS_TRY((run<kGated>(a, {{{x}, {gate, up}, n, f, nullptr, 0}}, {d}, false, false)));
        Args b{};
        return run<kOut>(b, {{{h}, {down}, n, o, q.y, q.y_stride}}, {f}, false, false);
    }

    cudaError_t backward()
    {
        const hiss_ffn &w = q.w;
        const hiss_ffn_grad &g = q.g;
        const int64_t n = q.n, f = w.hidden, d = w.width, o = w.out_width;
        if (n == 0) {
            auto zero = [&](void *p, int64_t stride, int64_t rows, int64_t cols) {
                const size_t e = dtype_bytes(dtype);
                return p && ws ? cudaMemset2DAsync(p, e * stride, 0, e * cols, rows, s) : cudaSuccess;
            };
            HISS_TRY(zero(g.dgate, g.dgate_stride, f, d));
            HISS_TRY(zero(g.dup, g.dup_stride, f, d));
            return zero(g.ddown, g.ddown_stride, o, f);
        }
        const Operand x = g.x ? matrix(g.x, g.x_stride, n, d) : unpacked(q.x8, n, d), dy = matrix(g.dy, g.dy_stride, n, o);
        const Operand gate = matrix(w.gate, w.gate_stride, f, d), up = matrix(w.up, w.up_stride, f, d);
        const Operand down = matrix(w.down, w.down_stride, o, f);
        HISS_TRY(run_stages());
        const Operand da = room(n, f), db = room(n, f), h = room(n, f);
        Args a{};
        a.act = w.activation;
        a.keeps = q.keeps;
        a.kept[0] = q.kept[0];
        a.kept[1] = q.kept[1];
        if (!q.keeps) {
            a.raw = static_cast<float *>(take(8 * (size_t)((n + 31) / 32 * 32) * ((f + 31) / 32 * 32)));
            HISS_TRY((run<kGated>(a, {{{x}, {gate, up}, n, f, nullptr, 0}}, {d}, false, false)));
        }
        if (ws) {
            const int cols = planes == 3 ? kGradCols<3> : kGradCols<1>;
            HISS_TRY(store_map(&a.h, h, planes, false, bf16, planes, cols));
            HISS_TRY(store_map(&a.da, da, planes, false, bf16, planes, cols));
            HISS_TRY(store_map(&a.db, db, planes, false, bf16, planes, cols));
        }
        if (planes == 1 && o > fold_blocks<kGrad, 1>(0) * kBlockK)
            HISS_TRY((run<kGradLong>(a, {{{dy}, {down}, n, f, nullptr, 0}}, {o}, false, true)));
        else
            HISS_TRY((run<kGrad>(a, {{{dy}, {down}, n, f, nullptr, 0}}, {o}, false, true)));
        Args b{};
        HISS_TRY((run<kOut>(b, {{{da, db}, {gate, up}, n, d, g.dx, g.dx_stride}}, {f, f}, false, true)));
        Args c{};
        return run<kOut>(c,
                         {{{da}, {x}, f, d, g.dgate, g.dgate_stride},
                          {{db}, {x}, f, d, g.dup, g.dup_stride},
                          {{dy}, {h}, o, f, g.ddown, g.ddown_stride}},
                         {n}, true, true);
    }
};

}  // namespace

size_t ffn_tmp_bytes(const FfnArgs &a)
{
    Plan p(a, nullptr, nullptr, nullptr, nullptr);
    (void)(a.backward ? p.backward() : p.forward());
    return p.used;
}

cudaError_t feed_forward(const FfnArgs &a, void *tmp, int *bad, cudaStream_t s, int64_t *launches)
{
    return Plan(a, tmp, bad, s, launches).forward();
}

cudaError_t feed_forward_grad(const FfnArgs &a, void *tmp, int *bad, cudaStream_t s, int64_t *launches)
{
    return Plan(a, tmp, bad, s, launches).backward();
}

}  // namespace hiss
