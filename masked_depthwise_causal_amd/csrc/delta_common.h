// delta_common.h -- what the kernels of the gated delta rule share: the chunk, the operands' images, and
// numbers in two 16-bit terms.
//
// In chunks of C = 64 rows, with G the running sum of the log decays within the chunk, M[i,j] =
// exp(G[i] - G[j]) for j <= i, and S0 the state before the chunk, the recurrence is
//
//   L = diag(beta) tril(M o Kn Kn^T, -1),   X = (I + L)^-1,   A = scale tril(M o Qn Kn^T)
//   U = X diag(beta) (V - exp(G) Kn S0),    out = scale exp(G) Qn S0 + A U
//   S = exp(G[C-1]) S0 + Kn^T diag(exp(G[C-1] - G)) U
//
// (Kn, Qn: the normalized rows.) X and A need no state, so every chunk's are made at once by one kernel;
// another then walks over the chunks with the state in registers.
//
// Numbers. Products run on the matrix units in fp16, in as many terms as they need to come out as in fp32:
// rows of q and k are exact in one (with a power of two a row taken out, bf16's 8 bits fit wherever fp16 is
// normal; values below 2^-28 of the row's largest lose 2^-40 of it); everything that is computed is split
// in two, hi + lo, 22 bits (a power of two a column, a row of A, or a matrix, taken out; what is lost is below
// 2^-22 of a value or 2^-40 of the largest that it shares a power with, so that factors which make up for a
// value's size stay out of what is split). An exact operand with a split
// one takes two products, two split ones three (lo lo is below 2^-22). On this card that is 8 and 5 times
// the rate of the fp32 matrix instructions; in bf16 terms it would take three and six products.
#pragma once

#include "mccb_delta.h"
#include "ssm_common.h"

namespace delta {

using namespace ssm;

constexpr int kC = 64;              // rows of a chunk
constexpr float kNormEps = 1e-6f;   // in the rows' norms
constexpr int kSquare = kC * kC;    // values of X, of A

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------------------------
// What one kernel hands to the next for a chunk. A key head's: the images of its rows of k and q, the factors
// that make them normalized rows, kn = kr k~, qn = qr q~ (without the scale), and those of k~ = k 2^-e and
// q~ = q 2^-e, negative for a row of zeros. A value head's: the images of X and A in two terms each, and what
// belongs to single rows.
// ---------------------------------------------------------------------------------------------
struct RowCoef {
    float p[kC];        // exp(G) kr: V - p (K~ S0)
    float beta[kC];
    float q[kC];        // scale exp(G) qr
    float u[kC];        // exp(G[C-1] - G) kr
    float whole;        // exp(G[C-1])
    float x;            // X = x (hi + lo)
    float pad[14];
    double cum[kC];     // G in units of log 2
    float a[kC];        // A's rows = a (hi + lo): as small as the rows of q, and as what they make
    float pad2[48];
};
static_assert(sizeof(RowCoef) == 2048, "two of the walks' loads");

constexpr size_t key_bytes(int kp) { return 2 * kC * kp * sizeof(uint16_t) + 4 * kC * sizeof(float); }
// X hi, X lo, A hi, A lo, of each the three 32x32 blocks on and below the diagonal
constexpr int kTriangle = 3 * 32 * 32;
constexpr size_t kXaBytes = 4 * kTriangle * sizeof(uint16_t);

// An image row R holds its chunks of 8 values in the order c ^ swizzle(R). The matrix instructions' rows m
// stand for rows 32 j + 8 (m / 4) + 4 p + m % 4 (below); sixteen of those read one chunk each from
// different banks, and a transposing read's four rows too.
template <int COLS>
__device__ static inline int swizzle(int row) {
    static_assert(COLS == 64 || COLS == 128, "images have 8 or 16 chunks a row");
    return COLS == 128 ? ((row >> 3) & 3) | ((row & 3) << 2) : ((row >> 3) & 3) | ((row & 2) << 1);
}
template <int COLS>
__device__ static inline int image_at(int row, int chunk) {  // in 16-bit values
    return row * COLS + ((chunk ^ swizzle<COLS>(row)) << 3);
}

// Rows of 16x16 results. Two neighbouring tiles, p = 0 and 1, cover 32 rows so that lane group g = lane / 16
// holds rows 8 g + 4 p + i in its four registers i: both tiles' registers, one after the other, are then
// eight consecutive rows, just what the next product wants of its right operand.
__device__ static inline int row_of(int tile, int m) { return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3); }

// Instructions stay on their side of this: operands are read a few products ahead, and not all of a loop's at once,
// which would take more registers than there are.
__device__ static inline void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// The same number, as a new one: what is computed from it is computed where it stands, not ahead of all loops, to
// be kept in registers that are needed.
__device__ static inline int anew(int v) {
    asm volatile("" : "+v"(v));
    return v;
}
__device__ static inline f4 anew(h4 v) {
    auto u = __builtin_bit_cast(uint2, v);
    asm volatile("" : "+v"(u.x), "+v"(u.y));
    v = __builtin_bit_cast(h4, u);
    return f4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

// Operands from images. Where a lane reads is a place of its own (left_place and so on, once a kernel) with
// a step or tile exclusive-or'ed in and constants added: the swizzle does not depend on those.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds4;

// Left operand, rows of `tile`, step s of 32 along the image's columns.
template <int COLS>
__device__ static inline int left_place(int lane) {
    return image_at<COLS>(row_of(0, lane & 15), lane >> 4);
}
template <int COLS>
__device__ static inline h8 left(const uint16_t *image, int place, int tile, int s) {
    return *(const h8 *)(image + (place ^ s << 5) + row_of(tile, 0) * COLS);
}
// Of a triangle's blocks, whose rows have four chunks in the order c ^ (row / 8): likewise, step s up to tile / 2.
__device__ static inline int block_at(int row, int chunk) { return row * 32 + ((chunk ^ (row >> 3)) << 3); }
__device__ static inline int block_of(int row, int col) { return (row * (row + 1) / 2 + col) * 1024; }
__device__ static inline int triangle_place(int lane) { return block_at(row_of(0, lane & 15), lane >> 4); }
__device__ static inline h8 triangle(const uint16_t *image, int place, int tile, int s) {
    return *(const h8 *)(image + place + block_of(tile >> 1, s) + 4 * (tile & 1) * 32);
}
// The transposed image's: its columns as rows (`tile` of them), step s of 32 along its rows.
// A transposing read gives lane i of 16 column i of the four rows that those lanes read 8 bytes of.
template <int COLS>
__device__ static inline int turned_place(int lane) {
    return image_at<COLS>(8 * (lane >> 4) + (lane >> 2 & 3), lane & 3);
}
template <int COLS>
__device__ static inline h8 turned_at(const uint16_t *__restrict__ p) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + 4 * COLS));
    return __builtin_bit_cast(h8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int COLS>
__device__ static inline h8 left_turned(const uint16_t *image, int place, int tile, int s) {
    return turned_at<COLS>(image + (place ^ (tile >> 1) << 5) + 32 * s * COLS + 4 * (tile & 1));
}
// And the transposed triangle's, step s from tile / 2 on.
__device__ static inline int triangle_turned_place(int lane) {
    return block_at(8 * (lane >> 4) + (lane >> 2 & 3), lane & 3);
}
__device__ static inline h8 triangle_turned(const uint16_t *image, int place, int tile, int s) {
    return turned_at<32>(image + place + block_of(s, tile >> 1) + 4 * (tile & 1));
}
// Right operand: columns 16 tile.. of an image, step s of 32 along its rows.
template <int COLS>
__device__ static inline int right_place(int lane) {
    return image_at<COLS>(8 * (lane >> 4) + (lane >> 2 & 3), lane >> 1 & 1) + 4 * (lane & 1);
}
template <int COLS>
__device__ static inline h8 right_turned(const uint16_t *image, int place, int tile, int s) {
    return turned_at<COLS>(image + (place ^ tile << 4) + 32 * s * COLS);
}

__device__ static inline f4 mma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// ---------------------------------------------------------------------------------------------
// Two terms.
// ---------------------------------------------------------------------------------------------
struct Split {
    h8 hi, lo;
};
// hi = fp16(v inv), lo = fp16(v inv - hi), each a mixed-precision multiply-add that rounds once. (The empty asm, which
// has no instruction, keeps the pair hi together: the compiler would round its halves a second time.)
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
__device__ static inline void split2(float a, float b, float inv, uint32_t &hi, uint32_t &lo) {
    const h2 first = {(_Float16)__builtin_fmaf(a, inv, 0.0f), (_Float16)__builtin_fmaf(b, inv, 0.0f)};
    uint32_t h = __builtin_bit_cast(uint32_t, first);
    asm("" : "+v"(h));
    const h2 t = __builtin_bit_cast(h2, h);
    const h2 l = {(_Float16)__builtin_fmaf(a, inv, -(float)t[0]), (_Float16)__builtin_fmaf(b, inv, -(float)t[1])};
    hi = h;
    lo = __builtin_bit_cast(uint32_t, l);
}
__device__ static inline Split split(const f4 &a, const f4 &b, float inv) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    uint32_t h[4], l[4];
    split2(a[0], a[1], inv, h[0], l[0]);
    split2(a[2], a[3], inv, h[1], l[1]);
    split2(b[0], b[1], inv, h[2], l[2]);
    split2(b[2], b[3], inv, h[3], l[3]);
    Split s;
    s.hi = __builtin_bit_cast(h8, u4{h[0], h[1], h[2], h[3]});
    s.lo = __builtin_bit_cast(h8, u4{l[0], l[1], l[2], l[3]});
    return s;
}

// What brings the largest value m to 2^14..2^15, a power of two, and its inverse. (So high, since the others' last bits
// are then fp16's smallest, 2^-24: a column of Y may hold rows whose sizes are a chunk's whole decay apart, and the small
// ones count, where their factors are the large ones.) From 2^-112 on down m counts as 2^-112; infinities stay what
// they are; NaN is not counted by the maximum that comes in.
struct Power {
    float back, inv;
};
__device__ static inline Power power_of(float m) {
    uint32_t e = __float_as_uint(m) >> 23;
    e = e < 15 ? 15 : e > 254 ? 254 : e;
    Power p;
    p.back = __uint_as_float((e - 14) << 23);
    p.inv = __uint_as_float((268 - e) << 23);
    return p;
}

// The matrix instruction cuts the sum of its 32 products off towards minus infinity (its addition to the accumulator
// is rounded). Such errors have one sign, and states, keys and queries have means that are not zero: <gS, S> and what
// else sums over many of them would collect it (2.5e-6 of gradA, at S=448 B=4 H=12 K=128 V=64; 2e-7 without). So
// half of the columns go through the products with their sign turned, for nothing, since a power of two is taken out
// of each in any case.
__device__ static inline Power turned_sign(Power p, int lane) {
    const uint32_t sign = (uint32_t)__builtin_popcount(lane & 15) << 31;
    p.back = __uint_as_float(__float_as_uint(p.back) ^ sign);
    p.inv = __uint_as_float(__float_as_uint(p.inv) ^ sign);
    return p;
}

// Over the four lanes that hold a column, 16 apart: the largest value, and the sum.
struct Pair {
    uint32_t a, b;
};
template <int LANES>
__device__ static inline Pair swapped(uint32_t v) {
    if constexpr (LANES == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return {r[0], r[1]};
    } else {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return {r[0], r[1]};
    }
}
__device__ static inline float column_max(float m) {
    Pair p = swapped<32>(__float_as_uint(m));
    m = __builtin_fmaxf(__uint_as_float(p.a), __uint_as_float(p.b));
    p = swapped<16>(__float_as_uint(m));
    return __builtin_fmaxf(__uint_as_float(p.a), __uint_as_float(p.b));
}
__device__ static inline float column_sum(float v) {
    Pair p = swapped<32>(__float_as_uint(v));
    v = __uint_as_float(p.a) + __uint_as_float(p.b);
    p = swapped<16>(__float_as_uint(v));
    return __uint_as_float(p.a) + __uint_as_float(p.b);
}
template <int LANES>
__device__ static inline double swapped_sum(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const Pair lo = swapped<LANES>((uint32_t)u), hi = swapped<LANES>((uint32_t)(u >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi.a << 32 | lo.a) + __builtin_bit_cast(double, (uint64_t)hi.b << 32 | lo.b);
}
__device__ static inline double column_sum(double v) { return swapped_sum<16>(swapped_sum<32>(v)); }
template <int N>
__device__ static inline Power column_power(const f4 (&v)[N], int lane) {
    float m = 0.0f;
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[t][i]));
    return turned_sign(power_of(column_max(m)), lane);
}

// A triangle of two terms times 64 rows of 16 columns, s0 and s1; TURNED: the transposed matrix. The terms go by in
// turns, since a product waits for the last one with the same sum.
template <bool TURNED>
__device__ static inline void triangle_times(const uint16_t *hi, const uint16_t *lo, int place, const Split &s0,
                                             const Split &s1, f4 (&r)[4]) {
    h8 h[4][2], l[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (TURNED ? s < t / 2 : s > t / 2) continue;
            h[t][s] = TURNED ? triangle_turned(hi, place, t, s) : triangle(hi, place, t, s);
            l[t][s] = TURNED ? triangle_turned(lo, place, t, s) : triangle(lo, place, t, s);
        }
#pragma unroll
    for (int t = 0; t < 4; ++t) r[t] = f4{};
#pragma unroll
    for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (TURNED ? s < t / 2 : s > t / 2) continue;
                const Split &x = s ? s1 : s0;
                r[t] = mma(term == 0 ? l[t][s] : h[t][s], term == 1 ? x.lo : x.hi, r[t]);
            }
}

// Sums and maxima over the 8 or 16 lanes of a group, on all of them: across pairs, quads, halves and the row, all within
// the vector unit (a shuffle by way of LDS is some 100 cycles).
template <int CTRL>
__device__ static inline float moved(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL, int ROWS = 0xf>
__device__ static inline double moved(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
constexpr int kPairs = 0xB1, kQuads = 0x4E, kHalves = 0x141, kRow = 0x140;
template <int LANES, typename T>
__device__ static inline T sum_over(T v) {
    v += moved<kPairs>(v);
    v += moved<kQuads>(v);
    if (LANES > 4) v += moved<kHalves>(v);
    if (LANES > 8) v += moved<kRow>(v);
    return v;
}
template <int LANES>
__device__ static inline float max_over(float v) {
    v = __builtin_fmaxf(v, moved<kPairs>(v));
    v = __builtin_fmaxf(v, moved<kQuads>(v));
    if (LANES > 4) v = __builtin_fmaxf(v, moved<kHalves>(v));
    if (LANES > 8) v = __builtin_fmaxf(v, moved<kRow>(v));
    return v;
}
__device__ static inline float sum16(float v) { return sum_over<16>(v); }
__device__ static inline float max16(float v) { return max_over<16>(v); }

// The sum over lanes 0 to this one, and its value on the last.
__device__ static inline double sum_up(double v) {
    v += moved<0x111>(v);       // rows of 16, by 1, 2, 4 and 8 lanes
    v += moved<0x112>(v);
    v += moved<0x114>(v);
    v += moved<0x118>(v);
    v += moved<0x142, 0xa>(v);  // a row's last to the next row; the second row's to the last two
    v += moved<0x143, 0xc>(v);
    return v;
}
__device__ static inline double last_lane(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, kWave - 1);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), kWave - 1);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// ---------------------------------------------------------------------------------------------
// Arguments.
// ---------------------------------------------------------------------------------------------
struct Delta {
    int S, B, H, G, K, V;
    int softplus, normalize;
    float scale;
    const uint16_t *q, *k, *v, *dt, *b;
    int64_t qs[3], ks[3], vs[3], ds[3], bs[3];
    const float *A, *bias;
    const int64_t *lengths;
};
__device__ static inline int length_of(const Delta &a, int b) {
    if (!a.lengths) return a.S;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.S ? a.S : (int)n;
}

// A head's step size and log2 decay for one row. A rate of -infinity is a decay of 0, and of 1 where there is
// no step; beyond e^-100000 a decay is 0 in any case, and a bound keeps sums and differences finite.
__device__ static inline float step_size(float raw, int softplus) { return softplus ? softplus_f(raw) : raw; }
__device__ static inline double log2_decay(float step, float rate) {
    const double g = step == 0.0f ? 0.0 : (double)step * (double)rate * 1.4426950408889634;
    return g < -1.5e5 ? -1.5e5 : g;
}

// The records of chunk n: [batch, head][chunk].
struct Records {
    uint8_t *key;       // key_bytes each
    uint8_t *xa;        // kXaBytes each
    RowCoef *coef;
    int64_t chunks;     // of a head
};
__host__ __device__ static inline uint64_t records_bytes(uint64_t key_heads, uint64_t heads, uint64_t chunks, int kp) {
    return chunks * (key_heads * key_bytes(kp) + heads * (kXaBytes + sizeof(RowCoef)));
}
__host__ static inline Records records_at(void *p, uint64_t key_heads, uint64_t heads, uint64_t chunks, int kp) {
    Records r;
    r.key = (uint8_t *)p;
    r.xa = r.key + chunks * key_heads * key_bytes(kp);
    r.coef = (RowCoef *)(r.xa + chunks * heads * kXaBytes);
    r.chunks = (int64_t)chunks;
    return r;
}

// Buffers of 16-bit values whose bounds the hardware keeps: loads past them give 0, stores past them are dropped.
// A lane whose column is not there starts at kNowhere, past any bound (bounds are below 2^31, and so is what is
// added to it).
constexpr uint32_t kNowhere = 0x80000000u;
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ static inline Buffer buffer_of(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, bytes, 0x00027000);
}

// Rows of S and V's width in memory: V's tensors are read through strides, the walks' own are padded to whole blocks
// of 64 columns and KP rows, so that nothing needs a check.
constexpr int kBlockV = 64;
__host__ __device__ static inline int padded_v(int V) { return (V + kBlockV - 1) / kBlockV * kBlockV; }

// A wave's 16 columns of a chunk's 64 rows, 16 values a lane, in the products' layout. WIDE: rows so far apart, or so
// close, that one chunk's are no buffer of their own.
struct Column16 {
    const uint16_t *base;       // of the head's first row
    int64_t stride;             // of a row
    int col, V;
};
__host__ __device__ static inline bool row_buffer(int64_t stride, int V) { return stride >= V && stride < (1 << 24); }
template <bool WIDE>
__device__ static inline void load_rows(const Column16 &c, int row0, int rows, int lane, uint16_t (&v)[4][4]) {
    const int grp = lane >> 4;
    const uint16_t *p = c.base + row0 * c.stride;
    const uint32_t st = 2 * (uint32_t)c.stride;
    const Buffer b = buffer_of(p, WIDE || rows <= 0 ? 0 : (rows < kC ? rows - 1 : kC - 1) * st + 2 * c.V);
    const uint32_t at = c.col < c.V ? 8 * grp * st + 2 * c.col : kNowhere;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row_of(t, 4 * grp + i);
            if (WIDE) v[t][i] = r < rows && c.col < c.V ? p[r * c.stride + c.col] : 0;
            else v[t][i] = __builtin_amdgcn_raw_buffer_load_b16(b, at + (row_of(t, 0) + i) * st, 0, 0);
        }
}

// A chunk's operands on their way to LDS: read into registers when the last chunk begins, written when it ends. (Loads
// straight to LDS need no registers, but while one is under way the compiler has any use of any other load wait
// for all of them.)
// OUTPUTS: false where none are made: neither A nor the image of q then.
template <int KP, int W, bool OUTPUTS>
struct Staged {
    static constexpr int kThreads = W * kWave, kKeys = (OUTPUTS ? 2 : 1) * kC * KP * 2, kXa = (OUTPUTS ? 4 : 2) * kTriangle * 2;
    static constexpr int kBytes = kKeys + kXa + (int)sizeof(RowCoef);
    static constexpr int kOfKeys = kKeys / 16 / kThreads, kOfXa = kXa / 16 / kThreads;
    static constexpr int kRest = (kXa - kOfXa * 16 * kThreads) / 8 / kThreads, kOfCoef = (int)sizeof(RowCoef) / 4 / kThreads;
    static_assert(kOfXa * 16 * kThreads + kRest * 8 * kThreads == kXa && kOfCoef * 4 * kThreads == (int)sizeof(RowCoef) &&
                  kOfKeys * 16 * kThreads == kKeys, "whole loads");
    typedef float f2 __attribute__((ext_vector_type(2)));
    f4 keys[kOfKeys], xa[kOfXa];
    f2 rest[kRest > 0 ? kRest : 1];
    float coef[kOfCoef];

    __device__ void load(const uint8_t *k, const uint8_t *x, const RowCoef *c) {
#pragma unroll
        for (int i = 0; i < kOfKeys; ++i) keys[i] = *lane_at((const f4 *)k + i * kThreads, threadIdx.x);
#pragma unroll
        for (int i = 0; i < kOfXa; ++i) xa[i] = *lane_at((const f4 *)x + i * kThreads, threadIdx.x);
#pragma unroll
        for (int i = 0; i < kRest; ++i) rest[i] = *lane_at((const f2 *)(x + kOfXa * 16 * kThreads) + i * kThreads, threadIdx.x);
#pragma unroll
        for (int i = 0; i < kOfCoef; ++i) coef[i] = *lane_at((const float *)c + i * kThreads, threadIdx.x);
    }
    __device__ void store(uint8_t *to) const {
#pragma unroll
        for (int i = 0; i < kOfKeys; ++i) ((f4 *)to)[i * kThreads + threadIdx.x] = keys[i];
#pragma unroll
        for (int i = 0; i < kOfXa; ++i) ((f4 *)(to + kKeys))[i * kThreads + threadIdx.x] = xa[i];
#pragma unroll
        for (int i = 0; i < kRest; ++i) ((f2 *)(to + kKeys + kOfXa * 16 * kThreads))[i * kThreads + threadIdx.x] = rest[i];
#pragma unroll
        for (int i = 0; i < kOfCoef; ++i) ((float *)(to + kKeys + kXa))[i * kThreads + threadIdx.x] = coef[i];
    }
};

// Blocks of one head, and heads of one key head, next to each other on one of the 8 dies, which have an L2 each.
__device__ static inline int same_die(int id, int all) { return all % 8 ? id : id % 8 * (all / 8) + id / 8; }

// A walk's blocks have four waves with states, or two where those all have a CU to themselves (for K above 64 LDS holds
// one block of either): more CUs then share what is read and written, and there are SIMDs left for more.
__host__ static inline bool half_blocks(const Delta &d, int segments) {
    return (int64_t)segments * d.B * d.H * (padded_v(d.V) / 32) <= 256;
}

__host__ static inline int padded(int64_t K) { return K <= 64 ? 64 : 128; }

// ---------------------------------------------------------------------------------------------
// Host side, of both directions.
// ---------------------------------------------------------------------------------------------
constexpr int kMaxK = 128;

inline uint64_t chunks_of(const mccb_delta_t *a) { return (uint64_t)((a->S + kC - 1) / kC); }
inline uint64_t state_bytes(const mccb_delta_t *a) { return (uint64_t)(a->B * a->H) * (uint64_t)(a->K * a->V) * 4; }
// fp32 values of every chunk: states, and rows
inline uint64_t chunk_states_bytes(const mccb_delta_t *a) {
    return chunks_of(a) * (uint64_t)(a->B * a->H) * (uint64_t)(padded(a->K) * padded_v((int)a->V)) * 4;
}
inline uint64_t chunk_rows_bytes(const mccb_delta_t *a) {
    return chunks_of(a) * (uint64_t)(a->B * a->H) * (uint64_t)(kC * padded_v((int)a->V)) * 4;
}
Delta delta_of(const mccb_delta_t *a);
int check_delta(const mccb_delta_t *a, bool token);
int delta_inputs(const mccb_delta_t *a, bool token, Span *in, int *count);
uint64_t records_size(const mccb_delta_t *a, uint64_t chunks);


}  // namespace delta
