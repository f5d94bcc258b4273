// delta_rule.hip -- the gated delta rule forward: chunks of 64 rows for prompts and training, and the
// single-token form. The formulas and the numbers' two 16-bit terms are in delta_common.h.
//
// delta_prepare makes what a chunk has without a state: the images of its rows of k and q, X and A. One
// block a chunk and key head; all chunks at once.
// delta_walk goes over a head's chunks with the state in registers. A wave owns 16 columns of V,
// and nothing passes between waves (but to second ones that make outputs, where heads are few): results of one product are the right operand of the next as they stand
// in the registers (row_of in delta_common.h), and the left operands, the same for all of a head's columns,
// come from LDS, where the next chunk's are written when this one's are done with, from loads that
// ran meanwhile.
// delta_one reads and writes the state once.
#include "delta_common.h"

using namespace delta;

namespace delta {

Delta delta_of(const mccb_delta_t *a) {
    Delta d{};
    d.S = (int)a->S, d.B = (int)a->B, d.H = (int)a->H, d.G = (int)a->G, d.K = (int)a->K, d.V = (int)a->V;
    d.softplus = a->softplus, d.normalize = a->normalize, d.scale = a->scale;
    d.q = (const uint16_t *)a->q, d.k = (const uint16_t *)a->k, d.v = (const uint16_t *)a->v;
    d.dt = (const uint16_t *)a->dt, d.b = (const uint16_t *)a->b;
    for (int i = 0; i < 3; ++i)
        d.qs[i] = a->q_stride[i], d.ks[i] = a->k_stride[i], d.vs[i] = a->v_stride[i], d.ds[i] = a->dt_stride[i],
        d.bs[i] = a->b_stride[i];
    d.A = a->A, d.bias = a->dt_bias, d.lengths = a->lengths;
    return d;
}

int check_delta(const mccb_delta_t *a, bool token) {
    if (!a) return MCCB_ERR_PARAM_NULLPTR;
    if (a->dtype != MCCB_BF16 && a->dtype != MCCB_FP16) return MCCB_ERR_PARAM_INVALID;
    if (a->S < 0 || a->S >= (1 << 28) || (token && a->S != 1) || a->B < 1 || a->H < 1 || a->B > 65535 ||
        a->H > 65535 || a->B * a->H > 65535 || a->G < 1 || a->G > a->H || a->H % a->G != 0 || a->K < 1 ||
        a->K > kMaxK || a->V < 1 || a->V > 256)
        return MCCB_ERR_SHAPE;
    if (!(a->scale >= -3.0e38f && a->scale <= 3.0e38f)) return MCCB_ERR_PARAM_INVALID;
    return MCCB_OK;
}

// Spans of the inputs; token: without a row axis.
int delta_inputs(const mccb_delta_t *a, bool token, Span *in, int *count) {
    if (!a->A || (a->S > 0 && (!a->q || !a->k || !a->v || !a->dt || !a->b))) return MCCB_ERR_PARAM_NULLPTR;
    const void *const p[5] = {a->q, a->k, a->v, a->dt, a->b};
    const int64_t *const st[5] = {a->q_stride, a->k_stride, a->v_stride, a->dt_stride, a->b_stride};
    const int64_t heads[5] = {a->G, a->G, a->H, a->H, a->H}, width[5] = {a->K, a->K, a->V, 1, 1};
    int n = 0;
    for (int i = 0; i < 5; ++i) {
        const int64_t size[4] = {token ? 1 : a->S, a->B, heads[i], width[i]};
        const int64_t stride[4] = {token ? 0 : st[i][0], st[i][1], st[i][2], 1};
        uint64_t bytes;
        if (!extent(4, size, stride, 2, &bytes) || misaligned(p[i], 2)) return MCCB_ERR_PARAM_INVALID;
        in[n++] = {p[i], bytes};
    }
    if (misaligned(a->A, 4) || misaligned(a->dt_bias, 4) || misaligned(a->lengths, 8) || misaligned(a->state, 4))
        return MCCB_ERR_PARAM_INVALID;
    in[n++] = {a->A, (uint64_t)a->H * 4};
    in[n++] = {a->dt_bias, (uint64_t)a->H * 4};
    in[n++] = {a->lengths, (uint64_t)a->B * 8};
    in[n++] = {a->state, state_bytes(a)};
    *count = n;
    return MCCB_OK;
}

uint64_t records_size(const mccb_delta_t *a, uint64_t chunks) {
    return align16(records_bytes((uint64_t)(a->B * a->G), (uint64_t)(a->B * a->H), chunks, padded(a->K)));
}

}  // namespace delta

namespace {

// ---------------------------------------------------------------------------------------------
// Preparation.
// ---------------------------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kLd = kC + 4;         // fp32 row of the triangular matrices in LDS

// One 16-bit row chunk of 8 values, zeros past K.
__device__ static inline HVec<8>::t row_chunk(const uint16_t *p, int left) {
    HVec<8>::t v = {};
    if (left >= 8) v = *(const HVec<8>::t *)p;
    else
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) v[i] = p[i];
    return v;
}

// The 64 rows of q or k: read all at once, then made an image in LDS and in memory, and the rows' factors.
template <int DT, int KP>
struct RawRows {
    static constexpr int kLanes = KP / 8, kRows = kPrepThreads / kLanes, kTurns = kC / kRows;
    HVec<8>::t raw[kTurns];

    __device__ void load(const Delta &a, const uint16_t *base, const int64_t (&st)[3], int b, int g, int row0, int live) {
        const int lane = threadIdx.x % kLanes;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int r = threadIdx.x / kLanes + i * kRows;
            raw[i] = HVec<8>::t{};
            if (r < live)
                raw[i] = row_chunk(base + (int64_t)(row0 + r) * st[0] + b * st[1] + g * st[2] + 8 * lane, a.K - 8 * lane);
        }
    }
    __device__ void image(const Delta &a, uint16_t *lds, uint16_t *to, float *factor, float *factor_out, float *power_out) const {
        const int lane = threadIdx.x % kLanes;
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int r = threadIdx.x / kLanes + t * kRows;
            float v[8], m = 0.0f, ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_f32<DT>(raw[t][i]), m = __builtin_fmaxf(m, __builtin_fabsf(v[i]));
            // the row's largest value is brought to 2^14..2^15
            m = max_over<kLanes>(m);
            int e = m > 0.0f ? ((__float_as_uint(m) >> 23) & 255) - 127 - 14 : -10;
            e = e < -100 ? -100 : e > 126 ? 126 : e;
            h8 h;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = __builtin_ldexpf(v[i], -e);
                ss = __builtin_fmaf(v[i], v[i], ss);
                h[i] = (_Float16)v[i];
            }
            ss = sum_over<kLanes>(ss);
            const int at = image_at<KP>(r, lane);
            *(h8 *)(lds + at) = h;
            *(h8 *)(to + at) = h;
            if (lane == 0) {
                // eps next to the row's square in whichever scale has them both as numbers
                float f = __builtin_ldexpf(1.0f, e);
                if (a.normalize)
                    f = e < 0 ? f / __builtin_sqrtf(__builtin_ldexpf(ss, 2 * e) + kNormEps)
                              : 1.0f / __builtin_sqrtf(ss + __builtin_ldexpf(kNormEps, -2 * e));
                // a row of zeros gets zeros from whatever its factor meets here, and must not be the largest of what is
                // split; its gradient has the factor, and a sign that says so
                factor[r] = m > 0.0f ? f : 0.0f;
                factor_out[r] = f;
                power_out[r] = __builtin_ldexpf(m > 0.0f ? 1.0f : -1.0f, -e);
            }
        }
    }
};

// A triangular 64x64 matrix in LDS as two terms in memory; returns the power of two taken out, of the whole matrix or
// (ROWS) of the thread's row, tid / 4.
template <bool ROWS>
__device__ static __forceinline__ float image_square(const float *m, uint16_t *hi, uint16_t *lo, float *part, int tid) {
    const int row = tid / 4, c0 = tid % 4 * 16;
    f4 v[4];
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = *(const f4 *)(m + row * kLd + c0 + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) big = __builtin_fmaxf(big, __builtin_fabsf(v[i][j]));
    }
    if (ROWS) {
        big = max_over<4>(big);
    } else {
        big = column_max(max16(big));
        if (tid % kWave == 0) part[tid / kWave] = big;
        lds_barrier();
        big = __builtin_fmaxf(__builtin_fmaxf(part[0], part[1]), __builtin_fmaxf(part[2], part[3]));
    }
    const Power p = power_of(big);
    if (c0 / 32 <= row / 32)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Split s = split(v[2 * i], v[2 * i + 1], p.inv);
            const int at = block_of(row / 32, c0 / 32) + block_at(row % 32, c0 % 32 / 8 + i);
            *(h8 *)(hi + at) = s.hi;
            *(h8 *)(lo + at) = s.lo;
        }
    return p.back;
}

// One 16x16 block of a product of fp32 matrices in LDS, added to c: rows r0.. of `l` from column k0 times `y`
// (registers of a lane: rows 4 (lane / 16) + i of column lane % 16, as the instruction leaves them).
__device__ static inline f4 block_product(const float *l, int r0, int k0, f4 y, f4 c, int lane) {
    const f4 a = *(const f4 *)(l + (r0 + (lane & 15)) * kLd + k0 + 4 * (lane >> 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], y[i], c, 0, 0, 0);
    return c;
}
__device__ static inline f4 square_at(const float *m, int r0, int c0, int lane) {
    f4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = m[(r0 + 4 * (lane >> 4) + i) * kLd + c0 + (lane & 15)];
    return v;
}
__device__ static inline void block_to(float *m, int r0, int c0, f4 v, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m[(r0 + 4 * (lane >> 4) + i) * kLd + c0 + (lane & 15)] = -v[i];
}

// X = (I + L)^-1 of a strictly lower triangular L: the diagonal blocks of 16 by substitution (a lane each
// column), then twice the lower left quarter, -X2 L21 X1, on the fp32 matrix units. All of X is written.
__device__ static __forceinline__ void invert(const float *L, float *X, int wave, int tid) {
    const int lane = tid % kWave;
    for (int i = tid; i < kC * kC / 4; i += kPrepThreads) *(f4 *)(X + i / 16 * kLd + i % 16 * 4) = f4{};
    lds_barrier();
    if (wave == 0) {
        const int d0 = 16 * (lane >> 4), c = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
#pragma unroll
        for (int j4 = 0; j4 < 16; j4 += 4) {  // a row that is done goes into all later ones at once
            f4 l[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i > j4) l[i] = *(const f4 *)(L + (d0 + i) * kLd + d0 + j4);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i > j4 + j) x[i] = __builtin_fmaf(-l[i][j], x[j4 + j], x[i]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) X[(d0 + i) * kLd + d0 + c] = x[i];
    }
    lds_barrier();
    if (wave < 2) {
        const int a = 32 * wave, b = a + 16;
        const f4 y = block_product(L, b, a, square_at(X, a, a, lane), f4{}, lane);
        block_to(X, b, a, block_product(X, b, b, y, f4{}, lane), lane);
    }
    lds_barrier();
    if (wave < 2) {
        const int c = 16 * wave;
        const f4 x0 = square_at(X, 0, c, lane), x1 = square_at(X, 16, c, lane);
        f4 y2 = block_product(L, 32, 0, x0, f4{}, lane), y3 = block_product(L, 48, 0, x0, f4{}, lane);
        y2 = block_product(L, 32, 16, x1, y2, lane), y3 = block_product(L, 48, 16, x1, y3, lane);
        const f4 x2 = block_product(X, 32, 32, y2, f4{}, lane);
        f4 x3 = block_product(X, 48, 32, y2, f4{}, lane);
        x3 = block_product(X, 48, 48, y3, x3, lane);
        block_to(X, 32, c, x2, lane);
        block_to(X, 48, c, x3, lane);
    }
    lds_barrier();
}

// Bound by what it writes, and by the chain of products in X's blocks where there are few chunks: S=4096 B=4 H=32 G=16
// K=V=128, 4096 blocks, 144 us for 373 MB written and 141 read (3.6 TB/s; 4 registers are spilled); S=513 B=2 H=6 G=3 K=64, 54
// blocks, 13 us.
template <int DT, int KP>
__global__ void __launch_bounds__(kPrepThreads, 4) delta_prepare(Delta a, Records rec, int n0) {
    constexpr int kImages = 2 * kC * KP * (int)sizeof(uint16_t), kSquares = 2 * kC * kLd * (int)sizeof(float);
    __shared__ __align__(16) uint8_t smem[kImages > kSquares ? kImages : kSquares];  // rows first, then L, X
    __shared__ float kr[kC], qr[kC], beta[kC], part[4];
    __shared__ double cum[kC];
    const int n = blockIdx.x, b = blockIdx.y / a.G, g = blockIdx.y % a.G;
    const int row0 = (n0 + n) * kC, live = length_of(a, b) - row0;
    if (live <= 0) return;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int heads = a.H / a.G;
    // a head's step sizes and gates, ahead of its turn: a lane each row, the first wave's
    uint16_t raw = 0, gate = 0;
    auto read_gates = [&](int h) {
        const int64_t row = row0 + (int)(threadIdx.x % kWave);
        if ((int)(threadIdx.x % kWave) < live) {
            raw = a.dt[row * a.ds[0] + b * a.ds[1] + h * a.ds[2]];
            gate = a.b[row * a.bs[0] + b * a.bs[1] + h * a.bs[2]];
        }
    };
    if (wave == 0) read_gates(g * heads);
    uint16_t *kt = (uint16_t *)smem, *qt = kt + kC * KP;
    {
        uint8_t *key = rec.key + ((int64_t)(b * a.G + g) * rec.chunks + n) * key_bytes(KP);
        uint16_t *images = (uint16_t *)key;
        float *factors = (float *)(images + 2 * kC * KP);
        RawRows<DT, KP> k, q;
        k.load(a, a.k, a.ks, b, g, row0, live);
        q.load(a, a.q, a.qs, b, g, row0, live);
        k.image(a, kt, images, kr, factors, factors + 2 * kC);
        q.image(a, qt, images + kC * KP, qr, factors + kC, factors + 3 * kC);
    }
    lds_barrier();
    // K~ K~^T and Q~ K~^T: wave w has rows 16 w.. of both, up to the diagonal block
    f4 kk[4] = {}, qk[4] = {};
    const int m = lane & 15, grp = lane >> 4;
#pragma unroll
    for (int s = 0; s < KP / 32; ++s) {
        const int c = 4 * s + grp;
        const h8 ak = *(const h8 *)(kt + image_at<KP>(16 * wave + m, c));
        const h8 aq = *(const h8 *)(qt + image_at<KP>(16 * wave + m, c));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= wave) {
                const h8 bk = *(const h8 *)(kt + image_at<KP>(16 * j + m, c));
                kk[j] = mma(ak, bk, kk[j]);
                qk[j] = mma(aq, bk, qk[j]);
            }
    }
    float *P = (float *)smem, *X = P + kC * kLd;
    for (int hh = 0; hh < heads; ++hh) {
        const int tid = anew(threadIdx.x), lane = tid % kWave, m = lane & 15, grp = lane >> 4;
        const int h = g * heads + hh;
        const int64_t at = (int64_t)(b * a.H + h) * rec.chunks + n;
        RowCoef *coef = rec.coef + at;
        uint16_t *xa = (uint16_t *)(rec.xa + at * kXaBytes);
        double total = 0.0, mine = 0.0;
        if (wave == 0) {
            if (lane < live)
                mine = log2_decay(step_size(to_f32<DT>(raw) + (a.bias ? a.bias[h] : 0.0f), a.softplus), a.A[h]);
            const float bt = lane < live ? sigmoid_f(to_f32<DT>(gate)) : 0.0f;
            if (hh + 1 < heads) read_gates(h + 1);
            mine = sum_up(mine);
            total = last_lane(mine);
            cum[lane] = mine, beta[lane] = bt;
        }
        lds_barrier();  // also: the last head's reads of P and X, or the rows' reads above, are done
        double gi[4];
        float bi[4], ki[4], qi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * wave + 4 * grp + i;
            gi[i] = cum[r], bi[i] = beta[r], ki[i] = kr[r], qi[i] = qr[r] * a.scale;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 16 * j + m;
            const double gj = cum[c];
            const float kj = kr[c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * wave + 4 * grp + i;
                const float decay = c <= r ? exp2_f((float)(gi[i] - gj)) * kj : 0.0f;
                P[r * kLd + c] = c <= r ? decay * qi[i] * qk[j][i] : 0.0f;
                X[r * kLd + c] = c < r ? decay * ki[i] * bi[i] * kk[j][i] : 0.0f;
            }
        }
        lds_barrier();
        const float sa = image_square<true>(P, xa + 2 * kTriangle, xa + 3 * kTriangle, part, tid);
        if (tid % 4 == 0) coef->a[tid / 4] = sa;
        lds_barrier();
        invert(X, P, wave, tid);
        const float sx = image_square<false>(P, xa, xa + kTriangle, part, tid);
        if (wave == 0) {
            const float ek = exp2_f((float)mine), k1 = kr[lane];
            coef->p[lane] = ek * k1;
            coef->beta[lane] = beta[lane];
            coef->q[lane] = a.scale * ek * qr[lane];
            coef->u[lane] = exp2_f((float)(total - mine)) * k1;
            coef->cum[lane] = mine;
            if (lane == 0) coef->whole = exp2_f((float)total), coef->x = sx;
        }
    }
}

// ---------------------------------------------------------------------------------------------
// The walk.
// ---------------------------------------------------------------------------------------------
// What a wave with a state hands to the one that makes its outputs.
template <int KP, int W>
struct Handed {
    h8 s[W][KP / 32][2][kWave];     // S0 as a right operand
    f4 u[W][4][kWave];
    float s_back[W][16], u_up[W][16];
};

struct Walk {
    const float *state_in;          // [B,H,K,V] or NULL
    float *state_out;               // or NULL
    uint16_t *out;                  // [S,B,H,V]
    float *states, *u;              // kept for the backward, padded: [B,H][chunk][K,V] and [B,H][chunk][64,V]; or NULL
    float *ends;                    // [segment][B,H][K, V + K], padded: what a first pass over segments finds
    float *carry;                   // [segment - 1][B,H][K,V], padded: the state before each segment but the first
    int chunks, per;                // chunks, and of a segment
    int segments;
    int blocks;                     // of columns, a head
};

// Bound by the vector and matrix instructions of one wave a SIMD, issued in 50 % of its cycles, and by what they wait for
// (one product's largest values, then the next one's operands): S=4096 B=4 H=32 G=16 K=V=128, 318 us, 5.0 a chunk.
// Training, S=2048 B=4 H=16, 143 us, of which the kept states and U (201 MB) are some 30.
// KEEP: the states and U are kept. (Two waves a SIMD would fit: with all of a SIMD's registers the compiler has the
// products' results in accumulation registers and moves each of them.)
// SEGMENTS: where there are few heads, the first pass of two over a sequence that is cut into segments, all at once:
// no outputs, but what a segment makes of the state before it, S -> T S + F. F is what the walk makes of a state of
// zeros, and T's columns are what it makes of the identity's where there is nothing to write (V = 0): K more columns.
// delta_carry then finds the states before the segments, and the second pass walks all of them at once with outputs.
// W: waves with states, four a block; or two where blocks are few (half_blocks), and then each has a second one (PAIRS)
// that makes the outputs of S0 and U as it finds them in LDS, and brings the operands: neither is on the way from one
// state to the next. Whole forwards: training, as above, 235 -> 187 us, S=777 B=5 H=6 K=96 V=80 75 -> 65; where they have no
// CU each 384 -> 488 (S=4096 B=4 H=32), 378 -> 416 (S=16384 H=16 in segments).
template <int DT, int KP, int W, bool KEEP, bool WIDE, bool SEGMENTS>
__global__ void __launch_bounds__((W == 2 ? 2 : 1) * W *kWave, 2) delta_walk(Delta a, Records rec, Walk w) {
    constexpr bool PAIRS = W == 2;
    constexpr int KT = KP / 16, KS = KP / 32;
    typedef Staged<KP, W, !SEGMENTS> Stage;
    typedef Handed<KP, W> Pairs;
    constexpr int kBuf = Stage::kBytes, kKeys = Stage::kKeys;
    __shared__ __align__(16) uint8_t smem[2 * kBuf + (PAIRS ? (int)sizeof(Pairs) : 0)];
    Pairs *const handed = (Pairs *)(smem + 2 * kBuf);
    const int lane = threadIdx.x % kWave, all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wave = PAIRS ? all_waves % W : all_waves;
    const int m = lane & 15, grp = lane >> 4;
    const int lk_at = left_place<KP>(lane), tk_at = turned_place<KP>(lane), ls_at = triangle_place(lane);
    const int id = same_die(blockIdx.x, gridDim.x);
    const int all = a.B * a.H, segment = id / (w.blocks * all), bh = id / w.blocks % all;
    const int b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int col = (id % w.blocks * W + wave) * 16 + m, VP = padded_v(a.V);
    const int n0 = segment * w.per, n1 = n0 + w.per < w.chunks ? n0 + w.per : w.chunks;
    const int length = length_of(a, b);
    const int chunks = (length + kC - 1) / kC, end = chunks < n1 ? chunks : n1;

    const uint8_t *key = rec.key + (int64_t)(b * a.G + g) * rec.chunks * key_bytes(KP);
    const uint8_t *xa = rec.xa + (int64_t)bh * rec.chunks * kXaBytes;
    const RowCoef *coefs = rec.coef + (int64_t)bh * rec.chunks;
    Stage stage;
    auto fetch = [&](int n) {
        stage.load(key + n * (int64_t)key_bytes(KP), xa + n * (int64_t)kXaBytes, coefs + n);
    };
    const Column16 vcol = {a.v + b * a.vs[1] + h * a.vs[2], a.vs[0], col, a.V};
    const uint32_t out_row = 2u * (uint32_t)(a.B * a.H) * a.V;       // bytes
    const uint32_t out_at = col < a.V ? 8 * grp * out_row + 2 * (h * a.V + col) : kNowhere;
    // out = q Q~ S0 + A U
    auto output = [&](int n, const uint8_t *buf, const f4 (&O)[4], float s_back, const f4 (&U)[4], float up) {
        const uint16_t *ah = (const uint16_t *)(buf + kKeys) + 2 * kTriangle, *al = ah + kTriangle;
        const RowCoef *coef = (const RowCoef *)(buf + kKeys + Stage::kXa);
        const Power p = column_power(U, lane);
        f4 AU[4];
        triangle_times<false>(ah, al, ls_at, split(U[0], U[1], p.inv), split(U[2], U[3], p.inv), AU);
        const float back = p.back * up;
        const int left_rows = length - n * kC;  // rows past the length are zeros, whatever the matrices' zeros meet
        const Buffer to = buffer_of(w.out + (int64_t)n * kC * (out_row / 2) + (int64_t)b * a.H * a.V,
                                    (left_rows < kC ? left_rows - 1 : kC - 1) * out_row + 2u * a.H * a.V);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f4 cq = *(const f4 *)(coef->q + row_of(t, 4 * grp)) * s_back;
            const f4 ca = *(const f4 *)(coef->a + row_of(t, 4 * grp)) * back;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                __builtin_amdgcn_raw_buffer_store_b16(from_f32<DT>(__builtin_fmaf(AU[t][i], ca[i], cq[i] * O[t][i])), to,
                                                      out_at + (row_of(t, 0) + i) * out_row, 0, 0);
        }
    };
    if constexpr (PAIRS)
        if (all_waves < W) {
            if (n0 < end) {
                fetch(n0);
                stage.store(smem + (n0 & 1) * kBuf);
                lds_barrier();
            }
            for (int n = n0; n < end; ++n) {
                const uint8_t *buf = smem + (n & 1) * kBuf;
                const uint16_t *qt = (const uint16_t *)buf + kC * KP;
                fetch(n + 1 < end ? n + 1 : n);
                lds_barrier();  // S0 is there
                f4 O[4] = {}, U[4];
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int term = 1; term >= 0; --term) {
                        const h8 x = handed->s[wave][s][term][lane];
#pragma unroll
                        for (int t = 0; t < 4; ++t) O[t] = mma(left<KP>(qt, lk_at, t, s), x, O[t]);
                    }
                const float s_back = handed->s_back[wave][m];
                lds_barrier();  // and U
#pragma unroll
                for (int t = 0; t < 4; ++t) U[t] = handed->u[wave][t][lane];
                output(n, buf, O, s_back, U, handed->u_up[wave][m]);
                stage.store(smem + (~n & 1) * kBuf);
                lds_barrier();  // as below
            }
            return;
        }
    f4 S[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = row_of(t, 4 * grp + i);
            if (SEGMENTS) S[t][i] = col == VP + k ? 1.0f : 0.0f;
            else if (segment > 0) S[t][i] = w.carry[(((int64_t)(segment - 1) * all + bh) * KP + k) * VP + col];
            else S[t][i] = w.state_in && k < a.K && col < a.V ? w.state_in[((int64_t)bh * a.K + k) * a.V + col] : 0.0f;
        }
    float *keep_s = KEEP ? w.states + ((int64_t)bh * rec.chunks * KP + 8 * grp) * VP + col : nullptr;
    float *keep_u = KEEP ? w.u + ((int64_t)bh * rec.chunks * kC + 8 * grp) * VP + col : nullptr;
    uint16_t v[4][4];
    if (n0 < end) {
        if (!PAIRS) fetch(n0);
        load_rows<WIDE>(vcol, n0 * kC, length - n0 * kC, lane, v);
        if (!PAIRS) stage.store(smem + (n0 & 1) * kBuf);
        lds_barrier();
    }
    for (int n = n0; n < end; ++n) {
        const uint8_t *buf = smem + (n & 1) * kBuf;
        const uint16_t *kt = (const uint16_t *)buf, *qt = kt + kC * KP;
        const uint16_t *xh = (const uint16_t *)(buf + kKeys), *xl = xh + kTriangle;
        const RowCoef *coef = (const RowCoef *)(buf + kKeys + Stage::kXa);
        if (!PAIRS) fetch(n + 1 < end ? n + 1 : n);
        if (KEEP) {
            float *to = keep_s + (int64_t)n * KP * VP;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) to[(row_of(t, 0) + i) * VP] = S[t][i];
        }
        // K~ S0 and Q~ S0
        f4 P[4] = {}, O[4] = {};
        const Power ps = column_power(S, lane);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const Split sp = split(S[2 * s], S[2 * s + 1], ps.inv);
            if constexpr (PAIRS) {
                handed->s[wave][s][0][lane] = sp.hi;
                handed->s[wave][s][1][lane] = sp.lo;
            }
            h8 lk[4], lq[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                lk[t] = left<KP>(kt, lk_at, t, s);
                if (!SEGMENTS && !PAIRS) lq[t] = left<KP>(qt, lk_at, t, s);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                P[t] = mma(lk[t], sp.lo, P[t]);
                if (!SEGMENTS && !PAIRS) O[t] = mma(lq[t], sp.lo, O[t]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                P[t] = mma(lk[t], sp.hi, P[t]);
                if (!SEGMENTS && !PAIRS) O[t] = mma(lq[t], sp.hi, O[t]);
            }
        }
        if constexpr (PAIRS) {
            if (grp == 0) handed->s_back[wave][m] = ps.back;
            lds_barrier();
        }
        // beta (V - p K~ S0)
        f4 R[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int r = row_of(t, 4 * grp);
            const f4 cp = *(const f4 *)(coef->p + r) * ps.back, cb = *(const f4 *)(coef->beta + r);
#pragma unroll
            for (int i = 0; i < 4; ++i) R[t][i] = cb[i] * __builtin_fmaf(-cp[i], P[t][i], to_f32<DT>(v[t][i]));
        }
        load_rows<WIDE>(vcol, (n + 1) * kC, length - (n + 1) * kC, lane, v);
        // U = X R, without the powers of two in `up`
        f4 U[4];
        float up;
        {
            const Power p = column_power(R, lane);
            up = p.back * coef->x;
            triangle_times<false>(xh, xl, ls_at, split(R[0], R[1], p.inv), split(R[2], R[3], p.inv), U);
        }
        if (KEEP) {
            float *to = keep_u + (int64_t)n * kC * VP;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) to[(row_of(t, 0) + i) * VP] = up * U[t][i];
        }
        if constexpr (PAIRS) {
#pragma unroll
            for (int t = 0; t < 4; ++t) handed->u[wave][t][lane] = U[t];
            if (grp == 0) handed->u_up[wave][m] = up;
            lds_barrier();
        } else if constexpr (!SEGMENTS) {
            output(n, buf, O, ps.back, U, up);
        }
        // S = whole S0 + K~^T u U
        {
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] *= *(const f4 *)(coef->u + row_of(t, 4 * grp));
            const Power p = column_power(U, lane);
            const Split s0 = split(U[0], U[1], p.inv), s1 = split(U[2], U[3], p.inv);
            const float whole = coef->whole, back = p.back * up;
#pragma unroll
            for (int t = 0; t < KT; t += 4) {
                f4 d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 0), s0.lo, f4{});
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 1), s1.lo, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 0), s0.hi, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 1), s1.hi, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[t + i][j] = __builtin_fmaf(whole, S[t + i][j], back * d[i][j]);
            }
        }
        if (!PAIRS) stage.store(smem + (~n & 1) * kBuf);
        lds_barrier();  // the next chunk's operands are there, and all waves are done with this one's
    }
    if (SEGMENTS) {
        const int wide = VP + KP;
        float *to = w.ends + (((int64_t)segment * all + bh) * KP + 8 * grp) * wide + col;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[(row_of(t, 0) + i) * wide] = S[t][i];
        return;
    }
    if (w.state_out && segment == w.segments - 1) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = row_of(t, 4 * grp + i);
                if (k < a.K && col < a.V) w.state_out[((int64_t)bh * a.K + k) * a.V + col] = S[t][i];
            }
    }
    // rows past the length are zeros
    const int from = length > n0 * kC ? length : n0 * kC, to = n1 * kC < a.S ? n1 * kC : a.S;
    for (int row = from + grp; row < to; row += 4)
        if (col < a.V) w.out[(((int64_t)row * a.B + b) * a.H + h) * a.V + col] = 0;
}

// The states before the segments, one after the other: S -> T S + F. A block has 16 columns, a wave 32 rows of them;
// what a segment needs of T and F does not depend on S and is read and split one segment ahead, and S goes from wave to
// wave in LDS as the products' right operand, with a power of two for each wave's rows of a column. Segments that begin
// past the sequence's length hand S on as it is, in all its bits. S=16384 B=1 H=16
// K=V=128, eight segments: 25 us; with all rows in one wave 63.
template <int KP>
__global__ void __launch_bounds__(KP / 32 * kWave, 1) delta_carry(Delta a, Walk w) {
    constexpr int KS = KP / 32;     // steps of a product, and waves
    __shared__ __align__(16) h8 parts[2][KS][2][kWave];
    __shared__ float backs[2][KS][16];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int m = lane & 15, grp = lane >> 4, all = a.B * a.H, VP = padded_v(a.V), wide = VP + KP, blocks = VP / 16;
    const int bh = blockIdx.x / blocks, col = blockIdx.x % blocks * 16 + m;
    f4 S[2], F[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = row_of(2 * wave + t, 4 * grp + i);
            S[t][i] = w.state_in && k < a.K && col < a.V ? w.state_in[((int64_t)bh * a.K + k) * a.V + col] : 0.0f;
        }
    f4 x[2][KS][2];                 // T's rows
    auto read = [&](int n) {
        const float *end = w.ends + ((int64_t)n * all + bh) * KP * wide;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float *row = end + row_of(2 * wave + t, m) * wide + VP + 8 * grp;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) x[t][s][j] = *(const f4 *)(row + 32 * s + 4 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) F[t][i] = end[(row_of(2 * wave + t, 4 * grp) + i) * wide + col];
        }
    };
    auto write = [&](int n) {
        float *to = w.carry + (((int64_t)n * all + bh) * KP + 8 * grp) * VP + col;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[(row_of(2 * wave + t, 0) + i) * VP] = S[t][i];
    };
    const int chunks = (length_of(a, bh / a.H) + kC - 1) / kC;
    const int live = (chunks + w.per - 1) / w.per, last = live < w.segments - 1 ? live : w.segments - 1;
    if (last > 0) read(0);
    for (int n = 0; n < last; ++n) {
        Split T[2][KS];
        float back[2];
        f4 next[2] = {F[0], F[1]};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float big = 0.0f;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    big = __builtin_fmaxf(big, __builtin_fmaxf(__builtin_fabsf(x[t][s][0][i]), __builtin_fabsf(x[t][s][1][i])));
            const Power p = power_of(column_max(max16(big)));
            back[t] = p.back;
#pragma unroll
            for (int s = 0; s < KS; ++s) T[t][s] = split(x[t][s][0], x[t][s][1], p.inv);
        }
        read(n + 1 < last ? n + 1 : n);
        const Power p = column_power(S, lane);
        const Split mine = split(S[0], S[1], p.inv);
        const int buf = n & 1;
        parts[buf][wave][0][lane] = mine.hi, parts[buf][wave][1][lane] = mine.lo;
        if (grp == 0) backs[buf][wave][m] = p.back;
        lds_barrier();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const h8 hi = parts[buf][s][0][lane], lo = parts[buf][s][1][lane];
            const float up = backs[buf][s][m];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f4 d = mma(T[t][s].lo, hi, f4{});
                d = mma(T[t][s].hi, lo, d);
                d = mma(T[t][s].hi, hi, d);
#pragma unroll
                for (int i = 0; i < 4; ++i) next[t][i] = __builtin_fmaf(d[i], back[t] * up, next[t][i]);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) S[t] = next[t];
        write(n);
    }
    for (int n = last; n + 1 < w.segments; ++n) write(n);
}

// ---------------------------------------------------------------------------------------------
// One token. A block has 32 columns of a head's state, a thread four of them in every 32nd row. With
// a = decay, p = a Kn^T S and o = a Qn^T S from one pass over the state: u = beta (v - p),
// out = o + (qn . kn) u, S = a S + kn u^T. Bound by the state's bytes, once in and once out: B=32 H=16 K=V=128, 67 MB in
// 13.6 us (4.9 TB/s); B=1 H=6 K=V=64 4.6 us, a launch.
// ---------------------------------------------------------------------------------------------
constexpr int kStepCols = 32, kStepThreads = 256;
constexpr int kStepRows = kMaxK / 32;

template <int DT>
__global__ void __launch_bounds__(kStepThreads) delta_one(Delta a, float *state, uint16_t *out) {
    __shared__ float kn[kMaxK], qn[kMaxK], norms[3][2];
    __shared__ __align__(16) float part[4][8][8];
    const int t = threadIdx.x, lane = t % kWave, wave = t / kWave;
    const int b = blockIdx.y / a.H, h = blockIdx.y % a.H, g = h / (a.H / a.G);
    const int c0 = blockIdx.x * kStepCols + (t & 7) * 4, r0 = t >> 3;
    float *S = state + (int64_t)blockIdx.y * a.K * a.V;
    typedef float row4 __attribute__((ext_vector_type(4), aligned(4)));
    row4 s[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int k = r0 + 32 * i;
        s[i] = row4{};
        if (k < a.K) {
            const float *p = S + (int64_t)k * a.V + c0;
            if (c0 + 4 <= a.V) s[i] = *(const row4 *)p;
            else
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j < a.V) s[i][j] = p[j];
        }
    }
    // the rows of k and q, a value a thread in the first two waves
    float kv = 0.0f, qv = 0.0f;
    if (t < a.K) {
        kv = to_f32<DT>(a.k[b * a.ks[1] + g * a.ks[2] + t]);
        qv = to_f32<DT>(a.q[b * a.qs[1] + g * a.qs[2] + t]);
    }
    const float raw = to_f32<DT>(a.dt[b * a.ds[1] + h * a.ds[2]]) + (a.bias ? a.bias[h] : 0.0f);
    const float decay = exp2_f((float)log2_decay(step_size(raw, a.softplus), a.A[h]));
    const float beta = sigmoid_f(to_f32<DT>(a.b[b * a.bs[1] + h * a.bs[2]]));
    auto sums = [&]() {
        if (t < kMaxK) {
            const float kk = column_sum(sum16(kv * kv)), qq = column_sum(sum16(qv * qv)), kq = column_sum(sum16(kv * qv));
            if (lane == 0) norms[0][wave] = kk, norms[1][wave] = qq, norms[2][wave] = kq;
        }
        __syncthreads();
    };
    sums();
    float ek = kNormEps, eq = kNormEps;
    const float most = 3.4e38f;
    const bool large_k = norms[0][0] + norms[0][1] > most, large_q = norms[1][0] + norms[1][1] > most;
    if (a.normalize && (large_k || large_q)) {  // squares past fp32's largest: the row as 2^-64 of itself, next to which eps is nothing
        if (large_k) kv *= 0x1p-64f, ek = 0.0f;
        if (large_q) qv *= 0x1p-64f, eq = 0.0f;
        __syncthreads();
        sums();
    }
    const float rk = a.normalize ? 1.0f / __builtin_sqrtf(norms[0][0] + norms[0][1] + ek) : 1.0f;
    const float rq = a.scale * (a.normalize ? 1.0f / __builtin_sqrtf(norms[1][0] + norms[1][1] + eq) : 1.0f);
    const float along = (norms[2][0] + norms[2][1]) * rk * rq;
    if (t < kMaxK) kn[t] = kv * rk, qn[t] = qv * rq;
    __syncthreads();
    float acc[8] = {};
    float kr[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int k = r0 + 32 * i;
        kr[i] = kn[k];
        const float q = qn[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = __builtin_fmaf(kr[i], s[i][j], acc[j]);
            acc[4 + j] = __builtin_fmaf(q, s[i][j], acc[4 + j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        acc[j] = column_sum(acc[j] + moved<0x128>(acc[j]));  // lanes 8, 16 and 32 apart
    }
    if (lane < 8) {
        *(f4 *)part[wave][lane] = f4{acc[0], acc[1], acc[2], acc[3]};
        *(f4 *)(part[wave][lane] + 4) = f4{acc[4], acc[5], acc[6], acc[7]};
    }
    __syncthreads();
    f4 p = {}, o = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) p += *(const f4 *)part[i][t & 7], o += *(const f4 *)(part[i][t & 7] + 4);
    f4 u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float v = c0 + j < a.V ? to_f32<DT>(a.v[b * a.vs[1] + h * a.vs[2] + c0 + j]) : 0.0f;
        u[j] = beta * __builtin_fmaf(-decay, p[j], v);
        if (r0 == 0 && c0 + j < a.V)
            out[(int64_t)blockIdx.y * a.V + c0 + j] = from_f32<DT>(__builtin_fmaf(decay, o[j], along * u[j]));
    }
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int k = r0 + 32 * i;
        if (k >= a.K) continue;
        row4 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __builtin_fmaf(decay, s[i][j], kr[i] * u[j]);
        float *to = S + (int64_t)k * a.V + c0;
        if (c0 + 4 <= a.V) *(row4 *)to = x;
        else
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j < a.V) to[j] = x[j];
    }
}

// ---------------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------------
template <int DT, int KP>
int prepare(const Delta &d, const Records &rec, int n0, int n1, hipStream_t st) {
    hipLaunchKernelGGL((delta_prepare<DT, KP>), dim3((unsigned)(n1 - n0), (unsigned)(d.B * d.G)), dim3(kPrepThreads),
                       0, st, d, rec, n0);
    return launched();
}
template <int DT, int KP, int W, bool KEEP, bool SEGMENTS>
int walk_of(const Delta &d, const Records &rec, Walk w, hipStream_t st) {
    w.blocks = (padded_v(d.V) + (SEGMENTS ? KP : 0)) / (16 * W);
    const int segments = w.segments - (SEGMENTS ? 1 : 0);  // nothing comes after the last one
    const dim3 grid((unsigned)(segments * d.B * d.H * w.blocks)), block((W == 2 ? 2 : 1) * W * kWave);
    if (row_buffer(d.vs[0], d.V))
        hipLaunchKernelGGL((delta_walk<DT, KP, W, KEEP, false, SEGMENTS>), grid, block, 0, st, d, rec, w);
    else
        hipLaunchKernelGGL((delta_walk<DT, KP, W, KEEP, true, SEGMENTS>), grid, block, 0, st, d, rec, w);
    return launched();
}
template <int DT, int KP, bool KEEP, bool SEGMENTS>
int walk(const Delta &d, const Records &rec, const Walk &w, hipStream_t st) {
    if constexpr (!SEGMENTS)
        if (half_blocks(d, w.segments)) return walk_of<DT, KP, 2, KEEP, false>(d, rec, w, st);
    return walk_of<DT, KP, 4, KEEP, SEGMENTS>(d, rec, w, st);
}
template <int DT, int KP>
int all_chunks(const Delta &d, const Records &rec, const Walk &w, hipStream_t st) {
    int rc = MCCB_OK;
    if (w.chunks > 0) rc = prepare<DT, KP>(d, rec, 0, w.chunks, st);
    if (rc == MCCB_OK && w.segments > 1) {
        rc = walk<DT, KP, false, true>(d, rec, w, st);
        if (rc != MCCB_OK) return rc;
        hipLaunchKernelGGL((delta_carry<KP>), dim3((unsigned)(d.B * d.H * (padded_v(d.V) / 16))), dim3(KP / 32 * kWave), 0, st,
                           d, w);
        rc = launched();
    }
    if (rc != MCCB_OK) return rc;
    return w.states ? walk<DT, KP, true, false>(d, rec, w, st) : walk<DT, KP, false, false>(d, rec, w, st);
}

// Segments of a walk, by what it costs: 3.2 us a chunk where a wave has a SIMD to itself, with outputs (2.8 with second
// waves, 3.9 in segments) and also without (two waves a SIMD then, of 1024 SIMDs), 3 us to carry a state over a segment,
// and 10 us for two more launches and their ends. Of 1 to 16 segments, at each of 11 sizes, it takes the fastest or one
// within 2 % of it. Whole forwards: S=16384 B=1 H=16 799 us as one segment, 357 as eight; S=4096 B=2 H=16 225 and 188
// (four); S=1300 B=1 H=2 K=64 60 and 39; S=2048 B=4 H=16 139 as one, 168 as two; S=777 B=5 H=6 64 and 76 (three).
struct Cut {
    int segments, per;
};
Cut cut_of(const mccb_delta_t *a) {
    const int64_t chunks = (int64_t)chunks_of(a), heads = a->B * a->H, VP = padded_v((int)a->V), KP = padded(a->K);
    Cut best = {1, (int)chunks};
    int64_t least = 32 * chunks;
    for (int64_t n = 2; n <= 16 && n <= chunks && n * heads * VP / 16 <= 1024; ++n) {
        const int64_t per = (chunks + n - 1) / n, rounds = ((n - 1) * heads * (VP + KP) / 16 + 2047) / 2048;
        const int64_t cost = 32 * per * (1 + rounds) + 30 * (n - 1) + 100;
        if (cost < least) least = cost, best.per = (int)per, best.segments = (int)((chunks + per - 1) / per);
    }
    return best;
}
uint64_t ends_floats(const mccb_delta_t *a, const Cut &c) {
    return (uint64_t)(c.segments - 1) * (uint64_t)(a->B * a->H) * (uint64_t)padded(a->K) * (uint64_t)(padded_v((int)a->V) + padded(a->K));
}
uint64_t carry_floats(const mccb_delta_t *a, const Cut &c) {
    return (uint64_t)(c.segments - 1) * (uint64_t)(a->B * a->H) * (uint64_t)padded(a->K) * (uint64_t)padded_v((int)a->V);
}
uint64_t cut_bytes(const mccb_delta_t *a) {
    const Cut c = cut_of(a);
    return (ends_floats(a, c) + carry_floats(a, c)) * sizeof(float);
}

template <int DT>
int forward(const mccb_delta_t *a, void *out, float *final_state, void *saved, void *ws, hipStream_t st) {
    const Delta d = delta_of(a);
    const uint64_t chunks = chunks_of(a);
    uint8_t *const at = (uint8_t *)(saved ? saved : ws);
    Records rec = records_at(at, (uint64_t)(a->B * a->G), (uint64_t)(a->B * a->H), chunks, padded(a->K));
    Walk w{};
    w.state_in = a->state, w.state_out = final_state, w.out = (uint16_t *)out;
    const Cut c = cut_of(a);
    w.chunks = (int)chunks, w.segments = c.segments, w.per = c.per;
    uint64_t used = records_size(a, chunks);
    if (saved) {
        w.states = (float *)(at + used);
        w.u = (float *)((uint8_t *)w.states + chunk_states_bytes(a));
        used += chunk_states_bytes(a) + chunk_rows_bytes(a);
    }
    w.ends = (float *)(at + used);
    w.carry = w.ends + ends_floats(a, c);
    return padded(a->K) == 64 ? all_chunks<DT, 64>(d, rec, w, st) : all_chunks<DT, 128>(d, rec, w, st);
}

}  // namespace

extern "C" {

int mccb_delta_saved_size(const mccb_delta_t *a, uint64_t *bytes) {
    if (!bytes) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_delta(a, false);
    if (rc != MCCB_OK) return rc;
    const uint64_t chunks = chunks_of(a);
    *bytes = records_size(a, chunks) + chunk_states_bytes(a) + chunk_rows_bytes(a) + cut_bytes(a);
    return MCCB_OK;
}

int mccb_delta_forward_get_workspace_size(const mccb_delta_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_delta(a, false);
    if (rc != MCCB_OK) return rc;
    *size = records_size(a, chunks_of(a)) + cut_bytes(a);
    return MCCB_OK;
}

int mccb_delta_forward(const mccb_delta_t *a, void *out, float *final_state, void *saved, void *ws, uint64_t ws_size,
                       void *stream) {
    int rc = check_delta(a, false);
    if (rc != MCCB_OK) return rc;
    Span in[9];
    int n;
    rc = delta_inputs(a, false, in, &n);
    if (rc != MCCB_OK) return rc;
    if (!out && a->S > 0) return MCCB_ERR_PARAM_NULLPTR;
    uint64_t need = 0, kept = 0;
    if (saved) mccb_delta_saved_size(a, &kept);
    else mccb_delta_forward_get_workspace_size(a, &need);
    rc = check_workspace(ws, ws_size, need);
    if (rc != MCCB_OK) return rc;
    const Span o[4] = {{out, (uint64_t)a->S * (uint64_t)(a->B * a->H) * (uint64_t)a->V * 2}, {final_state, state_bytes(a)},
                       {saved, kept}, {ws, need}};
    if (misaligned(out, 2) || misaligned(final_state, 4) || misaligned(saved, 16) || outputs_clash(in, n, o, 4))
        return MCCB_ERR_PARAM_INVALID;
    if (a->S == 0 && !final_state) return MCCB_OK;
    return a->dtype == MCCB_BF16 ? forward<MCCB_BF16>(a, out, final_state, saved, ws, (hipStream_t)stream)
                                 : forward<MCCB_FP16>(a, out, final_state, saved, ws, (hipStream_t)stream);
}

int mccb_delta_step(const mccb_delta_t *a, float *state, void *out, void *stream) {
    int rc = check_delta(a, true);
    if (rc != MCCB_OK) return rc;
    if (!state || !out) return MCCB_ERR_PARAM_NULLPTR;
    if (a->state || a->lengths) return MCCB_ERR_PARAM_INVALID;
    Span in[9];
    int n;
    rc = delta_inputs(a, true, in, &n);
    if (rc != MCCB_OK) return rc;
    const Span o[2] = {{out, (uint64_t)(a->B * a->H * a->V) * 2}, {state, state_bytes(a)}};
    if (misaligned(out, 2) || misaligned(state, 4) || outputs_clash(in, n, o, 2)) return MCCB_ERR_PARAM_INVALID;
    const dim3 grid((unsigned)((a->V + kStepCols - 1) / kStepCols), (unsigned)(a->B * a->H));
    if (a->dtype == MCCB_BF16)
        hipLaunchKernelGGL((delta_one<MCCB_BF16>), grid, dim3(kStepThreads), 0, (hipStream_t)stream, delta_of(a), state,
                           (uint16_t *)out);
    else
        hipLaunchKernelGGL((delta_one<MCCB_FP16>), grid, dim3(kStepThreads), 0, (hipStream_t)stream, delta_of(a), state,
                           (uint16_t *)out);
    return launched();
}

}  // extern "C"
