// delta_back.hip -- the gated delta rule's gradients. Notation as in delta_common.h; g marks a gradient, S1 is
// the state after a chunk.
//
// What depends on the state's gradient walks back over the chunks (delta_walk_back, the forward walk's
// counterpart, a wave 16 columns of V):
//
//   gU = A^T gO + diag(u) K~ gS1,   Y = X^T gU,   gV = beta Y
//   gS0 = whole gS1 + Q~^T (q gO) - K~^T (p beta Y)
//
// The rest is every chunk's own (delta_grads, a block a chunk and key head):
//
//   gQ~ = q gO S0^T + Z K~                           Z = scale tril(gO U^T) o M o qr kr^T
//   gK~ = u U gS1^T - p beta Y S0^T + Z^T Q~ + (W + W^T) K~     W = -tril(Y U^T, -1) o beta o M o kr kr^T
//   gb  = (1 - beta) Y.U  (U holds the factor beta)
//
// and the log decays, summed over a chunk's rows first (G): with E = tril(gO U^T, -1) o A - tril(Y U^T, -1) o L,
//
//   gG = E's row sums - its column sums + q Q~.(gO S0^T) - p beta K~.(Y S0^T) - e,   e = u K~.(U gS1^T),
//   gG[C-1] += sum(e) + whole gS1.S0,     and log a[t]'s is the sum of gG over rows from t on.
//
// E is Z o Q~ K~^T + W o K~ K~^T below the diagonal. (The diagonal, whose two sums cancel, is left out, and
// the sums are in fp64, since most of what they add cancels too: a row that has nothing before it gets
// exactly 0. The same gradient from gO.out - gV.V, which costs nothing, comes out to 1e-5 only.)
#include "delta_common.h"

using namespace delta;

namespace {

struct Back {
    const uint16_t *gout;           // [S,B,H,V]
    int64_t gs[3];                  // strides along S, B, H
    const float *gfinal;            // [B,H,K,V] or NULL
    uint16_t *gv;                   // [S,B,H,V]
    float *gstate;                  // [B,H,K,V] or NULL
    float *gstates, *y;             // [B,H][chunk][K,V], the gradient of S1; [B,H][chunk][64,V]
    const float *states, *u;        // the forward's
    uint16_t *gq, *gk, *gdt, *gb;   // [S,B,G,K], [S,B,H]
    double *part;                   // [2][chunk * B + b][H]: the chunks' parts of gA and gDtBias
    int chunks;
    int blocks;                     // of columns, a head
};

template <int DT, int KP, int W>
__global__ void __launch_bounds__(W *kWave) delta_walk_back(Delta a, Records rec, Back w) {
    constexpr int KT = KP / 16, KS = KP / 32;
    constexpr int kKeys = 2 * kC * KP * 2;
    constexpr int kBuf = kKeys + (int)kXaBytes + kStaged;
    __shared__ __align__(16) uint8_t smem[2 * kBuf];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int m = lane & 15, grp = lane >> 4;
    const int id = same_die(blockIdx.x, gridDim.x);
    const int bh = id / w.blocks, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int col = (id % w.blocks * W + wave) * 16 + m;
    const bool mine = col < a.V;
    const int length = length_of(a, b), chunks = (length + kC - 1) / kC;

    f4 S[KT];  // the gradient of the state
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = row_of(t, 4 * grp + i);
            S[t][i] = w.gfinal && k < a.K && mine ? w.gfinal[((int64_t)bh * a.K + k) * a.V + col] : 0.0f;
        }
    const uint8_t *keys = rec.key + (int64_t)(b * a.G + g) * rec.chunks * key_bytes(KP);
    const uint8_t *xas = rec.xa + (int64_t)bh * rec.chunks * kXaBytes;
    const RowCoef *coefs = rec.coef + (int64_t)bh * rec.chunks;
    auto fill = [&](int n) {
        uint8_t *to = smem + (n & 1) * kBuf;
        const uint8_t *key = keys + n * (int64_t)key_bytes(KP), *xa = xas + n * (int64_t)kXaBytes;
        const uint8_t *coef = (const uint8_t *)(coefs + n);
        for (int p = wave; p < kBuf / 1024; p += W) {
            const int o = p * 1024;
            to_lds(o < kKeys ? key + o : o < kKeys + (int)kXaBytes ? xa + (o - kKeys) : coef, to + o, lane);
        }
    };
    const uint16_t *gbase = w.gout + b * w.gs[1] + h * w.gs[2];
    uint16_t next[4][4];
    auto fetch = [&](int n) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = n * kC + row_of(t, 4 * grp + i);
                next[t][i] = row < length && mine ? gbase[(int64_t)row * w.gs[0] + col] : 0;
            }
    };
    if (chunks > 0) fill(chunks - 1), fetch(chunks - 1);
    for (int n = chunks - 1; n >= 0; --n) {
        __syncthreads();  // this chunk's operands are there, and all waves are done with the last one's
        const uint8_t *buf = smem + (n & 1) * kBuf;
        const uint16_t *kt = (const uint16_t *)buf, *qt = kt + kC * KP;
        const uint16_t *xh = (const uint16_t *)(buf + kKeys), *xl = xh + kSquare, *ah = xl + kSquare, *al = ah + kSquare;
        const float *coef = (const float *)(buf + kKeys + kXaBytes);
        const float whole = coefs[n].whole, sx = coefs[n].x, sa = coefs[n].a;
        f4 G[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) G[t][i] = to_f32<DT>(next[t][i]);
        if (n > 0) fill(n - 1), fetch(n - 1);
        float *keep = w.gstates + ((int64_t)bh * rec.chunks + n) * a.K * a.V;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = row_of(t, 4 * grp + i);
                if (k < a.K && mine) keep[(int64_t)k * a.V + col] = S[t][i];
            }
        // u K~ gS1
        f4 D[4] = {};
        {
            const Power p = column_power(S);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Split sp = split(S[2 * s], S[2 * s + 1], p.inv);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const h8 lk = left<KP>(kt, t, s, lane);
                    D[t] = mma(lk, sp.hi, D[t]);
                    D[t] = mma(lk, sp.lo, D[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f4 cu = *(const f4 *)(coef + 3 * kC + row_of(t, 4 * grp));
#pragma unroll
                for (int i = 0; i < 4; ++i) D[t][i] *= cu[i] * p.back;
            }
        }
        // + A^T gO, whose 16-bit values are exact in one term
        {
            const Power p = column_power(G);
            h8 one[2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i) one[s][i] = (_Float16)(G[2 * s + i / 4][i % 4] * p.inv);
            const float up = p.back * sa;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f4 d = {};
#pragma unroll
                for (int s = t / 2; s < 2; ++s) {
                    d = mma(left_turned<64>(ah, t, s, lane), one[s], d);
                    d = mma(left_turned<64>(al, t, s, lane), one[s], d);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) D[t][i] = __builtin_fmaf(d[i], up, D[t][i]);
            }
        }
        // Y = X^T gU
        f4 Y[4];
        {
            const Power p = column_power(D);
            Split sp[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) sp[s] = split(D[2 * s], D[2 * s + 1], p.inv);
            const float up = p.back * sx;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f4 d = {};
#pragma unroll
                for (int s = t / 2; s < 2; ++s) {
                    const h8 lh = left_turned<64>(xh, t, s, lane), ll = left_turned<64>(xl, t, s, lane);
                    d = mma(lh, sp[s].hi, d);
                    d = mma(ll, sp[s].hi, d);
                    d = mma(lh, sp[s].lo, d);
                }
                Y[t] = d * up;
            }
        }
        float *keep_y = w.y + ((int64_t)bh * rec.chunks + n) * kC * a.V;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int r = row_of(t, 4 * grp);
            const f4 cp = *(const f4 *)(coef + r), cb = *(const f4 *)(coef + kC + r), cq = *(const f4 *)(coef + 2 * kC + r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = n * kC + r + i;
                const float v = cb[i] * Y[t][i];
                if (mine) keep_y[(int64_t)(r + i) * a.V + col] = Y[t][i];
                if (mine && row < a.S) w.gv[(((int64_t)row * a.B + b) * a.H + h) * a.V + col] = from_f32<DT>(v);
                Y[t][i] = -cp[i] * v;
                G[t][i] *= cq[i];
            }
        }
        // gS0, both products in one sum: their columns have one power of two
        {
            float big = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    big = __builtin_fmaxf(big, __builtin_fmaxf(__builtin_fabsf(Y[t][i]), __builtin_fabsf(G[t][i])));
            const Power p = power_of(column_max(big));
            Split sy[2], sg[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                sy[s] = split(Y[2 * s], Y[2 * s + 1], p.inv);
                sg[s] = split(G[2 * s], G[2 * s + 1], p.inv);
            }
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                f4 d = {};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const h8 lk = left_turned<KP>(kt, t, s, lane), lq = left_turned<KP>(qt, t, s, lane);
                    d = mma(lk, sy[s].hi, d);
                    d = mma(lk, sy[s].lo, d);
                    d = mma(lq, sg[s].hi, d);
                    d = mma(lq, sg[s].lo, d);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) S[t][i] = __builtin_fmaf(whole, S[t][i], p.back * d[i]);
            }
        }
    }
    if (w.gstate) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = row_of(t, 4 * grp + i);
                if (k < a.K && mine) w.gstate[((int64_t)bh * a.K + k) * a.V + col] = S[t][i];
            }
    }
    for (int row = chunks * kC + grp; row < a.S; row += 4)  // rows that no chunk covers
        if (mine) w.gv[(((int64_t)row * a.B + b) * a.H + h) * a.V + col] = 0;
}

// Right operand from an image's columns 16 tile.., step s of 32 along its rows.
template <int COLS>
__device__ static inline h8 right_turned(const uint16_t *__restrict__ image, int tile, int s, int lane) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const int i = lane & 15, row = 32 * s + 8 * (lane >> 4) + (i >> 2);
    const int chunk = 2 * tile + (i >> 1 & 1), half = 4 * (i & 1);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(image + image_at<COLS>(row, chunk) + half));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(image + image_at<COLS>(row + 4, chunk) + half));
    return __builtin_bit_cast(h8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// 8 fp32 values of a row from column c, zeros past V.
__device__ static inline void eight(const float *row, int c, int V, bool on, f4 &x, f4 &y) {
    typedef float row4 __attribute__((ext_vector_type(4), aligned(4)));
    x = f4{}, y = f4{};
    if (!on) return;
    if (c + 8 <= V) {
        x = *(const row4 *)(row + c), y = *(const row4 *)(row + c + 4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c + i < V) x[i] = row[c + i];
            if (c + 4 + i < V) y[i] = row[c + 4 + i];
        }
    }
}
__device__ static inline HVec<8>::t eight16(const uint16_t *row, int c, int V, bool on) {
    HVec<8>::t v = {};
    if (!on) return v;
    if (c + 8 <= V) v = *(const HVec<8>::t *)(row + c);
    else
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < V) v[i] = row[c + i];
    return v;
}
__device__ static inline float largest(const f4 &x, const f4 &y, float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_fmaxf(m, __builtin_fmaxf(__builtin_fabsf(x[i]), __builtin_fabsf(y[i])));
    return m;
}

// A chunk's own gradients. V goes by in blocks of 64 columns: the block's rows of gO, U and Y are staged in LDS
// (a power of two a row taken out), the states' rows are the waves' right operands straight from memory, each
// wave with 16 rows of K. Of the 64x64 matrices a wave has a part of a row of tiles.
template <int DT, int KP>
__global__ void __launch_bounds__(KP / 16 * kWave) delta_grads(Delta a, Records rec, Back w) {
    constexpr int W = KP / 16, kThreads = W * kWave;
    constexpr int kSide = W / 4, NJ = 4 / kSide;         // waves that share a row of tiles, tiles of each
    constexpr int kPer = kThreads / kC, kCols = 64 / kPer;  // staging: threads of a row, columns of a thread
    __shared__ __align__(16) uint16_t kt[kC * KP], qt[kC * KP];
    __shared__ __align__(16) uint16_t stage[5 * kSquare];  // gO, U hi, U lo, Y hi, Y lo; then Z and W in two terms
    __shared__ __align__(16) float po[kC], pu[kC], py[kC], coef[4 * kC], kr[kC], qr[kC];
    __shared__ float rowf[W][kC], rowe[W][kC], yu[kC], big[2][W];
    __shared__ double cum[kC], dots[W], erow[kSide][kC], ecol[4][kC];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int m = lane & 15, grp = lane >> 4;
    const int rt = wave / kSide, j0 = wave % kSide * NJ; // the wave's row of tiles and its first tile
    const int kcol = 16 * wave + m;                      // the lane's row of K, a column of gQ~ and gK~
    const int n = blockIdx.x, b = blockIdx.y / a.G, g = blockIdx.y % a.G, heads = a.H / a.G;
    const int row0 = n * kC, live = length_of(a, b) - row0;
    const int rows = a.S - row0 < kC ? a.S - row0 : kC;
    if (live <= 0) {
        for (int i = threadIdx.x; i < rows * a.K; i += kThreads) {
            const int64_t at = (((int64_t)(row0 + i / a.K) * a.B + b) * a.G + g) * a.K + i % a.K;
            w.gq[at] = 0, w.gk[at] = 0;
        }
        for (int i = threadIdx.x; i < rows * heads; i += kThreads) {
            const int64_t at = ((int64_t)(row0 + i / heads) * a.B + b) * a.H + g * heads + i % heads;
            w.gdt[at] = 0, w.gb[at] = 0;
        }
        for (int i = threadIdx.x; i < heads; i += kThreads) {
            const int64_t at = ((int64_t)n * a.B + b) * a.H + g * heads + i;
            w.part[at] = 0.0, w.part[(int64_t)w.chunks * a.B * a.H + at] = 0.0;
        }
        return;
    }
    const uint8_t *key = rec.key + ((int64_t)(b * a.G + g) * rec.chunks + n) * key_bytes(KP);
    const float *factors = (const float *)(key + 2 * kC * KP * 2);
    for (int i = threadIdx.x; i < kC * KP / 8; i += kThreads) {
        ((h8 *)kt)[i] = ((const h8 *)key)[i];
        ((h8 *)qt)[i] = ((const h8 *)key)[kC * KP / 8 + i];
    }
    if (threadIdx.x < kC) kr[threadIdx.x] = factors[threadIdx.x], qr[threadIdx.x] = factors[kC + threadIdx.x];
    lds_barrier();
    auto value = [&](const uint16_t *image, int row) {
        return (float)__builtin_bit_cast(_Float16, image[image_at<KP>(row, kcol >> 3) + (kcol & 7)]);
    };
    // this lane's values of K~ and Q~ in the results' layout
    f4 kd[4], qd[4], aq[4] = {}, ak[4] = {};
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) kd[t][i] = value(kt, row_of(t, 4 * grp + i)), qd[t][i] = value(qt, row_of(t, 4 * grp + i));

    for (int hh = 0; hh < heads; ++hh) {
        const int h = g * heads + hh, bh = b * a.H + h;
        const int64_t at = (int64_t)bh * rec.chunks + n;
        const RowCoef *rc = rec.coef + at;
        const float whole = rc->whole;
        lds_barrier();  // the last head's reads are done
        if (threadIdx.x < 4 * kC) coef[threadIdx.x] = ((const float *)rc)[threadIdx.x];
        if (threadIdx.x < kC) cum[threadIdx.x] = rc->cum[threadIdx.x];
        f4 da[NJ] = {}, dl[NJ] = {}, er[4] = {}, fr[4] = {};
        float s0s1 = 0.0f, dot_u = 0.0f;
        for (int v0 = 0; v0 < a.V; v0 += 64) {
            // the wave's rows of both states, on their way while the rows are staged
            f4 st[2][2], gt[2][2];
            const float *s0 = w.states + (at * a.K + kcol) * a.V, *g1 = w.gstates + (at * a.K + kcol) * a.V;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                eight(s0, v0 + 32 * s + 8 * grp, a.V, kcol < a.K, st[s][0], st[s][1]);
                eight(g1, v0 + 32 * s + 8 * grp, a.V, kcol < a.K, gt[s][0], gt[s][1]);
            }
            {
                const int r = threadIdx.x / kPer, c0 = threadIdx.x % kPer * kCols;
                const uint16_t *go = w.gout + (int64_t)(row0 + r) * w.gs[0] + b * w.gs[1] + h * w.gs[2];
                const float *ur = w.u + (at * kC + r) * a.V, *yr = w.y + (at * kC + r) * a.V;
                f4 o[kCols / 4], u[kCols / 4], y[kCols / 4];
                float mo = 0.0f, mu = 0.0f, my = 0.0f;
#pragma unroll
                for (int j = 0; j < kCols / 8; ++j) {
                    const int c = v0 + c0 + 8 * j;
                    const auto og = eight16(go, c, a.V, r < live);
                    eight(ur, c, a.V, true, u[2 * j], u[2 * j + 1]);
                    eight(yr, c, a.V, true, y[2 * j], y[2 * j + 1]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[2 * j + i / 4][i % 4] = to_f32<DT>(og[i]);
                        dot_u = __builtin_fmaf(u[2 * j + i / 4][i % 4], y[2 * j + i / 4][i % 4], dot_u);
                    }
                    mo = largest(o[2 * j], o[2 * j + 1], mo);
                    mu = largest(u[2 * j], u[2 * j + 1], mu);
                    my = largest(y[2 * j], y[2 * j + 1], my);
                }
                auto row_power = [](float x) {
#pragma unroll
                    for (int i = 1; i < kPer; i *= 2) x = __builtin_fmaxf(x, __shfl_xor(x, i));
                    return power_of(x);
                };
                const Power ro = row_power(mo), ru = row_power(mu), ry = row_power(my);
                lds_barrier();  // the last block's, or head's, operands have been read
                if (threadIdx.x % kPer == 0) po[r] = ro.back, pu[r] = ru.back, py[r] = ry.back;
#pragma unroll
                for (int j = 0; j < kCols / 8; ++j) {
                    const int to = image_at<64>(r, c0 / 8 + j);
                    const Split su = split(u[2 * j], u[2 * j + 1], ru.inv), sy = split(y[2 * j], y[2 * j + 1], ry.inv);
                    h8 one;
#pragma unroll
                    for (int i = 0; i < 8; ++i) one[i] = (_Float16)(o[2 * j + i / 4][i % 4] * ro.inv);
                    *(h8 *)(stage + to) = one;
                    *(h8 *)(stage + kSquare + to) = su.hi;
                    *(h8 *)(stage + 2 * kSquare + to) = su.lo;
                    *(h8 *)(stage + 3 * kSquare + to) = sy.hi;
                    *(h8 *)(stage + 4 * kSquare + to) = sy.lo;
                }
                lds_barrier();
            }
            const uint16_t *oh = stage, *uh = stage + kSquare, *ul = uh + kSquare, *yh = ul + kSquare, *yl = yh + kSquare;
            {
                float ms = 0.0f, mg = 0.0f;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    ms = largest(st[s][0], st[s][1], ms), mg = largest(gt[s][0], gt[s][1], mg);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s0s1 = __builtin_fmaf(st[s][0][i], gt[s][0][i], s0s1);
                        s0s1 = __builtin_fmaf(st[s][1][i], gt[s][1][i], s0s1);
                    }
                }
                const Power ps = power_of(column_max(ms)), pg = power_of(column_max(mg));
                Split ss[2], sg[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    ss[s] = split(st[s][0], st[s][1], ps.inv);
                    sg[s] = split(gt[s][0], gt[s][1], pg.inv);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f4 x = {}, y = {}, z = {};
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const h8 lo = left<64>(oh, t, s, lane);
                        const h8 lyh = left<64>(yh, t, s, lane), lyl = left<64>(yl, t, s, lane);
                        const h8 luh = left<64>(uh, t, s, lane), lul = left<64>(ul, t, s, lane);
                        x = mma(lo, ss[s].hi, x);
                        y = mma(lyh, ss[s].hi, y);
                        z = mma(luh, sg[s].hi, z);
                        x = mma(lo, ss[s].lo, x);
                        y = mma(lyl, ss[s].hi, y);
                        z = mma(lul, sg[s].hi, z);
                        y = mma(lyh, ss[s].lo, y);
                        z = mma(luh, sg[s].lo, z);
                    }
                    const int r = row_of(t, 4 * grp);
                    const f4 fo = *(const f4 *)(po + r) * *(const f4 *)(coef + 2 * kC + r) * ps.back;
                    const f4 fy = *(const f4 *)(py + r) * *(const f4 *)(coef + r) * *(const f4 *)(coef + kC + r) * ps.back;
                    const f4 fu = *(const f4 *)(pu + r) * *(const f4 *)(coef + 3 * kC + r) * pg.back;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = fu[i] * z[i], o = fo[i] * x[i], l = fy[i] * y[i];
                        er[t][i] = __builtin_fmaf(e, kd[t][i], er[t][i]);
                        fr[t][i] = __builtin_fmaf(o, qd[t][i], __builtin_fmaf(-l, kd[t][i], fr[t][i]));
                        aq[t][i] += o;
                        ak[t][i] += e - l;
                    }
                }
            }
            // gO U^T and Y U^T
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if ((j0 + j) / 2 > rt / 2) continue;
                f4 x = {}, y = {};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const h8 lo = left<64>(oh, rt, s, lane);
                    const h8 lyh = left<64>(yh, rt, s, lane), lyl = left<64>(yl, rt, s, lane);
                    const h8 ruh = left<64>(uh, j0 + j, s, lane), rul = left<64>(ul, j0 + j, s, lane);
                    x = mma(lo, ruh, x);
                    y = mma(lyh, ruh, y);
                    x = mma(lo, rul, x);
                    y = mma(lyl, ruh, y);
                    y = mma(lyh, rul, y);
                }
                const int r = row_of(rt, 4 * grp);
                const float fu = pu[row_of(j0 + j, m)];
                const f4 fo = *(const f4 *)(po + r), fy = *(const f4 *)(py + r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    da[j][i] = __builtin_fmaf(fo[i] * fu, x[i], da[j][i]);
                    dl[j][i] = __builtin_fmaf(fy[i] * fu, y[i], dl[j][i]);
                }
            }
        }
        // sums over a row's columns, and of gS1.S0
#pragma unroll
        for (int i = 1; i < kPer; i *= 2) dot_u += __shfl_xor(dot_u, i);
        if (threadIdx.x % kPer == 0) yu[threadIdx.x / kPer] = dot_u;
        s0s1 = sum16(s0s1);
        s0s1 += __shfl_xor(s0s1, 16), s0s1 += __shfl_xor(s0s1, 32);
        if (lane == 0) dots[wave] = (double)s0s1;
        // Z, W and the sums of E
        float mz = 0.0f, mw = 0.0f;
        {
            const int r = row_of(rt, 4 * grp);
            double er_[4] = {};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                f4 qk = {}, kk = {};
                if ((j0 + j) / 2 <= rt / 2)
#pragma unroll
                    for (int s = 0; s < KP / 32; ++s) {
                        const h8 rk = left<KP>(kt, j0 + j, s, lane);
                        qk = mma(left<KP>(qt, rt, s, lane), rk, qk);
                        kk = mma(left<KP>(kt, rt, s, lane), rk, kk);
                    }
                const int c = row_of(j0 + j, m);
                const double gc = cum[c];
                const float kc = kr[c];
                double ec = 0.0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool on = c <= r + i, below = c < r + i;
                    const float decay = on ? exp2_f((float)(cum[r + i] - gc)) * kc : 0.0f;
                    da[j][i] = on ? a.scale * decay * qr[r + i] * da[j][i] : 0.0f;
                    dl[j][i] = below ? -coef[kC + r + i] * decay * kr[r + i] * dl[j][i] : 0.0f;
                    const double e = below ? (double)__builtin_fmaf(da[j][i], qk[i], dl[j][i] * kk[i]) : 0.0;
                    er_[i] += e, ec += e;
                    mz = __builtin_fmaxf(mz, __builtin_fabsf(da[j][i]));
                    mw = __builtin_fmaxf(mw, __builtin_fabsf(dl[j][i]));
                }
                ec += __shfl_xor(ec, 16);
                ec += __shfl_xor(ec, 32);
                if (grp == 0) ecol[rt][c] = ec;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int o = 1; o < 16; o *= 2) er_[i] += __shfl_xor(er_[i], o);
                if (m == 0) erow[wave % kSide][r + i] = er_[i];
            }
        }
        mz = column_max(max16(mz)), mw = column_max(max16(mw));
        if (lane == 0) big[0][wave] = mz, big[1][wave] = mw;
        // rows' sums over K
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row_of(t, 4 * grp + i);
                const float f = sum16(fr[t][i]), e = sum16(er[t][i]);
                if (m == 0) rowf[wave][r] = f, rowe[wave][r] = e;
            }
        lds_barrier();  // also: all reads of the staged rows are done
        mz = big[0][0], mw = big[1][0];
#pragma unroll
        for (int i = 1; i < W; ++i) mz = __builtin_fmaxf(mz, big[0][i]), mw = __builtin_fmaxf(mw, big[1][i]);
        const Power pz = power_of(mz), pw = power_of(mw);
        uint16_t *zh = stage, *zl = zh + kSquare, *wh = zl + kSquare, *wl = wh + kSquare;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row_of(rt, 4 * grp + i), c = row_of(j0 + j, m);
                const int to = image_at<64>(r, c >> 3) + (c & 7), across = image_at<64>(c, r >> 3) + (r & 7);
                const float z = da[j][i] * pz.inv, x = dl[j][i] * pw.inv;
                const _Float16 z0 = (_Float16)z, x0 = (_Float16)x;
                const _Float16 z1 = (_Float16)(z - (float)z0), x1 = (_Float16)(x - (float)x0);
                zh[to] = __builtin_bit_cast(uint16_t, z0), zl[to] = __builtin_bit_cast(uint16_t, z1);
                if (c <= r) {  // both halves; the diagonal's is zero
                    wh[to] = wh[across] = __builtin_bit_cast(uint16_t, x0);
                    wl[to] = wl[across] = __builtin_bit_cast(uint16_t, x1);
                }
            }
        lds_barrier();
        {
            h8 rk[2], rq[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) rk[s] = right_turned<KP>(kt, wave, s, lane), rq[s] = right_turned<KP>(qt, wave, s, lane);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f4 x = {}, y = {}, z = {};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s <= t / 2) {
                        x = mma(left<64>(zh, t, s, lane), rk[s], x);
                        x = mma(left<64>(zl, t, s, lane), rk[s], x);
                    }
                    if (s >= t / 2) {
                        y = mma(left_turned<64>(zh, t, s, lane), rq[s], y);
                        y = mma(left_turned<64>(zl, t, s, lane), rq[s], y);
                    }
                    z = mma(left<64>(wh, t, s, lane), rk[s], z);
                    z = mma(left<64>(wl, t, s, lane), rk[s], z);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    aq[t][i] = __builtin_fmaf(pz.back, x[i], aq[t][i]);
                    ak[t][i] = __builtin_fmaf(pz.back, y[i], __builtin_fmaf(pw.back, z[i], ak[t][i]));
                }
            }
        }
        if (wave == W - 1) {
            const int r = lane;
            const int64_t row = row0 + r;
            const float beta = coef[kC + r];
            double e = 0.0, f = 0.0, s0 = 0.0;
#pragma unroll
            for (int i = 0; i < W; ++i) e += (double)rowe[i][r], f += (double)rowf[i][r], s0 += dots[i];
            // gG, then its sum from a row on
            double s = f - e - (ecol[0][r] + ecol[1][r] + ecol[2][r] + ecol[3][r]);
#pragma unroll
            for (int i = 0; i < kSide; ++i) s += erow[i][r];
#pragma unroll
            for (int o = 32; o; o /= 2) e += __shfl_xor(e, o);
            e += (double)whole * s0;
#pragma unroll
            for (int o = 1; o < kC; o *= 2) {
                const double up = __shfl_down(s, o);
                if (lane + o < kC) s += up;
            }
            const double glog = s + e;  // of log a
            double pa = 0.0, pb = 0.0;
            if (r < live) {
                const float raw = to_f32<DT>(a.dt[row * a.ds[0] + b * a.ds[1] + h * a.ds[2]]) + (a.bias ? a.bias[h] : 0.0f);
                float slope = 1.0f;
                const float d = a.softplus ? softplus_f(raw, slope) : raw;
                // where nothing passes, nothing comes back, whatever the step or the rate
                pa = glog == 0.0 ? 0.0 : glog * (double)d;
                pb = glog == 0.0 ? 0.0 : glog * (double)a.A[h] * (double)slope;
            }
            if (r < rows) {
                const int64_t to = (row * a.B + b) * a.H + h;
                w.gdt[to] = from_f32<DT>((float)pb);
                w.gb[to] = r < live ? from_f32<DT>((1.0f - beta) * yu[r]) : 0;
            }
#pragma unroll
            for (int o = 32; o; o /= 2) pa += __shfl_xor(pa, o), pb += __shfl_xor(pb, o);
            if (lane == 0) {
                const int64_t to = ((int64_t)n * a.B + b) * a.H + h;
                w.part[to] = pa, w.part[(int64_t)w.chunks * a.B * a.H + to] = pb;
            }
        }
    }
    // through the norms: gk = 2^-e (gK~ - K~ kr^2 (K~.gK~))
    lds_barrier();
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row_of(t, 4 * grp + i);
            const float q = sum16(aq[t][i] * qd[t][i]), k = sum16(ak[t][i] * kd[t][i]);
            if (m == 0) rowf[wave][r] = q, rowe[wave][r] = k;
        }
    lds_barrier();
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = row_of(t, 4 * grp + i);
            if (r >= rows || kcol >= a.K) continue;
            const bool on = r < live;
            float q = 0.0f, k = 0.0f;
            if (a.normalize) {
#pragma unroll
                for (int j = 0; j < W; ++j) q += rowf[j][r], k += rowe[j][r];
                q *= qr[r] * qr[r], k *= kr[r] * kr[r];
            }
            const float k2 = factors[2 * kC + r], q2 = factors[3 * kC + r];
            const int64_t to = (((int64_t)(row0 + r) * a.B + b) * a.G + g) * a.K + kcol;
            w.gq[to] = on ? from_f32<DT>(q2 * __builtin_fmaf(-q, qd[t][i], aq[t][i])) : 0;
            w.gk[to] = on ? from_f32<DT>(k2 * __builtin_fmaf(-k, kd[t][i], ak[t][i])) : 0;
        }
}

// gA and gDtBias: the chunks' parts, in a fixed order.
constexpr int kSumSlots = 16;
__global__ void __launch_bounds__(kWave *kSumSlots)
    delta_sum(const double *__restrict__ part, int64_t rows, int H, float *gA, float *gbias) {
    __shared__ double s[kSumSlots][kWave];
    const int lane = threadIdx.x % kWave, slot = threadIdx.x / kWave, h = blockIdx.x * kWave + lane;
    const double *from = part + (blockIdx.y ? rows * H : 0);
    double v = 0.0;
    if (h < H)
        for (int64_t r = slot; r < rows; r += kSumSlots) v += from[r * H + h];
    s[slot][lane] = v;
    __syncthreads();
    float *to = blockIdx.y ? gbias : gA;
    if (slot == 0 && h < H && to) {
        for (int i = 1; i < kSumSlots; ++i) v += s[i][lane];
        to[h] = (float)v;
    }
}

// ---------------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------------
uint64_t part_bytes(const mccb_delta_t *a) { return 2 * chunks_of(a) * (uint64_t)(a->B * a->H) * sizeof(double); }

template <int DT, int KP>
int launch(const Delta &d, const Records &rec, Back w, hipStream_t st) {
    constexpr int W = 4;
    w.blocks = (d.V + 16 * W - 1) / (16 * W);
    hipLaunchKernelGGL((delta_walk_back<DT, KP, W>), dim3((unsigned)(d.B * d.H * w.blocks)), dim3(W * kWave), 0, st, d,
                       rec, w);
    int rc = launched();
    if (rc != MCCB_OK || w.chunks == 0) return rc;
    hipLaunchKernelGGL((delta_grads<DT, KP>), dim3((unsigned)w.chunks, (unsigned)(d.B * d.G)), dim3(KP / 16 * kWave), 0, st, d,
                       rec, w);
    return launched();
}

}  // namespace

extern "C" {

int mccb_delta_backward_get_workspace_size(const mccb_delta_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_delta(a, false);
    if (rc != MCCB_OK) return rc;
    *size = align16(part_bytes(a)) + chunks_of(a) * state_bytes(a) + chunk_rows_bytes(a);
    return MCCB_OK;
}

int mccb_delta_backward(const mccb_delta_t *a, const mccb_delta_grads_t *q, const void *saved, void *ws, uint64_t ws_size,
                        void *stream) {
    int rc = check_delta(a, false);
    if (rc != MCCB_OK) return rc;
    if (!q || !q->gradA) return MCCB_ERR_PARAM_NULLPTR;
    if (a->S > 0 && (!saved || !q->gradOut || !q->gradQ || !q->gradK || !q->gradV || !q->gradDt || !q->gradB))
        return MCCB_ERR_PARAM_NULLPTR;
    Span in[12];
    int n;
    rc = delta_inputs(a, false, in, &n);
    if (rc != MCCB_OK) return rc;
    const int64_t size[4] = {a->S, a->B, a->H, a->V}, stride[4] = {q->gout_stride[0], q->gout_stride[1], q->gout_stride[2], 1};
    uint64_t gout_bytes, need = 0, kept = 0;
    if (!extent(4, size, stride, 2, &gout_bytes)) return MCCB_ERR_PARAM_INVALID;
    mccb_delta_backward_get_workspace_size(a, &need);
    rc = check_workspace(ws, ws_size, need);
    if (rc != MCCB_OK) return rc;
    mccb_delta_saved_size(a, &kept);
    in[n++] = {q->gradOut, gout_bytes};
    in[n++] = {q->gradFinalState, state_bytes(a)};
    in[n++] = {saved, kept};
    const uint64_t rows = (uint64_t)a->S * (uint64_t)a->B;
    const Span out[9] = {{q->gradQ, rows * (uint64_t)(a->G * a->K) * 2}, {q->gradK, rows * (uint64_t)(a->G * a->K) * 2},
                         {q->gradV, rows * (uint64_t)(a->H * a->V) * 2}, {q->gradDt, rows * (uint64_t)a->H * 2},
                         {q->gradB, rows * (uint64_t)a->H * 2}, {q->gradA, (uint64_t)a->H * 4},
                         {q->gradDtBias, (uint64_t)a->H * 4}, {q->gradState, state_bytes(a)}, {ws, need}};
    for (int i = 0; i < 8; ++i)
        if (misaligned(out[i].p, i < 5 ? 2 : 4)) return MCCB_ERR_PARAM_INVALID;
    if (misaligned(q->gradOut, 2) || misaligned(q->gradFinalState, 4) || misaligned(saved, 16) ||
        outputs_clash(in, n, out, 9))
        return MCCB_ERR_PARAM_INVALID;

    const uint64_t chunks = chunks_of(a), heads = (uint64_t)(a->B * a->H);
    const Delta d = delta_of(a);
    const Records rec = records_at((void *)saved, (uint64_t)(a->B * a->G), heads, chunks, padded(a->K));
    Back w{};
    w.gout = (const uint16_t *)q->gradOut;
    for (int i = 0; i < 3; ++i) w.gs[i] = q->gout_stride[i];
    w.gfinal = q->gradFinalState, w.gv = (uint16_t *)q->gradV, w.gstate = q->gradState;
    w.part = (double *)ws;
    w.gstates = (float *)((uint8_t *)ws + align16(part_bytes(a)));
    w.y = w.gstates + chunks * heads * (uint64_t)(a->K * a->V);
    w.states = (const float *)((const uint8_t *)saved + records_size(a, chunks));
    w.u = w.states + chunks * heads * (uint64_t)(a->K * a->V);
    w.gq = (uint16_t *)q->gradQ, w.gk = (uint16_t *)q->gradK, w.gdt = (uint16_t *)q->gradDt, w.gb = (uint16_t *)q->gradB;
    w.chunks = (int)chunks;
    const hipStream_t st = (hipStream_t)stream;
    const bool narrow = padded(a->K) == 64;
    if (a->dtype == MCCB_BF16) rc = narrow ? launch<MCCB_BF16, 64>(d, rec, w, st) : launch<MCCB_BF16, 128>(d, rec, w, st);
    else rc = narrow ? launch<MCCB_FP16, 64>(d, rec, w, st) : launch<MCCB_FP16, 128>(d, rec, w, st);
    if (rc != MCCB_OK) return rc;
    hipLaunchKernelGGL(delta_sum, dim3((unsigned)((a->H + kWave - 1) / kWave), q->gradDtBias ? 2 : 1),
                       dim3(kWave * kSumSlots), 0, st, w.part, (int64_t)(chunks * (uint64_t)a->B), (int)a->H, q->gradA,
                       q->gradDtBias);
    return launched();
}

}  // extern "C"
