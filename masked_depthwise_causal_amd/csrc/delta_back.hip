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
//   gb  = sigmoid(-b) Y.U  (U holds the factor beta, and 1 - beta has nothing left where gates are open)
//
// and the log decays, summed over a chunk's rows first (G): with E = tril(gO U^T, -1) o A - tril(Y U^T, -1) o L,
//
//   gG = E's row sums - its column sums + q Q~.(gO S0^T) - p beta K~.(Y S0^T) - e,   e = u K~.(U gS1^T),
//   gG[C-1] += sum(e) + whole gS1.S0,     and log a[t]'s is the sum of gG over rows from t on.
//
// E is Z o Q~ K~^T + W o K~ K~^T below the diagonal. (The diagonal, whose two sums cancel, is left out, and
// the sums are in fp64, since most of what they add cancels too: a row that has nothing before it gets
// exactly 0. The same gradient from gO.out - gV.V, which costs nothing, comes out to 1e-5 only.)
//
// A row's kr and qr may be anything: 1/|k~|, 1000 times 2^e for a row whose square is below 1e-6, 2^e where nothing is
// normalized. Z and W, which are split with one power of two each, would hold the small rows' values next to the
// others', and gk = 2^-e gK~ would make up for it with nothing left. So kr = s c m: s a power of two for the chunk, c
// one for the row, 1 for the largest, and m, about the same for all. The rows' images are multiplied by c, what is
// called gK~ and gQ~ below is without c and s, and Z and W have m only.
#include "delta_common.h"

using namespace delta;

namespace {

struct Back {
    const uint16_t *gout;           // [S,B,H,V]
    int64_t gs[3];                  // strides along S, B, H
    const float *gfinal;            // [B,H,K,V] or NULL
    uint16_t *gv;                   // [S,B,H,V]
    float *gstate;                  // [B,H,K,V] or NULL
    float *gstates, *y;             // [B,H][chunk][K,V], the gradient of S1; [B,H][chunk][64,V]; padded
    const float *states, *u;        // the forward's
    uint16_t *gq, *gk, *gdt, *gb;   // [S,B,G,K], [S,B,H]
    double *part;                   // [2][chunk * B + b][H]: the chunks' parts of gA and gDtBias
    int chunks;
    int blocks;                     // of columns, a head
};

// What second waves make, and hand to those with the state's gradient: all that comes of gO alone.
template <int KP, int W>
struct Given {
    f4 u[W][4][kWave];              // A^T gO
    f4 s[W][KP / 16][kWave];        // Q~^T (q gO)
};
// Bound as the forward walk is, with a longer chain and twice as many transposed operands: S=2048 B=4 H=16 K=V=128, 141
// us, 4.4 a chunk, 235 MB written. W as there: a whole backward of that size 371 us, and 432 in blocks of four; S=513 B=2
// H=6 K=64 V=128 69 and 84; B H = 80 of V=128, where two waves have no CU each, 544 and 500. (Four and their seconds would need more than the LDS for K above 64.)
template <int DT, int KP, int W, bool WIDE>
__global__ void __launch_bounds__((W == 2 ? 2 : 1) * W *kWave, 1) delta_walk_back(Delta a, Records rec, Back w) {
    constexpr bool PAIRS = W == 2;
    constexpr int KT = KP / 16, KS = KP / 32;
    typedef Staged<KP, W, true> Stage;
    constexpr int kBuf = Stage::kBytes, kKeys = Stage::kKeys;
    __shared__ __align__(16) uint8_t smem[2 * kBuf + (PAIRS ? (int)sizeof(Given<KP, W>) : 0)];
    Given<KP, W> *const given = (Given<KP, W> *)(smem + 2 * kBuf);
    const int lane = threadIdx.x % kWave, all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wave = PAIRS ? all_waves % W : all_waves;
    const int m = lane & 15, grp = lane >> 4;
    const int lk_at = left_place<KP>(lane), tk_at = turned_place<KP>(lane), ts_at = triangle_turned_place(lane);
    const int id = same_die(blockIdx.x, gridDim.x);
    const int bh = id / w.blocks, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int col = (id % w.blocks * W + wave) * 16 + m, VP = padded_v(a.V);
    const bool mine = col < a.V;
    const int length = length_of(a, b), chunks = (length + kC - 1) / kC;

    const uint8_t *key = rec.key + (int64_t)(b * a.G + g) * rec.chunks * key_bytes(KP);
    const uint8_t *xa = rec.xa + (int64_t)bh * rec.chunks * kXaBytes;
    const RowCoef *coefs = rec.coef + (int64_t)bh * rec.chunks;
    Stage stage;
    auto fetch = [&](int n) { stage.load(key + n * (int64_t)key_bytes(KP), xa + n * (int64_t)kXaBytes, coefs + n); };
    const Column16 gcol = {w.gout + b * w.gs[1] + h * w.gs[2], w.gs[0], col, a.V};
    uint16_t v[4][4];
    auto begin = [&]() {  // the last chunk's operands
        const int n = chunks - 1;
        if (!PAIRS || all_waves < W) {
            fetch(n);
            load_rows<WIDE>(gcol, n * kC, length - n * kC, lane, v);
            stage.store(smem + (n & 1) * kBuf);
        }
        lds_barrier();
    };
    // A^T gO, whose 16-bit values, with A's powers of two, are exact in one term
    auto from_outputs = [&](const uint8_t *buf, const f4 (&G)[4], f4 (&D)[4]) {
        const uint16_t *ah = (const uint16_t *)(buf + kKeys) + 2 * kTriangle, *al = ah + kTriangle;
        const RowCoef *coef = (const RowCoef *)(buf + kKeys + Stage::kXa);
        f4 R[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) R[t] = G[t] * *(const f4 *)(coef->a + row_of(t, 4 * grp));
        const Power p = column_power(R, lane);
        h8 one[2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) one[s][i] = (_Float16)(R[2 * s + i / 4][i % 4] * p.inv);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f4 d = {};
#pragma unroll
            for (int s = t / 2; s < 2; ++s) {
                d = mma(triangle_turned(al, ts_at, t, s), one[s], d);
                d = mma(triangle_turned(ah, ts_at, t, s), one[s], d);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) D[t][i] = __builtin_fmaf(d[i], p.back, D[t][i]);
        }
    };
    if constexpr (PAIRS)
        if (all_waves < W) {
            if (chunks > 0) begin();
            for (int n = chunks - 1; n >= 0; --n) {
                const uint8_t *buf = smem + (n & 1) * kBuf;
                const uint16_t *qt = (const uint16_t *)buf + kC * KP;
                const RowCoef *coef = (const RowCoef *)(buf + kKeys + Stage::kXa);
                const int next = n > 0 ? n - 1 : 0;
                fetch(next);
                f4 G[4], D[4] = {};
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) G[t][i] = to_f32<DT>(v[t][i]);
                load_rows<WIDE>(gcol, next * kC, length - next * kC, lane, v);
                from_outputs(buf, G, D);
#pragma unroll
                for (int t = 0; t < 4; ++t) given->u[wave][t][lane] = D[t];
                lds_barrier();  // A^T gO is there
#pragma unroll
                for (int t = 0; t < 4; ++t) G[t] *= *(const f4 *)(coef->q + row_of(t, 4 * grp));
                const Power p = column_power(G, lane);
                const Split g0 = split(G[0], G[1], p.inv), g1 = split(G[2], G[3], p.inv);
#pragma unroll
                for (int t = 0; t < KT; t += 4) {
                    f4 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mma(left_turned<KP>(qt, tk_at, t + i, 0), g0.lo, f4{});
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mma(left_turned<KP>(qt, tk_at, t + i, 1), g1.lo, x[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mma(left_turned<KP>(qt, tk_at, t + i, 0), g0.hi, x[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mma(left_turned<KP>(qt, tk_at, t + i, 1), g1.hi, x[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) given->s[wave][t + i][lane] = p.back * x[i];
                }
                lds_barrier();  // and Q~^T (q gO)
                stage.store(smem + (~n & 1) * kBuf);
                lds_barrier();  // as below
            }
            return;
        }
    f4 S[KT];  // the gradient of the state
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = row_of(t, 4 * grp + i);
            S[t][i] = w.gfinal && k < a.K && mine ? w.gfinal[((int64_t)bh * a.K + k) * a.V + col] : 0.0f;
        }
    const uint32_t gv_row = 2u * (uint32_t)(a.B * a.H) * a.V;  // bytes
    const uint32_t gv_at = mine ? 8 * grp * gv_row + 2 * (h * a.V + col) : kNowhere;
    float *keep_s = w.gstates + ((int64_t)bh * rec.chunks * KP + 8 * grp) * VP + col;
    float *keep_y = w.y + ((int64_t)bh * rec.chunks * kC + 8 * grp) * VP + col;
    if (chunks > 0) begin();
    for (int n = chunks - 1; n >= 0; --n) {
        const uint8_t *buf = smem + (n & 1) * kBuf;
        const uint16_t *kt = (const uint16_t *)buf, *qt = kt + kC * KP;
        const uint16_t *xh = (const uint16_t *)(buf + kKeys), *xl = xh + kTriangle;
        const RowCoef *coef = (const RowCoef *)(buf + kKeys + Stage::kXa);
        const int next = n > 0 ? n - 1 : 0;
        if (!PAIRS) fetch(next);
        {
            float *to = keep_s + (int64_t)n * KP * VP;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) to[(row_of(t, 0) + i) * VP] = S[t][i];
        }
        f4 G[4], D[4] = {};
        if constexpr (!PAIRS) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) G[t][i] = to_f32<DT>(v[t][i]);
            load_rows<WIDE>(gcol, next * kC, length - next * kC, lane, v);
        }
        // u K~ gS1
        {
            const Power p = column_power(S, lane);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Split sp = split(S[2 * s], S[2 * s + 1], p.inv);
                h8 lk[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) lk[t] = left<KP>(kt, lk_at, t, s);
#pragma unroll
                for (int t = 0; t < 4; ++t) D[t] = mma(lk[t], sp.lo, D[t]);
#pragma unroll
                for (int t = 0; t < 4; ++t) D[t] = mma(lk[t], sp.hi, D[t]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) D[t] *= *(const f4 *)(coef->u + row_of(t, 4 * grp)) * p.back;
        }
        // + A^T gO
        if constexpr (PAIRS) {
            lds_barrier();
#pragma unroll
            for (int t = 0; t < 4; ++t) D[t] += given->u[wave][t][lane];
        } else {
            from_outputs(buf, G, D);
        }
        // Y = X^T gU
        f4 Y[4];
        {
            const Power p = column_power(D, lane);
            const float up = p.back * coef->x;
            triangle_times<true>(xh, xl, ts_at, split(D[0], D[1], p.inv), split(D[2], D[3], p.inv), Y);
#pragma unroll
            for (int t = 0; t < 4; ++t) Y[t] *= up;
        }
        {
            float *to = keep_y + (int64_t)n * kC * VP;
            const int left_rows = length - n * kC;  // rows past the length are zeros
            const Buffer gv = buffer_of(w.gv + (int64_t)n * kC * (gv_row / 2) + (int64_t)b * a.H * a.V,
                                        (left_rows < kC ? left_rows - 1 : kC - 1) * gv_row + 2u * a.H * a.V);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int r = row_of(t, 4 * grp);
                const f4 cp = *(const f4 *)(coef->p + r), cb = *(const f4 *)(coef->beta + r);
                const f4 x = cb * Y[t];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    to[(row_of(t, 0) + i) * VP] = Y[t][i];
                    __builtin_amdgcn_raw_buffer_store_b16(from_f32<DT>(x[i]), gv, gv_at + (row_of(t, 0) + i) * gv_row, 0, 0);
                }
                Y[t] = -cp * x;
                if (!PAIRS) G[t] *= *(const f4 *)(coef->q + r);
            }
        }
        if constexpr (PAIRS) {
            lds_barrier();  // Q~^T (q gO) is there
            const Power p = column_power(Y, lane);
            const Split y0 = split(Y[0], Y[1], p.inv), y1 = split(Y[2], Y[3], p.inv);
            const float whole = coef->whole;
#pragma unroll
            for (int t = 0; t < KT; t += 4) {
                f4 d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 0), y0.lo, f4{});
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 1), y1.lo, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 0), y0.hi, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 1), y1.hi, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f4 more = given->s[wave][t + i][lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        S[t + i][j] = __builtin_fmaf(whole, S[t + i][j], __builtin_fmaf(p.back, d[i][j], more[j]));
                }
            }
        } else {  // both products in one sum: their columns have one power of two
            float big = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    big = __builtin_fmaxf(big, __builtin_fmaxf(__builtin_fabsf(Y[t][i]), __builtin_fabsf(G[t][i])));
            const Power p = turned_sign(power_of(column_max(big)), lane);
            const Split y0 = split(Y[0], Y[1], p.inv), y1 = split(Y[2], Y[3], p.inv);
            const Split g0 = split(G[0], G[1], p.inv), g1 = split(G[2], G[3], p.inv);
            const float whole = coef->whole;
#pragma unroll
            for (int t = 0; t < KT; t += 4) {
                f4 d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 0), y0.lo, f4{});
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 1), y1.lo, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(qt, tk_at, t + i, 0), g0.lo, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(qt, tk_at, t + i, 1), g1.lo, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 0), y0.hi, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(kt, tk_at, t + i, 1), y1.hi, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(qt, tk_at, t + i, 0), g0.hi, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mma(left_turned<KP>(qt, tk_at, t + i, 1), g1.hi, d[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[t + i][j] = __builtin_fmaf(whole, S[t + i][j], p.back * d[i][j]);
            }
        }
        if (!PAIRS) stage.store(smem + (~n & 1) * kBuf);
        lds_barrier();  // the next chunk's operands are there, and all waves are done with this one's
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
    for (int row = length + grp; row < a.S; row += 4)  // rows past the length
        if (mine) w.gv[(((int64_t)row * a.B + b) * a.H + h) * a.V + col] = 0;
}

// 8 values of a row from column c, zeros past V and where the row is not there. ROWS8: V is a multiple of 8.
template <bool ROWS8>
__device__ static inline HVec<8>::t eight16(const uint16_t *row, int c, int V, bool on) {
    HVec<8>::t v = {};
    if (ROWS8) {
        if (on && c < V) v = *(const HVec<8>::t *)(row + c);
    } else if (on) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < V) v[i] = row[c + i];
    }
    return v;
}
// One of 16 values that every lane holds, by its number.
__device__ static inline float pick(const f4 (&v)[4], int n) {
    f4 r = v[0];
#pragma unroll
    for (int t = 1; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = n >> 2 == t ? v[t][i] : r[i];
    const float x = n & 1 ? r[1] : r[0], y = n & 1 ? r[3] : r[2];
    return n & 2 ? y : x;
}
__device__ static inline int exponent(float v) { return (int)(__float_as_uint(v) >> 23 & 255) - 127; }
__device__ static inline float uniform(float v) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v))); }
__device__ static inline float largest(const f4 &x, const f4 &y, float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_fmaxf(m, __builtin_fmaxf(__builtin_fabsf(x[i]), __builtin_fabsf(y[i])));
    return m;
}

// A chunk's own gradients. V goes by in blocks of 64 columns: the block's rows of gO, U and Y are staged in LDS
// (a power of two a row taken out), the states' rows are the waves' right operands straight from memory, each
// wave with 16 rows of K. Of the 64x64 matrices a wave has a part of a row of tiles. Bound by latency: all of a SIMD's
// registers go to two waves, one block a CU, whose loads, staging and products wait for each other (vector
// instructions in 40 % of the cycles): S=2048 B=4 H=16 K=V=128, 252 us for 539 MB read and 98 written. 7 registers are
// spilled (none where V is no multiple of 8); the next block of columns read ahead spills 47: 300 us. 16.4e6 of 42.4e6
// LDS cycles are bank conflicts, most of them (9.4e6) of 16-byte reads of operands with 64 columns, whose rows are half of
// the banks long; 1.6e6 each of those with 128 columns and of transposing reads, 1e6 each of the scattered Z, W and results.
template <int DT, int KP, bool ROWS8>
__global__ void __launch_bounds__(KP / 16 * kWave) delta_grads(Delta a, Records rec, Back w) {
    constexpr int W = KP / 16, kThreads = W * kWave;
    constexpr int kSide = W / 4, NJ = 4 / kSide;         // waves that share a row of tiles, tiles of each
    constexpr int kPer = kThreads / kC, kCols = 64 / kPer;  // staging: threads of a row, columns of a thread
    __shared__ __align__(16) uint16_t kt[kC * KP], qt[kC * KP];
    __shared__ __align__(16) uint16_t stage[5 * kSquare];  // gO, U hi, U lo, Y hi, Y lo; then Z and W in two terms
    __shared__ __align__(16) float po[kC], pu[kC], py[kC], coef[4 * kC], kr[kC], qr[kC], unit[2][kC];
    __shared__ float rowf[W][kC], rowe[W][kC], yu[kC], big[2][W], size[3];
    __shared__ double cum[kC], dots[W], erow[kSide][kC], ecol[4][kC];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    int lane = threadIdx.x % kWave, m = lane & 15, grp = lane >> 4;
    int lk_at, rk_at, ls_at, ts_at;                      // where the lane reads operands
    const int rt = wave / kSide, j0 = wave % kSide * NJ; // the wave's row of tiles and its first tile
    int kcol = 16 * wave + m;                            // the lane's row of K, a column of gQ~ and gK~
    const int n = blockIdx.x, b = blockIdx.y / a.G, g = blockIdx.y % a.G, heads = a.H / a.G, VP = padded_v(a.V);
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
    constexpr int kTurns = kC * KP / 8 / kThreads;
    h8 kraw[kTurns], qraw[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        kraw[i] = ((const h8 *)key)[threadIdx.x + i * kThreads];
        qraw[i] = ((const h8 *)key)[kC * KP / 8 + threadIdx.x + i * kThreads];
    }
    if (wave < 2) {  // the rows' factors, of k and of q
        const float *factors = (const float *)(key + 2 * kC * KP * 2);
        const float f = factors[wave * kC + lane], back = factors[(2 + wave) * kC + lane];
        const float most = column_max(max16(back > 0.0f ? f : 0.0f));
        // m is 2^-15..2^-14. s stays where its square is a number; c is above 1 for rows of zeros only
        int s = most > 0.0f ? exponent(most) + 15 : 0;
        s = s < -60 ? -60 : s > 60 ? 60 : s;
        int c = exponent(f) + 15 - s;
        if (back > 0.0f && c > 0) c = 0;
        (wave ? qr : kr)[lane] = __builtin_ldexpf(f, -s - c);
        unit[wave][lane] = __builtin_ldexpf(__builtin_fabsf(back), s + c);
        coef[wave * kC + lane] = __builtin_ldexpf(1.0f, c < 0 ? c : 0);
        if (lane == 0) size[wave] = __builtin_ldexpf(1.0f, s);
    }
    lds_barrier();
    if (threadIdx.x == 0) size[2] = size[1] / size[0];  // kept here: registers are all taken
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int at = threadIdx.x + i * kThreads, r = at / (KP / 8);
        ((h8 *)kt)[at] = kraw[i] * (_Float16)coef[r];
        ((h8 *)qt)[at] = qraw[i] * (_Float16)coef[kC + r];
    }
    lds_barrier();
    // this lane's values of K~ and Q~ in the results' layout
    h4 kd[4], qd[4];
    f4 aq[4] = {}, ak[4] = {};
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int to = image_at<KP>(row_of(t, 4 * grp + i), kcol >> 3) + (kcol & 7);
            kd[t][i] = __builtin_bit_cast(_Float16, kt[to]), qd[t][i] = __builtin_bit_cast(_Float16, qt[to]);
        }

    for (int hh = 0; hh < heads; ++hh) {
        const int h = g * heads + hh, bh = b * a.H + h;
        const int64_t at = (int64_t)bh * rec.chunks + n;
        const RowCoef *rc = rec.coef + at;
        const float whole = rc->whole;
        lds_barrier();  // the last head's reads are done
        if (threadIdx.x < 4 * kC) {  // as RowCoef has them, but for c and s
            const int tid = anew(threadIdx.x), r = tid % kC, which = tid / kC;
            const double G = rc->cum[r];
            if (which == 0) cum[r] = G, coef[r] = exp2_f((float)G) * kr[r];
            if (which == 1) coef[kC + r] = rc->beta[r];
            if (which == 2) coef[2 * kC + r] = a.scale * exp2_f((float)G) * qr[r];
            if (which == 3) coef[3 * kC + r] = exp2_f((float)(rc->cum[kC - 1] - G)) * kr[r];
        }
        f4 da[NJ] = {}, dl[NJ] = {}, er[4] = {}, fr[4] = {};
        float s0s1 = 0.0f, dot_u = 0.0f;
        for (int v0 = 0; v0 < a.V; v0 += 64) {
            lane = anew(threadIdx.x % kWave), m = lane & 15, grp = lane >> 4, kcol = 16 * wave + m;
            ls_at = left_place<64>(lane);
            // the wave's rows of both states, on their way while the rows are staged
            f4 st[2][2], gt[2][2];
            const float *s0 = w.states + (at * KP + kcol) * VP + v0 + 8 * grp, *g1 = w.gstates + (at * KP + kcol) * VP + v0 + 8 * grp;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    st[s][i] = *(const f4 *)(s0 + 32 * s + 4 * i), gt[s][i] = *(const f4 *)(g1 + 32 * s + 4 * i);
            {
                const int r = threadIdx.x / kPer, c0 = threadIdx.x % kPer * kCols;
                const uint16_t *go = w.gout + (int64_t)(row0 + r) * w.gs[0] + b * w.gs[1] + h * w.gs[2];
                const float *ur = w.u + (at * kC + r) * VP + v0 + c0, *yr = w.y + (at * kC + r) * VP + v0 + c0;
                f4 o[kCols / 4], u[kCols / 4], y[kCols / 4];
                float mo = 0.0f, mu = 0.0f, my = 0.0f;
#pragma unroll
                for (int j = 0; j < kCols / 8; ++j) {
                    const auto og = eight16<ROWS8>(go, v0 + c0 + 8 * j, a.V, r < live);
#pragma unroll
                    for (int i = 2 * j; i < 2 * j + 2; ++i) u[i] = *(const f4 *)(ur + 4 * i), y[i] = *(const f4 *)(yr + 4 * i);
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
                    return power_of(max_over<kPer>(x));
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
                const Power ps = turned_sign(power_of(column_max(ms)), lane), pg = turned_sign(power_of(column_max(mg)), lane);
                Split ss[2], sg[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    ss[s] = split(st[s][0], st[s][1], ps.inv);
                    sg[s] = split(gt[s][0], gt[s][1], pg.inv);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    keep_order();
                    f4 x = {}, y = {}, z = {};
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const h8 lo = left<64>(oh, ls_at, t, s);
                        const h8 lyh = left<64>(yh, ls_at, t, s), lyl = left<64>(yl, ls_at, t, s);
                        const h8 luh = left<64>(uh, ls_at, t, s), lul = left<64>(ul, ls_at, t, s);
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
                    // sizes that cancel first: gradients may be as small as states are large
                    const f4 fo = *(const f4 *)(po + r) * ps.back * *(const f4 *)(coef + 2 * kC + r);
                    const f4 fy = *(const f4 *)(py + r) * ps.back * *(const f4 *)(coef + r) * *(const f4 *)(coef + kC + r);
                    const f4 fu = *(const f4 *)(pu + r) * pg.back * *(const f4 *)(coef + 3 * kC + r);
                    const f4 kf = anew(kd[t]), qf = anew(qd[t]) * uniform(size[2]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = fu[i] * z[i], o = fo[i] * x[i], l = fy[i] * y[i];
                        er[t][i] = __builtin_fmaf(e, kf[i], er[t][i]);
                        fr[t][i] = __builtin_fmaf(o, qf[i], __builtin_fmaf(-l, kf[i], fr[t][i]));
                        aq[t][i] += o;
                        ak[t][i] += e - l;
                    }
                }
            }
            // gO U^T and Y U^T (those above the diagonal too: the waves that have them would wait for the others)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                keep_order();
                f4 x = {}, y = {};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const h8 lo = left<64>(oh, ls_at, rt, s);
                    const h8 lyh = left<64>(yh, ls_at, rt, s), lyl = left<64>(yl, ls_at, rt, s);
                    const h8 ruh = left<64>(uh, ls_at, j0 + j, s), rul = left<64>(ul, ls_at, j0 + j, s);
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
        lane = anew(threadIdx.x % kWave), m = lane & 15, grp = lane >> 4, kcol = 16 * wave + m;
        lk_at = left_place<KP>(lane);
        dot_u = sum_over<kPer>(dot_u);
        if (threadIdx.x % kPer == 0) yu[threadIdx.x / kPer] = dot_u;
        s0s1 = column_sum(sum16(s0s1));
        if (lane == 0) dots[wave] = (double)s0s1;
        // Z, W and the sums of E
        float mz = 0.0f, mw = 0.0f;
        const float sk = uniform(size[0]), sq = uniform(size[1]);
        {
            const int r = row_of(rt, 4 * grp);
            double er_[4] = {};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                keep_order();
                f4 qk = {}, kk = {};
#pragma unroll
                for (int s = 0; s < KP / 32; ++s) {
                    const h8 rk = left<KP>(kt, lk_at, j0 + j, s);
                    qk = mma(left<KP>(qt, lk_at, rt, s), rk, qk);
                    kk = mma(left<KP>(kt, lk_at, rt, s), rk, kk);
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
                    const double e = below ? (double)__builtin_fmaf(da[j][i], sq * sk * qk[i], dl[j][i] * (sk * sk * kk[i])) : 0.0;
                    er_[i] += e, ec += e;
                    mz = __builtin_fmaxf(mz, __builtin_fabsf(da[j][i]));
                    mw = __builtin_fmaxf(mw, __builtin_fabsf(dl[j][i]));
                }
                ec = column_sum(ec);
                if (grp == 0) ecol[rt][c] = ec;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                er_[i] = sum_over<16>(er_[i]);
                if (m == 0) erow[wave % kSide][r + i] = er_[i];
            }
        }
        mz = column_max(max16(mz)), mw = column_max(max16(mw));
        if (lane == 0) big[0][wave] = mz, big[1][wave] = mw;
        // rows' sums over K
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) fr[t][i] = sum16(fr[t][i]), er[t][i] = sum16(er[t][i]);
        rowf[wave][row_of(m >> 2, 4 * grp + (m & 3))] = pick(fr, m);
        rowe[wave][row_of(m >> 2, 4 * grp + (m & 3))] = pick(er, m);
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
                const int to = image_at<64>(r, c >> 3) + (c & 7);
                const float z = da[j][i] * pz.inv, x = dl[j][i] * pw.inv;
                const _Float16 z0 = (_Float16)z, x0 = (_Float16)x;
                const _Float16 z1 = (_Float16)(z - (float)z0), x1 = (_Float16)(x - (float)x0);
                zh[to] = __builtin_bit_cast(uint16_t, z0), zl[to] = __builtin_bit_cast(uint16_t, z1);
                wh[to] = __builtin_bit_cast(uint16_t, x0), wl[to] = __builtin_bit_cast(uint16_t, x1);
            }
        lds_barrier();
        {
            lane = anew(threadIdx.x % kWave), m = lane & 15, grp = lane >> 4, kcol = 16 * wave + m;
            ls_at = left_place<64>(lane), ts_at = turned_place<64>(lane), rk_at = right_place<KP>(lane);
            h8 rk[2], rq[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) rk[s] = right_turned<KP>(kt, rk_at, wave, s), rq[s] = right_turned<KP>(qt, rk_at, wave, s);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                keep_order();
                f4 x = {}, y = {}, z = {};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s <= t / 2) {
                        x = mma(left<64>(zl, ls_at, t, s), rk[s], x);
                        z = mma(left<64>(wl, ls_at, t, s), rk[s], z);
                        x = mma(left<64>(zh, ls_at, t, s), rk[s], x);
                        z = mma(left<64>(wh, ls_at, t, s), rk[s], z);
                    }
                    if (s >= t / 2) {
                        y = mma(left_turned<64>(zl, ts_at, t, s), rq[s], y);
                        z = mma(left_turned<64>(wl, ts_at, t, s), rk[s], z);
                        y = mma(left_turned<64>(zh, ts_at, t, s), rq[s], y);
                        z = mma(left_turned<64>(wh, ts_at, t, s), rk[s], z);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    aq[t][i] = __builtin_fmaf(pz.back * sk, x[i], aq[t][i]);
                    ak[t][i] = __builtin_fmaf(pz.back * sq, y[i], __builtin_fmaf(pw.back * sk, z[i], ak[t][i]));
                }
            }
        }
        if (wave == W - 1) {
            const int r = lane;
            const int64_t row = row0 + r;
            double e = 0.0, f = 0.0, s0 = 0.0;
#pragma unroll
            for (int i = 0; i < W; ++i) e += (double)rowe[i][r], f += (double)rowf[i][r], s0 += dots[i];
            e *= (double)sk, f *= (double)sk;
            // gG, then its sum from a row on
            double s = f - e - (ecol[0][r] + ecol[1][r] + ecol[2][r] + ecol[3][r]);
#pragma unroll
            for (int i = 0; i < kSide; ++i) s += erow[i][r];
            e = last_lane(sum_up(e)) + (double)whole * s0;
            const double up = sum_up(s);
            s += last_lane(up) - up;
            const double glog = s + e;  // of log a
            double pa = 0.0, pb = 0.0;
            float shut = 0.0f;
            if (r < live) {
                shut = sigmoid_f(-to_f32<DT>(a.b[row * a.bs[0] + b * a.bs[1] + h * a.bs[2]]));
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
                w.gb[to] = r < live ? from_f32<DT>(shut * yu[r]) : 0;
            }
            pa = last_lane(sum_up(pa)), pb = last_lane(sum_up(pb));
            if (lane == 0) {
                const int64_t to = ((int64_t)n * a.B + b) * a.H + h;
                w.part[to] = pa, w.part[(int64_t)w.chunks * a.B * a.H + to] = pb;
            }
        }
    }
    lane = anew(threadIdx.x % kWave), m = lane & 15, grp = lane >> 4, kcol = 16 * wave + m;
    // through the norms: gk = 2^-e s c (gK~ - K~ (s m)^2 (K~.gK~))
    f4 qs[4], ks[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) qs[t][i] = sum16(aq[t][i] * (float)qd[t][i]), ks[t][i] = sum16(ak[t][i] * (float)kd[t][i]);
    lds_barrier();  // the last head's sums, operands and matrices have been read
    rowf[wave][row_of(m >> 2, 4 * grp + (m & 3))] = pick(qs, m);
    rowe[wave][row_of(m >> 2, 4 * grp + (m & 3))] = pick(ks, m);
    lds_barrier();
    if (threadIdx.x < kC) {  // what a row's values lose along themselves, and the factor of what is left
        const int r = threadIdx.x;
        float q = 0.0f, k = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) q += rowf[j][r], k += rowe[j][r];
        const float sk = size[0], sq = size[1];
        coef[r] = a.normalize ? q * (sq * qr[r]) * (sq * qr[r]) : 0.0f;
        coef[kC + r] = a.normalize ? k * (sk * kr[r]) * (sk * kr[r]) : 0.0f;
        coef[2 * kC + r] = unit[1][r];
        coef[3 * kC + r] = unit[0][r];
    }
    lds_barrier();
    // by way of LDS, in rows
    constexpr int kLd = KP + 8;
    static_assert(kC * kLd <= 5 * kSquare, "one result at a time");
#pragma unroll
    for (int both = 0; both < 2; ++both) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int r = row_of(t, 4 * grp);
            const f4 along = *(const f4 *)(coef + both * kC + r), f = *(const f4 *)(coef + (2 + both) * kC + r);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                stage[(r + i) * kLd + kcol] =
                    both ? from_f32<DT>(f[i] * __builtin_fmaf(-along[i], (float)kd[t][i], ak[t][i]))
                         : from_f32<DT>(f[i] * __builtin_fmaf(-along[i], (float)qd[t][i], aq[t][i]));
        }
        lds_barrier();
        uint16_t *to = both ? w.gk : w.gq;
        for (int i = threadIdx.x; i < rows * (KP / 8); i += kThreads) {
            const int r = i / (KP / 8), c = i % (KP / 8) * 8;
            HVec<8>::t x = *(const HVec<8>::t *)(stage + r * kLd + c);
            if (r >= live) x = HVec<8>::t{};
            uint16_t *p = to + (((int64_t)(row0 + r) * a.B + b) * a.G + g) * a.K + c;
            if (c + 8 <= a.K) *(HVec<8>::t *)p = x;
            else
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < a.K) p[j] = x[j];
        }
        lds_barrier();
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

template <int DT, int KP, int W>
void walk_back(const Delta &d, const Records &rec, Back w, hipStream_t st) {
    w.blocks = padded_v(d.V) / (16 * W);
    const dim3 grid((unsigned)(d.B * d.H * w.blocks)), block((W == 2 ? 2 : 1) * W * kWave);
    if (row_buffer(w.gs[0], d.V)) hipLaunchKernelGGL((delta_walk_back<DT, KP, W, false>), grid, block, 0, st, d, rec, w);
    else hipLaunchKernelGGL((delta_walk_back<DT, KP, W, true>), grid, block, 0, st, d, rec, w);
}
template <int DT, int KP>
int launch(const Delta &d, const Records &rec, const Back &w, hipStream_t st) {
    if (half_blocks(d, 1)) walk_back<DT, KP, 2>(d, rec, w, st);
    else walk_back<DT, KP, 4>(d, rec, w, st);
    int rc = launched();
    if (rc != MCCB_OK || w.chunks == 0) return rc;
    const dim3 all((unsigned)w.chunks, (unsigned)(d.B * d.G)), threads(KP / 16 * kWave);
    if (d.V % 8 == 0) hipLaunchKernelGGL((delta_grads<DT, KP, true>), all, threads, 0, st, d, rec, w);
    else hipLaunchKernelGGL((delta_grads<DT, KP, false>), all, threads, 0, st, d, rec, w);
    return launched();
}

}  // namespace

extern "C" {

int mccb_delta_backward_get_workspace_size(const mccb_delta_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_delta(a, false);
    if (rc != MCCB_OK) return rc;
    *size = align16(part_bytes(a)) + chunk_states_bytes(a) + chunk_rows_bytes(a);
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
    w.y = (float *)((uint8_t *)w.gstates + chunk_states_bytes(a));
    w.states = (const float *)((const uint8_t *)saved + records_size(a, chunks));
    w.u = (const float *)((const uint8_t *)w.states + chunk_states_bytes(a));
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
