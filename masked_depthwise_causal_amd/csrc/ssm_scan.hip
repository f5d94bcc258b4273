// ssm_scan.hip -- selective state space scan for MI355X (gfx950): forward over prompts, backward and
// the single-token step (mccb_ssm.h).
//
//   d = softplus(dt + dt_bias), a[n] = exp(d A[n]), s[n] = a[n] s[n] + (d x) B[n],
//   y = sum_n C[n] s[n] + D x, out = y silu(z)           (per batch, channel and row)
//
// Backward, from gy = gout silu(z), with gs[t] the gradient of s[t]:
//   gs[t,n] = C[t,n] gy[t] + a[t+1,n] gs[t+1,n]
//   gC[t,n] = sum_h gy s[t,n],   gB[t,n] = sum_h gs[t,n] d x
//   q[n] = gs[t,n] a[t,n] s[t-1,n]  (the gradient of d A[n]),   u = sum_n gs[t,n] B[n]
//   gx = u d + D gy,  gd = sum_n q[n] A[n] + u x,  gdt = gd softplus'(dt + dt_bias)
//   gA[n] = sum q[n] d,  gD = sum gy x,  gz = gout y silu'(z)
//
// Layout: a block has 64 channels (one a lane) of one group and batch, and a wave for every four
// states, so that a lane keeps its states, decay rates and (backward) a tile's history of them in
// registers, sums over states are NW terms in LDS, and a channel's work is spread over NW waves.
// Rows go by tiles of 16: the block's threads first turn the tile's x and dt into d and d x in LDS
// (each row once, though NW waves need it) and B and C into fp32, then every wave walks the 16 rows,
// then the threads add the waves' sums, gate and store. The next tile's loads are in flight
// meanwhile.
//
// A long sequence with few channels is cut into chunks, a block each: a first kernel runs every
// chunk from a zero state and keeps its end state and sum of d; since the decay over a chunk is
// exp(A sum d), the second kernel's blocks fold the chunks before theirs into their initial state.
// The backward does the same from the other end for the gradient of the state.
//
// Bound by vector instructions, not by memory: each of N states of each element takes an exp (8.5 cycles
// of a SIMD for 64 lanes, measured) and, forward, about 4 multiply-adds, backward 12 (2.8 cycles with
// three vector registers, 4.4 with a scalar one). S=2048 B=8 H=4096 N=16 bf16, gated: forward 326 us
// (1.6 TB/s), backward 775 us, sums of gB, gC and the parameters 34. By the counters a wave takes 480
// vector instructions a tile forward and 1420 backward, at 4.7 and 4.5 cycles on average; they are
// active in 72 and 89 % of the cycles. The single token (B=64 H=5120) is bound by its state: 9.2 us,
// 4.9 TB/s, of which the last-level cache has most from call to call.
#include "ssm_common.h"

using namespace ssm;

namespace {

constexpr int kTile = 16;  // rows; the forward keeps the state before each tile for the backward
constexpr int kPer = 4;    // states a lane holds

// How a thread takes its channels of a row: one by one, or by one load, since they are adjacent and every
// block has as many; then, in LDS, at any channel or (as where it takes them one by one) at a multiple of
// its vectors' four floats (of two, where it takes two).
enum { kApart, kAdjacent, kWide };

struct Rows {  // a strided [S,B,H] input
    const uint16_t *p;
    int64_t s, b, h;
};
struct Coef {  // a strided [S,B,G,N] input
    const uint16_t *p;
    int64_t s, b, g, n;
};

struct ScanIn {
    Rows x, dt, z;
    Coef B, C;
    const float *A, *D, *bias, *state;
    const int64_t *lengths;
    int64_t S, nb, H, K;  // rows, batches, channels, channels of a group
    int N, G, per_group;  // states, groups, blocks of a group
    int softplus, chunks;
    int64_t chunk_rows;  // whole tiles
};

// What a block works on. Its threads have two roles: in the recurrence a lane has one channel and its
// wave four states; in preparing and finishing a tile a thread has JR = 16 / NW adjacent channels
// of one of the 16 rows, so that rows are read and written by wide loads and stores.
struct Place {
    int lane, wave;
    int64_t b, h;  // batch; the lane's channel, clamped into the group
    int g;
    bool on;              // whether the lane has a channel of its own
    int row, c;           // the thread's row of a tile and its first channel of the block
    int64_t h0;           // the block's first channel
    int channels;         // of the block
    int64_t r0, r1, end;  // the chunk's rows, and where its live rows end
};

// Two blocks share a compute unit, and the older one's waves win every issue slot that both want: it
// ends a quarter earlier and leaves the other alone at half of the rate. So blocks take the higher
// wave priority in turn, four tiles each, blocks a whole round of the 256 compute units apart in
// opposite turns (S=2048 B=8 H=4096: backward 941 -> 905 us, forward unchanged within its noise).
__device__ static inline void take_turn(int tile) {
    const uint32_t block = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
    if (((tile >> 2) + (block >> 8)) & 1) __builtin_amdgcn_s_setprio(1);
    else __builtin_amdgcn_s_setprio(0);
}

template <int NW, int ROWS>
__device__ static inline Place place(const ScanIn &a) {
    constexpr int JR = kTile / NW;
    Place p;
    p.lane = threadIdx.x % kWave;
    p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    p.g = blockIdx.x / a.per_group;
    const int64_t k0 = (int64_t)(blockIdx.x % a.per_group) * kWave;
    p.channels = a.K - k0 < kWave ? (int)(a.K - k0) : kWave;
    p.on = p.lane < p.channels;
    p.h0 = p.g * a.K + k0;
    p.h = p.h0 + (p.on ? p.lane : p.channels - 1);
    p.row = threadIdx.x / (kWave / JR);
    p.c = threadIdx.x % (kWave / JR) * JR;
    // in a block with fewer channels the last threads take the last JR, twice
    if (ROWS != kApart && p.c > p.channels - JR) p.c = p.channels - JR;
    p.b = blockIdx.y;
    int64_t len = a.S;
    if (a.lengths) {
        len = a.lengths[p.b];
        len = len < 0 ? 0 : len > a.S ? a.S : len;
    }
    p.r0 = (int64_t)blockIdx.z * a.chunk_rows;
    p.r1 = p.r0 + a.chunk_rows < a.S ? p.r0 + a.chunk_rows : a.S;
    p.end = len < p.r1 ? len : p.r1;
    return p;
}

// Step sizes d of v = dt + dt_bias, and (SLOPE) their derivatives by v.
template <bool SLOPE, int JR>
__device__ static inline void step_sizes(const ScanIn &a, const float (&v)[JR], float (&d)[JR],
                                         float (&slope)[JR]) {
    if (a.softplus) {
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            if (SLOPE) d[j] = softplus_f(v[j], slope[j]);
            else d[j] = softplus_f(v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < JR; ++j) d[j] = v[j], slope[j] = 1.0f;
    }
}

// An infinite rate as the largest one: its decay over a step is the same 0, and a row without a step
// (past the length, or of a step size of 0) has the decay 1, not the NaN of zero times infinity.
__device__ static inline float finite_rate(float v) {
    constexpr float kMost = 3.402823466e38f;
    return v < -kMost ? -kMost : v > kMost ? kMost : v;
}

// A [N,H] times log2(e), so that the decay is one exp2; zero for states past N, which then stay 0.
__device__ static inline void load_rates(const ScanIn &a, const Place &p, float (&A2)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = p.wave * kPer + i;
        A2[i] = n < a.N ? finite_rate(a.A[(int64_t)n * a.H + p.h] * kLog2e) : 0.0f;
    }
}

// A [B,N,H] buffer of states (or zeros), for the lane's four.
__device__ static inline void load_state(const float *st, const ScanIn &a, const Place &p,
                                         float (&s)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = p.wave * kPer + i;
        s[i] = st && n < a.N ? st[(p.b * a.N + n) * a.H + p.h] : 0.0f;
    }
}
__device__ static inline void store_state(float *st, const ScanIn &a, const Place &p,
                                          const float (&s)[kPer]) {
    if (!p.on) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = p.wave * kPer + i;
        if (n < a.N) st[(p.b * a.N + n) * a.H + p.h] = s[i];
    }
}

// s = state handed from chunk to chunk: for each of `n` chunks from `first` in direction `dir`,
// s = exp2(A2 dsum) s + end state.
__device__ static inline void fold_chunks(const float *ends, const float *dsum, const ScanIn &a,
                                          const Place &p, int first, int dir, int n,
                                          const float (&A2)[kPer], float (&s)[kPer]) {
    const int64_t states = a.nb * a.N * a.H;
    constexpr int kAhead = 8;  // chunks whose values are loaded together; missing ones change nothing
    for (int j0 = 0; j0 < n; j0 += kAhead) {
        float d[kAhead], e[kAhead][kPer];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int c = first + dir * (j0 + j < n ? j0 + j : n - 1);
            d[j] = dsum[((int64_t)c * a.nb + p.b) * a.H + p.h];
            load_state(ends + c * states, a, p, e[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (j0 + j >= n) break;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                s[i] = __builtin_fmaf(exp2_f(d[j] * A2[i]), s[i], e[j][i]);
        }
    }
}

// A thread's way through a [S,B,H] tensor, tile by tile from one that is whole or the chunk's last:
// JR channels of its row; one by one channels past the group's last repeat it.
template <int NW, int ROWS>
struct Walk {
    static constexpr int JR = kTile / NW;
    typedef typename HVec<JR>::t vec;
    const uint16_t *p;  // the thread's row of the tile
    int64_t step, s, h;
    __device__ inline Walk(const Rows &r, const Place &q, int64_t row, int dir)
        : p(r.p ? r.p + (row + q.row) * r.s + q.b * r.b + q.h0 * r.h + (ROWS != kApart ? q.c : 0) : nullptr),
          step(dir * kTile * r.s), s(r.s), h(r.h) {}
    // The tile's values. `last`: its last live row; rows past it repeat it
    __device__ inline vec fetch(const Place &q, int last) const {
        const uint16_t *at = p;
        if (last < kTile - 1) at -= (q.row > last ? q.row - last : 0) * s;
        if (ROWS != kApart) return *(const vec *)at;
        vec v;
#pragma unroll
        for (int i = 0; i < JR; ++i) {
            const int c = q.c + i < q.channels ? q.c + i : q.channels - 1;
            v[i] = at[c * h];
        }
        return v;
    }
    __device__ inline void move(bool on) { p += on ? step : 0; }
};

// The same channels of the thread's row to a contiguous [S,B,H] output.
template <int ROWS, int JR>
__device__ static inline void store_rows(uint16_t *p, const Place &q, const typename HVec<JR>::t v) {
    if (ROWS != kApart) {
        *(typename HVec<JR>::t *)p = v;
    } else {
#pragma unroll
        for (int i = 0; i < JR; ++i)
            if (q.c + i < q.channels) p[i] = v[i];
    }
}

// JR adjacent floats of LDS, from where their vectors are aligned or (kAdjacent) from any float, of which
// the compiler then takes two at a time.
template <int ROWS, int JR>
__device__ static inline void load_floats(const float *p, float (&f)[JR]) {
    if constexpr (ROWS == kAdjacent) {
#pragma unroll
        for (int i = 0; i < JR; ++i) f[i] = p[i];
    } else if constexpr (JR == 2) {
        const float2 q = *(const float2 *)p;
        f[0] = q.x, f[1] = q.y;
    } else {
#pragma unroll
        for (int i = 0; i < JR; i += 4) {
            const float4 q = *(const float4 *)(p + i);
            f[i] = q.x, f[i + 1] = q.y, f[i + 2] = q.z, f[i + 3] = q.w;
        }
    }
}
template <int ROWS, int JR>
__device__ static inline void store_floats(float *p, const float (&f)[JR]) {
    if constexpr (ROWS == kAdjacent) {
#pragma unroll
        for (int i = 0; i < JR; ++i) p[i] = f[i];
    } else if constexpr (JR == 2) {
        *(float2 *)p = make_float2(f[0], f[1]);
    } else {
#pragma unroll
        for (int i = 0; i < JR; i += 4) *(float4 *)(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
}
// A per-channel fp32 parameter (or zeros) of the thread's channels.
template <int JR>
__device__ static inline void load_param(const float *v, const Place &q, float (&f)[JR]) {
#pragma unroll
    for (int i = 0; i < JR; ++i) {
        const int c = q.c + i < q.channels ? q.c + i : q.channels - 1;
        f[i] = v ? v[q.h0 + c] : 0.0f;
    }
}

// The same for B and C: each of the block's threads has one value of 16 rows of NW*4 states.
template <int DT, int NW>
struct CoefWalk {
    int n, t;
    const uint16_t *bp, *cp;  // the thread's row of the tile
    int64_t bs, cs;
    int dir;
    bool has;
    uint16_t bv, cv;
    __device__ inline CoefWalk(const ScanIn &a, const Place &p, int64_t row, int d)
        : bs(a.B.s), cs(a.C.s), dir(d * kTile) {
        n = threadIdx.x % (NW * kPer);
        t = threadIdx.x / (NW * kPer);
        has = n < a.N;
        const int nc = has ? n : 0;
        bp = a.B.p + p.b * a.B.b + p.g * a.B.g + nc * a.B.n + (row + t) * bs;
        cp = a.C.p + p.b * a.C.b + p.g * a.C.g + nc * a.C.n + (row + t) * cs;
    }
    template <bool USE_B, bool USE_C>
    __device__ inline void fetch(int last) {
        const uint16_t *b = bp, *c = cp;
        if (last < kTile - 1) {
            const int over = t > last ? t - last : 0;
            b -= over * bs;
            c -= over * cs;
        }
        if (USE_B) bv = *b;
        if (USE_C) cv = *c;
    }
    __device__ inline void move(bool on) {
        bp += on ? dir * bs : 0;
        cp += on ? dir * cs : 0;
    }
    __device__ inline float b(int last) const { return has && t <= last ? to_f32<DT>(bv) : 0.0f; }
    __device__ inline float c(int last) const { return has && t <= last ? to_f32<DT>(cv) : 0.0f; }
};

__device__ static inline void load4(const float *p, float (&f)[kPer]) {
    const float4 q = *(const float4 *)p;
    f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
}

// Forward. ENDS: only the end state of each chunk from a zero state, and its sum of d (the last
// chunk's is not needed). One barrier a tile: while the waves scan tile k, whose operands one half
// of the LDS buffers holds, tile k+1 is prepared in the other half.
template <int DT, int NW, bool ENDS, bool GATE, int ROWS>
__global__ void __launch_bounds__(NW *kWave)
    scan_fwd(ScanIn a, uint16_t *__restrict__ out, float *__restrict__ final_state,
             float *__restrict__ saved, float *__restrict__ ends, float *__restrict__ dsum) {
    constexpr int NP = NW * kPer, JR = kTile / NW;
    typedef typename HVec<JR>::t vec;
    __shared__ __align__(16) float sd[2][kTile][2][kWave];  // d, d x
    __shared__ __align__(16) float sB[2][kTile][NP], sC[ENDS ? 1 : 2][kTile][NP];
    __shared__ __align__(16) float sy[ENDS ? 1 : 2][ENDS ? 1 : NW][ENDS ? 1 : kTile][kWave];
    const Place p = place<NW, ROWS>(a);
    float A2[kPer], s[kPer], total = 0.0f;
    load_rates(a, p, A2);
    load_state(ENDS ? nullptr : a.state, a, p, s);
    if (!ENDS) fold_chunks(ends, dsum, a, p, 0, 1, blockIdx.z, A2, s);
    float bias[JR], D[JR];
    load_param(a.bias, p, bias);
    load_param(ENDS ? nullptr : a.D, p, D);
    Walk<NW, ROWS> xw(a.x, p, p.r0, 1), dw(a.dt, p, p.r0, 1), zw(a.z, p, p.r0, 1);
    CoefWalk<DT, NW> coef(a, p, p.r0, 1);
    const int64_t BH = a.nb * a.H, states = BH * a.N;
    uint16_t *op = ENDS ? nullptr : out + (p.r0 + p.row) * BH + p.b * a.H + p.h0 + p.c;
    float *kept = saved ? saved + p.r0 / kTile * states + (p.b * a.N + p.wave * kPer) * a.H + p.h : nullptr;
    // fetched values; the next tile's, and the last one's, that finishing them needs
    vec xr, dr, zr, xn, zn, xc, zc;
    const int64_t live_rows = p.end - p.r0;
    const int tiles = live_rows > 0 ? (int)((live_rows + kTile - 1) / kTile) : 0;
    const int tail = (int)(live_rows - (int64_t)(tiles - 1) * kTile) - 1;  // the last tile's last row
    auto fetch = [&](int k) {
        const int last = k + 1 < tiles ? kTile - 1 : tail;
        xr = xw.fetch(p, last);
        dr = dw.fetch(p, last);
        if (GATE) zr = zw.fetch(p, last);
        coef.template fetch<true, !ENDS>(last);
        const bool more = k + 1 < tiles;  // the last tile is fetched again instead of one past it
        xw.move(more), dw.move(more), coef.move(more);
        if (GATE) zw.move(more);
    };
    auto prepare = [&](int k) {
        const int at = k & 1, last = k + 1 < tiles ? kTile - 1 : tail;
        float v[JR], d[JR], dx[JR], slope[JR];
#pragma unroll
        for (int j = 0; j < JR; ++j) v[j] = to_f32<DT>(dr[j]) + bias[j];
        step_sizes<false>(a, v, d, slope);
#pragma unroll
        for (int j = 0; j < JR; ++j) dx[j] = d[j] * to_f32<DT>(xr[j]);
        if (p.row > last) {  // past the length: d = 0 leaves the state alone
#pragma unroll
            for (int j = 0; j < JR; ++j) d[j] = dx[j] = 0.0f;
        }
        store_floats<ROWS>(&sd[at][p.row][0][p.c], d);
        store_floats<ROWS>(&sd[at][p.row][1][p.c], dx);
        sB[at][coef.t][coef.n] = coef.b(last);
        if (!ENDS) sC[at][coef.t][coef.n] = coef.c(last);
    };
    // Tile k's output, from the sums its waves left in LDS.
    auto finish = [&](int k) {
        float y[JR];
#pragma unroll
        for (int j = 0; j < JR; ++j) y[j] = D[j] * to_f32<DT>(xc[j]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            float f[JR];
            load_floats<ROWS>(&sy[k & 1][w][p.row][p.c], f);
#pragma unroll
            for (int j = 0; j < JR; ++j) y[j] += f[j];
        }
        vec v;
#pragma unroll
        for (int j = 0; j < JR; ++j)
            v[j] = from_f32<DT>(GATE ? y[j] * silu_f(to_f32<DT>(zc[j])) : y[j]);
        if (p.row <= (k + 1 < tiles ? kTile - 1 : tail)) store_rows<ROWS, JR>(op, p, v);
        op += kTile * BH;
    };
    if (ROWS != kApart && p.channels < kWave) {  // columns that no thread writes
        for (int r = p.wave; r < 2 * kTile * 2; r += NW)
            if (!p.on) (&sd[0][0][0][0])[r * kWave + p.lane] = 0.0f;
    }
    if (tiles > 0) {
        fetch(0);
        prepare(0);
        xn = xr, zn = zr;
        fetch(tiles > 1 ? 1 : 0);
        lds_barrier();
    }
    // The order matters: a wave's wait counts take loads and stores in order, and a store or load
    // under a condition makes the wait for an older one wait for it as well. So the loads are issued
    // last, without a condition, a whole tile before they are waited for (measured at S=16384
    // H=4096: 418 us with the stores after the loads, 371 us so).
    for (int k = 0; k < tiles; ++k) {
        const int half = k & 1;
        take_turn(k);
        const vec xk = xn, zk = zn;
        xn = xr, zn = zr;
        if (k + 1 < tiles) prepare(k + 1);
        if (!ENDS && k > 0) finish(k - 1);
        xc = xk, zc = zk;
        if (!ENDS && kept) {
            if (p.on) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (p.wave * kPer + i < a.N) kept[i * a.H] = s[i];
            }
            kept += states;
        }
        fetch(k + 2 < tiles ? k + 2 : tiles - 1);
        // Rows by groups, with the next group's operands on their way from LDS while this one's are
        // used.
        constexpr int kGroup = 4;
        float dd[2][kGroup], dx[2][kGroup];
        float Bt[2][kGroup][kPer], Ct[2][kGroup][kPer];
        auto operands = [&](int g, int to) {
#pragma unroll
            for (int r = 0; r < kGroup; ++r) {
                const int t = g * kGroup + r;
                dd[to][r] = sd[half][t][0][p.lane];
                dx[to][r] = sd[half][t][1][p.lane];
                load4(&sB[half][t][p.wave * kPer], Bt[to][r]);
                if (!ENDS) load4(&sC[half][t][p.wave * kPer], Ct[to][r]);
            }
        };
        operands(0, 0);
#pragma unroll
        for (int g = 0; g < kTile / kGroup; ++g) {
            const int at = g & 1;
            if (g + 1 < kTile / kGroup) operands(g + 1, at ^ 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < kGroup; ++r) {
                float y = 0.0f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    s[i] = __builtin_fmaf(exp2_f(dd[at][r] * A2[i]), s[i], dx[at][r] * Bt[at][r][i]);
                    if (!ENDS) y = __builtin_fmaf(Ct[at][r][i], s[i], y);
                }
                if (ENDS) total += dd[at][r];
                else sy[half][p.wave][g * kGroup + r][p.lane] = y;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        lds_barrier();
    }
    if (!ENDS && tiles > 0) finish(tiles - 1);
    if (ENDS) {
        store_state(ends + (int64_t)blockIdx.z * a.nb * a.N * a.H, a, p, s);
        if (p.wave == 0 && p.on) dsum[((int64_t)blockIdx.z * a.nb + p.b) * a.H + p.h] = total;
        return;
    }
    if (p.on)  // rows past the length
        for (int64_t t = (p.end > p.r0 ? p.end : p.r0) + p.wave; t < p.r1; t += NW)
            out[(t * a.nb + p.b) * a.H + p.h] = 0;
    if (final_state && (int)blockIdx.z == a.chunks - 1) store_state(final_state, a, p, s);
}

// ---------------------------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------------------------
struct ScanGrad {
    Rows go;
    const float *gfinal, *saved;
    uint16_t *gx, *gdt, *gz;
    float *gstate;
    float *pbc;     // [block of channels][pbc_rows][B][2][NP]: sums over the block's channels
    int64_t pbc_rows;  // S in whole tiles
    double *pa;     // [chunk][B][(N+2) H]: gA, gD, gdt_bias of a chunk
    float *ends, *dsum;
};

template <int CTRL>
__device__ static inline float dpp(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
constexpr int kRor8 = 0x128, kHalfMirror = 0x141, kXor2 = 0x4e, kXor1 = 0xb1;

__device__ static inline float swap_add32(float a, float b) {  // lanes < 32: a's sum, others: b's
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ static inline float swap_add16(float a, float b) {  // even rows of 16: a's, odd: b's
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// a's sum over lanes that CTRL joins where `second` is false, b's where it is true
template <int CTRL>
__device__ static inline float join(float a, float b, bool second) {
    const float x = a + dpp<CTRL>(a), y = b + dpp<CTRL>(b);
    return second ? y : x;
}

// Carry of a chunk from a zero gradient behind it: gs a at its first row, and its sum of d.
template <int DT, int NW, bool GATE, int ROWS>
__global__ void __launch_bounds__(NW *kWave)
    scan_bwd_ends(ScanIn a, ScanGrad q) {
    constexpr int NP = NW * kPer, JR = kTile / NW;
    typedef typename HVec<JR>::t vec;
    __shared__ __align__(16) float sd[2][kTile][2][kWave];  // d, gy
    __shared__ __align__(16) float sC[2][kTile][NP];
    const Place p = place<NW, ROWS>(a);
    float A2[kPer], carry[kPer] = {0.0f, 0.0f, 0.0f, 0.0f}, total = 0.0f, bias[JR];
    load_rates(a, p, A2);
    load_param(a.bias, p, bias);
    const int tiles = p.end > p.r0 ? (int)((p.end - p.r0 + kTile - 1) / kTile) : 0;
    const int64_t t0 = p.r0 + (int64_t)(tiles - 1) * kTile;
    Walk<NW, ROWS> dw(a.dt, p, t0, -1), zw(a.z, p, t0, -1), gw(q.go, p, t0, -1);
    CoefWalk<DT, NW> coef(a, p, t0, -1);
    const int tail = (int)(p.end - t0) - 1;  // the last tile may be partial, the others are whole
    vec dr, zr, gr;
    auto fetch = [&](int k) {
        const int last = k + 1 < tiles ? kTile - 1 : tail;
        dr = dw.fetch(p, last);
        gr = gw.fetch(p, last);
        if (GATE) zr = zw.fetch(p, last);
        coef.template fetch<false, true>(last);
        const bool more = k > 0;
        dw.move(more), gw.move(more), coef.move(more);
        if (GATE) zw.move(more);
    };
    auto prepare = [&](int k) {
        const int at = k & 1, last = k + 1 < tiles ? kTile - 1 : tail;
        float v[JR], d[JR], gy[JR], slope[JR];
#pragma unroll
        for (int j = 0; j < JR; ++j) v[j] = to_f32<DT>(dr[j]) + bias[j];
        step_sizes<false>(a, v, d, slope);
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            gy[j] = to_f32<DT>(gr[j]);
            if (GATE) gy[j] *= silu_f(to_f32<DT>(zr[j]));
        }
        if (p.row > last) {
#pragma unroll
            for (int j = 0; j < JR; ++j) d[j] = gy[j] = 0.0f;
        }
        store_floats<ROWS>(&sd[at][p.row][0][p.c], d);
        store_floats<ROWS>(&sd[at][p.row][1][p.c], gy);
        sC[at][coef.t][coef.n] = coef.c(last);
    };
    if (ROWS != kApart && p.channels < kWave) {
        for (int r = p.wave; r < 2 * kTile * 2; r += NW)
            if (!p.on) (&sd[0][0][0][0])[r * kWave + p.lane] = 0.0f;
    }
    if (tiles > 0) {
        fetch(tiles - 1);
        prepare(tiles - 1);
        fetch(tiles > 1 ? tiles - 2 : 0);
        lds_barrier();
    }
    for (int k = tiles - 1; k >= 0; --k) {
        take_turn(k);
        const int half = k & 1;
        if (k > 0) prepare(k - 1);
        fetch(k > 1 ? k - 2 : 0);
        constexpr int kGroup = 4;  // as in the forward
        float dd[2][kGroup], gy[2][kGroup];
        float Ct[2][kGroup][kPer];
        auto operands = [&](int g, int to) {
#pragma unroll
            for (int r = 0; r < kGroup; ++r) {
                const int t = g * kGroup + r;
                dd[to][r] = sd[half][t][0][p.lane];
                gy[to][r] = sd[half][t][1][p.lane];
                load4(&sC[half][t][p.wave * kPer], Ct[to][r]);
            }
        };
        operands(kTile / kGroup - 1, (kTile / kGroup - 1) & 1);
#pragma unroll
        for (int g = kTile / kGroup - 1; g >= 0; --g) {
            const int at = g & 1;
            if (g > 0) operands(g - 1, at ^ 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = kGroup - 1; r >= 0; --r) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    carry[i] = __builtin_fmaf(Ct[at][r][i], gy[at][r], carry[i]) *
                               exp2_f(dd[at][r] * A2[i]);
                total += dd[at][r];
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        lds_barrier();
    }
    store_state(q.ends + (int64_t)blockIdx.z * a.nb * a.N * a.H, a, p, carry);
    if (p.wave == 0 && p.on) q.dsum[((int64_t)blockIdx.z * a.nb + p.b) * a.H + p.h] = total;
}

// Two waves a SIMD: a single one issues a multiply-add every 5.1 cycles, two together one every 3.3, four
// every 2.8. The tile's history takes 128 registers of the 256 that leaves. Up to 8 states (two waves
// with eight channels a thread) the rest does not: 66 registers are spilled, 36 without a gate, and 143
// and 89 where channels are taken one by one (16 states: none; one by one 24 and 5).
template <int DT, int NW, bool GATE, int ROWS>
__global__ void __launch_bounds__(NW *kWave, 2)
    scan_bwd(ScanIn a, ScanGrad q) {
    constexpr int NP = NW * kPer, JR = kTile / NW;
    typedef typename HVec<JR>::t vec;
    __shared__ __align__(16) float sd[kTile][3][kWave];  // d, d x, gy
    __shared__ __align__(16) float sB[kTile][NP], sC[kTile][NP];
    // sums over a wave's states: u, w and (with a gate) y
    __shared__ __align__(16) float su[NW][kTile][kWave], sw[NW][kTile][kWave];
    __shared__ __align__(16) float sy[GATE ? NW : 1][GATE ? kTile : 1][kWave];
    __shared__ __align__(16) float sparam[2][kWave];  // dt_bias, D
    const Place p = place<NW, ROWS>(a);
    if (p.wave == 0) {
        sparam[0][p.lane] = a.bias ? a.bias[p.h] : 0.0f;
        sparam[1][p.lane] = a.D ? a.D[p.h] : 0.0f;
    }
    float A2[kPer], carry[kPer];
    double gA[kPer] = {0.0, 0.0, 0.0, 0.0};
    load_rates(a, p, A2);
    load_state(q.gfinal, a, p, carry);
    fold_chunks(q.ends, q.dsum, a, p, a.chunks - 1, -1, a.chunks - 1 - (int)blockIdx.z, A2, carry);
    // gD and gdt_bias of the thread's channels: fp32 sums of 32 rows, and of those sums
    float gD[2][JR], gb[2][JR];
#pragma unroll
    for (int j = 0; j < JR; ++j) gD[0][j] = gD[1][j] = gb[0][j] = gb[1][j] = 0.0f;
    const int tiles = p.end > p.r0 ? (int)((p.end - p.r0 + kTile - 1) / kTile) : 0;
    const int64_t t0 = p.r0 + (int64_t)(tiles - 1) * kTile;
    const int tail = (int)(p.end - t0) - 1;  // the last tile may be partial, the others are whole
    const int64_t BH = a.nb * a.H, states = BH * a.N;
    if (p.on)  // rows past the length
        for (int64_t t = (p.end > p.r0 ? p.end : p.r0) + p.wave; t < p.r1; t += NW) {
            const int64_t o = t * BH + p.b * a.H + p.h;
            q.gx[o] = 0;
            q.gdt[o] = 0;
            if (GATE) q.gz[o] = 0;
        }
    Walk<NW, ROWS> xw(a.x, p, t0, -1), dw(a.dt, p, t0, -1), zw(a.z, p, t0, -1), gw(q.go, p, t0, -1);
    CoefWalk<DT, NW> coef(a, p, t0, -1);
    // the lane's state n before the tile at kept[n H]
    const float *kept = q.saved + t0 / kTile * states + (p.b * a.N + p.wave * kPer) * a.H + p.h;
    int64_t to = (t0 + p.row) * BH + p.b * a.H + p.h0 + p.c;  // where the thread's row goes
    const int64_t pbc_row = a.nb * 2 * NP;
    // the sums over channels that this lane ends up with (see below): value n of B or C, row sum_t
    // of a half tile
    const int sum_t = ((p.lane >> 2) & 1) + (p.lane & 2) + (p.lane & 1) * 4;
    float *pbc = q.pbc + (((int64_t)blockIdx.x * q.pbc_rows + t0 + sum_t) * a.nb + p.b) * 2 * NP +
                 ((p.lane >> 3) & 1) * NP + p.wave * kPer + (p.lane >> 5) + ((p.lane >> 4) & 1) * 2;
    vec xr, dr, zr, gr;  // fetched; then the tile's and the last one's, which finishing it needs
    vec xc, zc, gc;
    float first[kPer];  // the state before the tile
    float slope[JR];
    auto fetch = [&](int k, int last) {
        xr = xw.fetch(p, last);
        dr = dw.fetch(p, last);
        gr = gw.fetch(p, last);
        if (GATE) zr = zw.fetch(p, last);
        coef.template fetch<true, true>(last);
        // states past N have no place: the first of the wave's (or of all) is read and not used
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            first[i] = kept[p.wave * kPer + i < a.N ? i * a.H : p.wave * kPer < a.N ? 0 : -(int64_t)(p.wave * kPer) * a.H];
        const bool more = k > 0;
        xw.move(more), dw.move(more), gw.move(more), coef.move(more);
        if (GATE) zw.move(more);
        kept -= more ? states : 0;
    };
    // Tile k's operands in LDS.
    auto prepare = [&](int k) {
        const int last = k + 1 < tiles ? kTile - 1 : tail;
        float v[JR], d[JR], dx[JR], gy[JR];
        load_floats<ROWS>(&sparam[0][p.c], v);
#pragma unroll
        for (int j = 0; j < JR; ++j) v[j] += to_f32<DT>(dr[j]);
        step_sizes<true>(a, v, d, slope);
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            dx[j] = d[j] * to_f32<DT>(xr[j]);
            gy[j] = to_f32<DT>(gr[j]);
            if (GATE) gy[j] *= silu_f(to_f32<DT>(zr[j]));
        }
        if (p.row > last || (ROWS == kApart && p.channels < kWave)) {
#pragma unroll
            for (int j = 0; j < JR; ++j)
                if (p.row > last || p.c + j >= p.channels) d[j] = dx[j] = gy[j] = 0.0f;
        }
        store_floats<ROWS>(&sd[p.row][0][p.c], d);
        store_floats<ROWS>(&sd[p.row][1][p.c], dx);
        store_floats<ROWS>(&sd[p.row][2][p.c], gy);
        sB[coef.t][coef.n] = coef.b(last);
        sC[coef.t][coef.n] = coef.c(last);
    };
    // Tile k's gradients, from the sums its waves left in LDS; d and gy are its rows', read before
    // the next tile's took their place.
    auto finish = [&](int k, const float (&d)[JR], const float (&gy)[JR], const float (&slope)[JR]) {
        float D[JR], u[JR], w[JR], y[JR], f[JR];
        load_floats<ROWS>(&sparam[1][p.c], D);
        load_floats<ROWS>(&su[0][p.row][p.c], u);
        load_floats<ROWS>(&sw[0][p.row][p.c], w);
        if (GATE) load_floats<ROWS>(&sy[0][p.row][p.c], y);
#pragma unroll
        for (int i = 1; i < NW; ++i) {
            load_floats<ROWS>(&su[i][p.row][p.c], f);
#pragma unroll
            for (int j = 0; j < JR; ++j) u[j] += f[j];
            load_floats<ROWS>(&sw[i][p.row][p.c], f);
#pragma unroll
            for (int j = 0; j < JR; ++j) w[j] += f[j];
            if (GATE) {
                load_floats<ROWS>(&sy[i][p.row][p.c], f);
#pragma unroll
                for (int j = 0; j < JR; ++j) y[j] += f[j];
            }
        }
        if (p.row <= (k + 1 < tiles ? kTile - 1 : tail)) {
            vec gx, gdt, gz;
#pragma unroll
            for (int j = 0; j < JR; ++j) {
                const float x = to_f32<DT>(xc[j]);
                const float gd = __builtin_fmaf(w[j], kLn2, u[j] * x) * slope[j];
                gx[j] = from_f32<DT>(__builtin_fmaf(u[j], d[j], D[j] * gy[j]));
                gdt[j] = from_f32<DT>(gd);
                gD[0][j] = __builtin_fmaf(gy[j], x, gD[0][j]);
                gb[0][j] += gd;
                if (GATE)
                    gz[j] = from_f32<DT>(to_f32<DT>(gc[j]) * __builtin_fmaf(D[j], x, y[j]) *
                                         silu_slope_f(to_f32<DT>(zc[j])));
            }
            store_rows<ROWS, JR>(q.gx + to, p, gx);
            store_rows<ROWS, JR>(q.gdt + to, p, gdt);
            if (GATE) store_rows<ROWS, JR>(q.gz + to, p, gz);
        }
        to -= kTile * BH;
        if (k % 32 == 0) {
#pragma unroll
            for (int j = 0; j < JR; ++j) {
                gD[1][j] += gD[0][j], gD[0][j] = 0.0f;
                gb[1][j] += gb[0][j], gb[0][j] = 0.0f;
            }
        }
    };
    if (ROWS != kApart && p.channels < kWave) {  // columns that no thread writes add nothing to the sums
        for (int r = p.wave; r < kTile * 3; r += NW)
            if (!p.on) (&sd[0][0][0])[r * kWave + p.lane] = 0.0f;
    }
    if (tiles > 0) fetch(tiles - 1, tail);
    lds_barrier();
    for (int k = tiles - 1; k >= 0; --k) {
        take_turn(k);
        float d[JR], gy[JR], last_slope[JR], s0[kPer];
        load_floats<ROWS>(&sd[p.row][0][p.c], d);
        load_floats<ROWS>(&sd[p.row][2][p.c], gy);
#pragma unroll
        for (int j = 0; j < JR; ++j) last_slope[j] = slope[j];
#pragma unroll
        for (int i = 0; i < kPer; ++i) s0[i] = p.wave * kPer + i < a.N ? first[i] : 0.0f;
        prepare(k);  // waits for the tile's loads, so before any store (see the forward)
        if (k + 1 < tiles) finish(k + 1, d, gy, last_slope);
        xc = xr, zc = zr, gc = gr;
        if (k > 0) fetch(k - 1, kTile - 1);
        lds_barrier();
        // the tile's states and decays again, kept in registers
        float S[kTile][kPer], E[kTile][kPer];
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            const float dd = sd[t][0][p.lane], dx = sd[t][1][p.lane];
            float Bt[kPer], Ct[kPer], y = 0.0f;
            load4(&sB[t][p.wave * kPer], Bt);
            if (GATE) load4(&sC[t][p.wave * kPer], Ct);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                E[t][i] = exp2_f(dd * A2[i]);
                S[t][i] = __builtin_fmaf(E[t][i], t ? S[t - 1][i] : s0[i], dx * Bt[i]);
                if (GATE) y = __builtin_fmaf(Ct[i], S[t][i], y);
            }
            if (GATE) sy[p.wave][t][p.lane] = y;
            // keep the reads of later rows from being taken up front: registers are what is short
            if (t % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
        float tA[kPer] = {0.0f, 0.0f, 0.0f, 0.0f};
        // Sums over the wave's channels. A row has eight values (four of gB, four of gC) in 64 lanes:
        // halving the values while adding lanes 32, 16 and 8 apart leaves a register a row, and eight
        // rows' registers join the same way over the last eight lanes. Value v of row t ends in lane
        // bits 5, 4, 3 = v's bits 0, 1, 2 and lane bits 2, 1, 0 = t's bits 0, 1, 2.
        float part[kTile / 2];
#pragma unroll
        for (int t = kTile - 1; t >= 0; --t) {
            const float dd = sd[t][0][p.lane], dx = sd[t][1][p.lane], gy = sd[t][2][p.lane];
            float Bt[kPer], Ct[kPer], u = 0.0f, w = 0.0f, v[2 * kPer];
            load4(&sB[t][p.wave * kPer], Bt);
            load4(&sC[t][p.wave * kPer], Ct);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float gs = __builtin_fmaf(Ct[i], gy, carry[i]);
                v[i] = gs * dx;
                v[kPer + i] = gy * S[t][i];
                u = __builtin_fmaf(gs, Bt[i], u);
                carry[i] = gs * E[t][i];
                const float g = carry[i] * (t ? S[t - 1][i] : s0[i]);
                w = __builtin_fmaf(g, A2[i], w);
                tA[i] = __builtin_fmaf(g, dd, tA[i]);
            }
            su[p.wave][t][p.lane] = u;
            sw[p.wave][t][p.lane] = w;
            float r4[4], r2[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) r4[i] = swap_add32(v[2 * i], v[2 * i + 1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) r2[i] = swap_add16(r4[2 * i], r4[2 * i + 1]);
            part[t % 8] = join<kRor8>(r2[0], r2[1], p.lane & 8);
            if (t % 8 == 0) {
                float h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    h[i] = join<kHalfMirror>(part[2 * i], part[2 * i + 1], p.lane & 4);
                const float m0 = join<kXor2>(h[0], h[1], p.lane & 2);
                const float m1 = join<kXor2>(h[2], h[3], p.lane & 2);
                const float m = join<kXor1>(m0, m1, p.lane & 1);
                pbc[t * pbc_row] = m;  // rows past the length too: their place is never read
            }
            if (t % 2 == 0) __builtin_amdgcn_sched_barrier(0);
        }
        pbc -= kTile * pbc_row;
#pragma unroll
        for (int i = 0; i < kPer; ++i) gA[i] += (double)tA[i];
        lds_barrier();
    }
    if (tiles > 0) {
        float d[JR], gy[JR];
        load_floats<ROWS>(&sd[p.row][0][p.c], d);
        load_floats<ROWS>(&sd[p.row][2][p.c], gy);
        finish(0, d, gy, slope);
        lds_barrier();  // the sums below take the place of what finish read
    }
    if (blockIdx.z == 0 && q.gstate) store_state(q.gstate, a, p, carry);
    double *pa = q.pa + ((int64_t)blockIdx.z * a.nb + p.b) * (a.N + 2) * a.H;
    store_floats<ROWS>(&su[0][p.row][p.c], gD[1]);
    store_floats<ROWS>(&sw[0][p.row][p.c], gb[1]);
    lds_barrier();
    if (!p.on) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = p.wave * kPer + i;
        if (n < a.N) pa[(int64_t)n * a.H + p.h] = gA[i];
    }
    if (p.wave == 0) {
        double d = 0.0, b = 0.0;
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            d += (double)su[0][t][p.lane];
            b += (double)sw[0][t][p.lane];
        }
        pa[(int64_t)a.N * a.H + p.h] = d;
        pa[(int64_t)(a.N + 1) * a.H + p.h] = b;
    }
}

// gB and gC: the sums of each group's blocks (fp32, of 64 channels each) in their order, in fp64: there may
// be 2^18 of them. (row, batch, group, which, n), n fastest, go round the threads.
template <int DT>
__global__ void __launch_bounds__(256)
    scan_sum_bc(const float *__restrict__ pbc, const int64_t *__restrict__ lengths, int64_t S,
                int64_t pbc_rows, int64_t nb, int N, int NP, int G, int per_group, uint16_t *__restrict__ gB,
                uint16_t *__restrict__ gC) {
    const int64_t rows = S * nb, all = rows * G * 2 * NP;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < all; id += (int64_t)gridDim.x * 256) {
        const int n = (int)(id % NP), which = (int)(id / NP % 2);
        const int64_t rg = id / (2 * NP);  // group slowest, so that neighbours read one block's sums
        const int64_t row = rg % rows, g = rg / rows;
        if (n >= N) continue;
        const int64_t t = row / nb, b = row - t * nb;
        double s = 0.0;
        if (!lengths || t < lengths[b]) {
            const int64_t block = pbc_rows * nb;
            const float *p = pbc + ((g * per_group * block + row) * 2 + which) * NP + n;
#pragma unroll 8
            for (int i = 0; i < per_group; ++i) s += (double)p[(int64_t)i * block * 2 * NP];
        }
        (which ? gC : gB)[(row * G + g) * N + n] = from_f32<DT>((float)s);
    }
}

// gA, gD and gdt_bias: [P][(N+2) H] doubles over P.
__global__ void __launch_bounds__(256)
    scan_sum_params(const double *__restrict__ pa, int64_t P, int64_t N, int64_t H,
                    float *__restrict__ gA, float *__restrict__ gD, float *__restrict__ gbias) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x, n_all = (N + 2) * H;
    if (c >= n_all) return;
    double s = 0.0;
#pragma unroll 8
    for (int64_t p = 0; p < P; ++p) s += pa[p * n_all + c];
    if (c < N * H)
        gA[c] = (float)s;
    else if (c < (N + 1) * H) {
        if (gD) gD[c - N * H] = (float)s;
    } else if (gbias) {
        gbias[c - (N + 1) * H] = (float)s;
    }
}

// ---------------------------------------------------------------------------------------------
// Single token: a lane has a channel of one batch and all its states; the state is read and written
// once, by rows of 64 channels (two channels a lane were slower: 10.5 us against 9.5 for B=64 H=5120
// N=16, 4.4 TB/s). Where the wave's channels are of one group its lanes load all of B and C at once,
// a value each (N is at most 32), and hand them round (12.5 us with a load a value).
// ---------------------------------------------------------------------------------------------
template <int DT, int NMAX>
__global__ void __launch_bounds__(kWave)
    scan_one(ScanIn a, float *__restrict__ state, uint16_t *__restrict__ out) {
    const int64_t b = blockIdx.y, h0 = (int64_t)blockIdx.x * kWave;
    const bool on = h0 + threadIdx.x < a.H;
    const int64_t h = on ? h0 + threadIdx.x : a.H - 1;
    const int64_t g0 = h0 / a.K, last = h0 + kWave < a.H ? h0 + kWave - 1 : a.H - 1;
    const bool one_group = g0 == last / a.K;
    float s[NMAX], r[NMAX];
    float *sp = state + b * a.N * a.H + h;
#pragma unroll
    for (int n = 0; n < NMAX; ++n)  // rows past N repeat the last and are not stored
        s[n] = sp[(int64_t)(n < a.N ? n : a.N - 1) * a.H];
    float mine = 0.0f;
    if (one_group) {
        const int n = threadIdx.x % 32;
        if (n < a.N)
            mine = to_f32<DT>(threadIdx.x < 32 ? a.B.p[b * a.B.b + g0 * a.B.g + n * a.B.n]
                                               : a.C.p[b * a.C.b + g0 * a.C.g + n * a.C.n]);
    }
#pragma unroll
    for (int n = 0; n < NMAX; ++n) r[n] = a.A[(int64_t)(n < a.N ? n : a.N - 1) * a.H + h];
    const float x = to_f32<DT>(a.x.p[b * a.x.b + h * a.x.h]);
    const float t = to_f32<DT>(a.dt.p[b * a.dt.b + h * a.dt.h]) + (a.bias ? a.bias[h] : 0.0f);
    const float z = a.z.p ? to_f32<DT>(a.z.p[b * a.z.b + h * a.z.h]) : 0.0f;
    const float d = a.softplus ? softplus_f(t) : t;
    float y = a.D ? a.D[h] * x : 0.0f;
    const float dx = d * x, d2 = d * kLog2e;
    // No step leaves the state alone, also with an infinite rate. Rates are bounded where a lane has none:
    // always, the token is 5 to 10 % slower.
    if (__builtin_amdgcn_ballot_w64(d == 0.0f)) {
#pragma unroll
        for (int n = 0; n < NMAX; ++n) r[n] = finite_rate(r[n]);
    }
    if (one_group) {
#pragma unroll
        for (int n = 0; n < NMAX; ++n) {
            const float Bn = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), n));
            const float Cn = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), n + 32));
            s[n] = __builtin_fmaf(exp2_f(d2 * r[n]), s[n], dx * Bn);
            if (n < a.N) y = __builtin_fmaf(Cn, s[n], y);
        }
    } else {
        const int64_t g = h / a.K;
#pragma unroll
        for (int n = 0; n < NMAX; ++n) {
            const int row = n < a.N ? n : a.N - 1;
            const float Bn = to_f32<DT>(a.B.p[b * a.B.b + g * a.B.g + row * a.B.n]);
            const float Cn = to_f32<DT>(a.C.p[b * a.C.b + g * a.C.g + row * a.C.n]);
            s[n] = __builtin_fmaf(exp2_f(d2 * r[n]), s[n], dx * Bn);
            if (n < a.N) y = __builtin_fmaf(Cn, s[n], y);
        }
    }
    if (!on) return;
#pragma unroll
    for (int n = 0; n < NMAX; ++n)
        if (n < a.N) sp[(int64_t)n * a.H] = s[n];
    out[b * a.H + h] = from_f32<DT>(a.z.p ? y * silu_f(z) : y);
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------
int check_scan(const mccb_scan_t *a, bool token) {
    if (!a) return MCCB_ERR_PARAM_NULLPTR;
    if (a->dtype != MCCB_BF16 && a->dtype != MCCB_FP16) return MCCB_ERR_PARAM_INVALID;
    // a group has a block of 128 to 512 threads at least, and a grid less than 2^32 along an axis
    if (a->B < 1 || a->B > kMaxBatch || a->S < 0 || a->S >= kMaxRows || a->H < 1 ||
        a->H > kMaxWidth || a->N < 1 || a->N > 32 || a->G < 1 || a->G > (int64_t)1 << 22 || a->H % a->G ||
        a->B * a->H >= kMaxRows || (token && a->S != 1))
        return MCCB_ERR_SHAPE;
    return MCCB_OK;
}

uint64_t row_bytes(const mccb_scan_t *a) { return (uint64_t)a->S * (uint64_t)(a->B * a->H) * 2; }
uint64_t coef_bytes(const mccb_scan_t *a) { return (uint64_t)a->S * (uint64_t)(a->B * a->G * a->N) * 2; }
uint64_t state_bytes(const mccb_scan_t *a) { return (uint64_t)(a->B * a->H) * (uint64_t)a->N * 4; }

int check_scan_inputs(const mccb_scan_t *a, Span *in, int *n) {
    if (!a->A || (a->S > 0 && (!a->x || !a->dt || !a->Bm || !a->Cm))) return MCCB_ERR_PARAM_NULLPTR;
    const int64_t rows[3] = {a->S, a->B, a->H}, coef[4] = {a->S, a->B, a->G, a->N};
    uint64_t x, dt, z = 0, b, c;
    if (!extent(3, rows, a->x_stride, 2, &x) || !extent(3, rows, a->dt_stride, 2, &dt) ||
        (a->z && !extent(3, rows, a->z_stride, 2, &z)) || !extent(4, coef, a->b_stride, 2, &b) ||
        !extent(4, coef, a->c_stride, 2, &c))
        return MCCB_ERR_PARAM_INVALID;
    if (misaligned(a->x, 2) || misaligned(a->dt, 2) || misaligned(a->z, 2) || misaligned(a->Bm, 2) ||
        misaligned(a->Cm, 2) || misaligned(a->A, 4) || misaligned(a->D, 4) ||
        misaligned(a->dt_bias, 4) || misaligned(a->state, 4) || misaligned(a->lengths, 8))
        return MCCB_ERR_PARAM_INVALID;
    const Span all[10] = {{a->x, x},
                          {a->dt, dt},
                          {a->z, z},
                          {a->Bm, b},
                          {a->Cm, c},
                          {a->A, (uint64_t)(a->N * a->H) * 4},
                          {a->D, (uint64_t)a->H * 4},
                          {a->dt_bias, (uint64_t)a->H * 4},
                          {a->lengths, (uint64_t)a->B * 8},
                          {a->state, state_bytes(a)}};
    for (int i = 0; i < 10; ++i) in[i] = all[i];
    *n = 10;
    return MCCB_OK;
}

// How the work is cut: a function of the sizes alone.
struct ScanPlan {
    int waves, chunks;
    int64_t per_group, blocks, chunk_rows;
};

ScanPlan plan_of(const mccb_scan_t *a) {
    ScanPlan p;
    p.waves = a->N <= 8 ? 2 : a->N <= 16 ? 4 : 8;
    const int64_t K = a->H / a->G;
    p.per_group = (K + kWave - 1) / kWave;
    p.blocks = p.per_group * a->G;
    // Chunks cost a second pass over the recurrence, so they pay only where they multiply the waves
    // well beyond that: at most half the card's SIMDs busy without them. Then as many as give six
    // waves a SIMD (three at a time; 24 chunks of S=16384 H=4096 take 570 us, 8 take 640), of three
    // tiles at least (S=777 B=5 H=1000 N=8: 32 us, four tiles 34, two 35).
    const int64_t waves = p.blocks * a->B * p.waves, tiles = (a->S + kTile - 1) / kTile;
    int64_t chunks = 1;
    if (waves <= 512) {
        chunks = 6144 / waves;
        if (chunks > tiles / 3) chunks = tiles / 3;
        if (chunks > 64) chunks = 64;
        if (chunks < 4) chunks = 1;
    }
    const int64_t per = tiles > 0 ? (tiles + chunks - 1) / chunks : 1;
    p.chunk_rows = per * kTile;
    p.chunks = tiles > 0 ? (int)((tiles + per - 1) / per) : 1;
    return p;
}

ScanIn device_args(const mccb_scan_t *a, const ScanPlan &p) {
    ScanIn in;
    auto rows = [](const void *q, const int64_t *s) {
        return Rows{(const uint16_t *)q, s[0], s[1], s[2]};
    };
    in.x = rows(a->x, a->x_stride);
    in.dt = rows(a->dt, a->dt_stride);
    in.z = rows(a->z, a->z_stride);
    in.B = {(const uint16_t *)a->Bm, a->b_stride[0], a->b_stride[1], a->b_stride[2], a->b_stride[3]};
    in.C = {(const uint16_t *)a->Cm, a->c_stride[0], a->c_stride[1], a->c_stride[2], a->c_stride[3]};
    in.A = a->A, in.D = a->D, in.bias = a->dt_bias, in.state = a->state;
    in.lengths = a->lengths;
    in.S = a->S, in.nb = a->B, in.H = a->H, in.K = a->H / a->G;
    in.N = (int)a->N, in.G = (int)a->G, in.per_group = (int)p.per_group;
    in.softplus = a->softplus, in.chunks = p.chunks;
    in.chunk_rows = p.chunk_rows;
    return in;
}

// How a block's threads take their channels of a row (`out` is the gradient of the output, or NULL).
int rows_form(const mccb_scan_t *a, const ScanPlan &p, const int64_t *out) {
    const int64_t K = a->H / a->G, JR = kTile / p.waves, tail = K % kWave;
    if (a->x_stride[2] != 1 || a->dt_stride[2] != 1 || (a->z && a->z_stride[2] != 1) ||
        (out && out[2] != 1) || (tail && tail < JR))
        return kApart;
    // the last threads of the last block start at its channel tail - JR
    return tail % (JR < 4 ? JR : 4) ? kAdjacent : kWide;
}

// Workspace for handing states between chunks.
uint64_t chunk_bytes(const mccb_scan_t *a, const ScanPlan &p) {
    if (p.chunks == 1) return 0;
    return (uint64_t)p.chunks * align16(state_bytes(a) + (uint64_t)(a->B * a->H) * 4);
}

uint64_t pbc_bytes(const mccb_scan_t *a, const ScanPlan &p) {
    const uint64_t rows = (uint64_t)((a->S + kTile - 1) / kTile * kTile);
    return (uint64_t)p.blocks * rows * (uint64_t)a->B * (2 * p.waves * kPer) * 4;
}
uint64_t pa_bytes(const mccb_scan_t *a, const ScanPlan &p) {
    return (uint64_t)p.chunks * (uint64_t)a->B * (uint64_t)((a->N + 2) * a->H) * 8;
}

template <typename F>
int by_waves(int waves, F f) {
    switch (waves) {
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}
template <typename F>
int by_rows(int form, F f) {
    switch (form) {
        case kApart: return f(std::integral_constant<int, kApart>{});
        case kAdjacent: return f(std::integral_constant<int, kAdjacent>{});
        default: return f(std::integral_constant<int, kWide>{});
    }
}
template <typename F>
int by_flag(bool v, F f) {
    return v ? f(std::true_type{}) : f(std::false_type{});
}
template <typename F>
int by_dtype(int dtype, F f) {
    return dtype == MCCB_BF16 ? f(std::integral_constant<int, MCCB_BF16>{})
                              : f(std::integral_constant<int, MCCB_FP16>{});
}

}  // namespace

extern "C" {

int mccb_scan_saved_size(const mccb_scan_t *a, uint64_t *bytes) {
    if (!bytes) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_scan(a, false);
    if (rc != MCCB_OK) return rc;
    *bytes = (uint64_t)((a->S + kTile - 1) / kTile) * state_bytes(a);
    return MCCB_OK;
}

int mccb_scan_forward_get_workspace_size(const mccb_scan_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_scan(a, false);
    if (rc != MCCB_OK) return rc;
    *size = chunk_bytes(a, plan_of(a));
    return MCCB_OK;
}

int mccb_scan_forward(const mccb_scan_t *a, void *out, float *final_state, void *saved, void *ws,
                      uint64_t ws_size, void *stream) {
    int rc = check_scan(a, false);
    if (rc != MCCB_OK) return rc;
    if (!out && a->S > 0) return MCCB_ERR_PARAM_NULLPTR;
    Span in[10];
    int n;
    rc = check_scan_inputs(a, in, &n);
    if (rc != MCCB_OK) return rc;
    const ScanPlan p = plan_of(a);
    const uint64_t need = chunk_bytes(a, p);
    uint64_t saved_bytes = 0;
    mccb_scan_saved_size(a, &saved_bytes);
    rc = check_workspace(ws, ws_size, need);
    if (rc != MCCB_OK) return rc;
    const Span outs[4] = {{out, row_bytes(a)},
                          {final_state, state_bytes(a)},
                          {saved, saved_bytes},
                          {ws, need}};
    if (misaligned(out, 2) || misaligned(final_state, 4) || misaligned(saved, 16) ||
        outputs_clash(in, n, outs, 4))
        return MCCB_ERR_PARAM_INVALID;
    if (a->S == 0 && !final_state) return MCCB_OK;
    const ScanIn da = device_args(a, p);
    float *ends = (float *)ws;
    float *dsum = p.chunks > 1 ? ends + (uint64_t)p.chunks * (uint64_t)(a->B * a->N * a->H) : nullptr;
    const dim3 grid((unsigned)p.blocks, (unsigned)a->B, (unsigned)p.chunks);
    const dim3 first((unsigned)p.blocks, (unsigned)a->B, (unsigned)(p.chunks - 1));
    const hipStream_t st = (hipStream_t)stream;
    return by_dtype(a->dtype, [&](auto dt) {
        return by_waves(p.waves, [&](auto nw) {
            return by_rows(rows_form(a, p, nullptr), [&](auto rows) {
                constexpr int DT = decltype(dt)::value, NW = decltype(nw)::value;
                constexpr int R = decltype(rows)::value;
                const dim3 block(NW * kWave);
                if (p.chunks > 1) {
                    hipLaunchKernelGGL((scan_fwd<DT, NW, true, false, R>), first, block, 0, st, da,
                                       (uint16_t *)nullptr, (float *)nullptr, (float *)nullptr, ends,
                                       dsum);
                    const int r = launched();
                    if (r != MCCB_OK) return r;
                }
                return by_flag(a->z != nullptr, [&](auto gate) {
                    hipLaunchKernelGGL((scan_fwd<DT, NW, false, decltype(gate)::value, R>), grid, block,
                                       0, st, da, (uint16_t *)out, final_state, (float *)saved, ends,
                                       dsum);
                    return launched();
                });
            });
        });
    });
}

int mccb_scan_backward_get_workspace_size(const mccb_scan_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_scan(a, false);
    if (rc != MCCB_OK) return rc;
    const ScanPlan p = plan_of(a);
    *size = pa_bytes(a, p) + align16(pbc_bytes(a, p)) + chunk_bytes(a, p);
    return MCCB_OK;
}

int mccb_scan_backward(const mccb_scan_t *a, const mccb_scan_grads_t *g, const void *saved, void *ws,
                       uint64_t ws_size, void *stream) {
    int rc = check_scan(a, false);
    if (rc != MCCB_OK) return rc;
    if (!g || !g->gradA) return MCCB_ERR_PARAM_NULLPTR;
    if (a->S > 0 && (!g->gradOut || !g->gradX || !g->gradDt || !g->gradB || !g->gradC || !saved ||
                     (a->z && !g->gradZ)))
        return MCCB_ERR_PARAM_NULLPTR;
    if (!a->z && g->gradZ) return MCCB_ERR_PARAM_INVALID;
    Span in[13];
    int n;
    rc = check_scan_inputs(a, in, &n);
    if (rc != MCCB_OK) return rc;
    const int64_t rows[3] = {a->S, a->B, a->H};
    uint64_t go_bytes, need = 0, saved_bytes = 0;
    if (!extent(3, rows, g->gout_stride, 2, &go_bytes)) return MCCB_ERR_PARAM_INVALID;
    mccb_scan_backward_get_workspace_size(a, &need);
    mccb_scan_saved_size(a, &saved_bytes);
    rc = check_workspace(ws, ws_size, need);
    if (rc != MCCB_OK) return rc;
    in[n++] = {g->gradOut, go_bytes};
    in[n++] = {g->gradFinalState, state_bytes(a)};
    in[n++] = {saved, saved_bytes};
    const uint64_t r = row_bytes(a), c = coef_bytes(a), h4 = (uint64_t)a->H * 4;
    const Span outs[10] = {{g->gradX, r},     {g->gradDt, r},     {g->gradZ, r},
                           {g->gradB, c},     {g->gradC, c},      {g->gradA, (uint64_t)a->N * h4},
                           {g->gradD, h4},    {g->gradDtBias, h4}, {g->gradState, state_bytes(a)},
                           {ws, need}};
    for (int i = 0; i < 5; ++i)
        if (misaligned(outs[i].p, 2)) return MCCB_ERR_PARAM_INVALID;
    for (int i = 5; i < 9; ++i)
        if (misaligned(outs[i].p, 4)) return MCCB_ERR_PARAM_INVALID;
    if (misaligned(g->gradOut, 2) || misaligned(g->gradFinalState, 4) || misaligned(saved, 16) ||
        outputs_clash(in, n, outs, 10))
        return MCCB_ERR_PARAM_INVALID;
    const ScanPlan p = plan_of(a);
    const ScanIn da = device_args(a, p);
    ScanGrad q;
    q.go = {(const uint16_t *)g->gradOut, g->gout_stride[0], g->gout_stride[1], g->gout_stride[2]};
    q.gfinal = g->gradFinalState, q.saved = (const float *)saved;
    q.gx = (uint16_t *)g->gradX, q.gdt = (uint16_t *)g->gradDt, q.gz = (uint16_t *)g->gradZ;
    q.gstate = g->gradState;
    uint8_t *at = (uint8_t *)ws;
    q.pa = (double *)at;
    at += pa_bytes(a, p);
    q.pbc = (float *)at;
    q.pbc_rows = (a->S + kTile - 1) / kTile * kTile;
    at += align16(pbc_bytes(a, p));
    q.ends = p.chunks > 1 ? (float *)at : nullptr;
    q.dsum = p.chunks > 1 ? q.ends + (uint64_t)p.chunks * (uint64_t)(a->B * a->N * a->H) : nullptr;
    const dim3 grid((unsigned)p.blocks, (unsigned)a->B, (unsigned)p.chunks);
    const hipStream_t st = (hipStream_t)stream;
    rc = by_dtype(a->dtype, [&](auto dt) {
        return by_waves(p.waves, [&](auto nw) {
            constexpr int DT = decltype(dt)::value, NW = decltype(nw)::value;
            const dim3 block(NW * kWave);
            int e = by_rows(rows_form(a, p, g->gout_stride), [&](auto form) {
                return by_flag(a->z != nullptr, [&](auto gate) {
                    constexpr int R = decltype(form)::value;
                    constexpr bool GATE = decltype(gate)::value;
                    if (p.chunks > 1) {
                        hipLaunchKernelGGL((scan_bwd_ends<DT, NW, GATE, R>), grid, block, 0, st, da, q);
                        const int r = launched();
                        if (r != MCCB_OK) return r;
                    }
                    hipLaunchKernelGGL((scan_bwd<DT, NW, GATE, R>), grid, block, 0, st, da, q);
                    return launched();
                });
            });
            if (e != MCCB_OK || a->S == 0) return e;
            // a grid has less than 2^32 threads along an axis
            const int64_t ids = a->S * a->B * a->G * 2 * NW * kPer, wanted = (ids + 255) / 256;
            const int64_t most = (int64_t)1 << 22;
            hipLaunchKernelGGL((scan_sum_bc<DT>), dim3((unsigned)(wanted < most ? wanted : most)), dim3(256), 0,
                               st, q.pbc, a->lengths, a->S, q.pbc_rows, a->B, (int)a->N, NW * kPer, (int)a->G,
                               (int)p.per_group, (uint16_t *)g->gradB, (uint16_t *)g->gradC);
            return launched();
        });
    });
    if (rc != MCCB_OK) return rc;
    const int64_t n_all = (a->N + 2) * a->H;
    hipLaunchKernelGGL(scan_sum_params, dim3((unsigned)((n_all + 255) / 256)), dim3(256), 0, st, q.pa,
                       (int64_t)p.chunks * a->B, a->N, a->H, g->gradA, g->gradD, g->gradDtBias);
    return launched();
}

int mccb_scan_step(const mccb_scan_t *a, float *state, void *out, void *stream) {
    int rc = check_scan(a, true);
    if (rc != MCCB_OK) return rc;
    if (!state || !out) return MCCB_ERR_PARAM_NULLPTR;
    if (a->state || a->lengths) return MCCB_ERR_PARAM_INVALID;
    Span in[10];
    int n;
    rc = check_scan_inputs(a, in, &n);
    if (rc != MCCB_OK) return rc;
    const Span outs[2] = {{out, row_bytes(a)}, {state, state_bytes(a)}};
    if (misaligned(out, 2) || misaligned(state, 4) || outputs_clash(in, n, outs, 2))
        return MCCB_ERR_PARAM_INVALID;
    const ScanIn da = device_args(a, plan_of(a));
    const dim3 grid((unsigned)((a->H + kWave - 1) / kWave), (unsigned)a->B);
    return by_dtype(a->dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const hipStream_t st = (hipStream_t)stream;
        uint16_t *o = (uint16_t *)out;
        if (a->N <= 8)
            hipLaunchKernelGGL((scan_one<DT, 8>), grid, dim3(kWave), 0, st, da, state, o);
        else if (a->N <= 16)
            hipLaunchKernelGGL((scan_one<DT, 16>), grid, dim3(kWave), 0, st, da, state, o);
        else
            hipLaunchKernelGGL((scan_one<DT, 32>), grid, dim3(kWave), 0, st, da, state, o);
        return launched();
    });
}

}  // extern "C"
