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
#include "ssm_common.h"

using namespace ssm;

namespace {

constexpr int kTile = 16;  // rows; the forward keeps the state before each tile for the backward
constexpr int kPer = 4;    // states a lane holds

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

// What a block works on.
struct Place {
    int lane, wave;
    int64_t b, h;  // batch; the lane's channel, clamped into the group
    int g;
    bool on;  // whether the lane has a channel of its own
    int64_t r0, r1, end;  // the chunk's rows, and where its live rows end
};

__device__ static inline Place place(const ScanIn &a) {
    Place p;
    p.lane = threadIdx.x % kWave;
    p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    p.g = blockIdx.x / a.per_group;
    const int64_t k = (int64_t)(blockIdx.x % a.per_group) * kWave + p.lane;
    p.on = k < a.K;
    p.h = p.g * a.K + (p.on ? k : a.K - 1);
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

__device__ static inline float step_size(const ScanIn &a, float v, float &slope) {
    slope = 1.0f;
    return a.softplus ? softplus_f(v, slope) : v;
}

// A [N,H] times log2(e), so that the decay is one exp2; zero for states past N, which then stay 0.
__device__ static inline void load_rates(const ScanIn &a, const Place &p, float (&A2)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = p.wave * kPer + i;
        A2[i] = n < a.N ? a.A[(int64_t)n * a.H + p.h] * kLog2e : 0.0f;
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
    for (int j = 0; j < n; ++j) {
        const int c = first + dir * j;
        const float d = dsum[((int64_t)c * a.nb + p.b) * a.H + p.h];
        float e[kPer];
        load_state(ends + c * states, a, p, e);
#pragma unroll
        for (int i = 0; i < kPer; ++i) s[i] = __builtin_fmaf(exp2_f(d * A2[i]), s[i], e[i]);
    }
}

// One value of B and of C for each of the block's threads: 16 rows of NW*4 states.
template <int DT, int NW>
struct CoefTile {
    int n, t;
    const uint16_t *bp, *cp;
    bool has;
    uint16_t bv, cv;
    __device__ inline CoefTile(const ScanIn &a, const Place &p) {
        n = threadIdx.x % (NW * kPer);
        t = threadIdx.x / (NW * kPer);
        has = n < a.N;
        const int nc = has ? n : 0;
        bp = a.B.p + p.b * a.B.b + p.g * a.B.g + nc * a.B.n;
        cp = a.C.p + p.b * a.C.b + p.g * a.C.g + nc * a.C.n;
    }
    __device__ inline void fetch(const ScanIn &a, int64_t t0, int64_t end) {
        const int64_t r = t0 + t < end ? t0 + t : end - 1;
        bv = bp[r * a.B.s];
        cv = cp[r * a.C.s];
    }
    __device__ inline float b(int64_t t0, int64_t end) const {
        return has && t0 + t < end ? to_f32<DT>(bv) : 0.0f;
    }
    __device__ inline float c(int64_t t0, int64_t end) const {
        return has && t0 + t < end ? to_f32<DT>(cv) : 0.0f;
    }
};

__device__ static inline void load4(const float *p, float (&f)[kPer]) {
    const float4 q = *(const float4 *)p;
    f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
}

// Forward. ENDS: only the end state of each chunk from a zero state, and its sum of d (the last
// chunk's is not needed).
template <int DT, int NW, bool ENDS>
__global__ void __launch_bounds__(NW *kWave)
    scan_fwd(ScanIn a, uint16_t *__restrict__ out, float *__restrict__ final_state,
             float *__restrict__ saved, float *__restrict__ ends, float *__restrict__ dsum) {
    constexpr int NP = NW * kPer, JR = kTile / NW;
    __shared__ float2 sd[kTile][kWave];  // d, d x
    __shared__ __align__(16) float sB[kTile][NP], sC[kTile][NP];
    __shared__ float sy[ENDS ? 1 : NW][ENDS ? 1 : kTile][kWave];
    const Place p = place(a);
    float A2[kPer], s[kPer], total = 0.0f;
    load_rates(a, p, A2);
    load_state(ENDS ? nullptr : a.state, a, p, s);
    if (!ENDS) fold_chunks(ends, dsum, a, p, 0, 1, blockIdx.z, A2, s);
    const float bias = a.bias ? a.bias[p.h] : 0.0f, D = a.D ? a.D[p.h] : 0.0f;
    const uint16_t *xp = a.x.p + p.b * a.x.b + p.h * a.x.h;
    const uint16_t *dp = a.dt.p + p.b * a.dt.b + p.h * a.dt.h;
    const uint16_t *zp = a.z.p ? a.z.p + p.b * a.z.b + p.h * a.z.h : nullptr;
    CoefTile<DT, NW> coef(a, p);
    uint16_t xr[JR], dr[JR], zr[JR];
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int64_t t = t0 + p.wave + NW * j, r = t < p.end ? t : p.end - 1;
            xr[j] = xp[r * a.x.s];
            dr[j] = dp[r * a.dt.s];
            if (!ENDS && zp) zr[j] = zp[r * a.z.s];
        }
        coef.fetch(a, t0, p.end);
    };
    int64_t t0 = p.r0;
    if (t0 < p.end) fetch(t0);
    for (; t0 < p.end; t0 += kTile) {
        float xf[JR], zf[JR];
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int t = p.wave + NW * j;
            const bool live = t0 + t < p.end;
            float slope;
            const float d = live ? step_size(a, to_f32<DT>(dr[j]) + bias, slope) : 0.0f;
            xf[j] = live ? to_f32<DT>(xr[j]) : 0.0f;
            zf[j] = to_f32<DT>(zr[j]);
            sd[t][p.lane] = make_float2(d, d * xf[j]);
        }
        sB[coef.t][coef.n] = coef.b(t0, p.end);
        if (!ENDS) sC[coef.t][coef.n] = coef.c(t0, p.end);
        __syncthreads();
        if (t0 + kTile < p.end) fetch(t0 + kTile);
        if (!ENDS && saved) store_state(saved + t0 / kTile * a.nb * a.N * a.H, a, p, s);
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            const float2 dd = sd[t][p.lane];
            float Bt[kPer], Ct[kPer], y = 0.0f;
            load4(&sB[t][p.wave * kPer], Bt);
            if (!ENDS) load4(&sC[t][p.wave * kPer], Ct);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                s[i] = __builtin_fmaf(exp2_f(dd.x * A2[i]), s[i], dd.y * Bt[i]);
                if (!ENDS) y = __builtin_fmaf(Ct[i], s[i], y);
            }
            if (ENDS) total += dd.x;
            else sy[p.wave][t][p.lane] = y;
        }
        __syncthreads();
        if (ENDS) continue;
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int t = p.wave + NW * j;
            float y = D * xf[j];
#pragma unroll
            for (int w = 0; w < NW; ++w) y += sy[w][t][p.lane];
            if (zp) y *= silu_f(zf[j]);
            if (p.on && t0 + t < p.r1)
                out[((t0 + t) * a.nb + p.b) * a.H + p.h] = t0 + t < p.end ? from_f32<DT>(y) : 0;
        }
    }
    if (ENDS) {
        store_state(ends + (int64_t)blockIdx.z * a.nb * a.N * a.H, a, p, s);
        if (p.wave == 0 && p.on) dsum[((int64_t)blockIdx.z * a.nb + p.b) * a.H + p.h] = total;
        return;
    }
    if (p.on)
        for (int64_t t = t0 + p.wave; t < p.r1; t += NW) out[(t * a.nb + p.b) * a.H + p.h] = 0;
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
    float *pbc;     // [block of channels][S][B][2][NP]: sums over the block's channels
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
template <int DT, int NW>
__global__ void __launch_bounds__(NW *kWave)
    scan_bwd_ends(ScanIn a, ScanGrad q) {
    constexpr int NP = NW * kPer, JR = kTile / NW;
    __shared__ float2 sd[kTile][kWave];  // d, gy
    __shared__ __align__(16) float sC[kTile][NP];
    const Place p = place(a);
    float A2[kPer], carry[kPer] = {0.0f, 0.0f, 0.0f, 0.0f}, total = 0.0f;
    load_rates(a, p, A2);
    const float bias = a.bias ? a.bias[p.h] : 0.0f;
    const uint16_t *dp = a.dt.p + p.b * a.dt.b + p.h * a.dt.h;
    const uint16_t *zp = a.z.p ? a.z.p + p.b * a.z.b + p.h * a.z.h : nullptr;
    const uint16_t *gp = q.go.p + p.b * q.go.b + p.h * q.go.h;
    CoefTile<DT, NW> coef(a, p);
    uint16_t dr[JR], zr[JR], gr[JR];
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int64_t t = t0 + p.wave + NW * j, r = t < p.end ? t : p.end - 1;
            dr[j] = dp[r * a.dt.s];
            gr[j] = gp[r * q.go.s];
            if (zp) zr[j] = zp[r * a.z.s];
        }
        coef.fetch(a, t0, p.end);
    };
    const int64_t tiles = p.end > p.r0 ? (p.end - p.r0 + kTile - 1) / kTile : 0;
    if (tiles) fetch(p.r0 + (tiles - 1) * kTile);
    for (int64_t k = tiles - 1; k >= 0; --k) {
        const int64_t t0 = p.r0 + k * kTile;
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int t = p.wave + NW * j;
            const bool live = t0 + t < p.end;
            float slope;
            const float d = live ? step_size(a, to_f32<DT>(dr[j]) + bias, slope) : 0.0f;
            float gy = to_f32<DT>(gr[j]);
            if (zp) gy *= silu_f(to_f32<DT>(zr[j]));
            sd[t][p.lane] = make_float2(d, live ? gy : 0.0f);
        }
        sC[coef.t][coef.n] = coef.c(t0, p.end);
        __syncthreads();
        if (k > 0) fetch(t0 - kTile);
#pragma unroll
        for (int t = kTile - 1; t >= 0; --t) {
            const float2 dd = sd[t][p.lane];
            float Ct[kPer];
            load4(&sC[t][p.wave * kPer], Ct);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                carry[i] = __builtin_fmaf(Ct[i], dd.y, carry[i]) * exp2_f(dd.x * A2[i]);
            total += dd.x;
        }
        __syncthreads();
    }
    store_state(q.ends + (int64_t)blockIdx.z * a.nb * a.N * a.H, a, p, carry);
    if (p.wave == 0 && p.on) q.dsum[((int64_t)blockIdx.z * a.nb + p.b) * a.H + p.h] = total;
}

template <int DT, int NW, bool GATE>
__global__ void __launch_bounds__(NW *kWave)
    scan_bwd(ScanIn a, ScanGrad q) {
    constexpr int NP = NW * kPer, JR = kTile / NW;
    __shared__ float2 sd[kTile][kWave];  // d, d x
    __shared__ float sg[kTile][kWave];   // gy
    __shared__ __align__(16) float sB[kTile][NP], sC[kTile][NP];
    __shared__ float su[NW][kTile][kWave], sq[NW][kTile][kWave];  // sums over a wave's states
    __shared__ float sy[GATE ? NW : 1][GATE ? kTile : 1][kWave];
    const Place p = place(a);
    float A2[kPer], carry[kPer];
    double gA[kPer] = {0.0, 0.0, 0.0, 0.0}, gD = 0.0, gbias = 0.0;
    load_rates(a, p, A2);
    load_state(q.gfinal, a, p, carry);
    fold_chunks(q.ends, q.dsum, a, p, a.chunks - 1, -1, a.chunks - 1 - (int)blockIdx.z, A2, carry);
    const float bias = a.bias ? a.bias[p.h] : 0.0f, D = a.D ? a.D[p.h] : 0.0f;
    const uint16_t *xp = a.x.p + p.b * a.x.b + p.h * a.x.h;
    const uint16_t *dp = a.dt.p + p.b * a.dt.b + p.h * a.dt.h;
    const uint16_t *zp = GATE ? a.z.p + p.b * a.z.b + p.h * a.z.h : nullptr;
    const uint16_t *gp = q.go.p + p.b * q.go.b + p.h * q.go.h;
    CoefTile<DT, NW> coef(a, p);
    uint16_t xr[JR], dr[JR], zr[JR], gr[JR];
    float first[kPer];  // the state before the tile
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int64_t t = t0 + p.wave + NW * j, r = t < p.end ? t : p.end - 1;
            xr[j] = xp[r * a.x.s];
            dr[j] = dp[r * a.dt.s];
            gr[j] = gp[r * q.go.s];
            if (GATE) zr[j] = zp[r * a.z.s];
        }
        coef.fetch(a, t0, p.end);
        load_state(q.saved + t0 / kTile * a.nb * a.N * a.H, a, p, first);
    };
    // rows past the length
    const int64_t tiles = p.end > p.r0 ? (p.end - p.r0 + kTile - 1) / kTile : 0;
    const int64_t at = p.b * a.H + p.h, BH = a.nb * a.H;
    if (p.on)
        for (int64_t t = p.r0 + tiles * kTile + p.wave; t < p.r1; t += NW) {
            q.gx[t * BH + at] = 0;
            q.gdt[t * BH + at] = 0;
            if (GATE) q.gz[t * BH + at] = 0;
        }
    if (tiles) fetch(p.r0 + (tiles - 1) * kTile);
    for (int64_t k = tiles - 1; k >= 0; --k) {
        const int64_t t0 = p.r0 + k * kTile;
        float xf[JR], df[JR], slope[JR], gf[JR], zf[JR], gyf[JR];
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int t = p.wave + NW * j;
            const bool live = p.on && t0 + t < p.end;
            const float d = step_size(a, to_f32<DT>(dr[j]) + bias, slope[j]);
            df[j] = live ? d : 0.0f;
            xf[j] = live ? to_f32<DT>(xr[j]) : 0.0f;
            gf[j] = live ? to_f32<DT>(gr[j]) : 0.0f;
            zf[j] = GATE && live ? to_f32<DT>(zr[j]) : 0.0f;
            gyf[j] = GATE ? gf[j] * silu_f(zf[j]) : gf[j];
            sd[t][p.lane] = make_float2(df[j], df[j] * xf[j]);
            sg[t][p.lane] = gyf[j];
        }
        sB[coef.t][coef.n] = coef.b(t0, p.end);
        sC[coef.t][coef.n] = coef.c(t0, p.end);
        float s0[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) s0[i] = first[i];
        __syncthreads();
        if (k > 0) fetch(t0 - kTile);
        // the tile's states and decays again, kept in registers
        float S[kTile][kPer], E[kTile][kPer];
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
            const float2 dd = sd[t][p.lane];
            float Bt[kPer], Ct[kPer], y = 0.0f;
            load4(&sB[t][p.wave * kPer], Bt);
            if (GATE) load4(&sC[t][p.wave * kPer], Ct);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                E[t][i] = exp2_f(dd.x * A2[i]);
                S[t][i] = __builtin_fmaf(E[t][i], t ? S[t - 1][i] : s0[i], dd.y * Bt[i]);
                if (GATE) y = __builtin_fmaf(Ct[i], S[t][i], y);
            }
            if (GATE) sy[p.wave][t][p.lane] = y;
        }
        float tA[kPer] = {0.0f, 0.0f, 0.0f, 0.0f};
        float part[kTile];  // a row's eight sums, each over eight lanes
#pragma unroll
        for (int t = kTile - 1; t >= 0; --t) {
            const float2 dd = sd[t][p.lane];
            const float gy = sg[t][p.lane];
            float Bt[kPer], Ct[kPer], u = 0.0f, w = 0.0f, v[2 * kPer];
            load4(&sB[t][p.wave * kPer], Bt);
            load4(&sC[t][p.wave * kPer], Ct);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float gs = __builtin_fmaf(Ct[i], gy, carry[i]);
                v[i] = gs * dd.y;
                v[kPer + i] = gy * S[t][i];
                u = __builtin_fmaf(gs, Bt[i], u);
                carry[i] = gs * E[t][i];
                const float g = carry[i] * (t ? S[t - 1][i] : s0[i]);
                w = __builtin_fmaf(g, A2[i], w);
                tA[i] = __builtin_fmaf(g, dd.x, tA[i]);
            }
            su[p.wave][t][p.lane] = u;
            sq[p.wave][t][p.lane] = w;
            float r4[4], r2[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) r4[i] = swap_add32(v[2 * i], v[2 * i + 1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) r2[i] = swap_add16(r4[2 * i], r4[2 * i + 1]);
            part[t] = join<kRor8>(r2[0], r2[1], p.lane & 8);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) gA[i] += (double)tA[i];
        // 16 rows of 8 sums over 8 lanes: two values a lane. Value v of row t ends in lane bits
        // 5, 4, 3 = v's bits 0, 1, 2 and lane bits 2, 1, 0 = t's bits 0, 1, 2; t's bit 3 is `half`.
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[i] = join<kHalfMirror>(part[half * 8 + 2 * i], part[half * 8 + 2 * i + 1], p.lane & 4);
            const float m0 = join<kXor2>(r[0], r[1], p.lane & 2), m1 = join<kXor2>(r[2], r[3], p.lane & 2);
            const float m = join<kXor1>(m0, m1, p.lane & 1);
            const int l = p.lane;
            const int t = half * 8 + ((l >> 2) & 1) + (l & 2) + (l & 1) * 4;
            const int n = (l >> 5) + ((l >> 4) & 1) * 2, which = (l >> 3) & 1;
            if (t0 + t < p.end)
                q.pbc[((((int64_t)blockIdx.x * a.S + t0 + t) * a.nb + p.b) * 2 + which) * NP +
                      p.wave * kPer + n] = m;
        }
        __syncthreads();
        float tD = 0.0f, tb = 0.0f;
#pragma unroll
        for (int j = 0; j < JR; ++j) {
            const int t = p.wave + NW * j;
            float u = 0.0f, w = 0.0f, y = D * xf[j];
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                u += su[i][t][p.lane];
                w += sq[i][t][p.lane];
                if (GATE) y += sy[i][t][p.lane];
            }
            const float gd = __builtin_fmaf(w, kLn2, u * xf[j]) * slope[j];
            const bool live = p.on && t0 + t < p.end;
            tD = __builtin_fmaf(gyf[j], xf[j], tD);
            tb += live ? gd : 0.0f;
            if (p.on && t0 + t < p.r1) {
                const int64_t o = (t0 + t) * BH + at;
                q.gx[o] = live ? from_f32<DT>(__builtin_fmaf(u, df[j], D * gyf[j])) : 0;
                q.gdt[o] = live ? from_f32<DT>(gd) : 0;
                if (GATE) q.gz[o] = live ? from_f32<DT>(gf[j] * y * silu_slope_f(zf[j])) : 0;
            }
        }
        gD += (double)tD;
        gbias += (double)tb;
    }
    if (blockIdx.z == 0 && q.gstate) store_state(q.gstate, a, p, carry);
    double *pa = q.pa + ((int64_t)blockIdx.z * a.nb + p.b) * (a.N + 2) * a.H + p.h;
    __syncthreads();
    double *sums = (double *)&su[0][0][0];  // [NW][2][64] doubles: 1 KiB a wave, of its 4 KiB
    sums[(p.wave * 2 + 0) * kWave + p.lane] = gD;
    sums[(p.wave * 2 + 1) * kWave + p.lane] = gbias;
    __syncthreads();
    if (!p.on) return;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = p.wave * kPer + i;
        if (n < a.N) pa[(int64_t)n * a.H] = gA[i];
    }
    if (p.wave == 0) {
        double d = 0.0, b = 0.0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            d += sums[(w * 2 + 0) * kWave + p.lane];
            b += sums[(w * 2 + 1) * kWave + p.lane];
        }
        pa[(int64_t)a.N * a.H] = d;
        pa[(int64_t)(a.N + 1) * a.H] = b;
    }
}

// gB and gC: the sums of each group's blocks, in their order; a thread for each (row, batch, group,
// which, n), n fastest.
template <int DT>
__global__ void __launch_bounds__(256)
    scan_sum_bc(const float *__restrict__ pbc, const int64_t *__restrict__ lengths, int64_t S,
                int64_t nb, int N, int NP, int G, int per_group, uint16_t *__restrict__ gB,
                uint16_t *__restrict__ gC) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t rows = S * nb;
    const int n = (int)(id % NP), which = (int)(id / NP % 2);
    const int64_t rg = id / (2 * NP);  // group slowest, so that neighbours read one block's sums
    const int64_t row = rg % rows, g = rg / rows;
    if (g >= G || n >= N) return;
    const int64_t t = row / nb, b = row - t * nb;
    float s = 0.0f;
    if (!lengths || t < lengths[b]) {
        const float *p = pbc + ((g * per_group * rows + row) * 2 + which) * NP + n;
#pragma unroll 8
        for (int i = 0; i < per_group; ++i) s += p[(int64_t)i * rows * 2 * NP];
    }
    (which ? gC : gB)[(row * G + g) * N + n] = from_f32<DT>(s);
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
// Single token: a lane has a channel of one batch and all its states; the state is read and
// written once, a wave's 64 channels at a time.
// ---------------------------------------------------------------------------------------------
template <int DT, int NMAX>
__global__ void __launch_bounds__(kWave)
    scan_one(ScanIn a, float *__restrict__ state, uint16_t *__restrict__ out) {
    const int64_t h = (int64_t)blockIdx.x * kWave + threadIdx.x, b = blockIdx.y;
    if (h >= a.H) return;
    float s[NMAX], r[NMAX];
    float *sp = state + b * a.N * a.H + h;
#pragma unroll
    for (int n = 0; n < NMAX; ++n) {
        s[n] = n < a.N ? sp[(int64_t)n * a.H] : 0.0f;
        r[n] = n < a.N ? a.A[(int64_t)n * a.H + h] : 0.0f;
    }
    const int64_t g = h / a.K;
    const uint16_t *bp = a.B.p + b * a.B.b + g * a.B.g, *cp = a.C.p + b * a.C.b + g * a.C.g;
    const float x = to_f32<DT>(a.x.p[b * a.x.b + h * a.x.h]);
    float slope;
    const float d = step_size(
        a, to_f32<DT>(a.dt.p[b * a.dt.b + h * a.dt.h]) + (a.bias ? a.bias[h] : 0.0f), slope);
    float y = a.D ? a.D[h] * x : 0.0f;
    const float dx = d * x, d2 = d * kLog2e;
#pragma unroll
    for (int n = 0; n < NMAX; ++n) {
        if (n >= a.N) break;
        s[n] = __builtin_fmaf(exp2_f(d2 * r[n]), s[n], dx * to_f32<DT>(bp[n * a.B.n]));
        y = __builtin_fmaf(to_f32<DT>(cp[n * a.C.n]), s[n], y);
        sp[(int64_t)n * a.H] = s[n];
    }
    if (a.z.p) y *= silu_f(to_f32<DT>(a.z.p[b * a.z.b + h * a.z.h]));
    out[b * a.H + h] = from_f32<DT>(y);
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------
int check_scan(const mccb_scan_t *a, bool token) {
    if (!a) return MCCB_ERR_PARAM_NULLPTR;
    if (a->dtype != MCCB_BF16 && a->dtype != MCCB_FP16) return MCCB_ERR_PARAM_INVALID;
    if (a->B < 1 || a->B > kMaxBatch || a->S < 0 || a->S >= kMaxRows || a->H < 1 ||
        a->H > kMaxWidth || a->N < 1 || a->N > 32 || a->G < 1 || a->H % a->G ||
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
    p.waves = a->N <= 4 ? 1 : a->N <= 8 ? 2 : a->N <= 16 ? 4 : 8;
    const int64_t K = a->H / a->G;
    p.per_group = (K + kWave - 1) / kWave;
    p.blocks = p.per_group * a->G;
    // Chunks cost a second pass over the recurrence, so they pay only where they multiply the waves
    // well beyond that: at most half the card's SIMDs busy without them. Then as many as give two
    // waves a SIMD, no shorter than four tiles.
    const int64_t waves = p.blocks * a->B * p.waves, tiles = (a->S + kTile - 1) / kTile;
    int64_t chunks = 1;
    if (waves <= 512) {
        chunks = 2048 / waves;
        if (chunks > tiles / 4) chunks = tiles / 4;
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

// Workspace for handing states between chunks.
uint64_t chunk_bytes(const mccb_scan_t *a, const ScanPlan &p) {
    if (p.chunks == 1) return 0;
    return (uint64_t)p.chunks * align16(state_bytes(a) + (uint64_t)(a->B * a->H) * 4);
}

uint64_t pbc_bytes(const mccb_scan_t *a, const ScanPlan &p) {
    return (uint64_t)p.blocks * (uint64_t)a->S * (uint64_t)a->B * (2 * p.waves * kPer) * 4;
}
uint64_t pa_bytes(const mccb_scan_t *a, const ScanPlan &p) {
    return (uint64_t)p.chunks * (uint64_t)a->B * (uint64_t)((a->N + 2) * a->H) * 8;
}

template <typename F>
int by_waves(int waves, F f) {
    switch (waves) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 8>{});
    }
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
            constexpr int DT = decltype(dt)::value, NW = decltype(nw)::value;
            if (p.chunks > 1) {
                hipLaunchKernelGGL((scan_fwd<DT, NW, true>), first, dim3(NW * kWave), 0, st, da,
                                   (uint16_t *)nullptr, (float *)nullptr, (float *)nullptr, ends,
                                   dsum);
                const int r = launched();
                if (r != MCCB_OK) return r;
            }
            hipLaunchKernelGGL((scan_fwd<DT, NW, false>), grid, dim3(NW * kWave), 0, st, da,
                               (uint16_t *)out, final_state, (float *)saved, ends, dsum);
            return launched();
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
    at += align16(pbc_bytes(a, p));
    q.ends = p.chunks > 1 ? (float *)at : nullptr;
    q.dsum = p.chunks > 1 ? q.ends + (uint64_t)p.chunks * (uint64_t)(a->B * a->N * a->H) : nullptr;
    const dim3 grid((unsigned)p.blocks, (unsigned)a->B, (unsigned)p.chunks);
    const hipStream_t st = (hipStream_t)stream;
    rc = by_dtype(a->dtype, [&](auto dt) {
        return by_waves(p.waves, [&](auto nw) {
            constexpr int DT = decltype(dt)::value, NW = decltype(nw)::value;
            const dim3 block(NW * kWave);
            if (p.chunks > 1) {
                hipLaunchKernelGGL((scan_bwd_ends<DT, NW>), grid, block, 0, st, da, q);
                const int e = launched();
                if (e != MCCB_OK) return e;
            }
            if (a->z)
                hipLaunchKernelGGL((scan_bwd<DT, NW, true>), grid, block, 0, st, da, q);
            else
                hipLaunchKernelGGL((scan_bwd<DT, NW, false>), grid, block, 0, st, da, q);
            int e = launched();
            if (e != MCCB_OK || a->S == 0) return e;
            const int64_t ids = a->S * a->B * a->G * 2 * NW * kPer;
            hipLaunchKernelGGL((scan_sum_bc<DT>), dim3((unsigned)((ids + 255) / 256)), dim3(256), 0,
                               st, q.pbc, a->lengths, a->S, a->B, (int)a->N, NW * kPer, (int)a->G,
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
        if (a->N <= 8)
            hipLaunchKernelGGL((scan_one<DT, 8>), grid, dim3(kWave), 0, st, da, state, (uint16_t *)out);
        else if (a->N <= 16)
            hipLaunchKernelGGL((scan_one<DT, 16>), grid, dim3(kWave), 0, st, da, state, (uint16_t *)out);
        else
            hipLaunchKernelGGL((scan_one<DT, 32>), grid, dim3(kWave), 0, st, da, state, (uint16_t *)out);
        return launched();
    });
}

}  // extern "C"
