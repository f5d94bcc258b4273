// ssm_conv.hip -- causal depthwise convolution with bias, activation and carried rows, for MI355X
// (gfx950): forward, backward and the single-token step (mccb_ssm.h).
//
//   pre[t] = bias + sum_k w[k] x[t-W+1+k],  y[t] = act(pre[t])            (per batch and channel)
//   g[t]   = gy[t] act'(pre[t]),            gx[t] = sum_k g[t+k] w[W-1-k]
//   gw[k]  = sum_t g[t] x[t-W+1+k],         gbias = sum_t g[t]
//
// Rows x[-W+1..-1] come from the carried state. All three kernels are bound by HBM: a row element
// is read once and written once (backward: two read, one written) for about 20 lane operations.
// S=4096 B=4 H=4096 bf16, W=4 with silu: forward 53 us (5.0 TB/s), backward 101 us (4.0 TB/s) and 5 for
// the partial sums of gw and gbias; a large copy reaches 4.8 TB/s. The single token (B=8 H=5120) is 3 us,
// a launch's own time.
// A lane owns V adjacent channels of one batch and walks down a strip of rows, with the last W-1
// rows in registers; the next rows' loads are in flight while it computes. Channels have no
// alignment to keep (loads of 16-bit vectors may start at any element), and where V does not
// divide H the last lane takes the last V channels, computing the ones it shares with its
// neighbour a second time to the same values.
#include "ssm_common.h"

#include <type_traits>

using namespace ssm;

namespace {

constexpr int kThreads = 256;
constexpr int kFwdVec = 8, kBwdVec = 4;
constexpr int kFwdBatch = 4, kBwdBatch = 4;  // rows whose loads are issued together

struct Rows {  // a strided [S,B,H] input
    const uint16_t *p;
    int64_t s, b, h;
};

template <int DT, int V>
__device__ static inline void widen(const typename HVec<V>::t q, float (&f)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = to_f32<DT>(q[v]);
}

template <int DT, int V>
__device__ static inline typename HVec<V>::t narrow(const float (&f)[V]) {
    typename HVec<V>::t q;
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = from_f32<DT>(f[v]);
    return q;
}

template <int V>
__device__ static inline typename HVec<V>::t load(const uint16_t *p) {
    return *(const typename HVec<V>::t *)p;
}
template <int V>
__device__ static inline void store(uint16_t *p, const typename HVec<V>::t q) {
    *(typename HVec<V>::t *)p = q;
}

// Lane id's batch and first channel; false past the last lane.
template <int V>
__device__ static inline bool lane_place(uint32_t id, int64_t B, int64_t H, uint32_t per_batch,
                                         int64_t &b, int64_t &h) {
    const uint32_t j = id / per_batch;
    b = h = 0;
    if (j >= B) return false;
    const int64_t first = (int64_t)(id - j * per_batch) * V;
    b = j;
    h = first < H - V ? first : H - V;
    return true;
}

__device__ static inline int64_t clamp_len(const int64_t *lengths, int64_t b, int64_t S) {
    if (!lengths) return S;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n > S ? S : n;
}

// Row r of x, or of the carried state where r < 0, as fp32.
template <int DT, int W, int V>
__device__ static inline void row_before(const Rows &x, const uint16_t *state, int64_t r, int64_t B,
                                         int64_t H, int64_t b, int64_t h, float (&f)[V]) {
    if (r >= 0) {
        widen<DT, V>(load<V>(x.p + r * x.s + b * x.b + h * x.h), f);
    } else if (state) {
        widen<DT, V>(load<V>(state + ((r + W - 1) * B + b) * H + h), f);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.0f;
    }
}

template <int DT, int W, bool SILU, int V>
__global__ void __launch_bounds__(kThreads)
    conv_act_fwd(Rows x, const uint16_t *__restrict__ weight, const uint16_t *__restrict__ bias,
                 const int64_t *__restrict__ lengths, const uint16_t *__restrict__ state,
                 uint16_t *__restrict__ y, uint16_t *__restrict__ final_state, int64_t S, int64_t B,
                 int64_t H, uint32_t per_batch, int rows) {
    typedef typename HVec<V>::t vec;
    int64_t b, h;
    if (!lane_place<V>(blockIdx.x * (uint32_t)kThreads + threadIdx.x, B, H, per_batch, b, h)) return;
    const int64_t len = clamp_len(lengths, b, S);
    const int64_t t0 = (int64_t)blockIdx.y * rows, t1 = t0 + rows < S ? t0 + rows : S;
    if (W > 1 && blockIdx.y == 0 && final_state) {
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
            float f[V];
            row_before<DT, W, V>(x, state, len - (W - 1) + r, B, H, b, h, f);
            store<V>(final_state + (r * B + b) * H + h, narrow<DT, V>(f));
        }
    }
    const int64_t BH = B * H;
    uint16_t *yp = y + t0 * BH + b * H + h;
    int64_t i = t0;
    const int64_t end = len < t1 ? len : t1;
    if (i < end) {
        float w[W][V], bv[V], win[W][V];
#pragma unroll
        for (int k = 0; k < W; ++k) widen<DT, V>(load<V>(weight + k * H + h), w[k]);
#pragma unroll
        for (int v = 0; v < V; ++v) bv[v] = 0.0f;
        if (bias) widen<DT, V>(load<V>(bias + h), bv);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            row_before<DT, W, V>(x, state, t0 - (W - 1) + k, B, H, b, h, win[k]);
        const uint16_t *xp = x.p + b * x.b + h * x.h;
        auto row = [&](const vec q) {
            widen<DT, V>(q, win[W - 1]);
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = bv[v];
#pragma unroll
                for (int k = 0; k < W; ++k) o[v] = __builtin_fmaf(w[k][v], win[k][v], o[v]);
                if (SILU) o[v] = silu_f(o[v]);
            }
            store<V>(yp, narrow<DT, V>(o));
            yp += BH;
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v];
        };
        vec next[kFwdBatch];
        // loads past the strip's end stay on its last row and are not used
        auto fetch = [&](int64_t from) {
#pragma unroll
            for (int r = 0; r < kFwdBatch; ++r) {
                const int64_t t = from + r < end ? from + r : end - 1;
                next[r] = load<V>(xp + t * x.s);
            }
        };
        fetch(i);
        while (i + kFwdBatch <= end) {
            vec cur[kFwdBatch];
#pragma unroll
            for (int r = 0; r < kFwdBatch; ++r) cur[r] = next[r];
            fetch(i + kFwdBatch);
#pragma unroll
            for (int r = 0; r < kFwdBatch; ++r) row(cur[r]);
            i += kFwdBatch;
        }
#pragma unroll
        for (int r = 0; r < kFwdBatch - 1; ++r)
            if (i < end) {
                row(next[r]);
                ++i;
            }
    }
    vec zero;
#pragma unroll
    for (int v = 0; v < V; ++v) zero[v] = 0;
    for (; i < t1; ++i, yp += BH) store<V>(yp, zero);
}

// Backward. A strip's lane walks its rows and the W-1 after it: g of row i completes gx of row
// i-W+1. Its own rows add to the weight's and bias's sums, in fp32 over the strip's rows (64 at most, up
// to S of 4 million). A block has 64 lanes' columns and four consecutive strips, a wave each, whose sums
// it adds in fp32 and writes to the workspace as [block of strips][b][W+1][H]; the second kernel adds
// them over blocks and batches in fp64, in a fixed order. (With a wave for every strip's sums they were a fifth of the traffic.)
template <int DT, int W, bool SILU, int V>
__global__ void __launch_bounds__(kThreads)
    conv_act_bwd(Rows x, Rows gy, const uint16_t *__restrict__ weight,
                 const uint16_t *__restrict__ bias, const int64_t *__restrict__ lengths,
                 const uint16_t *__restrict__ state, const uint16_t *__restrict__ gfinal,
                 uint16_t *__restrict__ gx, uint16_t *__restrict__ gstate,
                 float *__restrict__ partial, int64_t S, int64_t B, int64_t H, uint32_t per_batch,
                 int rows) {
    typedef typename HVec<V>::t vec;
    constexpr int kWaves = kThreads / kWave;
    __shared__ float part[kWaves][(W + 1) * V][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    int64_t b, h;
    const uint32_t column = blockIdx.z * gridDim.x + blockIdx.x;  // of 64 lanes
    const bool on = lane_place<V>(column * (uint32_t)kWave + lane, B, H, per_batch, b, h);
    const int64_t strip = (int64_t)blockIdx.y * kWaves + wave;
    const int64_t t0 = strip * rows, t1 = t0 + rows < S ? t0 + rows : S;
    const int64_t BH = B * H, at = b * H + h;
    float gw[W][V], gb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        gb[v] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) gw[k][v] = 0.0f;
    }
    // strip 0 is walked without rows too: it has the carried rows' gradient
    if (on && (t0 < S || strip == 0)) {
        const int64_t len = clamp_len(lengths, b, S);
        float w[W][V], bv[V], win[W][V], g[W][V];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            widen<DT, V>(load<V>(weight + k * H + h), w[k]);
#pragma unroll
            for (int v = 0; v < V; ++v) g[k][v] = 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) bv[v] = 0.0f;
        if (bias) widen<DT, V>(load<V>(bias + h), bv);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            // rows past the length are in no live row's window, and may hold anything
            if (t0 - (W - 1) + k < len) {
                row_before<DT, W, V>(x, state, t0 - (W - 1) + k, B, H, b, h, win[k]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = 0.0f;
            }
        }
        const uint16_t *xp = x.p + b * x.b + h * x.h, *gp = gy.p + b * gy.b + h * gy.h;

        // gx of row t = i-W+1 from g of rows t..i (g[0] the oldest). Unless `all` of them are rows from 0
        // to the length, the sum leaves the others out: a zero times an infinite weight is not zero.
        auto gradient = [&](int64_t t, auto all, float (&o)[V]) {
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k)
                if (decltype(all)::value || (t + k >= 0 && t + k < len))
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        o[v] = __builtin_fmaf(g[k][v], w[W - 1 - k][v], o[v]);
            // the last W-1 rows before the length are the final state
            if (W > 1 && gfinal && t < len && t >= len - (W - 1)) {
                float f[V];
                widen<DT, V>(load<V>(gfinal + (t - len + (W - 1)) * BH + at), f);
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] += f[v];
            }
        };
        auto emit = [&](int64_t i, auto all) {
            const int64_t t = i - (W - 1);
            float o[V];
            if (t >= t0) {
                gradient(t, all, o);
                store<V>(gx + t * BH + at, narrow<DT, V>(o));
            } else if (W > 1 && t < 0 && gstate) {
                gradient(t, std::false_type{}, o);
                store<V>(gstate + (t + W - 1) * BH + at, narrow<DT, V>(o));
            }
        };
        auto shift = [&]() {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    win[k][v] = win[k + 1][v];
                    g[k][v] = g[k + 1][v];
                }
        };
        auto row = [&](const vec qx, const vec qg, bool mine) {
            widen<DT, V>(qx, win[W - 1]);
            widen<DT, V>(qg, g[W - 1]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (SILU) {
                    float pre = bv[v];
#pragma unroll
                    for (int k = 0; k < W; ++k) pre = __builtin_fmaf(w[k][v], win[k][v], pre);
                    g[W - 1][v] *= silu_slope_f(pre);
                }
                if (mine) {
                    gb[v] += g[W - 1][v];
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        gw[k][v] = __builtin_fmaf(g[W - 1][v], win[k][v], gw[k][v]);
                }
            }
        };
        int64_t i = t0;
        const int64_t end = len < t1 ? len : t1;
        vec nx[kBwdBatch], ng[kBwdBatch];
        if (i < end) {
            auto fetch = [&](int64_t from) {
#pragma unroll
                for (int r = 0; r < kBwdBatch; ++r) {
                    const int64_t t = from + r < end ? from + r : end - 1;
                    nx[r] = load<V>(xp + t * x.s);
                    ng[r] = load<V>(gp + t * gy.s);
                }
            };
            fetch(i);
            while (i + kBwdBatch <= end) {
                vec cx[kBwdBatch], cg[kBwdBatch];
#pragma unroll
                for (int r = 0; r < kBwdBatch; ++r) cx[r] = nx[r], cg[r] = ng[r];
                fetch(i + kBwdBatch);
#pragma unroll
                for (int r = 0; r < kBwdBatch; ++r) {
                    row(cx[r], cg[r], true);
                    emit(i + r, std::true_type{});
                    shift();
                }
                i += kBwdBatch;
            }
#pragma unroll
            for (int r = 0; r < kBwdBatch - 1; ++r)
                if (i < end) {
                    row(nx[r], ng[r], true);
                    emit(i, std::true_type{});
                    shift();
                    ++i;
                }
        }
        // rows after the strip that are still live, then rows past the length
        for (; i < t1 + (W - 1); ++i) {
            if (i >= t1 && i < len) {
                row(load<V>(xp + i * x.s), load<V>(gp + i * gy.s), false);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) g[W - 1][v] = win[W - 1][v] = 0.0f;
            }
            emit(i, std::false_type{});
            shift();
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) part[wave][k * V + v][lane] = gw[k][v];
        part[wave][W * V + v][lane] = gb[v];
    }
    __syncthreads();
    if (!on) return;
    float *pp = partial + ((int64_t)blockIdx.y * B + b) * (W + 1) * H + h;
#pragma unroll
    for (int i = wave; i < (W + 1) * V; i += kWaves) {
        float f = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) f += part[q][i][lane];
        pp[i / V * H + i % V] = f;
    }
}

// partial [P][W+1][H] summed over P: 64 columns of [W+1][H] a block, its four waves taking every
// fourth entry.
template <int DT>
__global__ void __launch_bounds__(kThreads)
    conv_act_sum(const float *__restrict__ partial, int64_t P, int64_t n_weight, int64_t n_all,
                 uint16_t *__restrict__ gw, uint16_t *__restrict__ gb) {
    __shared__ double part[kThreads / kWave][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWave + lane;
    double s = 0.0;
    if (c < n_all) {
#pragma unroll 8
        for (int64_t p = wave; p < P; p += kThreads / kWave) s += (double)partial[p * n_all + c];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < n_all) {
        const float f = (float)((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]));
        if (c < n_weight)
            gw[c] = from_f32<DT>(f);
        else if (gb)
            gb[c - n_weight] = from_f32<DT>(f);
    }
}

// One token: the W-1 carried rows and x give y; the rows move up by one.
template <int DT, int W, bool SILU, int V>
__global__ void __launch_bounds__(kThreads)
    conv_act_one(Rows x, const uint16_t *__restrict__ weight, const uint16_t *__restrict__ bias,
                 uint16_t *__restrict__ state, uint16_t *__restrict__ y, int64_t B, int64_t H,
                 uint32_t per_batch) {
    typedef typename HVec<V>::t vec;
    const uint32_t id = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
    const uint32_t j = id / per_batch;
    // the state is read and written here, so no two lanes may share channels: the last lane of a
    // batch takes its channels one by one where V does not divide H
    const int64_t b = j, h0 = (int64_t)(id - j * per_batch) * V;
    if (b >= B) return;
    auto channels = [&](auto width, int64_t h) {
        constexpr int N = decltype(width)::value;
        typedef typename HVec<N>::t nvec;
        nvec q[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) q[k] = load<N>(state + (k * B + b) * H + h);
        q[W - 1] = load<N>(x.p + b * x.b + h * x.h);
        float o[N], w[N], f[N];
#pragma unroll
        for (int v = 0; v < N; ++v) o[v] = 0.0f;
        if (bias) widen<DT, N>(load<N>(bias + h), o);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            widen<DT, N>(load<N>(weight + k * H + h), w);
            widen<DT, N>(q[k], f);
#pragma unroll
            for (int v = 0; v < N; ++v) o[v] = __builtin_fmaf(w[v], f[v], o[v]);
        }
#pragma unroll
        for (int v = 0; v < N; ++v)
            if (SILU) o[v] = silu_f(o[v]);
        store<N>(y + b * H + h, narrow<DT, N>(o));
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store<N>(state + (k * B + b) * H + h, q[k + 1]);
    };
    if (h0 + V <= H) {
        channels(std::integral_constant<int, V>{}, h0);
    } else {
        for (int64_t h = h0; h < H; ++h) channels(std::integral_constant<int, 1>{}, h);
    }
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------
struct Strips {
    int64_t rows, n;
};

// Rows of a strip: whole batches of loads, as long as leaves 8192 waves (8 a SIMD), within [lo, hi]: a
// strip reads W-1 rows of its neighbours again (forward, S=8192 B=1 H=1024: 9.4 us with at least 8
// rows, 11.4 with 4, 10.0 with 12).
Strips strips(int64_t S, int64_t lanes, int64_t lo, int64_t hi) {
    const int64_t across = (lanes + kWave - 1) / kWave;
    int64_t rows = S * across / 8192 / 4 * 4;
    rows = rows < lo ? lo : rows > hi ? hi : rows;
    while ((S + rows - 1) / rows > 65535) rows *= 2;
    return {rows, (S + rows - 1) / rows};
}

int64_t lanes_of(int64_t H, int V) { return (H + V - 1) / V; }

bool vector_ok(int64_t H, int64_t hs, int V) { return H >= V && hs == 1; }

int check_conv(const mccb_conv_t *a, bool token) {
    if (!a) return MCCB_ERR_PARAM_NULLPTR;
    if (a->dtype != MCCB_BF16 && a->dtype != MCCB_FP16) return MCCB_ERR_PARAM_INVALID;
    if (a->activation != MCCB_ACT_NONE && a->activation != MCCB_ACT_SILU)
        return MCCB_ERR_PARAM_INVALID;
    if (a->B < 1 || a->B > kMaxBatch || a->S < 0 || a->S >= kMaxRows || a->H < 1 ||
        a->H > kMaxWidth || a->W < 1 || a->W > 4 || a->B * a->H >= kMaxRows || (token && a->S != 1))
        return MCCB_ERR_SHAPE;
    return MCCB_OK;
}

// The inputs' extents, and their pointers where they hold elements.
int check_conv_inputs(const mccb_conv_t *a, Span *in, int *n) {
    if (!a->weight || (!a->x && a->S > 0)) return MCCB_ERR_PARAM_NULLPTR;
    const int64_t size[3] = {a->S, a->B, a->H};
    uint64_t bytes;
    if (!extent(3, size, a->x_stride, 2, &bytes)) return MCCB_ERR_PARAM_INVALID;
    if (misaligned(a->x, 2) || misaligned(a->weight, 2) || misaligned(a->bias, 2) ||
        misaligned(a->state, 2) || misaligned(a->lengths, 8))
        return MCCB_ERR_PARAM_INVALID;
    in[0] = {a->x, bytes};
    in[1] = {a->weight, (uint64_t)(a->W * a->H) * 2};
    in[2] = {a->bias, (uint64_t)a->H * 2};
    in[3] = {a->lengths, (uint64_t)a->B * 8};
    in[4] = {a->state, (uint64_t)((a->W - 1) * a->B * a->H) * 2};
    *n = 5;
    return MCCB_OK;
}

Rows rows_of(const void *p, const int64_t *st) { return {(const uint16_t *)p, st[0], st[1], st[2]}; }

// Of the backward, n counts blocks of four strips.
Strips bwd_strips(const mccb_conv_t *a) {
    Strips s = strips(a->S > 0 ? a->S : 1, a->B * lanes_of(a->H, kBwdVec), 8, 64);
    s.n = (s.n + kThreads / kWave - 1) / (kThreads / kWave);
    return s;
}

template <typename F>
int by_window(int64_t W, F f) {
    switch (W) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        default: return f(std::integral_constant<int, 4>{});
    }
}

// f(dtype, window, whether silu) with compile-time values
template <typename F>
int by_form(const mccb_conv_t *a, F f) {
    return by_window(a->W, [&](auto w) {
        auto act = [&](auto dt) {
            return a->activation == MCCB_ACT_SILU ? f(dt, w, std::true_type{})
                                                  : f(dt, w, std::false_type{});
        };
        return a->dtype == MCCB_BF16 ? act(std::integral_constant<int, MCCB_BF16>{})
                                     : act(std::integral_constant<int, MCCB_FP16>{});
    });
}

template <int V>
int launch_fwd(const mccb_conv_t *a, void *y, void *final_state, hipStream_t st) {
    const int64_t per = lanes_of(a->H, V), lanes = a->B * per;
    const Strips s = strips(a->S > 0 ? a->S : 1, lanes, 8, 16);
    const dim3 grid((unsigned)((lanes + kThreads - 1) / kThreads), (unsigned)s.n);
    return by_form(a, [&](auto dt, auto w, auto silu) {
        hipLaunchKernelGGL((conv_act_fwd<decltype(dt)::value, decltype(w)::value,
                                         decltype(silu)::value, V>),
                           grid, dim3(kThreads), 0, st, rows_of(a->x, a->x_stride),
                           (const uint16_t *)a->weight, (const uint16_t *)a->bias, a->lengths,
                           (const uint16_t *)a->state, (uint16_t *)y, (uint16_t *)final_state, a->S,
                           a->B, a->H, (uint32_t)per, (int)s.rows);
        return launched();
    });
}

template <int V>
int launch_bwd(const mccb_conv_t *a, const void *gy, const int64_t *gs, const void *gfinal, void *gx,
               void *gstate, float *partial, const Strips &s, hipStream_t st) {
    const int64_t per = lanes_of(a->H, V), lanes = a->B * per;
    // a grid has less than 2^32 threads along an axis; the rest goes along z
    const int64_t columns = (lanes + kWave - 1) / kWave, most = (int64_t)1 << 23;
    const int64_t deep = (columns + most - 1) / most, across = (columns + deep - 1) / deep;
    const dim3 grid((unsigned)across, (unsigned)s.n, (unsigned)deep);
    return by_form(a, [&](auto dt, auto w, auto silu) {
        hipLaunchKernelGGL((conv_act_bwd<decltype(dt)::value, decltype(w)::value,
                                         decltype(silu)::value, V>),
                           grid, dim3(kThreads), 0, st, rows_of(a->x, a->x_stride), rows_of(gy, gs),
                           (const uint16_t *)a->weight, (const uint16_t *)a->bias, a->lengths,
                           (const uint16_t *)a->state, (const uint16_t *)gfinal, (uint16_t *)gx,
                           (uint16_t *)gstate, partial, a->S, a->B, a->H, (uint32_t)per,
                           (int)s.rows);
        return launched();
    });
}

template <int V>
int launch_one(const mccb_conv_t *a, void *state, void *y, hipStream_t st) {
    const int64_t per = lanes_of(a->H, V), lanes = a->B * per;
    const dim3 grid((unsigned)((lanes + kThreads - 1) / kThreads));
    return by_form(a, [&](auto dt, auto w, auto silu) {
        hipLaunchKernelGGL((conv_act_one<decltype(dt)::value, decltype(w)::value,
                                         decltype(silu)::value, V>),
                           grid, dim3(kThreads), 0, st, rows_of(a->x, a->x_stride),
                           (const uint16_t *)a->weight, (const uint16_t *)a->bias,
                           (uint16_t *)state, (uint16_t *)y, a->B, a->H, (uint32_t)per);
        return launched();
    });
}

}  // namespace

extern "C" {

int mccb_conv_act_forward(const mccb_conv_t *a, void *y, void *final_state, void *stream) {
    int rc = check_conv(a, false);
    if (rc != MCCB_OK) return rc;
    if (!y && a->S > 0) return MCCB_ERR_PARAM_NULLPTR;
    Span in[5];
    int n;
    rc = check_conv_inputs(a, in, &n);
    if (rc != MCCB_OK) return rc;
    const Span out[2] = {{y, (uint64_t)a->S * (uint64_t)(a->B * a->H) * 2},
                         {final_state, (uint64_t)((a->W - 1) * a->B * a->H) * 2}};
    if (misaligned(y, 2) || misaligned(final_state, 2) || outputs_clash(in, n, out, 2))
        return MCCB_ERR_PARAM_INVALID;
    if (a->S == 0 && (!final_state || a->W == 1)) return MCCB_OK;
    return vector_ok(a->H, a->x_stride[2], kFwdVec)
               ? launch_fwd<kFwdVec>(a, y, final_state, (hipStream_t)stream)
               : launch_fwd<1>(a, y, final_state, (hipStream_t)stream);
}

int mccb_conv_act_backward_get_workspace_size(const mccb_conv_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_conv(a, false);
    if (rc != MCCB_OK) return rc;
    *size = (uint64_t)bwd_strips(a).n * (uint64_t)(a->B * (a->W + 1) * a->H) * sizeof(float);
    return MCCB_OK;
}

int mccb_conv_act_backward(const mccb_conv_t *a, const void *gy, const int64_t *gy_stride,
                           const void *gfinal, void *gx, void *gw, void *gb, void *gstate,
                           void *ws, uint64_t ws_size, void *stream) {
    int rc = check_conv(a, false);
    if (rc != MCCB_OK) return rc;
    if (!gy_stride || !gw || ((!gy || !gx) && a->S > 0)) return MCCB_ERR_PARAM_NULLPTR;
    Span in[8];
    int n;
    rc = check_conv_inputs(a, in, &n);
    if (rc != MCCB_OK) return rc;
    const int64_t size[3] = {a->S, a->B, a->H};
    uint64_t gy_bytes, need = 0;
    if (!extent(3, size, gy_stride, 2, &gy_bytes)) return MCCB_ERR_PARAM_INVALID;
    mccb_conv_act_backward_get_workspace_size(a, &need);
    rc = check_workspace(ws, ws_size, need);
    if (rc != MCCB_OK) return rc;
    const uint64_t n_state = (uint64_t)((a->W - 1) * a->B * a->H) * 2;
    in[n++] = {gy, gy_bytes};
    in[n++] = {gfinal, n_state};
    const Span out[5] = {{gx, (uint64_t)a->S * (uint64_t)(a->B * a->H) * 2},
                         {gw, (uint64_t)(a->W * a->H) * 2},
                         {gb, (uint64_t)a->H * 2},
                         {gstate, n_state},
                         {ws, need}};
    if (misaligned(gy, 2) || misaligned(gfinal, 2) || misaligned(gx, 2) || misaligned(gw, 2) ||
        misaligned(gb, 2) || misaligned(gstate, 2) || outputs_clash(in, n, out, 5))
        return MCCB_ERR_PARAM_INVALID;
    const hipStream_t st = (hipStream_t)stream;
    const Strips s = bwd_strips(a);
    float *partial = (float *)ws;
    const bool vec = vector_ok(a->H, a->x_stride[2], kBwdVec) && gy_stride[2] == 1;
    rc = vec ? launch_bwd<kBwdVec>(a, gy, gy_stride, gfinal, gx, gstate, partial, s, st)
             : launch_bwd<1>(a, gy, gy_stride, gfinal, gx, gstate, partial, s, st);
    if (rc != MCCB_OK) return rc;
    const int64_t n_weight = a->W * a->H, n_all = n_weight + a->H;
    const dim3 grid((unsigned)((n_all + kWave - 1) / kWave));
    if (a->dtype == MCCB_BF16)
        hipLaunchKernelGGL((conv_act_sum<MCCB_BF16>), grid, dim3(kThreads), 0, st, partial,
                           s.n * a->B, n_weight, n_all, (uint16_t *)gw, (uint16_t *)gb);
    else
        hipLaunchKernelGGL((conv_act_sum<MCCB_FP16>), grid, dim3(kThreads), 0, st, partial,
                           s.n * a->B, n_weight, n_all, (uint16_t *)gw, (uint16_t *)gb);
    return launched();
}

int mccb_conv_act_step(const mccb_conv_t *a, void *state, void *y, void *stream) {
    int rc = check_conv(a, true);
    if (rc != MCCB_OK) return rc;
    if (!y || (!state && a->W > 1)) return MCCB_ERR_PARAM_NULLPTR;
    if (a->state || a->lengths) return MCCB_ERR_PARAM_INVALID;
    Span in[5];
    int n;
    rc = check_conv_inputs(a, in, &n);
    if (rc != MCCB_OK) return rc;
    const Span out[2] = {{y, (uint64_t)(a->B * a->H) * 2},
                         {state, (uint64_t)((a->W - 1) * a->B * a->H) * 2}};
    if (misaligned(y, 2) || misaligned(state, 2) || outputs_clash(in, n, out, 2))
        return MCCB_ERR_PARAM_INVALID;
    return vector_ok(a->H, a->x_stride[2], kFwdVec)
               ? launch_one<kFwdVec>(a, state, y, (hipStream_t)stream)
               : launch_one<1>(a, state, y, (hipStream_t)stream);
}

}  // extern "C"
