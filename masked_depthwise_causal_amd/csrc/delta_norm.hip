// delta_norm.hip -- the norms before and after a block, with what stands next to them: the scaled residual
// addition before (prenorm), and weight, gate, residual scale and addition after (postnorm).
//
//   prenorm   r = residual + scale x,  out = r rstd w                  rstd = 1/sqrt(mean(r^2) + eps)
//   postnorm  out = residual + scale (x rstd w silu(z))                over each of a row's groups
//
// Backward, with n the normalized value, gn the gradient that reaches it (all factors behind the norm) and
// D the group's width: the gradient of what is normalized is rstd (gn - n mean(gn n)), so one reduction
// of two sums (r^2 and gn r) is all that a group needs; gradients of weight and scale are sums over rows.
//
// All of it is bound by HBM: each value is read once, kept in registers as it was read (16 bits) between
// the reduction and its use, and each result written once. A team of T lanes takes a group, so many that
// a lane has one or two vectors of 8 values; teams keep their group and walk over rows, with the
// weights of their columns in registers, and in the backward also the columns' sums.
#include "mccb_delta.h"
#include "ssm_common.h"

using namespace ssm;

namespace {

constexpr int kVec = 8;             // 16-bit values of a load
constexpr int kBlock = 256;         // threads of a block whose teams are a wave or less
constexpr int kMaxTeam = 1024, kMaxPer = 2;
constexpr int64_t kMaxGroup = (int64_t)kMaxTeam * kMaxPer * kVec;

struct Norm {
    int64_t R;                      // rows
    int D, G;                       // a group's width, groups
    int weight_step;                // from one group's weights to the next: D, or 0 where they are shared
    float eps, inv;                 // inv = 1 / D
    const uint16_t *x, *residual, *z, *w, *scale;
    int64_t x_ld, residual_ld, z_ld;
};

// ---------------------------------------------------------------------------------------------
// Vectors of 8 values; the last one of a group may hold fewer.
// ---------------------------------------------------------------------------------------------
typedef HVec<kVec>::t vec8;

// p is a group's column c, of which n are left. A last vector of fewer is read as the last 8 values and moved down.
__device__ static inline vec8 load8(const uint16_t *p, int n, int c) {
    if (n >= kVec) return *(const vec8 *)p;
    vec8 v = {};
    if (n <= 0) return v;
    if (c >= kVec) {
        const auto last = __builtin_bit_cast(unsigned __int128, *(const vec8 *)(p - (kVec - n)));
        return __builtin_bit_cast(vec8, last >> (16 * (kVec - n)));
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) v[i] = p[i];
    return v;
}
__device__ static inline void store8(uint16_t *p, vec8 v, int n) {
    if (n >= kVec) {
        *(vec8 *)p = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = v[i];
}

// The sums of a and b over a team's lanes, on every one of them, in a fixed order. Teams of more than a
// wave are the whole block and meet in LDS (`slot` alternates, so one barrier a reduction is enough).
template <int CTRL>
__device__ static inline float row_add(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
template <int T>
__device__ static inline void team_sum(float &a, float &b, float (*part)[2 * kMaxTeam / kWave], int slot) {
    a = row_add<0x128>(a), b = row_add<0x128>(b);  // within 16 lanes: by rotations of 8, 4, 2, 1
    a = row_add<0x124>(a), b = row_add<0x124>(b);
    a = row_add<0x122>(a), b = row_add<0x122>(b);
    a = row_add<0x121>(a), b = row_add<0x121>(b);
    if constexpr (T > 16) {
        a += __shfl_xor(a, 16), b += __shfl_xor(b, 16);
        a += __shfl_xor(a, 32), b += __shfl_xor(b, 32);
    }
    if constexpr (T > kWave) {
        const int waves = blockDim.x / kWave, wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0) part[slot][2 * wave] = a, part[slot][2 * wave + 1] = b;
        lds_barrier();
        a = b = 0.0f;
        for (int i = 0; i < waves; ++i) a += part[slot][2 * i], b += part[slot][2 * i + 1];
    }
}

// Which group and rows a team takes: blocks along x are sets of `groups` groups, along y strips of rows;
// within a block `slots` teams share a group and take its rows in turn.
struct Teams {
    int groups, slots;              // of a block
    int64_t strip;                  // rows of a block
};

struct Place {
    int g, slot, lane;              // lane: within the team
    bool on;
};
template <int T>
__device__ static inline Place place(const Norm &n, const Teams &t) {
    Place p;
    const int team = T > kWave ? 0 : threadIdx.x / T;
    p.lane = T > kWave ? threadIdx.x : threadIdx.x % T;
    p.g = blockIdx.x * t.groups + team % t.groups;
    p.slot = team / t.groups;
    p.on = p.slot < t.slots && p.g < n.G;
    return p;
}

// T: lanes of a team (over a wave: the block, of any number of waves). E: vectors of a lane.
// T lanes' vectors lie next to each other: vector e of a lane starts at column 8 (lane + e team).
// 16384 rows of bf16: prenorm of 4096 with residual, scale and sum 96 us (537 MB, 5.6 TB/s), postnorm in 32 groups with a
// gate 79 us (403 MB, 5.1 TB/s), of 5120 with gate, scale and residual 135 us (671 MB, 5.0 TB/s). Narrow groups leave lanes of
// a team idle: 64 groups of 64 84 us, 256 of 16 288.
template <int DT, bool POST, int T, int E>
__global__ void __launch_bounds__(T > kWave ? kMaxTeam : kBlock)
    norm_forward(Norm n, Teams t, uint16_t *__restrict__ out, uint16_t *__restrict__ sum) {
    __shared__ float part[2][2 * kMaxTeam / kWave];
    const Place p = place<T>(n, t);
    if (T <= kWave && !p.on) return;
    const int team = T > kWave ? blockDim.x : T;
    const int64_t H = (int64_t)n.D * n.G, first = (int64_t)p.g * n.D;
    vec8 w[E], s[E];
    int have[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = kVec * (p.lane + e * team);
        have[e] = n.D - c;
        w[e] = load8(n.w + (int64_t)p.g * n.weight_step + c, have[e], c);
        s[e] = n.scale ? load8(n.scale + first + c, have[e], c) : vec8{};
    }
    const int64_t end = min(n.R, (blockIdx.y + 1) * t.strip);
    int turn = 0;
    for (int64_t r = blockIdx.y * t.strip + p.slot; r < end; r += t.slots, turn ^= 1) {
        vec8 x[E], res[E], z[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int col = kVec * (p.lane + e * team);
            const int64_t c = first + col;
            x[e] = load8(n.x + r * n.x_ld + c, have[e], col);
            res[e] = n.residual ? load8(n.residual + r * n.residual_ld + c, have[e], col) : vec8{};
            z[e] = POST && n.z ? load8(n.z + r * n.z_ld + c, have[e], col) : vec8{};
        }
        float a = 0.0f, unused = 0.0f;
        float v[E][kVec];
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                v[e][i] = to_f32<DT>(x[e][i]);
                if (!POST) {
                    if (n.scale) v[e][i] *= to_f32<DT>(s[e][i]);
                    if (n.residual) v[e][i] += to_f32<DT>(res[e][i]);
                }
                a = __builtin_fmaf(v[e][i], v[e][i], a);
            }
        team_sum<T>(a, unused, part, turn);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(a, n.inv, n.eps));
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t c = r * H + first + kVec * (p.lane + e * team);
            vec8 y, total;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                float o = v[e][i] * rstd * to_f32<DT>(w[e][i]);
                if (POST) {
                    if (n.z) o *= silu_f(to_f32<DT>(z[e][i]));
                    if (n.scale) o *= to_f32<DT>(s[e][i]);
                    if (n.residual) o += to_f32<DT>(res[e][i]);
                }
                y[i] = from_f32<DT>(o);
                total[i] = from_f32<DT>(v[e][i]);
            }
            if (have[e] > 0) {
                store8(out + c, y, have[e]);
                if (!POST && sum) store8(sum + c, total, have[e]);
            }
        }
    }
}

struct NormGrads {
    const uint16_t *g, *gsum;       // gsum: prenorm's gradient into the sum
    int64_t g_ld, gsum_ld;
    uint16_t *gx, *gres, *gz;       // gres: prenorm's, where it is not gx
    float *pw, *ps;                 // sums over a block's rows, of weight and scale
};

// A row's values as they were read.
template <int E>
struct Row {
    vec8 x[E], g[E], other[E], gsum[E];  // other: residual, or the gate
};
template <bool POST, int E>
__device__ static inline void load_row(const Norm &n, const NormGrads &q, int64_t r, int64_t first, int lane, int team,
                                       const int (&have)[E], Row<E> &row) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int col = kVec * (lane + e * team);
        const int64_t c = first + col;
        row.x[e] = load8(n.x + r * n.x_ld + c, have[e], col);
        row.g[e] = load8(q.g + r * q.g_ld + c, have[e], col);
        row.other[e] = row.gsum[e] = vec8{};
        if (POST) {
            if (n.z) row.other[e] = load8(n.z + r * n.z_ld + c, have[e], col);
        } else {
            if (n.residual) row.other[e] = load8(n.residual + r * n.residual_ld + c, have[e], col);
            if (q.gsum) row.gsum[e] = load8(q.gsum + r * q.gsum_ld + c, have[e], col);
        }
    }
}

// The next row is on its way while one is worked on, where a lane has one vector; with two, in blocks that leave a
// lane 128 registers, there is no room for it, nor for the weights, which are read again with each row, and 68 to 198
// registers are spilled all the same: groups above 8192 values, of which there is no other form, run at 0.8 to 1.5 TB/s
// (8192 rows of 8200: prenorm 551 us, postnorm 852). 16-lane teams with a gate spill 7 and 14.
// 16384 rows of bf16: prenorm of 4096 with residual, scale and the sum's gradient 182 us (805 MB, 4.4 TB/s),
// postnorm of 5120 with gate and scale 223 to 235 us (839 MB, 3.6 to 3.8 TB/s).
template <int DT, bool POST, int T, int E>
__global__ void __launch_bounds__(T > kWave ? kMaxTeam : kBlock, T == 16 && E == 1 ? 4 : 1)
    norm_backward(Norm n, Teams t, NormGrads q) {
    constexpr int kTeams = T > kWave ? 1 : kBlock / T;
    constexpr bool kAhead = T <= kWave || E == 1;
    __shared__ float part[2][2 * kMaxTeam / kWave];
    __shared__ float meet[kTeams > 1 ? kTeams : 1][kTeams > 1 ? T * E * kVec : 1];
    const Place p = place<T>(n, t);
    const int team = T > kWave ? blockDim.x : T;
    const int64_t H = (int64_t)n.D * n.G, first = (int64_t)p.g * n.D;
    vec8 w[E], s[E];
    int have[E];
    float sw[E][kVec], ss[E][kVec];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = kVec * (p.lane + e * team);
        have[e] = p.on ? n.D - c : 0;
        w[e] = load8(n.w + (int64_t)p.g * n.weight_step + c, have[e], c);
        s[e] = n.scale ? load8(n.scale + first + c, have[e], c) : vec8{};
#pragma unroll
        for (int i = 0; i < kVec; ++i) sw[e][i] = ss[e][i] = 0.0f;
    }
    const int64_t end = p.on ? min(n.R, (blockIdx.y + 1) * t.strip) : 0;
    int turn = 0;
    Row<E> next;
    int64_t r = blockIdx.y * t.strip + p.slot;
    if (kAhead && r < end) load_row<POST>(n, q, r, first, p.lane, team, have, next);
    for (; r < end; r += t.slots, turn ^= 1) {
        Row<E> row;
        if (kAhead) {
            row = next;
            if (r + t.slots < end) load_row<POST>(n, q, r + t.slots, first, p.lane, team, have, next);
        } else {
            load_row<POST>(n, q, r, first, p.lane, team, have, row);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = kVec * (p.lane + e * team);
                w[e] = load8(n.w + (int64_t)p.g * n.weight_step + c, have[e], c);
                if (n.scale) s[e] = load8(n.scale + first + c, have[e], c);
            }
        }
        // what is normalized, and the gradient at the normalized value; the gate's logistic function is kept
        float sig[POST ? E : 1][kVec];
        auto at = [&](int e, int i, float &v, float &gn) {
            v = to_f32<DT>(row.x[e][i]);
            gn = to_f32<DT>(row.g[e][i]) * to_f32<DT>(w[e][i]);
            if (POST) {
                if (n.scale) gn *= to_f32<DT>(s[e][i]);
                if (n.z) gn *= to_f32<DT>(row.other[e][i]) * sig[e][i];
            } else {
                if (n.scale) v *= to_f32<DT>(s[e][i]);
                if (n.residual) v += to_f32<DT>(row.other[e][i]);
            }
        };
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                float v, gn;
                if (POST && n.z) sig[e][i] = sigmoid_f(to_f32<DT>(row.other[e][i]));
                at(e, i, v, gn);
                a = __builtin_fmaf(v, v, a);
                b = __builtin_fmaf(v, gn, b);
            }
        team_sum<T>(a, b, part, turn);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(a, n.inv, n.eps));
        const float mean = b * rstd * n.inv;  // of gn n
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t c = r * H + first + kVec * (p.lane + e * team);
            vec8 o, ores, oz;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                float v, gn;
                at(e, i, v, gn);
                const float nv = v * rstd;
                float gr = rstd * __builtin_fmaf(-nv, mean, gn);
                const float gv = to_f32<DT>(row.g[e][i]);
                if (POST) {
                    const float wv = to_f32<DT>(w[e][i]), sv = n.scale ? to_f32<DT>(s[e][i]) : 1.0f;
                    const float zv = to_f32<DT>(row.other[e][i]), gate = n.z ? zv * sig[e][i] : 1.0f;
                    const float gy = gv * nv;  // the gradient of every factor behind the norm, save itself
                    sw[e][i] = __builtin_fmaf(gy * sv, gate, sw[e][i]);
                    ss[e][i] = __builtin_fmaf(gy * wv, gate, ss[e][i]);
                    if (n.z)
                        oz[i] = from_f32<DT>(gy * sv * wv * sig[e][i] * __builtin_fmaf(bounded(zv), 1.0f - sig[e][i], 1.0f));
                } else {
                    sw[e][i] = __builtin_fmaf(gv, nv, sw[e][i]);
                    if (q.gsum) gr += to_f32<DT>(row.gsum[e][i]);
                    ss[e][i] = __builtin_fmaf(gr, to_f32<DT>(row.x[e][i]), ss[e][i]);
                    ores[i] = from_f32<DT>(gr);
                    if (n.scale) gr *= to_f32<DT>(s[e][i]);
                }
                o[i] = from_f32<DT>(gr);
            }
            if (have[e] > 0) {
                store8(q.gx + c, o, have[e]);
                if (POST && q.gz) store8(q.gz + c, oz, have[e]);
                if (!POST && q.gres) store8(q.gres + c, ores, have[e]);
            }
        }
    }
    // A block's sums are one partial row: its slots', and where all groups have one weight, the groups' too.
    auto meeting = [&](float (&v)[E][kVec], bool all) {
        if constexpr (kTeams > 1) {
            const int mine = threadIdx.x / T;
            lds_barrier();
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < kVec; ++i) meet[mine][(e * kVec + i) * T + p.lane] = v[e][i];
            lds_barrier();
            const int step = all ? 1 : t.groups, teams = t.groups * t.slots;
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    for (int k = mine + step; k < teams; k += step) v[e][i] += meet[k][(e * kVec + i) * T + p.lane];
        }
    };
    const bool shared = n.weight_step == 0 && n.G > 1;
    meeting(sw, shared);
    if (q.ps) meeting(ss, false);
    const int64_t row_w = shared ? ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * n.D : blockIdx.y * H + first;
    const bool writes = p.on && p.slot == 0, writes_w = shared ? threadIdx.x / (T > kWave ? kMaxTeam : T) == 0 : writes;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < have[e]) {
                const int c = kVec * (p.lane + e * team) + i;
                if (writes_w) q.pw[row_w + c] = sw[e][i];
                if (q.ps && writes) q.ps[blockIdx.y * H + first + c] = ss[e][i];
            }
}

// Column sums of the partial rows in 64 bits: 64 columns a block, 16 threads for each.
constexpr int kSumSlots = 16;
template <int DT>
__global__ void __launch_bounds__(kWave *kSumSlots)
    norm_sum(const float *__restrict__ pw, int64_t rows_w, int64_t width_w, uint16_t *__restrict__ gw,
             const float *__restrict__ ps, int64_t rows_s, int64_t width_s, uint16_t *__restrict__ gs) {
    __shared__ double part[kSumSlots][kWave];
    const int lane = threadIdx.x % kWave, slot = threadIdx.x / kWave;
    const int64_t blocks_w = (width_w + kWave - 1) / kWave;
    const bool second = blockIdx.x >= blocks_w;
    const float *from = second ? ps : pw;
    const int64_t rows = second ? rows_s : rows_w, width = second ? width_s : width_w;
    const int64_t c = (blockIdx.x - (second ? blocks_w : 0)) * kWave + lane;
    double v = 0.0;
    if (c < width)
#pragma unroll 8
        for (int64_t r = slot; r < rows; r += kSumSlots) v += (double)from[r * width + c];
    part[slot][lane] = v;
    __syncthreads();
    if (slot == 0 && c < width) {
        for (int i = 1; i < kSumSlots; ++i) v += part[i][lane];
        (second ? gs : gw)[c] = from_f32<DT>((float)v);
    }
}

// ---------------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------------
// A team is 16 lanes up to 256 values, a wave up to 1024, and above the smallest block whose lanes
// have two vectors each at most; `one`: one each, as far as that goes, as the gradients have it (registers), and
// where there are few rows, since then a row's latency is what counts and not the lanes that a reduction's barrier
// holds up.
struct Shape {
    int team, per;                  // lanes (16, 64, or a block's), vectors of a lane
    Teams t;
    unsigned gx, gy, threads;
};
Shape shape_of(const mccb_norm_t *a, bool one, int64_t blocks_wanted, int64_t least_rows) {
    Shape s;
    const int64_t D = a->H / a->groups, vecs = (D + kVec - 1) / kVec;
    const bool few = a->R * a->groups <= 1024;
    if (vecs <= 32) s.team = 16, s.per = vecs <= 16 ? 1 : 2;
    else if (vecs <= 128) s.team = kWave, s.per = vecs <= 64 ? 1 : 2;
    else {
        s.per = (few || one) && vecs <= kMaxTeam ? 1 : 2;
        const int64_t lanes = (vecs + s.per - 1) / s.per;
        s.team = (int)((lanes + kWave - 1) / kWave * kWave);
    }
    s.threads = s.team > kWave ? s.team : kBlock;
    const int teams = s.team > kWave ? 1 : kBlock / s.team;
    s.t.groups = a->groups < teams ? (int)a->groups : teams;
    s.t.slots = teams / s.t.groups;
    const int64_t gx = (a->groups + s.t.groups - 1) / s.t.groups;
    const int64_t turns = (a->R + s.t.slots - 1) / s.t.slots;  // of a block that took all rows
    int64_t strips = blocks_wanted / gx, most = (turns + least_rows - 1) / least_rows;
    strips = strips < 1 ? 1 : strips;
    strips = strips > most ? most : strips;
    strips = strips > 65535 ? 65535 : strips;
    strips = strips < 1 ? 1 : strips;
    const int64_t rows = (turns + strips - 1) / strips;         // turns of a strip
    s.t.strip = (rows < 1 ? 1 : rows) * s.t.slots;
    s.gx = (unsigned)gx;
    s.gy = (unsigned)(a->R > 0 ? (a->R + s.t.strip - 1) / s.t.strip : 0);
    return s;
}
Shape forward_shape(const mccb_norm_t *a) { return shape_of(a, false, 4096, 1); }
Shape backward_shape(const mccb_norm_t *a) { return shape_of(a, true, 1024, 4); }

Norm norm_of(const mccb_norm_t *a) {
    Norm n{};
    n.R = a->R, n.G = (int)a->groups, n.D = (int)(a->H / a->groups);
    n.weight_step = a->weight_shared ? 0 : n.D;
    n.eps = a->eps, n.inv = 1.0f / (float)n.D;
    n.x = (const uint16_t *)a->x, n.residual = (const uint16_t *)a->residual;
    n.z = (const uint16_t *)a->z, n.w = (const uint16_t *)a->weight, n.scale = (const uint16_t *)a->scale;
    n.x_ld = a->x_ld, n.residual_ld = a->residual_ld, n.z_ld = a->z_ld;
    return n;
}

int check_norm(const mccb_norm_t *a, bool post) {
    if (!a) return MCCB_ERR_PARAM_NULLPTR;
    if (a->dtype != MCCB_BF16 && a->dtype != MCCB_FP16) return MCCB_ERR_PARAM_INVALID;
    if (a->R < 0 || a->R > kMaxRows - 1 || a->H < 1 || a->groups < 1 || a->groups > 65535 ||
        a->H % a->groups != 0 || a->H / a->groups > kMaxGroup || a->H > kMaxWidth)
        return MCCB_ERR_SHAPE;
    // the hardware's reciprocal root takes subnormal numbers for 0, which would make NaN of a row of zeros
    if (!(a->eps >= 0x1p-126f) || a->eps > 3.0e38f) return MCCB_ERR_PARAM_INVALID;
    if (!post && (a->z || a->groups != 1)) return MCCB_ERR_PARAM_INVALID;
    return MCCB_OK;
}

// The inputs' spans, after the checks on each of them.
int norm_inputs(const mccb_norm_t *a, Span *in, int *count) {
    if (!a->weight || (!a->x && a->R > 0)) return MCCB_ERR_PARAM_NULLPTR;
    const int64_t size[2] = {a->R, a->H};
    const void *const rows[3] = {a->x, a->residual, a->z};
    const int64_t ld[3] = {a->x_ld, a->residual_ld, a->z_ld};
    int n = 0;
    for (int i = 0; i < 3; ++i) {
        if (!rows[i]) continue;
        const int64_t stride[2] = {ld[i], 1};
        uint64_t b;
        if (!extent(2, size, stride, 2, &b) || misaligned(rows[i], 2)) return MCCB_ERR_PARAM_INVALID;
        in[n++] = {rows[i], b};
    }
    if (misaligned(a->weight, 2) || misaligned(a->scale, 2)) return MCCB_ERR_PARAM_INVALID;
    in[n++] = {a->weight, (uint64_t)(a->weight_shared ? a->H / a->groups : a->H) * 2};
    in[n++] = {a->scale, (uint64_t)a->H * 2};
    *count = n;
    return MCCB_OK;
}

template <bool POST, int T, int E>
int launch_forward(const mccb_norm_t *a, const Shape &s, uint16_t *out, uint16_t *sum, hipStream_t st) {
    const dim3 grid(s.gx, s.gy), block(s.threads);
    if (a->dtype == MCCB_BF16)
        hipLaunchKernelGGL((norm_forward<MCCB_BF16, POST, T, E>), grid, block, 0, st, norm_of(a), s.t, out, sum);
    else
        hipLaunchKernelGGL((norm_forward<MCCB_FP16, POST, T, E>), grid, block, 0, st, norm_of(a), s.t, out, sum);
    return launched();
}
template <bool POST, int T, int E>
int launch_backward(const mccb_norm_t *a, const Shape &s, const NormGrads &q, hipStream_t st) {
    const dim3 grid(s.gx, s.gy), block(s.threads);
    if (a->dtype == MCCB_BF16)
        hipLaunchKernelGGL((norm_backward<MCCB_BF16, POST, T, E>), grid, block, 0, st, norm_of(a), s.t, q);
    else
        hipLaunchKernelGGL((norm_backward<MCCB_FP16, POST, T, E>), grid, block, 0, st, norm_of(a), s.t, q);
    return launched();
}

template <bool POST>
int forward(const mccb_norm_t *a, void *out, void *sum, void *stream) {
    int rc = check_norm(a, POST);
    if (rc != MCCB_OK) return rc;
    Span in[5];
    int n;
    rc = norm_inputs(a, in, &n);
    if (rc != MCCB_OK) return rc;
    if (!out && a->R > 0) return MCCB_ERR_PARAM_NULLPTR;
    const uint64_t b = (uint64_t)a->R * (uint64_t)a->H * 2;
    const Span o[2] = {{out, b}, {sum, b}};
    if (misaligned(out, 2) || misaligned(sum, 2) || outputs_clash(in, n, o, 2)) return MCCB_ERR_PARAM_INVALID;
    if (a->R == 0) return MCCB_OK;
    const Shape s = forward_shape(a);
    uint16_t *const po = (uint16_t *)out, *const pt = (uint16_t *)sum;
    const hipStream_t st = (hipStream_t)stream;
    if (s.team == 16)
        return s.per == 1 ? launch_forward<POST, 16, 1>(a, s, po, pt, st) : launch_forward<POST, 16, 2>(a, s, po, pt, st);
    if (s.team == kWave)
        return s.per == 1 ? launch_forward<POST, kWave, 1>(a, s, po, pt, st)
                          : launch_forward<POST, kWave, 2>(a, s, po, pt, st);
    return s.per == 1 ? launch_forward<POST, kMaxTeam, 1>(a, s, po, pt, st)
                      : launch_forward<POST, kMaxTeam, 2>(a, s, po, pt, st);
}

// Floats of the partial rows: of a shared weight one a block, else one a strip.
bool one_weight(const mccb_norm_t *a) { return a->weight_shared && a->groups > 1; }
uint64_t partial_w(const mccb_norm_t *a, const Shape &s) {
    return one_weight(a) ? (uint64_t)s.gx * s.gy * (uint64_t)(a->H / a->groups) : (uint64_t)s.gy * (uint64_t)a->H;
}

template <bool POST>
int backward_size(const mccb_norm_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_norm(a, POST);
    if (rc != MCCB_OK) return rc;
    const Shape s = backward_shape(a);
    *size = (partial_w(a, s) + (a->scale ? (uint64_t)s.gy * (uint64_t)a->H : 0)) * sizeof(float);
    return MCCB_OK;
}

template <bool POST>
int backward(const mccb_norm_t *a, NormGrads q, void *gw, void *gscale, void *ws, uint64_t ws_size, void *stream) {
    int rc = check_norm(a, POST);
    if (rc != MCCB_OK) return rc;
    Span in[8];
    int n;
    rc = norm_inputs(a, in, &n);
    if (rc != MCCB_OK) return rc;
    if (!gw || (a->R > 0 && (!q.g || !q.gx || (a->z && !q.gz))) || (a->scale && !gscale))
        return MCCB_ERR_PARAM_NULLPTR;
    if ((q.gz && !a->z) || (gscale && !a->scale) || (q.gres && !a->residual)) return MCCB_ERR_PARAM_INVALID;
    uint64_t need = 0, b;
    backward_size<POST>(a, &need);
    rc = check_workspace(ws, ws_size, need);
    if (rc != MCCB_OK) return rc;
    const int64_t size[2] = {a->R, a->H};
    const uint16_t *const rows[2] = {q.g, q.gsum};
    const int64_t ld[2] = {q.g_ld, q.gsum_ld};
    for (int i = 0; i < 2; ++i) {
        if (!rows[i]) continue;
        const int64_t stride[2] = {ld[i], 1};
        if (!extent(2, size, stride, 2, &b) || misaligned(rows[i], 2)) return MCCB_ERR_PARAM_INVALID;
        in[n++] = {rows[i], b};
    }
    const uint64_t all = (uint64_t)a->R * (uint64_t)a->H * 2;
    const int64_t n_weight = a->weight_shared ? a->H / a->groups : a->H;
    const Span o[6] = {{q.gx, all}, {q.gres, all}, {q.gz, all}, {gw, (uint64_t)n_weight * 2},
                       {gscale, (uint64_t)a->H * 2}, {ws, need}};
    for (int i = 0; i < 5; ++i)
        if (misaligned(o[i].p, 2)) return MCCB_ERR_PARAM_INVALID;
    if (outputs_clash(in, n, o, 6)) return MCCB_ERR_PARAM_INVALID;

    const Shape s = backward_shape(a);
    const hipStream_t st = (hipStream_t)stream;
    q.pw = (float *)ws;
    q.ps = a->scale ? q.pw + partial_w(a, s) : nullptr;
    if (a->R > 0) {
        if (s.team == 16)
            rc = s.per == 1 ? launch_backward<POST, 16, 1>(a, s, q, st) : launch_backward<POST, 16, 2>(a, s, q, st);
        else if (s.team == kWave)
            rc = s.per == 1 ? launch_backward<POST, kWave, 1>(a, s, q, st) : launch_backward<POST, kWave, 2>(a, s, q, st);
        else
            rc = s.per == 1 ? launch_backward<POST, kMaxTeam, 1>(a, s, q, st)
                            : launch_backward<POST, kMaxTeam, 2>(a, s, q, st);
        if (rc != MCCB_OK) return rc;
    }
    const int64_t rows_w = (int64_t)s.gy * (one_weight(a) ? s.gx : 1), rows_p = s.gy;
    const int64_t width_s = a->scale ? a->H : 0;
    const dim3 grid((unsigned)((n_weight + kWave - 1) / kWave + (width_s + kWave - 1) / kWave));
    const dim3 block(kWave * kSumSlots);
    if (a->dtype == MCCB_BF16)
        hipLaunchKernelGGL((norm_sum<MCCB_BF16>), grid, block, 0, st, q.pw, rows_w, n_weight, (uint16_t *)gw, q.ps,
                           rows_p, width_s, (uint16_t *)gscale);
    else
        hipLaunchKernelGGL((norm_sum<MCCB_FP16>), grid, block, 0, st, q.pw, rows_w, n_weight, (uint16_t *)gw, q.ps,
                           rows_p, width_s, (uint16_t *)gscale);
    return launched();
}

}  // namespace

extern "C" {

int mccb_prenorm_forward(const mccb_norm_t *a, void *out, void *sum, void *stream) {
    return forward<false>(a, out, sum, stream);
}
int mccb_postnorm_forward(const mccb_norm_t *a, void *out, void *stream) {
    return forward<true>(a, out, nullptr, stream);
}
int mccb_prenorm_backward_get_workspace_size(const mccb_norm_t *a, uint64_t *size) {
    return backward_size<false>(a, size);
}
int mccb_postnorm_backward_get_workspace_size(const mccb_norm_t *a, uint64_t *size) {
    return backward_size<true>(a, size);
}
int mccb_prenorm_backward(const mccb_norm_t *a, const void *gout, int64_t gout_ld, const void *gsum, int64_t gsum_ld,
                          void *gx, void *gres, void *gw, void *gscale, void *ws, uint64_t ws_size, void *stream) {
    NormGrads q{};
    q.g = (const uint16_t *)gout, q.gsum = (const uint16_t *)gsum, q.g_ld = gout_ld, q.gsum_ld = gsum_ld;
    q.gx = (uint16_t *)gx, q.gres = (uint16_t *)gres;
    return backward<false>(a, q, gw, gscale, ws, ws_size, stream);
}
int mccb_postnorm_backward(const mccb_norm_t *a, const void *gout, int64_t gout_ld, void *gx, void *gz, void *gw,
                           void *gscale, void *ws, uint64_t ws_size, void *stream) {
    NormGrads q{};
    q.g = (const uint16_t *)gout, q.g_ld = gout_ld;
    q.gx = (uint16_t *)gx, q.gz = (uint16_t *)gz;
    return backward<true>(a, q, gw, gscale, ws, ws_size, stream);
}

}  // extern "C"
