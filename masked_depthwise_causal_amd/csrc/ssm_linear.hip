// ssm_linear.hip -- matrix product with bias, activation and residual in its epilogue, and its
// backward, for MI355X (gfx950) (mccb_ssm.h).
//
//   out[m,n] = act(sum_k x[m,k] w[n,k] + bias[n]) + residual[m,n]
//   g = gout act'(pre),  gx[m,k] = sum_n g[m,n] w[n,k],  gw[n,k] = sum_m g[m,n] x[m,k]
//
// Two kernels carry the products, all of the form C = P Q^T:
//   tiles   (M above 64): a block computes a BM x BN tile with 32x32x16 matrix instructions from two
//           LDS buffers that are filled by loads straight to LDS, 64 of the contraction at a time.
//           Few tiles and a long contraction: the contraction is split over blocks, which leave fp32
//           partial tiles for `finish` to add in a fixed order. bf16 M=4096 K=4096 N=8192: 227 us,
//           1.21 PFLOP/s; M=4096 K=4096 N=5120: 140 us, 1.23.
//   skinny  (M up to 64): bound by reading w once. A wave takes 16 rows of w and every WAVES-th
//           part of the contraction, straight from memory into 16x16x32 matrix instructions.
//           M=4 K=5120 N=4096 with w not in any cache: 11.7 us, 3.6 TB/s.
// Rounded to 16 bits on the way to the gradients: g, a matrix instruction's operand (kept in two 16-bit
// terms it would double the backward's products), and pre, unless the caller asks for it in fp32. At
// M=4096 K=5120 N=4096 with silu, bf16, gx and gw are 0.0024 off in relation to their norm, of which
// their own rounding is 0.0017; pre in fp32 makes that 0.00235 and takes 12 us more of 535.
// The epilogue works on fp32 sums staged through LDS, so that bias, residual, pre and out are read
// and written as whole rows.
//
// Operands that the direct-to-LDS loads cannot take (rows not 16-byte aligned) go through registers
// instead, by loads that may start at any element. In the backward w, and g and x for gw, lie the other
// way round, with rows across the contraction; the tiles turn them as they read LDS. Only rows that are
// not aligned, and the skinny products, have them transposed into the workspace first (M=4096 K=5120
// N=4096, silu: 364 us with that, 335 without; M=1024 K=512 N=768: 34.6 and 25.0).
#include "ssm_common.h"

#include <type_traits>

using namespace ssm;

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

template <int DT>
__device__ static inline f32x16 mfma32(u16x8 a, u16x8 b, f32x16 c) {
    if constexpr (DT == MCCB_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <int DT>
__device__ static inline f32x4 mfma16(u16x8 a, u16x8 b, f32x4 c) {
    if constexpr (DT == MCCB_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

constexpr int kBK = 64;  // contraction a tile step takes: a row's 128 bytes, eight 16-byte chunks

__device__ __align__(16) const uint32_t zero_chunk[4] = {0, 0, 0, 0};

// What happens to a finished sum of out[m, n].
struct Epilogue {
    const uint16_t *bias, *residual;
    uint16_t *out;
    void *pre;  // of the dtype, or fp32
    int64_t residual_ld, N;
    int act, pre_fp32;
};

template <int ACT>
__device__ static inline void act8(float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_f(v[i], ACT);
}

// Eight adjacent values, `count` of them inside the matrix, the others 0.
template <int DT>
__device__ static inline void get8(const uint16_t *p, int count, float (&f)[8]) {
    if (count == 8) {
        const HVec<8>::t q = *(const HVec<8>::t *)p;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = to_f32<DT>(q[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < count ? to_f32<DT>(p[i]) : 0.0f;
    }
}

// Eight adjacent floats, from any one on.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
__device__ static inline void put_floats(float *p, int count, const float (&v)[8]) {
    if (count == 8) {
        *(f32x4_any *)p = f32x4_any{v[0], v[1], v[2], v[3]};
        *(f32x4_any *)(p + 4) = f32x4_any{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) p[i] = v[i];
    }
}
__device__ static inline void get_floats(const float *p, int count, float (&f)[8]) {
    if (count == 8) {
        const f32x4_any lo = *(const f32x4_any *)p, hi = *(const f32x4_any *)(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = lo[i], f[4 + i] = hi[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < count ? p[i] : 0.0f;
    }
}

// The sums v of eight adjacent columns of row m from column n, with the bias and the residual there.
template <int DT>
__device__ static inline void finish8(const Epilogue &e, int64_t m, int64_t n, int count, float (&v)[8],
                                      const float (&bias)[8], const float (&residual)[8]) {
    auto put = [&](uint16_t *p) {
        if (count == 8) {
            HVec<8>::t q;
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = from_f32<DT>(v[i]);
            *(HVec<8>::t *)p = q;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < count) p[i] = from_f32<DT>(v[i]);
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += bias[i];
    if (e.pre) {
        if (e.pre_fp32) put_floats((float *)e.pre + m * e.N + n, count, v);
        else put((uint16_t *)e.pre + m * e.N + n);
    }
    switch (e.act) {
        case MCCB_ACT_RELU: act8<MCCB_ACT_RELU>(v); break;
        case MCCB_ACT_SILU: act8<MCCB_ACT_SILU>(v); break;
        case MCCB_ACT_GELU: act8<MCCB_ACT_GELU>(v); break;
        case MCCB_ACT_SOFTPLUS: act8<MCCB_ACT_SOFTPLUS>(v); break;
        default: break;
    }
    if (e.residual) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += residual[i];
    }
    put(e.out + m * e.N + n);
}
template <int DT>
__device__ static inline void finish8(const Epilogue &e, int64_t m, int64_t n, int count, float (&v)[8]) {
    float bias[8] = {}, residual[8] = {};
    if (e.bias) get8<DT>(e.bias + n, count, bias);
    if (e.residual) get8<DT>(e.residual + m * e.residual_ld + n, count, residual);
    finish8<DT>(e, m, n, count, v, bias, residual);
}

// Operands as P [M,K] and Q [N,K]; an operand that lies the other way is [K,M] or [K,N].
struct Product {
    const uint16_t *p, *q;
    int64_t p_ld, q_ld;
    int64_t M, N, K;
    int tiles_m, tiles_n, splits, steps_per_split;  // steps of kBK
    float *partial;                                 // [splits][M][N] where splits > 1
};

// A block's tile: consecutive blocks go to different XCDs, so each XCD gets a run of tiles, and a
// run walks columns of eight tile rows, whose operands its L2 then holds.
__device__ static inline void tile_of(const Product &g, int &tm, int &tn) {
    constexpr int kXcd = 8, kGroup = 8;
    const int n = g.tiles_m * g.tiles_n, id = blockIdx.x;
    const int full = n / kXcd * kXcd;
    const int t = id < full ? id % kXcd * (n / kXcd) + id / kXcd : id;
    const int per = kGroup * g.tiles_n, grp = t / per, first = grp * kGroup;
    const int rows = g.tiles_m - first < kGroup ? g.tiles_m - first : kGroup;
    const int r = t - grp * per;
    tm = first + r % rows;
    tn = r / rows;
}

// Lane l's operand of 32x32x16 products, eight of the contraction from 8 (l / 32) of row l % 32, from LDS
// where the contraction's rows are `columns` apart. In each read a group of 16 lanes takes 16 columns of
// four rows, lane i the columns 4 (i % 4) .. + 3 of row i / 4, and gets column i of the four. (Without
// __restrict__, which holds until the barrier that lets the buffer be filled again, the compiler has every
// such read wait for all loads to LDS, the next step's too: backward of
// M=4096 K=4096 N=8192 578 us, 530 with.)
__device__ static inline u16x8 turned(const uint16_t *__restrict__ p, int columns) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + 4 * columns));
    return __builtin_bit_cast(u16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// DIRECT: both operands' rows are 16-byte aligned whole chunks. TP, TQ: that operand lies the other
// way, its rows along M or N, and is turned on its way from LDS to the registers.
template <int DT, int BM, int BN, int WM, int WN, bool DIRECT, bool TP, bool TQ>
__global__ void __launch_bounds__(WM *WN *kWave)
    product_tiles(Product g, Epilogue e) {
    constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;      // a wave's 32x32 tiles
    constexpr int kRows = BM + BN, kLoads = kRows / 8 / kWaves;  // a wave's load takes 8 rows
    constexpr int kBuf = kRows * kBK;                        // 16-bit values of a buffer
    // Tiles with a compute unit to themselves read the next operands while this one's products run,
    // over the step's end too: the one barrier of a step stands before its last products, whose
    // operands are in registers by then, and the loads of the step after the next go out behind them,
    // into the buffer that came free (M=4096 K=4096 N=8192: 254 us without; 241 with the barrier
    // first; 227; 233 with each load behind two products). The others have more waves to fill such
    // gaps, or (256x320 by way of registers or with operands turned) no registers left.
    constexpr bool kPipe = kWaves == 8 && (TM * TN <= 8 || (DIRECT && !TQ));
    constexpr int kStage = BN + 4;                           // fp32 row of the epilogue's staging
    constexpr int kRound = BM / WM;                          // rows it stages at a time
    constexpr size_t kBytes = sizeof(uint16_t) * 2 * kBuf > sizeof(float) * kRound * kStage
                                  ? sizeof(uint16_t) * 2 * kBuf
                                  : sizeof(float) * kRound * kStage;
    __shared__ __align__(16) uint8_t smem[kBytes];
    uint16_t *lds = (uint16_t *)smem;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    tile_of(g, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int all_steps = (int)((g.K + kBK - 1) / kBK);
    const int s0 = blockIdx.y * g.steps_per_split;
    const int s1 = s0 + g.steps_per_split < all_steps ? s0 + g.steps_per_split : all_steps;

    // Row r of a buffer (P's rows, then Q's) holds its eight chunks in the order c ^ (r / 2 % 8), so
    // that reading one chunk of 16 rows (256 bytes, all banks) meets every bank once. A load's lane i
    // fills place i % 8 of row i / 8 of a group of eight rows; groups go round the waves, P's before
    // Q's, so that a wave's groups are all even or all odd. Rows past the matrix repeat its last row.
    constexpr int kLoadsP = BM / 8 / kWaves;
    static_assert(BM / 8 % kWaves == 0 && BN / 8 % kWaves == 0 && kWaves % 2 == 0, "whole groups");
    static_assert(DIRECT || !(TP || TQ), "operands by way of registers are not turned");
    const int chunk = (lane % 8) ^ (lane / 16) ^ (wave % 2 * 4);
    // An operand that lies the other way fills its part of the buffer with 64 rows of BM or BN columns,
    // in the order of the loads. A read takes 64 bytes (32 columns) of four rows; those are moved by
    // `apart`, so that the four meet different banks whether a row is a multiple of all banks or not.
    auto apart = [](int row, int columns) { return columns % 128 == 0 ? row % 4 : row / 2 % 2; };
    auto row_across = [&](int i) {
        return (((i < kLoadsP ? i : i - kLoadsP) * kWaves + wave) * kWave + lane) /
               ((i < kLoadsP ? BM : BN) / 8);
    };
    uint32_t at[kLoads];  // bytes from the tile's first row of P or Q (DIRECT: below 2^32)
    const uint8_t *p0 = (const uint8_t *)(TP ? g.p + m0 : g.p + m0 * g.p_ld);
    const uint8_t *q0 = (const uint8_t *)(TQ ? g.q + n0 : g.q + n0 * g.q_ld);
    const int64_t p_step = (TP ? g.p_ld : 1) * kBK * 2, q_step = (TQ ? g.q_ld : 1) * kBK * 2;  // bytes
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const bool of_p = i < kLoadsP;
        const int64_t left = of_p ? g.M - m0 : g.N - n0, ld = of_p ? g.p_ld : g.q_ld;
        if (of_p ? TP : TQ) {
            const int across = (of_p ? BM : BN) / 8, r = row_across(i);
            const int id = ((of_p ? i : i - kLoadsP) * kWaves + wave) * kWave + lane;
            const int64_t c = ((id - r * across) ^ (apart(r, across * 8) * 4)) * 8;  // past: the last chunk
            at[i] = (uint32_t)((r * ld + (c < left ? c : left - 8)) * 2);
        } else {
            const int64_t r = ((of_p ? i : i - kLoadsP) * kWaves + wave) * 8 + lane / 8;
            at[i] = (uint32_t)((r < left ? r : left - 1) * ld * 2 + chunk * 16);
        }
    }
    typedef __attribute__((address_space(1))) const uint32_t gmem;
    typedef __attribute__((address_space(3))) uint32_t lmem;
    u16x8 held[DIRECT ? 1 : kLoads];
    auto place_of = [&](int i, int buf) {
        const int group = i < kLoadsP ? i * kWaves + wave : BM / 8 + (i - kLoadsP) * kWaves + wave;
        return lds + buf * kBuf + group * 8 * kBK;
    };
    auto fill_whole = [&](int step, int buf) {  // straight to LDS, 64 of the contraction
        const uint8_t *ps = p0 + step * p_step, *qs = q0 + step * q_step;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_global_load_lds((gmem *)lane_at(i < kLoadsP ? ps : qs, at[i]),
                                             (lmem *)place_of(i, buf), 16, 0, 0);
    };
    auto fill = [&](int step, int buf) {  // or what is left of it, and zeros
        const int64_t k = (int64_t)step * kBK;
        if (k + kBK <= g.K) {
            fill_whole(step, buf);
        } else {
            const uint8_t *ps = p0 + step * p_step, *qs = q0 + step * q_step;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const bool past = k + ((i < kLoadsP ? TP : TQ) ? row_across(i) : chunk * 8) >= g.K;
                const uint8_t *s = past ? (const uint8_t *)zero_chunk : (i < kLoadsP ? ps : qs) + at[i];
                __builtin_amdgcn_global_load_lds((gmem *)s, (lmem *)place_of(i, buf), 16, 0, 0);
            }
        }
    };
    // Operands that direct loads cannot take, by way of registers.
    auto row_of = [&](int i) {
        const bool of_p = i < kLoadsP;
        const int64_t r = ((of_p ? i : i - kLoadsP) * kWaves + wave) * 8 + lane / 8;
        const int64_t left = of_p ? g.M - m0 : g.N - n0;
        return (of_p ? g.p + (m0 + (r < left ? r : left - 1)) * g.p_ld
                     : g.q + (n0 + (r < left ? r : left - 1)) * g.q_ld) + chunk * 8;
    };
    auto take = [&](int step) {
        const int64_t k = (int64_t)step * kBK;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint16_t *s = row_of(i) + k;
            const int64_t left = g.K - k - chunk * 8;
            if (left >= 8) {
                held[i] = *(const HVec<8>::t *)s;
            } else {
                held[i] = u16x8{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int v = 0; v < 7; ++v)
                    if (v < left) held[i][v] = s[v];
            }
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) *(u16x8 *)(place_of(i, buf) + lane * 8) = held[i];
    };
    f32x16 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    // The operands of 16 of the contraction, and their products.
    u16x8 a[kPipe ? 2 : 1][TN], b[kPipe ? 2 : 1][TM];
    // Where operands lie the other way: what `turned` reads first for this lane, of a tile's columns and 16
    // of the contraction.
    auto across = [&](int ks, int tile, int columns) {
        const int r = lane % 16 / 4;
        return (ks * 16 + lane / 32 * 8 + r) * columns + (tile ^ apart(r, columns)) * 32 +
               lane / 16 % 2 * 16 + lane % 4 * 4;
    };
    auto operands = [&](int buf, int ks, int to) {
        const uint16_t *base = lds + buf * kBuf;
        const int c = (ks * 2 + lane / 32) ^ (lane / 2 % 8);  // rows below are lane % 32 modulo 32
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const int r = BM + (wn * TN + i) * 32 + lane % 32;
            if constexpr (TQ) a[to][i] = turned(base + BM * kBK + across(ks, wn * TN + i, BN), BN);
            else a[to][i] = *(const u16x8 *)(base + r * kBK + c * 8);
        }
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int r = (wm * TM + j) * 32 + lane % 32;
            if constexpr (TP) b[to][j] = turned(base + across(ks, wm * TM + j, BM), BM);
            else b[to][j] = *(const u16x8 *)(base + r * kBK + c * 8);
        }
    };
    auto multiply = [&](int from) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = mfma32<DT>(a[from][i], b[from][j], acc[i][j]);
    };
    auto landed = [&] {  // this wave's loads, and every wave is here
        __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        __syncthreads();
    };
    if (DIRECT) {
        fill(s0, 0);
    } else {
        take(s0);
        put(0);
    }
    if constexpr (kPipe) {
        auto next = [&](int step, int buf) { DIRECT ? fill(step, buf) : take(step); };
        // products from operands `from`, the reads of the next operands behind the first of them
        auto first = [&](int from) {
            acc[0][0] = mfma32<DT>(a[from][0], b[from][0], acc[0][0]);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto rest = [&](int from) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = i == 0 ? 1 : 0; j < TM; ++j)
                    acc[i][j] = mfma32<DT>(a[from][i], b[from][j], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        };
        constexpr int kLast = kBK / 16 - 1;
        landed();
        operands(0, 0, 0);
        if (s0 + 1 < s1) next(s0 + 1, 1);
        for (int s = s0; s < s1; ++s) {
            const int buf = (s - s0) & 1;
#pragma unroll
            for (int ks = 0; ks < kLast; ++ks) {
                first(ks & 1);
                operands(buf, ks + 1, (ks + 1) & 1);
                rest(ks & 1);
            }
            if (!DIRECT && s + 1 < s1) put(buf ^ 1);
            landed();
            first(kLast & 1);
            operands(buf ^ 1, 0, 0);  // behind the last step nothing that is used
            rest(kLast & 1);
            if (s + 2 < s1) next(s + 2, buf);
        }
    } else {
        for (int s = s0; s < s1; ++s) {
            const int buf = (s - s0) & 1;
            landed();
            if (s + 1 < s1) DIRECT ? fill(s + 1, buf ^ 1) : take(s + 1);
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks) {
                operands(buf, ks, 0);
                multiply(0);
            }
            if (!DIRECT && s + 1 < s1) put(buf ^ 1);
        }
    }
    // Epilogue, kRound rows at a time. A lane's 16 sums of a 32x32 tile are column lane % 32 (a row
    // of P) and rows 8 (v / 4) + 4 (lane / 32) + v % 4 (rows of Q, columns of the output).
    // The rows of the residual are on their way while the sums are staged (M=16384 K=2048 N=2048 with
    // bias, relu and residual: 141 us read where they are added, 130).
    float *stage = (float *)smem;
    constexpr int kAcross = BN / 8, kDown = kThreads / kAcross, kTimes = (kRound + kDown - 1) / kDown;
    const int n = threadIdx.x % kAcross * 8;
    const int64_t left = g.N - n0 - n;
    const int count = left < 8 ? (int)left : 8;
    float bias[8] = {};
    if (e.bias && left > 0) get8<DT>(e.bias + n0 + n, count, bias);
#pragma unroll
    for (int round = 0; round < WM; ++round) {
        const int64_t m1 = m0 + round * kRound;
        u16x8 rows[kTimes];
        const bool ahead = e.residual && !g.partial && left >= 8;
        if (ahead) {
#pragma unroll
            for (int t = 0; t < kTimes; ++t) {
                const int64_t m = m1 + threadIdx.x / kAcross + t * kDown;
                rows[t] = *(const HVec<8>::t *)(e.residual + (m < g.M ? m : g.M - 1) * e.residual_ld + n0 + n);
            }
        }
        __syncthreads();
        if (wm == round) {
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int row = j * 32 + lane % 32;
                        const int at_n = (wn * TN + i) * 32 + 8 * v + 4 * (lane / 32);
                        *(f32x4 *)(stage + row * kStage + at_n) =
                            f32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2],
                                  acc[i][j][4 * v + 3]};
                    }
        }
        __syncthreads();
        if (left <= 0) continue;
#pragma unroll
        for (int t = 0; t < kTimes; ++t) {
            const int r = threadIdx.x / kAcross + t * kDown;
            const int64_t m = m1 + r;
            if (r >= kRound || m >= g.M) break;
            float v[8], residual[8] = {};
            const f32x4 lo = *(const f32x4 *)(stage + r * kStage + n);
            const f32x4 hi = *(const f32x4 *)(stage + r * kStage + n + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
            if (g.partial) {
                float *q = g.partial + ((int64_t)blockIdx.y * g.M + m) * g.N + n0 + n;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < count) q[i] = v[i];
                continue;
            }
            if (ahead) {
#pragma unroll
                for (int i = 0; i < 8; ++i) residual[i] = to_f32<DT>(rows[t][i]);
            } else if (e.residual) {
                get8<DT>(e.residual + m * e.residual_ld + n0 + n, count, residual);
            }
            finish8<DT>(e, m, n0 + n, count, v, bias, residual);
        }
    }
}

// The split contraction's partial sums, added in order, through the epilogue.
template <int DT>
__global__ void __launch_bounds__(256)
    finish(Product g, Epilogue e) {
    const int64_t across = (g.N + 7) / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = id / across, n = id % across * 8;
    if (m >= g.M) return;
    const int count = g.N - n < 8 ? (int)(g.N - n) : 8;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < g.splits; ++s) {
        const float *p = g.partial + ((int64_t)s * g.M + m) * g.N + n;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) v[i] += p[i];
    }
    finish8<DT>(e, m, n, count, v);
}

// M up to 16 MB: a block has 16 rows of Q; its waves take parts of 64 of the contraction in turn and
// add their sums in LDS. A lane reads 32 adjacent bytes of its row for two matrix instructions (the
// order of the contraction is free as long as P's is the same), so a wave takes whole lines of its
// 16 rows. Loads may start at any 2-byte address.
template <int DT, int MB, int WAVES>
__global__ void __launch_bounds__(WAVES *kWave)
    product_skinny(Product g, Epilogue e) {
    __shared__ __align__(16) float part[WAVES][MB * 16][16 + 4];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t n = n0 + lane % 16 < g.N ? n0 + lane % 16 : g.N - 1;
    const int64_t own = (lane / 16) * 16;  // the lane's 16 of a part
    const uint16_t *qp = g.q + n * g.q_ld, *pp[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t m = b * 16 + lane % 16;
        pp[b] = g.p + (m < g.M ? m : g.M - 1) * g.p_ld;
    }
    // Eight sums go to a thread at the end; its bias and residual are on their way from the start.
    static_assert(MB * 16 * 2 <= WAVES * kWave, "a thread for every eight sums");
    const int64_t own_m = threadIdx.x / 2, own_n = n0 + threadIdx.x % 2 * 8, left = g.N - own_n;
    const bool sums = threadIdx.x < MB * 16 * 2 && own_m < g.M && left > 0, ahead = sums && left >= 8;
    u16x8 bias8 = {}, residual8 = {};
    if (ahead && e.bias) bias8 = *(const HVec<8>::t *)(e.bias + own_n);
    if (ahead && e.residual) residual8 = *(const HVec<8>::t *)(e.residual + own_m * e.residual_ld + own_n);
    f32x4 acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto guarded = [&](const uint16_t *p, int64_t k) {
        u16x8 v;
        if (k + 8 <= g.K) {
            v = *(const HVec<8>::t *)(p + k);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = k + i < g.K ? p[k + i] : 0;
        }
        return v;
    };
    // several parts' loads in flight, without a check of bounds; then part by part
    constexpr int kAhead = MB == 1 ? 4 : 2;
    constexpr int64_t kStride = WAVES * 64;
    int64_t k = wave * 64;
    for (; k + (kAhead - 1) * kStride + 64 <= g.K; k += kAhead * kStride) {
        u16x8 q[kAhead][2], p[kAhead][MB][2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                q[i][h] = *(const HVec<8>::t *)(qp + k + i * kStride + own + h * 8);
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    p[i][b][h] = *(const HVec<8>::t *)(pp[b] + k + i * kStride + own + h * 8);
            }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int b = 0; b < MB; ++b) acc[b] = mfma16<DT>(q[i][h], p[i][b][h], acc[b]);
    }
    for (; k < g.K; k += kStride) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u16x8 q = guarded(qp, k + own + h * 8);
#pragma unroll
            for (int b = 0; b < MB; ++b)
                acc[b] = mfma16<DT>(q, guarded(pp[b], k + own + h * 8), acc[b]);
        }
    }
    // a lane's four sums: row lane % 16 of P, rows 4 (lane / 16) + 0..3 of Q
#pragma unroll
    for (int b = 0; b < MB; ++b)
        *(f32x4 *)&part[wave][b * 16 + lane % 16][lane / 16 * 4] = acc[b];
    __syncthreads();
    if (!sums) return;
    float v[8] = {}, bias[8] = {}, residual[8] = {};
    // not unrolled whole: that many sums on their way take registers which spill
#pragma unroll 4
    for (int w = 0; w < WAVES; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += part[w][own_m][threadIdx.x % 2 * 8 + i];
    if (ahead) {
#pragma unroll
        for (int i = 0; i < 8; ++i) bias[i] = to_f32<DT>(bias8[i]), residual[i] = to_f32<DT>(residual8[i]);
    } else {
        if (e.bias) get8<DT>(e.bias + own_n, (int)left, bias);
        if (e.residual) get8<DT>(e.residual + own_m * e.residual_ld + own_n, (int)left, residual);
    }
    finish8<DT>(e, own_m, own_n, left < 8 ? (int)left : 8, v, bias, residual);
}

// ---------------------------------------------------------------------------------------------
// Operands laid out for the products
// ---------------------------------------------------------------------------------------------
// What the backward makes of gout (or of a plain matrix, without `pre`): g = gout act'(pre), kept by
// rows and / or by columns, and the column sums of 64 rows. One 64x64 tile a block; bound by memory
// (4096 x 4096, g by rows and sums: 24 us, 4.2 TB/s).
struct Turn {
    const uint16_t *src;
    const void *pre;
    int64_t ld, R, C;
    uint16_t *rows;     // [R, rows_ld] or NULL
    uint16_t *columns;  // [C, columns_ld] or NULL, zeros past R
    float *sums;        // [row tiles][C] or NULL
    int64_t rows_ld, columns_ld;
    int act, pre_fp32;
};

// PRE: without pre, with one of the dtype, of fp32.
enum { kNoPre, kPre16, kPre32 };
template <int DT, int PRE>
__global__ void __launch_bounds__(256)
    turn(Turn t) {
    __shared__ uint16_t tile[64][64 + 2];
    __shared__ float sum[32][64];
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const int c = threadIdx.x % 8 * 8, rr = threadIdx.x / 8;  // eight columns, rows rr and rr + 32
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t left = t.C - c0 - c;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = rr + half * 32;
        u16x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
        if (r0 + r < t.R && left > 0) {
            const uint16_t *p = t.src + (r0 + r) * t.ld + c0 + c;
            const int64_t at = (r0 + r) * t.C + c0 + c;
            const int count = left < 8 ? (int)left : 8;
            if (count == 8) {
                v = *(const HVec<8>::t *)p;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < count) v[i] = p[i];
            }
            float z[8];
            if (PRE == kPre16) get8<DT>((const uint16_t *)t.pre + at, count, z);
            if (PRE == kPre32) get_floats((const float *)t.pre + at, count, z);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float f = to_f32<DT>(v[i]);
                if (PRE != kNoPre) {
                    f *= act_slope_f(z[i], t.act);
                    v[i] = from_f32<DT>(f);
                }
                s[i] += f;
            }
            if (t.rows) {
                // rows are padded to whole vectors, with zeros past C
                u16x8 w = v;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= left) w[i] = 0;
                *(u16x8 *)(t.rows + (r0 + r) * t.rows_ld + c0 + c) = w;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) tile[r][c + i] = v[i];
    }
    if (t.sums) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[rr][c + i] = s[i];
    }
    __syncthreads();
    if (t.sums && threadIdx.x < 64 && c0 + threadIdx.x < t.C) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += sum[i][threadIdx.x];
        t.sums[(int64_t)blockIdx.y * t.C + c0 + threadIdx.x] = a;
    }
    if (!t.columns) return;
    // column cc, rows r .. r + 7 of the tile as one vector
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int cc = rr + half * 32, r = c;
        if (c0 + cc >= t.C || r0 + r >= t.columns_ld) continue;
        u16x8 v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = tile[r + i][cc];
        *(u16x8 *)(t.columns + (c0 + cc) * t.columns_ld + r0 + r) = v;
    }
}

// bias gradient: [P][N] over P, in fp64.
template <int DT>
__global__ void __launch_bounds__(256)
    sum_columns(const float *__restrict__ sums, int64_t P, int64_t N, uint16_t *__restrict__ gb) {
    __shared__ double part[4][64];
    const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    double s = 0.0;
    if (c < N) {
#pragma unroll 8
        for (int64_t p = w; p < P; p += 4) s += (double)sums[p * N + c];
    }
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < N)
        gb[c] = from_f32<DT>((float)((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane])));
}

// ---------------------------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------------------------
int64_t up8(int64_t v) { return (v + 7) & ~(int64_t)7; }
uint64_t area(int64_t rows, int64_t ld) { return align16((uint64_t)rows * (uint64_t)ld * 2); }

// Rows that the loads straight to LDS can take: aligned chunks, a tile's rows within 32-bit offsets.
bool direct_rows(const void *p, int64_t ld, int64_t along) {
    return !misaligned(p, 16) && ld % 8 == 0 && along % 8 == 0 && ld <= (int64_t)1 << 22;
}

// How a product is cut; a function of its sizes alone.
enum { kSkinny, k256x256, k256x320, k256x192, k128x128, k64x64, kForms };
struct Tile {
    int m, n;
    // cycles of a compute unit a step of 64 of the contraction: with one tile on it, and its share
    // of several (the smaller tiles'), measured with bf16 over M, N, K from 64 to 16384
    double alone, shared;
};
constexpr Tile kTiles[kForms] = {{0, 0, 0, 0},           {256, 256, 4100, 4100}, {256, 320, 4570, 4570},
                                 {256, 192, 2930, 2930}, {128, 128, 1900, 1350}, {64, 64, 900, 440}};

struct Cut {
    int form, splits, steps_per_split;
    int64_t tiles_m, tiles_n;
    uint64_t partial;  // workspace bytes
};

// The form and split with the least estimated time, in cycles: a compute unit's share of the tiles,
// each its steps and its epilogue, and for a split contraction another launch and the partial sums'
// way through memory.
Cut cut_of(int64_t M, int64_t N, int64_t K) {
    Cut best{};
    best.splits = 1;
    if (M <= 64) return best;  // skinny: w is read once however few the rows
    const int64_t steps = (K + kBK - 1) / kBK;
    double least = 0.0;
    for (int f = k256x256; f < kForms; ++f) {
        const Tile &t = kTiles[f];
        const int64_t tm = (M + t.m - 1) / t.m, tn = (N + t.n - 1) / t.n;
        for (int64_t want = 1; want <= 32 && (want == 1 || want * 4 <= steps); want *= 2) {
            const int64_t per = (steps + want - 1) / want, splits = (steps + per - 1) / per;
            const double share = (double)((tm * tn * splits + 255) / 256);  // of 256 compute units
            double cost = share * (per * (share > 1.0 ? t.shared : t.alone) + t.m * t.n * 0.25);
            if (splits > 1) cost += 12000.0 + (double)M * N * splits * 8.0 / 900.0;
            if (best.tiles_m == 0 || cost < least) {
                least = cost;
                best = {f, (int)splits, (int)per, tm, tn,
                        splits > 1 ? (uint64_t)splits * (uint64_t)M * (uint64_t)N * 4 : 0};
            }
        }
    }
    return best;
}

template <int DT, bool DIRECT, bool TP = false, bool TQ = false>
void launch_tiles(const Cut &c, const Product &g, const Epilogue &e, hipStream_t st) {
    const dim3 grid((unsigned)(c.tiles_m * c.tiles_n), (unsigned)c.splits);
    auto launch = [&](auto kernel, int threads) {
        hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, g, e);
    };
    switch (c.form) {
        case k256x256: launch(product_tiles<DT, 256, 256, 2, 4, DIRECT, TP, TQ>, 512); break;
        case k256x320: launch(product_tiles<DT, 256, 320, 4, 2, DIRECT, TP, TQ>, 512); break;
        case k256x192: launch(product_tiles<DT, 256, 192, 4, 2, DIRECT, TP, TQ>, 512); break;
        case k128x128: launch(product_tiles<DT, 128, 128, 2, 2, DIRECT, TP, TQ>, 256); break;
        default: launch(product_tiles<DT, 64, 64, 2, 2, DIRECT, TP, TQ>, 256);
    }
}

template <int DT, int MB>
void launch_skinny(const Product &g, const Epilogue &e, hipStream_t st) {
    const dim3 grid((unsigned)((g.N + 15) / 16));
    // enough waves a block that each has a few parts of the contraction
    if (g.K >= 4096)
        hipLaunchKernelGGL((product_skinny<DT, MB, 16>), grid, dim3(1024), 0, st, g, e);
    else if (g.K >= 512)
        hipLaunchKernelGGL((product_skinny<DT, MB, 8>), grid, dim3(512), 0, st, g, e);
    else
        hipLaunchKernelGGL((product_skinny<DT, MB, 2>), grid, dim3(128), 0, st, g, e);
}

template <int DT>
int launch_product(const uint16_t *p, int64_t p_ld, const uint16_t *q, int64_t q_ld, int64_t M,
                   int64_t N, int64_t K, const Epilogue &e, void *partial, hipStream_t st, bool tp = false,
                   bool tq = false) {
    const Cut c = cut_of(M, N, K);
    Product g{p, q, p_ld, q_ld, M, N, K, (int)c.tiles_m, (int)c.tiles_n, c.splits, c.steps_per_split,
              c.splits > 1 ? (float *)partial : nullptr};
    if (c.form == kSkinny) {
        if (M <= 16) launch_skinny<DT, 1>(g, e, st);
        else if (M <= 32) launch_skinny<DT, 2>(g, e, st);
        else launch_skinny<DT, 4>(g, e, st);
        return launched();
    }
    if (tp) launch_tiles<DT, true, true, true>(c, g, e, st);
    else if (tq) launch_tiles<DT, true, false, true>(c, g, e, st);
    else if (direct_rows(p, p_ld, K) && direct_rows(q, q_ld, K)) launch_tiles<DT, true>(c, g, e, st);
    else launch_tiles<DT, false>(c, g, e, st);
    const int rc = launched();
    if (rc != MCCB_OK || c.splits == 1) return rc;
    const int64_t ids = M * ((N + 7) / 8);
    hipLaunchKernelGGL((finish<DT>), dim3((unsigned)((ids + 255) / 256)), dim3(256), 0, st, g, e);
    return launched();
}

template <int DT>
int launch_turn(const Turn &t, hipStream_t st) {
    const dim3 grid((unsigned)((t.C + 63) / 64), (unsigned)((t.R + 63) / 64));
    if (!t.pre) hipLaunchKernelGGL((turn<DT, kNoPre>), grid, dim3(256), 0, st, t);
    else if (!t.pre_fp32) hipLaunchKernelGGL((turn<DT, kPre16>), grid, dim3(256), 0, st, t);
    else hipLaunchKernelGGL((turn<DT, kPre32>), grid, dim3(256), 0, st, t);
    return launched();
}

int check_linear(const mccb_linear_t *a) {
    if (!a) return MCCB_ERR_PARAM_NULLPTR;
    if (a->dtype != MCCB_BF16 && a->dtype != MCCB_FP16) return MCCB_ERR_PARAM_INVALID;
    if (a->activation < MCCB_ACT_NONE || a->activation > MCCB_ACT_SOFTPLUS)
        return MCCB_ERR_PARAM_INVALID;
    // tiles of 64 rows and columns are counted in a grid's 65535 rows
    if (a->M < 0 || a->M > ((int64_t)1 << 22) - 64 || a->N < 1 || a->N > ((int64_t)1 << 22) - 64 ||
        a->K < 1 || a->K > ((int64_t)1 << 22) - 64)
        return MCCB_ERR_SHAPE;
    return MCCB_OK;
}

int check_linear_inputs(const mccb_linear_t *a, Span *in) {
    if (!a->weight || (!a->x && a->M > 0)) return MCCB_ERR_PARAM_NULLPTR;
    const int64_t xs[2] = {a->M, a->K}, ws[2] = {a->N, a->K};
    const int64_t xst[2] = {a->x_ld, 1}, wst[2] = {a->weight_ld, 1};
    uint64_t x, w;
    if (!extent(2, xs, xst, 2, &x) || !extent(2, ws, wst, 2, &w) || misaligned(a->x, 2) ||
        misaligned(a->weight, 2) || misaligned(a->bias, 2))
        return MCCB_ERR_PARAM_INVALID;
    in[0] = {a->x, x};
    in[1] = {a->weight, w};
    in[2] = {a->bias, (uint64_t)a->N * 2};
    return MCCB_OK;
}

// The backward's: g by rows and by columns, x and w by columns (columns for products that do not read
// them as they lie; the size is a matter of sizes alone, not of alignment), the column sums, and the
// larger of the two products' partial sums.
struct BwdLayout {
    uint64_t g_rows, g_cols, x_cols, w_cols, sums, partial, total;
};

BwdLayout bwd_layout(const mccb_linear_t *a) {
    BwdLayout l{};
    const int64_t Mp = up8(a->M), Np = up8(a->N);
    const Cut cx = cut_of(a->M, a->K, a->N), cw = cut_of(a->N, a->K, a->M);
    uint64_t at = 0;
    l.g_rows = at, at += area(a->M, Np);
    l.g_cols = at, at += area(a->N, Mp);
    l.x_cols = at, at += area(a->K, Mp);
    l.w_cols = at, at += area(a->K, Np);
    l.sums = at, at += align16((uint64_t)((a->M + 63) / 64) * (uint64_t)a->N * 4);
    l.partial = at, at += cx.partial > cw.partial ? cx.partial : cw.partial;
    l.total = at;
    return l;
}

template <typename F>
int by_dtype(int dtype, F f) {
    return dtype == MCCB_BF16 ? f(std::integral_constant<int, MCCB_BF16>{})
                              : f(std::integral_constant<int, MCCB_FP16>{});
}

// Zeros for a gradient that sums no rows.
__global__ void __launch_bounds__(256) fill_zero(uint16_t *p, int64_t n) {
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < n; id += (int64_t)gridDim.x * 256) p[id] = 0;
}
int zero(void *p, int64_t n, hipStream_t st) {
    if (!p) return MCCB_OK;
    const int64_t blocks = (n + 255) / 256, most = (int64_t)1 << 16;
    hipLaunchKernelGGL(fill_zero, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, st,
                       (uint16_t *)p, n);
    return launched();
}

}  // namespace

extern "C" {

int mccb_linear_forward_get_workspace_size(const mccb_linear_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_linear(a);
    if (rc != MCCB_OK) return rc;
    *size = a->M > 0 ? cut_of(a->M, a->N, a->K).partial : 0;
    return MCCB_OK;
}

int mccb_linear_forward(const mccb_linear_t *a, const void *residual, int64_t residual_ld, void *out,
                        void *pre, void *ws, uint64_t ws_size, void *stream) {
    int rc = check_linear(a);
    if (rc != MCCB_OK) return rc;
    if (!out && a->M > 0) return MCCB_ERR_PARAM_NULLPTR;
    Span in[4];
    rc = check_linear_inputs(a, in);
    if (rc != MCCB_OK) return rc;
    const int64_t size[2] = {a->M, a->N}, stride[2] = {residual_ld, 1};
    uint64_t r_bytes = 0;
    if (residual && (!extent(2, size, stride, 2, &r_bytes) || misaligned(residual, 2)))
        return MCCB_ERR_PARAM_INVALID;
    const uint64_t need = a->M > 0 ? cut_of(a->M, a->N, a->K).partial : 0;
    rc = check_workspace(ws, ws_size, need);
    if (rc != MCCB_OK) return rc;
    in[3] = {residual, r_bytes};
    const uint64_t n_out = (uint64_t)a->M * (uint64_t)a->N, pre_size = a->pre_fp32 ? 4 : 2;
    const Span outs[3] = {{out, n_out * 2}, {pre, n_out * pre_size}, {ws, need}};
    if (misaligned(out, 2) || misaligned(pre, pre_size) || outputs_clash(in, 4, outs, 3))
        return MCCB_ERR_PARAM_INVALID;
    if (a->M == 0) return MCCB_OK;
    const hipStream_t st = (hipStream_t)stream;
    const Epilogue e{(const uint16_t *)a->bias, (const uint16_t *)residual, (uint16_t *)out,
                     pre, residual_ld, a->N, a->activation, a->pre_fp32};
    return by_dtype(a->dtype, [&](auto dt) {
        return launch_product<decltype(dt)::value>((const uint16_t *)a->x, a->x_ld,
                                                   (const uint16_t *)a->weight, a->weight_ld, a->M,
                                                   a->N, a->K, e, ws, st);
    });
}

int mccb_linear_backward_get_workspace_size(const mccb_linear_t *a, uint64_t *size) {
    if (!size) return MCCB_ERR_PARAM_NULLPTR;
    const int rc = check_linear(a);
    if (rc != MCCB_OK) return rc;
    *size = a->M > 0 ? bwd_layout(a).total : 0;
    return MCCB_OK;
}

int mccb_linear_backward(const mccb_linear_t *a, const void *gout, int64_t gout_ld, const void *pre,
                         void *gx, void *gw, void *gb, void *ws, uint64_t ws_size, void *stream) {
    int rc = check_linear(a);
    if (rc != MCCB_OK) return rc;
    if (a->M > 0 && (!gout || (a->activation != MCCB_ACT_NONE && !pre))) return MCCB_ERR_PARAM_NULLPTR;
    Span in[5];
    rc = check_linear_inputs(a, in);
    if (rc != MCCB_OK) return rc;
    const int64_t size[2] = {a->M, a->N}, stride[2] = {gout_ld, 1};
    uint64_t g_bytes = 0, need = 0;
    const uint64_t pre_size = a->pre_fp32 ? 4 : 2;
    if (!extent(2, size, stride, 2, &g_bytes) || misaligned(gout, 2) || misaligned(pre, pre_size))
        return MCCB_ERR_PARAM_INVALID;
    mccb_linear_backward_get_workspace_size(a, &need);
    rc = check_workspace(ws, ws_size, need);
    if (rc != MCCB_OK) return rc;
    in[3] = {gout, g_bytes};
    in[4] = {pre, (uint64_t)a->M * (uint64_t)a->N * pre_size};
    const Span outs[4] = {{gx, (uint64_t)a->M * (uint64_t)a->K * 2},
                          {gw, (uint64_t)a->N * (uint64_t)a->K * 2},
                          {gb, (uint64_t)a->N * 2},
                          {ws, need}};
    if (misaligned(gx, 2) || misaligned(gw, 2) || misaligned(gb, 2) || outputs_clash(in, 5, outs, 4))
        return MCCB_ERR_PARAM_INVALID;
    const hipStream_t st = (hipStream_t)stream;
    if (a->M == 0) {
        rc = zero(gw, a->N * a->K, st);
        return rc != MCCB_OK ? rc : zero(gb, a->N, st);
    }
    const BwdLayout l = bwd_layout(a);
    uint8_t *at = (uint8_t *)ws;
    const int64_t Mp = up8(a->M), Np = up8(a->N);
    uint16_t *g_rows = (uint16_t *)(at + l.g_rows), *g_cols = (uint16_t *)(at + l.g_cols);
    uint16_t *x_cols = (uint16_t *)(at + l.x_cols), *w_cols = (uint16_t *)(at + l.w_cols);
    float *sums = (float *)(at + l.sums);
    return by_dtype(a->dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const bool slope = a->activation != MCCB_ACT_NONE;
        // without an activation g is gradOut, which the products can read where it is
        const uint16_t *g = slope ? g_rows : (const uint16_t *)gout;
        const int64_t g_ld = slope ? Np : gout_ld;
        const uint16_t *x = (const uint16_t *)a->x, *w = (const uint16_t *)a->weight;
        // tiles read w, g and x as they lie; skinny products and unaligned rows need them turned
        const bool w_lies = a->M > 64 && direct_rows(g, g_ld, a->N) && direct_rows(w, a->weight_ld, a->K);
        const bool x_lies = a->N > 64 && direct_rows(g, g_ld, a->N) && direct_rows(x, a->x_ld, a->K);
        const Turn tg{(const uint16_t *)gout, slope ? pre : nullptr, gout_ld, a->M, a->N,
                      slope && (gx || (gw && x_lies)) ? g_rows : nullptr, gw && !x_lies ? g_cols : nullptr,
                      gb ? sums : nullptr, Np, Mp, a->activation, a->pre_fp32};
        int r = tg.rows || tg.columns || tg.sums ? launch_turn<DT>(tg, st) : MCCB_OK;
        if (r == MCCB_OK && gb) {
            hipLaunchKernelGGL((sum_columns<DT>), dim3((unsigned)((a->N + 63) / 64)), dim3(256), 0, st,
                               sums, (a->M + 63) / 64, a->N, (uint16_t *)gb);
            r = launched();
        }
        if (r == MCCB_OK && gx) {
            const Turn tw{w, nullptr, a->weight_ld, a->N, a->K, nullptr, w_cols, nullptr, 0, Np, MCCB_ACT_NONE, 0};
            if (!w_lies) r = launch_turn<DT>(tw, st);
            const Epilogue e{nullptr, nullptr, (uint16_t *)gx, nullptr, 0, a->K, MCCB_ACT_NONE, 0};
            if (r == MCCB_OK)
                r = launch_product<DT>(g, g_ld, w_lies ? w : w_cols, w_lies ? a->weight_ld : Np, a->M, a->K,
                                       a->N, e, at + l.partial, st, false, w_lies);
        }
        if (r == MCCB_OK && gw) {
            const Turn tx{x, nullptr, a->x_ld, a->M, a->K, nullptr, x_cols, nullptr, 0, Mp, MCCB_ACT_NONE, 0};
            if (!x_lies) r = launch_turn<DT>(tx, st);
            const Epilogue e{nullptr, nullptr, (uint16_t *)gw, nullptr, 0, a->K, MCCB_ACT_NONE, 0};
            if (r == MCCB_OK)
                r = launch_product<DT>(x_lies ? g : g_cols, x_lies ? g_ld : Mp, x_lies ? x : x_cols,
                                       x_lies ? a->x_ld : Mp, a->N, a->K, a->M, e, at + l.partial, st,
                                       x_lies, x_lies);
        }
        return r;
    });
}

}  // extern "C"
