// ssm_common.h -- what the kernels of the state space block share: 16-bit formats, activations in
// fp32, and the host's argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "mccb_ssm.h"

namespace ssm {

constexpr int kWave = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------------------------
// 16-bit formats. Conversions to 16 bits round to nearest, ties to even.
// ---------------------------------------------------------------------------------------------
template <int DT>
struct F16;
template <>
struct F16<MCCB_BF16> {
    typedef __bf16 elem;
    __device__ static inline float to_f32(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }
};
template <>
struct F16<MCCB_FP16> {
    typedef _Float16 elem;
    __device__ static inline float to_f32(uint16_t u) {
        return (float)__builtin_bit_cast(_Float16, u);
    }
};
template <int DT>
__device__ static inline float to_f32(uint16_t u) {
    return F16<DT>::to_f32(u);
}
template <int DT>
__device__ static inline uint16_t from_f32(float f) {
    return __builtin_bit_cast(uint16_t, (typename F16<DT>::elem)f);
}

// V 16-bit values in one load. Global memory takes vectors at any 2-byte address on this target,
// so the type carries the elements' alignment: rows of odd lengths keep their wide loads.
template <int V>
struct HVec {
    typedef uint16_t t __attribute__((ext_vector_type(V), aligned(2)));
};
template <>
struct HVec<1> {
    struct t {
        uint16_t v;
        __device__ uint16_t &operator[](int) { return v; }
        __device__ uint16_t operator[](int) const { return v; }
    };
};

// A wave-uniform address plus a lane's 32-bit offset. The empty asm keeps the base in scalar
// registers, so that loads and stores take the form with a scalar base and a 32-bit lane offset
// instead of a 64-bit vector addition each. (Unoptimized builds do not keep it uniform.)
template <typename P>
__device__ static inline P *lane_at(P *base, uint32_t offset) {
#if defined(__OPTIMIZE__)
    asm("" : "+s"(base));
    typedef __attribute__((address_space(1))) P gP;
    return (P *)((gP *)base + offset);
#else
    return base + offset;
#endif
}

// A barrier for data in LDS: this wave's LDS accesses are done, its global loads and stores may stay
// in flight (__syncthreads waits for those too, which ends every prefetch at the barrier).
__device__ static inline void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---------------------------------------------------------------------------------------------
// fp32 functions. exp2, log and the reciprocal are the hardware's (about 1 ulp).
// ---------------------------------------------------------------------------------------------
__device__ static inline float exp2_f(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ static inline float exp_f(float v) { return exp2_f(v * kLog2e); }
__device__ static inline float rcp_f(float v) { return __builtin_amdgcn_rcpf(v); }

// 1/(1+exp(-v)): exp(-v) overflows to infinity below v = -88 and its reciprocal is 0, the limit.
__device__ static inline float sigmoid_f(float v) { return rcp_f(1.0f + exp_f(-v)); }

// log(1+e) for e in [0,1] to 2e-7 of itself: with u = 1+e rounded, log(1+e) = log(u) + (e-(u-1))/u,
// whose last term (below 2^-24, its division by u below 2^-25) matters where e is small and u near
// 1. Step sizes of 1e-3 come from e = 1e-3, of which log(1+e) alone keeps four digits.
__device__ static inline float log1p_unit(float e) {
    const float u = 1.0f + e;
    return __builtin_fmaf(__builtin_amdgcn_logf(u), kLn2, e - (u - 1.0f));
}

// softplus(v) = max(v,0) + log(1 + exp(-|v|)): 0 at -infinity, v itself from where the logarithm is
// below half a step of v (up to the largest values and infinity); the logarithm keeps NaN, which the
// maximum drops. `slope` gets its derivative, the logistic function.
__device__ static inline float softplus_f(float v, float &slope) {
    const float e = exp_f(-__builtin_fabsf(v));
    const float r = rcp_f(1.0f + e);
    slope = v >= 0.0f ? r : e * r;
    return __builtin_fmaxf(v, 0.0f) + log1p_unit(e);
}
__device__ static inline float softplus_f(float v) {
    float unused;
    return softplus_f(v, unused);
}

__device__ static inline float silu_f(float v) { return v * sigmoid_f(v); }
// Slopes are 0 and 1 at the ends. There sigmoid_f is exactly 0 or 1, and the factor v (in gelu's also
// v^2, which overflows from 2e19 on) is taken as +-128, so that it leaves no zero times infinity.
// (Of NaN it makes a number; sigmoid_f keeps it.)
__device__ static inline float bounded(float v) { return __builtin_amdgcn_fmed3f(v, -128.0f, 128.0f); }
__device__ static inline float silu_slope_f(float v) {
    const float g = sigmoid_f(v);
    return g * __builtin_fmaf(bounded(v), 1.0f - g, 1.0f);
}

// tanh-form gelu: 0.5 (1 + tanh u) is the logistic function of 2u, u = c (v + 0.044715 v^3).
constexpr float kGelu2c = 1.5957691216057308f;  // 2 sqrt(2/pi)
__device__ static inline float act_f(float v, int act) {
    switch (act) {
        case MCCB_ACT_RELU: return v < 0.0f ? 0.0f : v;
        case MCCB_ACT_SILU: return silu_f(v);
        case MCCB_ACT_GELU:
            return v * sigmoid_f(kGelu2c * v * __builtin_fmaf(0.044715f * v, v, 1.0f));
        case MCCB_ACT_SOFTPLUS: return softplus_f(v);
        default: return v;
    }
}
__device__ static inline float act_slope_f(float v, int act) {
    switch (act) {
        case MCCB_ACT_RELU: return v > 0.0f ? 1.0f : 0.0f;
        case MCCB_ACT_SILU: return silu_slope_f(v);
        case MCCB_ACT_GELU: {
            const float g = sigmoid_f(kGelu2c * v * __builtin_fmaf(0.044715f * v, v, 1.0f));
            const float c = bounded(v), du = kGelu2c * __builtin_fmaf(0.134145f * c, c, 1.0f);
            return __builtin_fmaf(c * g * (1.0f - g), du, g);
        }
        case MCCB_ACT_SOFTPLUS: return sigmoid_f(v);
        default: return 1.0f;
    }
}

// ---------------------------------------------------------------------------------------------
// Host side: checks shared by the entry points. Nothing here allocates or throws.
// ---------------------------------------------------------------------------------------------
constexpr int64_t kMaxBatch = 65535, kMaxRows = (int64_t)1 << 31, kMaxWidth = (int64_t)1 << 24;

inline uint64_t align16(uint64_t v) { return (v + 15u) & ~(uint64_t)15u; }

struct Span {
    const void *p;
    uint64_t bytes;
};

// Bytes from the base to one past the last element of a strided tensor (0 for an empty one); false
// if a stride is negative or the extent does not fit in 2^62 bytes.
inline bool extent(int n, const int64_t *size, const int64_t *stride, int64_t esz, uint64_t *out) {
    unsigned __int128 last = 0;
    for (int i = 0; i < n; ++i) {
        if (stride[i] < 0) return false;
        if (size[i] == 0) {
            *out = 0;
            return true;
        }
        last += (unsigned __int128)(uint64_t)(size[i] - 1) * (uint64_t)stride[i];
    }
    const unsigned __int128 bytes = (last + 1) * (uint64_t)esz;
    if (bytes >> 62) return false;
    *out = (uint64_t)bytes;
    return true;
}

inline bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}

// No output may overlap an input or another output.
inline bool outputs_clash(const Span *in, int n_in, const Span *out, int n_out) {
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (overlap(out[o], in[i])) return true;
        for (int q = 0; q < o; ++q)
            if (overlap(out[o], out[q])) return true;
    }
    return false;
}

inline bool misaligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

inline int launched() { return hipGetLastError() == hipSuccess ? MCCB_OK : MCCB_ERR_RUNTIME; }

// A workspace argument against the size needed.
inline int check_workspace(const void *ws, uint64_t have, uint64_t need) {
    if (need == 0) return MCCB_OK;
    if (!ws) return MCCB_ERR_PARAM_NULLPTR;
    return have < need || misaligned(ws, 16) ? MCCB_ERR_PARAM_INVALID : MCCB_OK;
}

}  // namespace ssm
