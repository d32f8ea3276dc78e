// train_dev.cuh -- device helpers of the training operators: 16-byte vectors of either
// activation type, the activations and their derivatives, the padded row order.
#pragma once

#include "common.cuh"
#include "train_internal.h"

namespace moe {
namespace {

// 16-byte vectors: 8 bf16 or 4 f32.
template <typename T> struct Vec;
template <> struct Vec<float> { static constexpr int N = 4; };
template <> struct Vec<__nv_bfloat16> { static constexpr int N = 8; };

template <typename T>
__device__ __forceinline__ void unpack_vec(const uint4 v, float (&f)[Vec<T>::N]) {
    if constexpr (Vec<T>::N == 8) {
        unpack8(v, f);
    } else {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
}
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[Vec<T>::N]) {
    unpack_vec<T>(*reinterpret_cast<const uint4*>(p), f);
}
template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float (&f)[Vec<T>::N]) {
    if constexpr (Vec<T>::N == 8) {
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            r[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    } else {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[Vec<T>::N]) {
    *reinterpret_cast<uint4*>(p) = pack_vec<T>(f);
}

// Logistic function. expf overflows to inf for z < -88, where 1 / (1 + inf) = 0 is the
// rounded value; FAST: the hardware exponential and divide (relative error about 2^-21),
// for results that are rounded to bf16 next. __fdividef returns 0 for a divisor in
// (2^126, 2^128), which is again the rounded value here.
template <bool FAST>
__device__ __forceinline__ float logistic(float z) {
    if constexpr (FAST) return __fdividef(1.0f, 1.0f + __expf(-z));
    else return 1.0f / (1.0f + expf(-z));
}

// Phi(z) and the normal density for results that are rounded to bf16 next: Phi(-|z|) =
// erfc(|z| / sqrt 2) / 2 by Abramowitz and Stegun 7.1.26, t (a1 + ... + a5 t^4) e^(-z^2 / 2) with
// t = 1 / (1 + p |z| / sqrt 2), absolute error below 1.5e-7; the exponential is the density's.
// 23.8 -> 10 us against erfcf in the derivative pass of 4097 x 2048 (the erfcf made it
// compute bound).
__device__ __forceinline__ void normal_fast(float z, float& Phi, float& phi) {
    const float e = __expf(-0.5f * z * z);
    const float t = __fdividef(1.0f, fmaf(0.3275911f * 0.70710678f, fabsf(z), 1.0f));
    const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f),
                             0.254829592f);
    const float tail = 0.5f * p * e;
    Phi = z > 0.0f ? 1.0f - tail : tail;
    phi = 0.39894228f * e;
}

// Activation of a linear layer and its derivative.
template <bool FAST>
__device__ __forceinline__ float linear_act(int act, float z) {
    if (act == MOE_LINEAR_SILU) return z * logistic<FAST>(z);
    // z Phi(z) with Phi(z) = erfc(-z / sqrt 2) / 2, which keeps its relative precision for z << 0
    if (act == MOE_LINEAR_GELU) {
        if constexpr (FAST) {
            float Phi, phi;
            normal_fast(z, Phi, phi);
            return z * Phi;
        }
        return z * 0.5f * erfcf(-z * 0.70710678f);
    }
    return z;
}
template <bool FAST>
__device__ __forceinline__ float linear_dact(int act, float z) {
    if (act == MOE_LINEAR_SILU) {
        const float p = logistic<FAST>(z);
        return p * (1.0f + z * (1.0f - p));
    }
    if (act == MOE_LINEAR_GELU) {
        if constexpr (FAST) {
            float Phi, phi;
            normal_fast(z, Phi, phi);
            return Phi + z * phi;
        }
        return 0.5f * erfcf(-z * 0.70710678f) + z * expf(-0.5f * z * z) * 0.39894228f;
    }
    return 1.0f;
}

// min(x, top) that keeps a NaN (fminf would return top).
__device__ __forceinline__ float clamp_above(float x, float top) { return x > top ? top : x; }

// Gated activation: SwiGLU h = g p v with p = sigma(g), or the clamped form
// h = g' p (v' + 1), g' = min(g, limit), v' = clamp(v, -limit, limit), p = sigma(alpha g').
template <bool FAST>
__device__ __forceinline__ float gated_h(int act, float g, float v, float limit, float alpha) {
    if (act == MOE_ACT_SWIGLU) return g * logistic<FAST>(g) * v;
    const float gc = clamp_above(g, limit), vc = -clamp_above(-clamp_above(v, limit), limit);
    return gc * logistic<FAST>(alpha * gc) * (vc + 1.0f);
}
// ... with dh/dg and dh/dv. At the clamp's borders the derivative is that of the inside.
template <bool FAST>
__device__ __forceinline__ void gated_grad(int act, float g, float v, float limit, float alpha, float& h, float& hg,
                                           float& hv) {
    if (act == MOE_ACT_SWIGLU) {
        const float p = logistic<FAST>(g);
        const float gp = g * p;
        h = gp * v;
        hg = (p + gp * (1.0f - p)) * v;
        hv = gp;
        return;
    }
    const float gc = clamp_above(g, limit), vc = -clamp_above(-clamp_above(v, limit), limit);
    const float p = logistic<FAST>(alpha * gc);
    const float gp = gc * p, v1 = vc + 1.0f;
    h = gp * v1;
    hg = g > limit ? 0.0f : (p + alpha * gp * (1.0f - p)) * v1;
    hv = (v < -limit || v > limit) ? 0.0f : gp;
}

// Expert of padded row r: the last e with poff[e] <= r.
__device__ __forceinline__ int expert_of_row(const int32_t* poff, int E, int r) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (poff[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

}  // namespace
}  // namespace moe
