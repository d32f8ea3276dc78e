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
// (2^126, 2^128), that is for z < -87.3, where the value is below 2^-125.
template <bool FAST>
__device__ __forceinline__ float logistic(float z) {
    if constexpr (FAST) return __fdividef(1.0f, 1.0f + __expf(-z));
    else return 1.0f / (1.0f + expf(-z));
}

// Phi(z) and the normal density for results that are rounded to bf16 next: Phi(-|z|) = t Q(t)
// e^(-z^2 / 2) with t = 1 / (1 + p |z|), the exponential being the density's. Q is fitted to
// erfcx(|z| / sqrt 2) / (2 t) over |z| <= 13.3, where e^(-z^2 / 2) leaves the f32 range (weighted least
// squares on Chebyshev nodes, the weights raised where the relative error is largest, p chosen for
// the smallest): relative error below 2^-20 in f32, so that a small Phi is right to bf16 too.
// erfcf here made the derivative pass of 4097 x 2048 compute bound (23.8 us against 15.2).
__device__ __forceinline__ void normal_fast(float z, float& Phi, float& phi) {
    const float e = __expf(-0.5f * z * z);
    const float t = __fdividef(1.0f, fmaf(0.2625f, fabsf(z), 1.0f));
    float q = fmaf(t, -0.0706492872f, 0.212851164f);
    q = fmaf(t, q, -0.087404421f);
    q = fmaf(t, q, 0.15532532f);
    q = fmaf(t, q, 0.0777212643f);
    q = fmaf(t, q, 0.107607208f);
    q = fmaf(t, q, 0.104548969f);
    const float tail = t * q * e;
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

// Two f32 operations per instruction (sm_100), for the passes that are bound by issue slots as
// much as by HBM.
__device__ __forceinline__ uint64_t bits2(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 pair2(uint64_t a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return pair2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}

// The hardware's exponential (base 2) and reciprocal: relative errors about 2^-22 and 2^-23.
__device__ __forceinline__ float ex2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// min and max that keep a NaN (fminf and fmaxf return the other operand).
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// 1 / (1 + 2^(c z)) for two values, c = -alpha log2(e).
__device__ __forceinline__ float2 logistic2(float2 z, float c) {
    const float2 x = mul2(z, make_float2(c, c));
    const float2 q = add2(make_float2(ex2_fast(x.x), ex2_fast(x.y)), make_float2(1.0f, 1.0f));
    return make_float2(rcp_fast(q.x), rcp_fast(q.y));
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
// ... with dh/dg and dh/dv, in full f32. At the clamp's borders the derivative is that of the inside.
__device__ __forceinline__ void gated_grad(int act, float g, float v, float limit, float alpha, float& h, float& hg,
                                           float& hv) {
    if (act == MOE_ACT_SWIGLU) {
        const float p = logistic<false>(g);
        const float gp = g * p;
        h = gp * v;
        hg = (p + gp * (1.0f - p)) * v;
        hv = gp;
        return;
    }
    const float gc = clamp_above(g, limit), vc = -clamp_above(-clamp_above(v, limit), limit);
    const float p = logistic<false>(alpha * gc);
    const float gp = gc * p, v1 = vc + 1.0f;
    h = gp * v1;
    hg = g > limit ? 0.0f : (p + alpha * gp * (1.0f - p)) * v1;
    hv = (v < -limit || v > limit) ? 0.0f : gp;
}

// gated_grad for two units at once, for results that are rounded to bf16 next (one call per unit
// with the activation chosen inside took 55 issue slots per unit, this about 15; the epilogue
// that calls it was longer than its product). cexp = -log2(e), or -alpha log2(e) clamped.
template <bool CLAMPED>
__device__ __forceinline__ void gated_grad2(float2 g, float2 v, float limit, float alpha, float cexp, float2& h, float2& hg,
                                            float2& hv) {
    float2 gc = g, v1 = v;
    if constexpr (CLAMPED) {
        gc = make_float2(min_nan(g.x, limit), min_nan(g.y, limit));
        v1 = add2(make_float2(max_nan(min_nan(v.x, limit), -limit), max_nan(min_nan(v.y, limit), -limit)),
                  make_float2(1.0f, 1.0f));
    }
    const float2 p = logistic2(gc, cexp);
    const float2 gp = mul2(gc, p);
    // p + alpha gp (1 - p)
    const float2 w = fma2(make_float2(-gp.x, -gp.y), p, gp);
    float2 t = CLAMPED ? fma2(w, make_float2(alpha, alpha), p) : add2(w, p);
    h = mul2(gp, v1);
    hg = mul2(t, v1);
    hv = gp;
    if constexpr (CLAMPED) {
        if (g.x > limit) hg.x = 0.0f;
        if (g.y > limit) hg.y = 0.0f;
        if (fabsf(v.x) > limit) hv.x = 0.0f;
        if (fabsf(v.y) > limit) hv.y = 0.0f;
    }
}
template <bool CLAMPED>
__device__ __forceinline__ float2 gated_h2(float2 g, float2 v, float limit, float cexp) {
    if constexpr (CLAMPED) {
        g = make_float2(min_nan(g.x, limit), min_nan(g.y, limit));
        v = add2(make_float2(max_nan(min_nan(v.x, limit), -limit), max_nan(min_nan(v.y, limit), -limit)),
                 make_float2(1.0f, 1.0f));
    }
    return mul2(mul2(g, logistic2(g, cexp)), v);
}

// Programmatic launch. Every kernel of the training operators lets the next launch on its stream
// start when its blocks leave, and itself waits for the launch before it to complete, with its
// memory visible, before it touches memory: what precedes the wait (barriers, TMEM, bringing
// weights into L2) runs in the other's tail. Every block waits, so that a launch's completion
// implies that of all before it. What it gives: 8192 tokens 7168 -> 3584 351 -> 337 us, dense gated
// backward (8192 x 7168 x 2048) 1227 -> 1190, one token 3584 -> 7168 12.3 -> 11.6, RMS norm 8192 x 3584
// 24.5 -> 23.0.
//
// Launches that follow a long tail and spread over the GPU by themselves stay plain: their blocks
// would crowd on the first SMs that are free (behind an expert product dtopk_kernel's 128 blocks took
// 23 us in place of 8.7, sum_slots_kernel's 2368 took 67 in place of 57; behind the plan
// copy_tokens_kernel took 83 in place of 68).
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Loads are plain, never .nc: what they read may be written while the kernel is already there.
__device__ __forceinline__ uint4 ld_once16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}

// The launches return their own error and leave none behind; what starts several returns the first
// (a launch that fails and one after it that does not is an error too).
#define MOE_LAUNCH(expr)                         \
    do {                                         \
        const cudaError_t e_ = (expr);           \
        if (e_ != cudaSuccess) return e_;        \
    } while (0)
template <typename... P, typename... A>
[[nodiscard]] cudaError_t launch_chained(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, P(args)...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}
// The same where the grid is small, else plain.
template <typename... P, typename... A>
[[nodiscard]] cudaError_t launch_spread(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
    if (int64_t(grid.x) * grid.y <= 64) return launch_chained(kern, grid, block, 0, s, args...);
    kern<<<grid, block, 0, s>>>(args...);
    return cudaGetLastError();
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
