// train_small.cu -- linear and gated products for a handful of tokens (serving single tokens):
// the weights stream through once, on the CUDA cores.
//
//   y[t, n] = act(sum_c x[t, c] W[n, c] + b[n]) + r[t, n]
//   h[t, i] = gated(sum_c x[t, c] Wg[i, c] + bg[i], sum_c x[t, c] Wv[i, c] + bv[i])
//
// Bound by HBM on the weights, in practice by how soon enough of them are in flight: a warp
// takes R rows (gated: the gate and up row of one unit) and issues U 16-byte loads per row and
// lane before it uses the first; where there are few rows, several warps of a block share a
// row's columns and add up through shared memory in warp order.
#include <algorithm>

#include "train_dev.cuh"

namespace moe {

namespace {

constexpr int kSmallThreads = 256;

// Vectors of up to U rounds of a row: lane's columns (w * 32 + lane) + 32 * ks * round.
// A full SM of warps with few loads each beats half of one with many for the linear form (3584 x
// 7168, weights cold: one token 14.3 -> 12.6 us, two 18.0 -> 14.4), not for the gated one (7168 x
// 2048: 30.4 us with 8 loads per row, 35.2 with 2).
template <typename T, int TT, bool GATED>
__global__ void __launch_bounds__(kSmallThreads, GATED ? 1 : TT <= 2 ? 8 : 4) small_kernel(const SmallArgs a) {
    constexpr int V = Vec<T>::N;
    constexpr bool FAST = V == 8;
    constexpr int R = GATED ? 2 : (TT <= 2 ? 1 : 2), U = GATED ? 8 / TT : TT == 1 ? 4 : 2;
    __shared__ float part[8][TT * R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ks = a.ks;                     // warps per row group
    const int group = blockIdx.x * (8 / ks) + warp / ks, kw = warp % ks;
    const int n0 = GATED ? group : group * R;
    const int vecs = a.K / V, step = 32 * ks;
    const T* w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        int64_t row;
        const void* base = a.w;
        if (GATED) {
            row = a.interleaved ? 2 * int64_t(n0) + r : n0;
            if (!a.interleaved && r == 1) base = a.w1;
            if (n0 >= a.N) row = 0;
        } else {
            row = min(n0 + r, a.N - 1);
        }
        w[r] = static_cast<const T*>(base) + row * a.K;
    }
    float acc[TT][R] = {};
    const bool live = n0 < a.N;
    launch_next();
    if (a.prefetch && live)  // the first weights come under way while the launch before ends
        for (int c = kw * 32 + lane; c < min(vecs, 2 * U * step); c += step)
#pragma unroll
            for (int r = 0; r < R; ++r) asm volatile("prefetch.global.L2 [%0];" ::"l"(w[r] + int64_t(c) * V));
    wait_before();
    if (live) {
        for (int c0 = kw * 32 + lane; c0 < vecs; c0 += U * step) {
            uint4 wv[U][R];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    wv[u][r] = c0 + u * step < vecs ? ld_once16(w[r] + int64_t(c0 + u * step) * V) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + u * step >= vecs) break;
                float wf[R][V];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if constexpr (V == 8) {
                        unpack8(wv[u][r], wf[r]);
                    } else {
                        wf[r][0] = __uint_as_float(wv[u][r].x); wf[r][1] = __uint_as_float(wv[u][r].y);
                        wf[r][2] = __uint_as_float(wv[u][r].z); wf[r][3] = __uint_as_float(wv[u][r].w);
                    }
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (t >= a.T) break;
                    float xf[V];
                    load_vec(static_cast<const T*>(a.x) + t * a.ldx + int64_t(c0 + u * step) * V, xf);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int q = 0; q < V; ++q) acc[t][r] = fmaf(xf[q], wf[r][q], acc[t][r]);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[t][r] = warp_sum(acc[t][r]);
    if (ks > 1) {
        if (lane == 0)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int r = 0; r < R; ++r) part[warp][t * R + r] = acc[t][r];
        __syncthreads();
        if (kw != 0) return;
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float s = part[warp][t * R + r];
                for (int i = 1; i < ks; ++i) s += part[warp + i][t * R + r];
                acc[t][r] = s;
            }
    }
    if (!live) return;
    // lane t (t * R + r) finishes token t (row r)
    if constexpr (GATED) {
        float g = 0.f, v = 0.f;
#pragma unroll
        for (int t = 0; t < TT; ++t)
            if (lane == t) {
                g = acc[t][0];
                v = acc[t][1];
            }
        if (lane >= min(TT, a.T)) return;
        const T *b0 = static_cast<const T*>(a.bias), *b1 = static_cast<const T*>(a.bias1);
        if (b0) {
            g += to_f<T>(a.interleaved ? b0[2 * n0] : b0[n0]);
            v += to_f<T>(a.interleaved ? b0[2 * n0 + 1] : b1[n0]);
        }
        if (a.pre) {
            T* p = static_cast<T*>(a.pre) + int64_t(lane) * 2 * a.N;
            p[a.interleaved ? 2 * n0 : n0] = from_f<T>(g);
            p[a.interleaved ? 2 * n0 + 1 : a.N + n0] = from_f<T>(v);
        }
        static_cast<T*>(a.y)[lane * a.ldy + n0] = from_f<T>(gated_h<FAST>(a.act, g, v, a.limit, a.alpha));
    } else {
        float z = 0.f;
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (lane == t * R + r) z = acc[t][r];
        const int t = lane / R, n = n0 + lane % R;
        if (t >= min(TT, a.T) || n >= a.N) return;
        if (a.bias) z += to_f<T>(static_cast<const T*>(a.bias)[n]);
        if (a.pre) static_cast<T*>(a.pre)[int64_t(t) * a.N + n] = from_f<T>(z);
        z = linear_act<FAST>(a.act, z);
        if (a.residual) z += to_f<T>(static_cast<const T*>(a.residual)[t * a.ldr + n]);
        static_cast<T*>(a.y)[t * a.ldy + n] = from_f<T>(z);
    }
}

template <typename T, int TT, bool GATED>
cudaError_t launch_tt(SmallArgs a, cudaStream_t s) {
    constexpr int R = GATED ? 1 : (TT <= 2 ? 1 : 2);  // outputs per warp group
    const int groups = (a.N + R - 1) / R, vecs = a.K / Vec<T>::N;
    // warps per row: until the launch has 8 warps for every SM sub-partition or the lanes run
    // out of columns
    a.ks = 1;
    while (a.ks < 8 && int64_t(groups) * a.ks < 148 * 32 && vecs >= 64 * a.ks) a.ks *= 2;
    const int per = 8 / a.ks;
    return launch_chained(small_kernel<T, TT, GATED>, dim3((groups + per - 1) / per), dim3(kSmallThreads), 0, s, a);
}

template <typename T, bool GATED>
cudaError_t launch_t(const SmallArgs& a, cudaStream_t s) {
    if (a.T == 1) return launch_tt<T, 1, GATED>(a, s);
    if (a.T == 2) return launch_tt<T, 2, GATED>(a, s);
    return launch_tt<T, kSmallT, GATED>(a, s);
}

}  // namespace

cudaError_t launch_small(const SmallArgs& a, cudaStream_t s) {
    if (a.dtype == MOE_DTYPE_F32) return a.gated ? launch_t<float, true>(a, s) : launch_t<float, false>(a, s);
    return a.gated ? launch_t<__nv_bfloat16, true>(a, s) : launch_t<__nv_bfloat16, false>(a, s);
}

}  // namespace moe
