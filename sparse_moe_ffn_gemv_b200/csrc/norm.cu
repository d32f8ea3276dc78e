// norm.cu -- layer norm and RMS norm, forward and backward.
//
//   y = xh w + b, xh = (x - mean) rstd            (RMS: mean = 0, no b)
//   dx = rstd (dy w - [mean(dy w)] - xh mean(dy w xh)),  dw = sum_t dy xh,  db = sum_t dy
//
// Statistics and sums in f32; the variance is taken about the mean in a second pass over the
// row, not as a difference of two large sums.
#include <algorithm>

#include "train_dev.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* sm) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) s += sm[i];
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_forward_kernel(const NormArgs a) {
    constexpr int V = Vec<T>::N;
    __shared__ float sm[kNormThreads / 32];
    const int n = a.H / V;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + t * a.ldx;
        float mean = 0.f;
        if (a.kind == MOE_NORM_LAYER) {
            float s = 0.f;
            for (int c = threadIdx.x; c < n; c += kNormThreads) {
                float f[V];
                load_vec(x + c * V, f);
#pragma unroll
                for (int q = 0; q < V; ++q) s += f[q];
            }
            mean = block_sum(s, sm) / float(a.H);
        }
        float s = 0.f;
        for (int c = threadIdx.x; c < n; c += kNormThreads) {
            float f[V];
            load_vec(x + c * V, f);
#pragma unroll
            for (int q = 0; q < V; ++q) s += (f[q] - mean) * (f[q] - mean);
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, sm) / float(a.H) + a.eps);
        T* y = static_cast<T*>(a.y) + t * a.ldy;
        for (int c = threadIdx.x; c < n; c += kNormThreads) {
            float f[V], w[V], b[V] = {};
            load_vec(x + c * V, f);
            load_vec(static_cast<const T*>(a.w) + c * V, w);
            if (a.b) load_vec(static_cast<const T*>(a.b) + c * V, b);
#pragma unroll
            for (int q = 0; q < V; ++q) f[q] = (f[q] - mean) * rstd * w[q] + b[q];
            store_vec(y + c * V, f);
        }
        if (a.stats && threadIdx.x == 0) {
            a.stats[2 * t] = mean;
            a.stats[2 * t + 1] = rstd;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_dx_kernel(const NormArgs a) {
    constexpr int V = Vec<T>::N;
    __shared__ float sm[kNormThreads / 32];
    const int n = a.H / V;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + t * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + t * a.lddy;
        const float mean = a.cstats[2 * t], rstd = a.cstats[2 * t + 1];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < n; c += kNormThreads) {
            float f[V], g[V], w[V];
            load_vec(x + c * V, f);
            load_vec(dy + c * V, g);
            load_vec(static_cast<const T*>(a.w) + c * V, w);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                s1 += g[q] * w[q];
                s2 += g[q] * w[q] * ((f[q] - mean) * rstd);
            }
        }
        s1 = a.kind == MOE_NORM_LAYER ? block_sum(s1, sm) / float(a.H) : 0.f;
        s2 = block_sum(s2, sm) / float(a.H);
        T* dx = static_cast<T*>(a.dx) + t * a.lddx;
        for (int c = threadIdx.x; c < n; c += kNormThreads) {
            float f[V], g[V], w[V];
            load_vec(x + c * V, f);
            load_vec(dy + c * V, g);
            load_vec(static_cast<const T*>(a.w) + c * V, w);
#pragma unroll
            for (int q = 0; q < V; ++q) f[q] = rstd * (g[q] * w[q] - s1 - (f[q] - mean) * rstd * s2);
            store_vec(dx + c * V, f);
        }
    }
}

// Column sums of dy xh and dy over a block of rows (blockIdx.y), 64 vectors of columns x 4 rows.
constexpr int kColVecs = 64, kColRows = 4;
template <typename T>
__global__ void __launch_bounds__(kColVecs * kColRows) norm_dw_kernel(const NormArgs a) {
    constexpr int V = Vec<T>::N;
    const int c = (blockIdx.x * kColVecs + threadIdx.x % kColVecs) * V;
    const int ry = threadIdx.x / kColVecs;
    const int64_t per = (a.T + gridDim.y - 1) / gridDim.y;
    const int64_t b = blockIdx.y * per, end = min(a.T, b + per);
    float aw[V] = {}, ab[V] = {};
    if (c < a.H) {
        for (int64_t t = b + ry; t < end; t += kColRows) {
            float f[V], g[V];
            load_vec(static_cast<const T*>(a.x) + t * a.ldx + c, f);
            load_vec(static_cast<const T*>(a.dy) + t * a.lddy + c, g);
            const float mean = a.cstats[2 * t], rstd = a.cstats[2 * t + 1];
#pragma unroll
            for (int q = 0; q < V; ++q) {
                aw[q] += g[q] * ((f[q] - mean) * rstd);
                ab[q] += g[q];
            }
        }
    }
    __shared__ float sm[2][kColRows][kColVecs][V + 1];
#pragma unroll
    for (int q = 0; q < V; ++q) {
        sm[0][ry][threadIdx.x % kColVecs][q] = aw[q];
        sm[1][ry][threadIdx.x % kColVecs][q] = ab[q];
    }
    __syncthreads();
    if (ry < 2 && c < a.H) {
        float* o = a.partial + (int64_t(blockIdx.y) * 2 + ry) * a.H + c;
#pragma unroll
        for (int q = 0; q < V; ++q) {
            float s = 0.f;
#pragma unroll
            for (int y = 0; y < kColRows; ++y) s += sm[ry][y][threadIdx.x % kColVecs][q];
            o[q] = s;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) norm_finish_kernel(const NormArgs a, int parts) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= 2 * a.H) return;
    const int which = i / a.H, c = i - which * a.H;
    T* o = static_cast<T*>(which ? a.db : a.dw);
    if (!o) return;
    float s = 0.f;
    for (int p = 0; p < parts; ++p) s += a.partial[(int64_t(p) * 2 + which) * a.H + c];
    o[c] = from_f<T>(s);
}

template <typename T>
cudaError_t backward_t(const NormArgs& a, cudaStream_t s) {
    constexpr int V = Vec<T>::N;
    if (a.dx) norm_dx_kernel<T><<<unsigned(std::min<int64_t>(a.T, 148 * 8)), kNormThreads, 0, s>>>(a);
    if (a.dw || a.db) {
        const int parts = norm_blocks(a.T, a.H);
        const dim3 grid((a.H / V + kColVecs - 1) / kColVecs, parts);
        norm_dw_kernel<T><<<grid, kColVecs * kColRows, 0, s>>>(a);
        norm_finish_kernel<T><<<(2 * a.H + 255) / 256, 256, 0, s>>>(a, parts);
    }
    return cudaGetLastError();
}

}  // namespace

int norm_blocks(int64_t T, int H) {
    const int64_t cb = (H + 511) / 512;
    return int(std::max<int64_t>(1, std::min<int64_t>(std::max<int64_t>(1, 592 / cb), T / 16)));
}

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s) {
    const unsigned grid = unsigned(std::min<int64_t>(a.T, 148 * 8));
    if (a.dtype == MOE_DTYPE_F32) norm_forward_kernel<float><<<grid, kNormThreads, 0, s>>>(a);
    else norm_forward_kernel<__nv_bfloat16><<<grid, kNormThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t s) {
    return a.dtype == MOE_DTYPE_F32 ? backward_t<float>(a, s) : backward_t<__nv_bfloat16>(a, s);
}

}  // namespace moe
