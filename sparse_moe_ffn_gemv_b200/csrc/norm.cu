// norm.cu -- layer norm and RMS norm, forward and backward.
//
//   y = xh w + b, xh = (x - mean) rstd            (RMS: mean = 0, no b)
//   dx = rstd (dy w - [mean(dy w)] - xh mean(dy w xh)),  dw = sum_t dy xh,  db = sum_t dy
//
// Statistics and sums in f32; the variance is taken about the mean in a second pass over the
// row, not as a difference of two large sums.
#include <algorithm>
#include <atomic>

#include "ptx.cuh"
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

// Sums of two values over the tpr threads of a row group (a multiple of 32), through red[warp].
// One block barrier; calls in a row alternate between two arrays.
__device__ __forceinline__ void group_sum2(float& x, float& y, int tpr, float2* red) {
    x = warp_sum(x);
    y = warp_sum(y);
    const int warp = threadIdx.x >> 5, nw = tpr >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(x, y);
    __syncthreads();
    const float2* g = red + warp / nw * nw;
    x = y = 0.f;
    for (int i = 0; i < nw; ++i) {
        x += g[i].x;
        y += g[i].y;
    }
}

// Rows of up to 4 vectors per thread, kept in registers: one read, one write. A group of tpr
// threads per row, 256 / tpr rows per block.
constexpr int kVpt = 4;
template <typename T, bool LAYER>
__global__ void __launch_bounds__(kNormThreads) norm_forward_rows_kernel(const NormArgs a, int tpr) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    __shared__ float2 red[2][kNormThreads / 32];
    const int n = a.H / V, g = threadIdx.x / tpr, c0 = threadIdx.x % tpr;
    const int64_t t = int64_t(blockIdx.x) * (kNormThreads / tpr) + g;
    const bool live = t < a.T;
    const T* x = static_cast<const T*>(a.x) + (live ? t : 0) * a.ldx;
    uint4 xv[kVpt];
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
        const int c = c0 + i * tpr;
        xv[i] = live && c < n ? ld_once16(x + c * V) : make_uint4(0, 0, 0, 0);
    }
    float mean = 0.f, s = 0.f, unused = 0.f;
    if constexpr (LAYER) {
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            float f[V];
            unpack_vec<T>(xv[i], f);
#pragma unroll
            for (int q = 0; q < V; ++q) s += f[q];
        }
        group_sum2(s, unused, tpr, red[0]);
        mean = s / float(a.H);
        s = unused = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
        if (c0 + i * tpr >= n) break;
        float f[V];
        unpack_vec<T>(xv[i], f);
#pragma unroll
        for (int q = 0; q < V; ++q) s = fmaf(f[q] - mean, f[q] - mean, s);
    }
    group_sum2(s, unused, tpr, red[1]);
    if (!live) return;
    const float rstd = 1.0f / sqrtf(s / float(a.H) + a.eps);
    T* y = static_cast<T*>(a.y) + t * a.ldy;
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
        const int c = c0 + i * tpr;
        if (c >= n) break;
        float f[V], w[V], b[V] = {};
        unpack_vec<T>(xv[i], f);
        load_vec(static_cast<const T*>(a.w) + c * V, w);
        if (LAYER && a.b) load_vec(static_cast<const T*>(a.b) + c * V, b);
#pragma unroll
        for (int q = 0; q < V; ++q) f[q] = (f[q] - mean) * rstd * w[q] + b[q];
        store_vec(y + c * V, f);
    }
    if (a.stats && c0 == 0) *reinterpret_cast<float2*>(a.stats + 2 * t) = make_float2(mean, rstd);
}

// Wider rows: read again (from L2) for each pass.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_forward_kernel(const NormArgs a) {
    pdl_begin();
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

// The thread's 16 bytes at src to its place in shared memory, asynchronously; read once.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t pol) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(pol) : "memory");
}
// Until at most n of the thread's groups of copies are under way (the instruction takes a constant).
__device__ __forceinline__ void copies_left(int n) {
    switch (n) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    }
}

// Backward for rows of up to 4 vectors per thread: one read of x and dy serves dx, dw and db.
// Two blocks per SM walk the rows; x and dy of the next rows are brought to shared memory
// meanwhile (registers hold the running column sums, so they cannot hold loads in flight as
// well). Each thread copies the vectors that it reads itself and waits for them in hardware, so
// that no wait can give up: the call has no status to say so in. Each thread keeps its columns'
// sums over all of the block's rows; the block's row groups add up in order at the end, then
// norm_finish_kernel adds the blocks.
constexpr int kNormStages = 8;
template <typename T, bool LAYER>
__global__ void __launch_bounds__(kNormThreads, 2) norm_backward_rows_kernel(const NormArgs a, int tpr, int stages) {
    constexpr int V = Vec<T>::N;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float2 red[2][kNormThreads / 32];
    const int n = a.H / V, G = kNormThreads / tpr, g = threadIdx.x / tpr, c0 = threadIdx.x % tpr;
    const uint32_t row_bytes = uint32_t(a.H) * sizeof(T);
    const uint4* sw = reinterpret_cast<const uint4*>(sm);
    uint8_t* ring = sm + (row_bytes + 127) / 128 * 128;
    const uint32_t stage_bytes = 2 * G * row_bytes;
    const int64_t groups = (a.T + G - 1) / G;
    pdl_begin();
    const uint64_t pol = policy_evict_first();
    // the thread's vectors of row group grp, one group of copies (empty past the last row)
    auto fill = [&](int64_t grp, int st) {
        const int64_t t = grp * G + g;
        if (t < a.T) {
            const uint32_t d = su32(ring + st * stage_bytes + g * 2 * row_bytes);
            const T* x = static_cast<const T*>(a.x) + t * a.ldx;
            const T* dy = static_cast<const T*>(a.dy) + t * a.lddy;
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                const int c = c0 + i * tpr;
                if (c >= n) break;
                copy16(d + c * 16, x + c * V, pol);
                copy16(d + row_bytes + c * 16, dy + c * V, pol);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < stages - 1; ++i) fill(blockIdx.x + int64_t(i) * gridDim.x, i);
    for (int c = threadIdx.x; c < n; c += kNormThreads)
        reinterpret_cast<uint4*>(sm)[c] = reinterpret_cast<const uint4*>(a.w)[c];
    __syncthreads();
    float2 aw[kVpt][V / 2], ab[kVpt][V / 2];
#pragma unroll
    for (int i = 0; i < kVpt; ++i)
#pragma unroll
        for (int q = 0; q < V / 2; ++q) aw[i][q] = ab[i][q] = make_float2(0.f, 0.f);
    int st = 0, it = 0;
    auto stats_of = [&](int64_t grp) {
        const int64_t t = grp * G + g;
        return t < a.T ? *reinterpret_cast<const float2*>(a.cstats + 2 * t) : make_float2(0.f, 0.f);
    };
    float2 ms = stats_of(blockIdx.x);
    for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x, ++it) {
        const int64_t t = grp * G + g;
        const bool live = t < a.T;
        const float mean = ms.x, rstd = ms.y;
        ms = stats_of(grp + gridDim.x);  // of the next row, while this one is worked on
        copies_left(stages - 2);
        const uint4* sx = reinterpret_cast<const uint4*>(ring + st * stage_bytes + g * 2 * row_bytes);
        const uint4* sd = reinterpret_cast<const uint4*>(ring + st * stage_bytes + g * 2 * row_bytes + row_bytes);
        float2 t1 = make_float2(0.f, 0.f), t2 = t1;  // sums of dy w and dy w (x - mean)
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int c = c0 + i * tpr;
            if (!live || c >= n) break;
            float f[V], d[V], w[V];
            unpack_vec<T>(sx[c], f);
            unpack_vec<T>(sd[c], d);
            unpack_vec<T>(sw[c], w);
#pragma unroll
            for (int q = 0; q < V; q += 2) {
                const float2 x2 = add2(make_float2(f[q], f[q + 1]), make_float2(-mean, -mean));
                const float2 d2 = make_float2(d[q], d[q + 1]);
                const float2 g2 = mul2(d2, make_float2(w[q], w[q + 1]));
                aw[i][q / 2] = fma2(mul2(d2, make_float2(rstd, rstd)), x2, aw[i][q / 2]);
                if (LAYER) {
                    ab[i][q / 2] = add2(ab[i][q / 2], d2);
                    t1 = add2(t1, g2);
                }
                t2 = fma2(g2, x2, t2);
            }
        }
        float s1 = t1.x + t1.y, s2 = (t2.x + t2.y) * rstd;
        group_sum2(s1, s2, tpr, red[it & 1]);
        // every thread is done with the rows before these: bring that stage's next rows
        fill(grp + int64_t(stages - 1) * gridDim.x, st == 0 ? stages - 1 : st - 1);
        if (++st == stages) st = 0;
        if (!live || !a.dx) continue;
        // dx = rstd g - rstd mean(g) - (x - mean) rstd^2 mean(g xh)
        const float k1 = -rstd * (s1 / float(a.H)), k2 = -rstd * rstd * (s2 / float(a.H));
        T* dx = static_cast<T*>(a.dx) + t * a.lddx;
#pragma unroll
        for (int i = 0; i < kVpt; ++i) {
            const int c = c0 + i * tpr;
            if (c >= n) break;
            float f[V], d[V], w[V];
            unpack_vec<T>(sx[c], f);
            unpack_vec<T>(sd[c], d);
            unpack_vec<T>(sw[c], w);
#pragma unroll
            for (int q = 0; q < V; q += 2) {
                const float2 x2 = add2(make_float2(f[q], f[q + 1]), make_float2(-mean, -mean));
                const float2 g2 = mul2(make_float2(d[q], d[q + 1]), make_float2(w[q], w[q + 1]));
                const float2 o = fma2(x2, make_float2(k2, k2), fma2(g2, make_float2(rstd, rstd), make_float2(k1, k1)));
                f[q] = o.x;
                f[q + 1] = o.y;
            }
            store_vec(dx + c * V, f);
        }
    }
    if (!a.partial) return;
    // the row groups' sums, one group after the other (the ring is free: the copies still under way are empty)
    __syncthreads();
    float* acc = reinterpret_cast<float*>(ring);
    for (int j = 0; j < G; ++j) {
        if (g == j) {
#pragma unroll
            for (int i = 0; i < kVpt; ++i) {
                const int c = c0 + i * tpr;
                if (c >= n) break;
#pragma unroll
                for (int q = 0; q < V / 2; ++q) {
                    float2* pw = reinterpret_cast<float2*>(acc + c * V + 2 * q);
                    float2* pb = reinterpret_cast<float2*>(acc + a.H + c * V + 2 * q);
                    *pw = j ? add2(*pw, aw[i][q]) : aw[i][q];
                    if (LAYER) *pb = j ? add2(*pb, ab[i][q]) : ab[i][q];
                }
            }
        }
        __syncthreads();
    }
    float* o = a.partial + int64_t(blockIdx.x) * 2 * a.H;
    for (int c = threadIdx.x; c < (LAYER ? 2 : 1) * a.H; c += kNormThreads) o[c] = acc[c];
}

// Wider rows.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_dx_kernel(const NormArgs a) {
    pdl_begin();
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
    pdl_begin();
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

// The blocks' partial sums: 32 columns per block, 8 threads per column each adding every 8th
// part, then those 8 in order; rounded once.
template <typename T>
__global__ void __launch_bounds__(256) norm_finish_kernel(const NormArgs a, int parts) {
    __shared__ float sm[8][33];
    pdl_begin();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    T* o = static_cast<T*>(blockIdx.y ? a.db : a.dw);
    if (!o) return;
    float s = 0.f;
    if (c < a.H)
#pragma unroll 8
        for (int p = y; p < parts; p += 8) s += a.partial[(int64_t(p) * 2 + blockIdx.y) * a.H + c];
    sm[y][x] = s;
    __syncthreads();
    if (y != 0 || c >= a.H) return;
    s = sm[0][x];
#pragma unroll
    for (int j = 1; j < 8; ++j) s += sm[j][x];
    o[c] = from_f<T>(s);
}

// Threads per row that hold it in registers, or 0 for wider rows.
int threads_per_row(int H, int V) {
    for (int tpr = 32; tpr <= kNormThreads; tpr *= 2)
        if (H / V <= tpr * kVpt) return tpr;
    return 0;
}

// Shared memory of the backward kernel: w, then as many stages as fit about 100 KB (two blocks
// per SM), which the final sums (2 H floats) reuse.
struct NormRing {
    int stages, bytes;
};
NormRing norm_ring(int H, int es, int tpr) {
    const int row = H * es, w = (row + 127) / 128 * 128, stage = 2 * (kNormThreads / tpr) * row;
    NormRing r;
    r.stages = std::max(2, std::min(kNormStages, (100 * 1024 - w) / stage));
    r.bytes = w + std::max(r.stages * stage, 2 * H * 4);
    return r;
}

int backward_parts(int64_t T, int H, int V, bool* rows) {
    const int tpr = threads_per_row(H, V);
    *rows = tpr > 0;
    if (tpr) return int(std::min<int64_t>((T + kNormThreads / tpr - 1) / (kNormThreads / tpr), 2 * 148));
    const int64_t cb = (H + 511) / 512;
    return int(std::max<int64_t>(1, std::min<int64_t>(std::max<int64_t>(1, 592 / cb), T / 16)));
}

template <typename T, bool LAYER>
cudaError_t backward_rows(const NormArgs& a, int parts, cudaStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    const int tpr = threads_per_row(a.H, Vec<T>::N);
    const NormRing ring = norm_ring(a.H, sizeof(T), tpr);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(allowed.load() & bit)) {
        e = cudaFuncSetAttribute(norm_backward_rows_kernel<T, LAYER>, cudaFuncAttributeMaxDynamicSharedMemorySize, 112 * 1024);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit);
    }
    return launch_chained(norm_backward_rows_kernel<T, LAYER>, parts, kNormThreads, ring.bytes, s, a, tpr, ring.stages);
}

template <typename T>
cudaError_t backward_t(NormArgs a, cudaStream_t s) {
    constexpr int V = Vec<T>::N;
    bool rows;
    const int parts = backward_parts(a.T, a.H, V, &rows);
    const bool sums = a.dw || a.db;
    if (!sums) a.partial = nullptr;
    if (!sums && !a.dx) return cudaSuccess;
    if (rows) {
        const cudaError_t e = a.kind == MOE_NORM_LAYER ? backward_rows<T, true>(a, parts, s) : backward_rows<T, false>(a, parts, s);
        if (e != cudaSuccess) return e;
    } else {
        if (a.dx) MOE_LAUNCH(launch_chained(norm_dx_kernel<T>, unsigned(std::min<int64_t>(a.T, 148 * 8)), kNormThreads, 0, s, a));
        if (sums) MOE_LAUNCH(launch_chained(norm_dw_kernel<T>, dim3((a.H / V + kColVecs - 1) / kColVecs, parts), kColVecs * kColRows, 0, s, a));
    }
    if (sums) MOE_LAUNCH(launch_chained(norm_finish_kernel<T>, dim3((a.H + 31) / 32, a.db ? 2 : 1), 256, 0, s, a, parts));
    return cudaSuccess;
}

template <typename T>
cudaError_t forward_t(const NormArgs& a, cudaStream_t s) {
    const int tpr = threads_per_row(a.H, Vec<T>::N);
    if (!tpr) {
        return launch_chained(norm_forward_kernel<T>, unsigned(std::min<int64_t>(a.T, 148 * 8)), kNormThreads, 0, s, a);
    }
    const unsigned grid = unsigned((a.T + kNormThreads / tpr - 1) / (kNormThreads / tpr));
    if (a.kind == MOE_NORM_LAYER) return launch_chained(norm_forward_rows_kernel<T, true>, grid, kNormThreads, 0, s, a, tpr);
    return launch_chained(norm_forward_rows_kernel<T, false>, grid, kNormThreads, 0, s, a, tpr);
}

}  // namespace

int norm_blocks(int64_t T, int H, int dtype) {
    bool rows;
    return backward_parts(T, H, dtype == MOE_DTYPE_F32 ? 4 : 8, &rows);
}

cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s) {
    return a.dtype == MOE_DTYPE_F32 ? forward_t<float>(a, s) : forward_t<__nv_bfloat16>(a, s);
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t s) {
    return a.dtype == MOE_DTYPE_F32 ? backward_t<float>(a, s) : backward_t<__nv_bfloat16>(a, s);
}

}  // namespace moe
