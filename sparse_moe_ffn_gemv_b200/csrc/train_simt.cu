// train_simt.cu -- matrix products on the CUDA cores, for f32 operands (the tensor cores have
// no 32-bit product) in every operand order the training operators need.
//
// 64 x 64 outputs per block, 16 reduction steps per shared-memory stage, a 4 x 4 register tile
// per thread; the next stage's operands are loaded into registers while the current one is
// multiplied. The tile is small because f32 blocks are small (a launch of few tiles leaves
// SMs idle sooner than it meets the FMA rate).
#include <algorithm>

#include "train_dev.cuh"

namespace moe {

namespace {

constexpr int kBM = 64, kBN = 64, kBR = 16, kThreads = 256;

// One operand tile [64 rows (m or n)][16 r] as 4 values per thread. RMAJOR: memory rows are
// reduction indices (element (i, r) at p[r * ld + i]), else (i, r) at p[i * ld + r].
template <typename T, bool RMAJOR>
__device__ __forceinline__ void fetch(float (&v)[4], const T* p, int64_t ld, int64_t i0, int64_t ni, int64_t r0,
                                      int64_t r1) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int idx = threadIdx.x + q * kThreads;
        const int i = RMAJOR ? idx % 64 : idx / kBR, r = RMAJOR ? idx / 64 : idx % kBR;
        const int64_t gi = i0 + i, gr = r0 + r;
        v[q] = gi < ni && gr < r1 ? to_f<T>(p[RMAJOR ? gr * ld + gi : gi * ld + gr]) : 0.0f;
    }
}
template <bool RMAJOR>
__device__ __forceinline__ void stash(float (&sm)[kBR][64 + 4], const float (&v)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int idx = threadIdx.x + q * kThreads;
        const int i = RMAJOR ? idx % 64 : idx / kBR, r = RMAJOR ? idx / 64 : idx % kBR;
        sm[r][i] = v[q];
    }
}

struct Shared {
    float a[kBR][kBM + 4], b[kBR][kBN + 4];
};

template <int KIND>
__device__ void simt_tile(const GemmArgs& a, int64_t m0, int64_t n0, int z, Shared& sh) {
    using T = float;
    constexpr bool AR = KIND == kTN, BR = KIND != kNT;  // operand rows are reduction indices
    auto& sa = sh.a;
    auto& sb = sh.b;
    const RowPlan& p = a.plan;
    const bool grouped = p.offsets != nullptr;
    int e = 0;
    int64_t M = a.M, r0 = 0, R = a.R;
    if (KIND == kTN) {
        e = z;
        if (grouped) {
            r0 = p.poff[e];
            R = r0 + (p.uoff[e + 1] - p.uoff[e]);
        }
    } else if (grouped) {
        M = p.poff[p.E];
        if (m0 >= M) return;
        e = expert_of_row(p.poff, p.E, int(m0));
    }
    const T* A = static_cast<const T*>(a.a);
    const T* B = static_cast<const T*>(a.b) + int64_t(e) * (KIND == kTN ? 0 : a.sb);
    const T* B1 = a.b1 ? static_cast<const T*>(a.b1) + int64_t(e) * a.sb : nullptr;
    // operand B's pointer and index shift for reduction step r (kNN split) / column n (kNT split):
    // splits are multiples of the tile only by chance, so the choice is made per element
    float va[4], vb[4], acc[4][4] = {};
    auto fetch_b = [&](int64_t r) {
        if (KIND == kNN && a.split) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int idx = threadIdx.x + q * kThreads;
                const int64_t gi = n0 + idx % 64, gr = r + idx / 64;
                vb[q] = 0.f;
                if (gi < a.N && gr < R) vb[q] = to_f<T>(gr < a.split ? B[gr * a.ldb + gi] : B1[(gr - a.split) * a.ldb + gi]);
            }
        } else if (KIND == kNT && a.split) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int idx = threadIdx.x + q * kThreads;
                const int64_t gi = n0 + idx / kBR, gr = r + idx % kBR;
                vb[q] = 0.f;
                if (gi < a.N && gr < R) vb[q] = to_f<T>(gi < a.split ? B[gi * a.ldb + gr] : B1[(gi - a.split) * a.ldb + gr]);
            }
        } else {
            fetch<T, BR>(vb, B, a.ldb, n0, a.N, r, R);
        }
    };
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    if (r0 < R) {
        fetch<T, AR>(va, A, a.lda, m0, M, r0, R);
        fetch_b(r0);
    }
    for (int64_t r = r0; r < R; r += kBR) {
        stash<AR>(sa, va);
        stash<BR>(sb, vb);
        __syncthreads();
        if (r + kBR < R) {
            fetch<T, AR>(va, A, a.lda, m0, M, r + kBR, R);
            fetch_b(r + kBR);
        }
#pragma unroll
        for (int q = 0; q < kBR; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(&sa[q][ty * 4]);
            const float4 y = *reinterpret_cast<const float4*>(&sb[q][tx * 4]);
            const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= M) continue;
        float rs = 1.0f;
        if (KIND != kTN && a.row_scale) {
            const int slot = p.row_slot[m];
            rs = slot < 0 ? 0.0f : a.row_scale[slot];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx * 4 + j;
            if (n >= a.N) continue;
            float z = acc[i][j];
            if (KIND == kTN) {
                T* o = a.split && m >= a.split ? static_cast<T*>(a.out1) + int64_t(e) * a.so + (m - a.split) * a.ldo
                                               : static_cast<T*>(a.out) + int64_t(e) * a.so + m * a.ldo;
                o[n] = from_f<T>(z);
                continue;
            }
            if (a.bias)
                z += a.split && n >= a.split ? to_f<T>(static_cast<const T*>(a.bias1)[int64_t(e) * a.sbias + n - a.split])
                                             : to_f<T>(static_cast<const T*>(a.bias)[int64_t(e) * a.sbias + n]);
            if (a.pre) static_cast<T*>(a.pre)[m * a.ldp + n] = from_f<T>(z);
            z = linear_act<false>(a.act, z) * rs;
            if (a.residual) z += to_f<T>(static_cast<const T*>(a.residual)[m * a.ldr + n]);
            static_cast<T*>(a.out)[m * a.ldo + n] = z;
        }
    }
}

struct Simt {
    GemmArgs p[kMaxSimt];
    int64_t end[kMaxSimt];  // first tile after problem i
    int tx[kMaxSimt], ty[kMaxSimt];
    int n;
};

__global__ void __launch_bounds__(kThreads) simt_gemm_kernel(const __grid_constant__ Simt S) {
    __shared__ Shared sh;
    int64_t t = blockIdx.x;
    int i = 0;
    while (i < S.n - 1 && t >= S.end[i]) ++i;
    if (i > 0) t -= S.end[i - 1];
    // row tiles fastest: neighbouring blocks share operand B
    const int64_t mt = t % S.tx[i], r = t / S.tx[i];
    const int nt = int(r % S.ty[i]), z = int(r / S.ty[i]);
    const GemmArgs& a = S.p[i];
    if (a.kind == kNT) simt_tile<kNT>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
    else if (a.kind == kNN) simt_tile<kNN>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
    else simt_tile<kTN>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
}

}  // namespace

cudaError_t launch_simt_gemm(const GemmArgs* a, int n, cudaStream_t s) {
    Simt S;
    S.n = n;
    int64_t tiles = 0;
    for (int i = 0; i < n; ++i) {
        const bool grouped = a[i].plan.offsets != nullptr;
        const int64_t rows = a[i].kind == kTN ? a[i].M : grouped ? a[i].plan.max_rows : a[i].M;
        S.p[i] = a[i];
        S.tx[i] = int((rows + kBM - 1) / kBM);
        S.ty[i] = (a[i].N + kBN - 1) / kBN;
        tiles += int64_t(S.tx[i]) * S.ty[i] * (a[i].kind == kTN && grouped ? a[i].plan.E : 1);
        S.end[i] = tiles;
    }
    if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    simt_gemm_kernel<<<unsigned(tiles), kThreads, 0, s>>>(S);
    return cudaGetLastError();
}

}  // namespace moe
