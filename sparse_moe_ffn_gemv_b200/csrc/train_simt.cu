// train_simt.cu -- matrix products on the CUDA cores, for f32 operands (the tensor cores have
// no 32-bit product) in every operand order the training operators need.
//
// 64 x 64 outputs per block, 32 reduction steps per shared-memory stage, a 4 x 4 register tile
// per thread; the next stage's operands are loaded into registers (16-byte vectors) while the
// current one is multiplied. The tile is small because f32 blocks are small (a launch of few tiles leaves
// SMs idle sooner than it meets the FMA rate).
#include <algorithm>

#include "train_dev.cuh"

namespace moe {

namespace {

constexpr int kBR = 32;

// TD x TD threads, 4 x 4 outputs each.
template <int TD> struct Shared {
    float a[2][kBR][4 * TD + 4], b[2][kBR][4 * TD + 4];
};

// One operand tile [4 TD i][32 r] as V 16-byte vectors per thread. RMAJOR: memory rows are
// reduction indices (vectors along i), else vectors along r. at(i, r) gives a vector's address,
// or null outside the operand (row lengths are multiples of 4, so a vector is in or out whole).
template <int TD> constexpr int kVecs = 4 * TD * kBR / 4 / (TD * TD);
template <int TD, bool RMAJOR, typename At>
__device__ __forceinline__ void fetch(float4 (&v)[kVecs<TD>], At at) {
#pragma unroll
    for (int q = 0; q < kVecs<TD>; ++q) {
        const int idx = threadIdx.x + q * TD * TD;
        const int i = RMAJOR ? idx % TD * 4 : idx / 8, r = RMAJOR ? idx / TD : idx % 8 * 4;
        const float* p = at(i, r);
        v[q] = p ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
template <int TD, bool RMAJOR>
__device__ __forceinline__ void stash(float (&sm)[kBR][4 * TD + 4], const float4 (&v)[kVecs<TD>]) {
#pragma unroll
    for (int q = 0; q < kVecs<TD>; ++q) {
        const int idx = threadIdx.x + q * TD * TD;
        if (RMAJOR) {
            *reinterpret_cast<float4*>(&sm[idx / TD][idx % TD * 4]) = v[q];
        } else {
            const int i = idx / 8, r = idx % 8 * 4;
            sm[r][i] = v[q].x;
            sm[r + 1][i] = v[q].y;
            sm[r + 2][i] = v[q].z;
            sm[r + 3][i] = v[q].w;
        }
    }
}

template <int TD, int KIND>
__device__ __forceinline__ void simt_tile(const GemmArgs& a, int64_t m0, int64_t n0, int z, Shared<TD>& sh) {
    constexpr bool AR = KIND == kTN, BR = KIND != kNT;  // operand rows are reduction indices
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
    const float* A = static_cast<const float*>(a.a);
    const float* B = static_cast<const float*>(a.b) + int64_t(e) * (KIND == kTN ? 0 : a.sb);
    const float* B1 = a.b1 ? static_cast<const float*>(a.b1) + int64_t(e) * a.sb : nullptr;
    // two stages of operands in registers ahead of the one in shared memory
    float4 va[2][kVecs<TD>], vb[2][kVecs<TD>];
    auto fetch_ab = [&](float4 (&xa)[kVecs<TD>], float4 (&xb)[kVecs<TD>], int64_t rb) {
        fetch<TD, AR>(xa, [&](int i, int r) -> const float* {
            const int64_t gi = m0 + i, gr = rb + r;
            return gi < M && gr < R ? A + (AR ? gr * a.lda + gi : gi * a.lda + gr) : nullptr;
        });
        fetch<TD, BR>(xb, [&](int i, int r) -> const float* {
            const int64_t gi = n0 + i, gr = rb + r;
            if (gi >= a.N || gr >= R) return nullptr;
            if (KIND == kNN && a.split && gr >= a.split) return B1 + (gr - a.split) * a.ldb + gi;
            if (KIND == kNT && a.split && gi >= a.split) return B1 + (gi - a.split) * a.ldb + gr;
            return B + (BR ? gr * a.ldb + gi : gi * a.ldb + gr);
        });
    };
    float acc[4][4] = {};
    const int ty = threadIdx.x / TD, tx = threadIdx.x % TD;
    fetch_ab(va[0], vb[0], r0);
    fetch_ab(va[1], vb[1], r0 + kBR);
    for (int64_t r = r0; r < R; r += 2 * kBR) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // one barrier per stage: the other buffer's readers are past the barrier before it
            stash<TD, AR>(sh.a[h], va[h]);
            stash<TD, BR>(sh.b[h], vb[h]);
            __syncthreads();
            fetch_ab(va[h], vb[h], r + (2 + h) * kBR);
#pragma unroll 8
            for (int q = 0; q < kBR; ++q) {
                const float4 x = *reinterpret_cast<const float4*>(&sh.a[h][q][ty * 4]);
                const float4 y = *reinterpret_cast<const float4*>(&sh.b[h][q][tx * 4]);
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
            }
        }
    }
    const int64_t n = n0 + tx * 4;
    if (n >= a.N) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= M) break;
        float o[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
        if (KIND == kTN) {
            float* d = static_cast<float*>(a.split && m >= a.split ? a.out1 : a.out) + int64_t(e) * a.so +
                       (a.split && m >= a.split ? m - a.split : m) * a.ldo + n;
            store_vec(d, o);
            continue;
        }
        if (a.bias) {
            const bool second = a.split && n >= a.split;
            float b[4];
            load_vec(static_cast<const float*>(second ? a.bias1 : a.bias) + int64_t(e) * a.sbias + (second ? n - a.split : n), b);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] += b[j];
        }
        if (a.pre) store_vec(static_cast<float*>(a.pre) + m * a.ldp + n, o);
        float rs = 1.0f;
        if (a.row_scale) {
            const int slot = p.row_slot[m];
            rs = slot < 0 ? 0.0f : a.row_scale[slot];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = linear_act<false>(a.act, o[j]) * rs;
        if (a.residual) {
            float b[4];
            load_vec(static_cast<const float*>(a.residual) + m * a.ldr + n, b);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] += b[j];
        }
        store_vec(static_cast<float*>(a.out) + m * a.ldo + n, o);
    }
}

struct Simt {
    GemmArgs p[kMaxSimt];
    int64_t end[kMaxSimt];  // first tile after problem i
    int tx[kMaxSimt], ty[kMaxSimt];
    int n;
};

// FWD: every problem is kNT; else kNN and kTN (one kernel per pass keeps its code small: a tiny
// launch spends much of its time fetching instructions).
template <int TD, bool FWD>
__global__ void __launch_bounds__(TD * TD) simt_gemm_kernel(const __grid_constant__ Simt S) {
    __shared__ Shared<TD> sh;
    constexpr int kBM = 4 * TD, kBN = 4 * TD;
    int64_t t = blockIdx.x;
    int i = 0;
    while (i < S.n - 1 && t >= S.end[i]) ++i;
    if (i > 0) t -= S.end[i - 1];
    // row tiles fastest: neighbouring blocks share operand B
    const int64_t mt = t % S.tx[i], r = t / S.tx[i];
    const int nt = int(r % S.ty[i]), z = int(r / S.ty[i]);
    const GemmArgs& a = S.p[i];
    if constexpr (FWD) simt_tile<TD, kNT>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
    else if (a.kind == kNN) simt_tile<TD, kNN>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
    else simt_tile<TD, kTN>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
}

template <int TD>
cudaError_t launch_td(Simt& S, cudaStream_t s) {
    constexpr int B = 4 * TD;
    int64_t tiles = 0;
    for (int i = 0; i < S.n; ++i) {
        const GemmArgs& a = S.p[i];
        const bool grouped = a.plan.offsets != nullptr;
        const int64_t rows = a.kind == kTN ? a.M : grouped ? a.plan.max_rows : a.M;
        S.tx[i] = int((rows + B - 1) / B);
        S.ty[i] = (a.N + B - 1) / B;
        tiles += int64_t(S.tx[i]) * S.ty[i] * (a.kind == kTN && grouped ? a.plan.E : 1);
        S.end[i] = tiles;
    }
    if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    if (S.p[0].kind == kNT) simt_gemm_kernel<TD, true><<<unsigned(tiles), TD * TD, 0, s>>>(S);
    else simt_gemm_kernel<TD, false><<<unsigned(tiles), TD * TD, 0, s>>>(S);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_simt_gemm(const GemmArgs* a, int n, cudaStream_t s) {
    Simt S;
    S.n = n;
    int64_t tiles = 0;  // of 64 x 64
    for (int i = 0; i < n; ++i) {
        S.p[i] = a[i];
        const bool grouped = a[i].plan.offsets != nullptr;
        const int64_t rows = a[i].kind != kTN && grouped ? a[i].plan.S : a[i].M;
        tiles += ((rows + 63) / 64) * ((a[i].N + 63) / 64) * (a[i].kind == kTN && grouped ? a[i].plan.E : 1);
    }
    return tiles >= 2 * 148 ? launch_td<16>(S, s) : launch_td<8>(S, s);
}

}  // namespace moe
