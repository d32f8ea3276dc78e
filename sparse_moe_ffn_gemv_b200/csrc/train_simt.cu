// train_simt.cu -- matrix products on the CUDA cores, for f32 operands (the tensor cores have
// no 32-bit product) in every operand order the training operators need.
//
// 4 x 4 outputs per thread, 64 x 64 per block, or 32 x 32 with the reduction shared by four groups
// of threads where 64 x 64 gives fewer than two blocks per SM (a small f32 block is bound by
// latency: 77 x 192 x 320 took 14.8 us on 10 blocks of 256 threads, 11.6 us on 30 of 64, 9.4 us on
// 30 of four groups of 64). The operands of two more stages wait in registers.
#include <algorithm>

#include "train_dev.cuh"

namespace moe {

namespace {

// TD x TD threads of 4 x 4 outputs each, in KG groups that take every KG-th stage of BR
// reduction steps.
template <int TD_, int KG_, int BR_> struct Form {
    static constexpr int TD = TD_, KG = KG_, BR = BR_;
    static constexpr int GROUP = TD * TD, THREADS = GROUP * KG, B = 4 * TD;
    static constexpr int VECS = B * BR / 4 / GROUP;  // 16-byte vectors of an operand per thread and stage
    struct Shared {
        float a[KG][2][BR][B + 4], b[KG][2][BR][B + 4];
    };
    static_assert(sizeof(Shared) <= 48 * 1024 && GROUP * 16 * 4 * (KG - 1) <= int(sizeof(Shared)), "shared memory");
};

// One operand tile [B i][BR r] as vectors. RMAJOR: memory rows are reduction indices (vectors
// along i), else vectors along r. at(i, r) gives a vector's address, or null outside the operand
// (row lengths are multiples of 4, so a vector is in or out whole).
template <typename F, bool RMAJOR, typename At>
__device__ __forceinline__ void fetch(float4 (&v)[F::VECS], int tid, At at) {
    constexpr int Q = F::BR / 4;
#pragma unroll
    for (int q = 0; q < F::VECS; ++q) {
        const int idx = tid + q * F::GROUP;
        const int i = RMAJOR ? idx % F::TD * 4 : idx / Q, r = RMAJOR ? idx / F::TD : idx % Q * 4;
        const float* p = at(i, r);
        v[q] = p ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
template <typename F, bool RMAJOR>
__device__ __forceinline__ void stash(float (&sm)[F::BR][F::B + 4], int tid, const float4 (&v)[F::VECS]) {
    constexpr int Q = F::BR / 4;
#pragma unroll
    for (int q = 0; q < F::VECS; ++q) {
        const int idx = tid + q * F::GROUP;
        if (RMAJOR) {
            *reinterpret_cast<float4*>(&sm[idx / F::TD][idx % F::TD * 4]) = v[q];
        } else {
            const int i = idx / Q, r = idx % Q * 4;
            sm[r][i] = v[q].x;
            sm[r + 1][i] = v[q].y;
            sm[r + 2][i] = v[q].z;
            sm[r + 3][i] = v[q].w;
        }
    }
}

template <typename F, int KIND>
__device__ __forceinline__ void simt_tile(const GemmArgs& a, int64_t m0, int64_t n0, int z, typename F::Shared& sh) {
    constexpr int TD = F::TD;
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
    const int g = threadIdx.x / F::GROUP, tid = threadIdx.x % F::GROUP;
    // two stages of operands in registers ahead of the one in shared memory
    float4 va[2][F::VECS], vb[2][F::VECS];
    auto fetch_ab = [&](float4 (&xa)[F::VECS], float4 (&xb)[F::VECS], int64_t rb) {
        fetch<F, AR>(xa, tid, [&](int i, int r) -> const float* {
            const int64_t gi = m0 + i, gr = rb + r;
            return gi < M && gr < R ? A + (AR ? gr * a.lda + gi : gi * a.lda + gr) : nullptr;
        });
        fetch<F, BR>(xb, tid, [&](int i, int r) -> const float* {
            const int64_t gi = n0 + i, gr = rb + r;
            if (gi >= a.N || gr >= R) return nullptr;
            if (KIND == kNN && a.split && gr >= a.split) return B1 + (gr - a.split) * a.ldb + gi;
            if (KIND == kNT && a.split && gi >= a.split) return B1 + (gi - a.split) * a.ldb + gr;
            return B + (BR ? gr * a.ldb + gi : gi * a.ldb + gr);
        });
    };
    float acc[4][4] = {};
    const int ty = tid / TD, tx = tid % TD;
    constexpr int64_t step = int64_t(F::KG) * F::BR;  // of one stage of every group
    const int64_t rg = r0 + g * F::BR;
    fetch_ab(va[0], vb[0], rg);
    fetch_ab(va[1], vb[1], rg + step);
    for (int64_t r = r0; r < R; r += 2 * step) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // one barrier per stage: the other buffer's readers are past the barrier before it
            stash<F, AR>(sh.a[g][h], tid, va[h]);
            stash<F, BR>(sh.b[g][h], tid, vb[h]);
            __syncthreads();
            fetch_ab(va[h], vb[h], r + g * F::BR + (2 + h) * step);
#pragma unroll 8
            for (int q = 0; q < F::BR; ++q) {
                const float4 x = *reinterpret_cast<const float4*>(&sh.a[g][h][q][ty * 4]);
                const float4 y = *reinterpret_cast<const float4*>(&sh.b[g][h][q][tx * 4]);
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
            }
        }
    }
    if constexpr (F::KG > 1) {  // the groups' sums in order, through shared memory
        float4* part = reinterpret_cast<float4*>(&sh);
        __syncthreads();
        if (g > 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[((g - 1) * 4 + i) * F::GROUP + tid] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        __syncthreads();
        if (g > 0) return;
#pragma unroll
        for (int j = 0; j < F::KG - 1; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = part[(j * 4 + i) * F::GROUP + tid];
                acc[i][0] += v.x; acc[i][1] += v.y; acc[i][2] += v.z; acc[i][3] += v.w;
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
template <typename F, bool FWD>
__global__ void __launch_bounds__(F::THREADS) simt_gemm_kernel(const __grid_constant__ Simt S) {
    __shared__ typename F::Shared sh;
    pdl_begin();
    constexpr int kBM = F::B, kBN = F::B;
    int64_t t = blockIdx.x;
    int i = 0;
    while (i < S.n - 1 && t >= S.end[i]) ++i;
    if (i > 0) t -= S.end[i - 1];
    // row tiles fastest: neighbouring blocks share operand B
    const int64_t mt = t % S.tx[i], r = t / S.tx[i];
    const int nt = int(r % S.ty[i]), z = int(r / S.ty[i]);
    const GemmArgs& a = S.p[i];
    if constexpr (FWD) simt_tile<F, kNT>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
    else if (a.kind == kNN) simt_tile<F, kNN>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
    else simt_tile<F, kTN>(a, mt * kBM, int64_t(nt) * kBN, z, sh);
}

template <typename F>
cudaError_t launch_form(Simt& S, cudaStream_t s) {
    constexpr int B = F::B;
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
    if (S.p[0].kind == kNT) return launch_chained(simt_gemm_kernel<F, true>, unsigned(tiles), F::THREADS, 0, s, S);
    return launch_chained(simt_gemm_kernel<F, false>, unsigned(tiles), F::THREADS, 0, s, S);
}

}  // namespace

cudaError_t launch_simt_gemm(const GemmArgs* a, int n, cudaStream_t s) {
    Simt S;
    S.n = 0;
    if (n > kMaxSimt) return cudaErrorInvalidValue;
    int64_t tiles = 0;  // of 64 x 64, of all products: the form, and with it the order of their sums, is the pass's
    for (int i = 0; i < n; ++i) {
        if (a[i].out) S.p[S.n++] = a[i];
        const bool grouped = a[i].plan.offsets != nullptr;
        const int64_t rows = a[i].kind != kTN && grouped ? a[i].plan.S : a[i].M;
        tiles += ((rows + 63) / 64) * ((a[i].N + 63) / 64) * (a[i].kind == kTN && grouped ? a[i].plan.E : 1);
    }
    if (S.n == 0) return cudaSuccess;
    return tiles >= 2 * 148 ? launch_form<Form<16, 1, 32>>(S, s) : launch_form<Form<8, 4, 16>>(S, s);
}

}  // namespace moe
