// train_internal.h -- host-side launchers of the training operators (moe_train.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_train.h"

namespace moe {

// Routed rows live in a padded order: expert e's rows start at poff[e], a multiple of
// kRowTile, so that no row tile holds rows of two experts. A reduction over an expert's rows
// runs to the next multiple of kRowPad (the matrix instruction's depth), over rows that are zero.
constexpr int kRowTile = 128, kRowPad = 16;

inline int64_t round_rows(int64_t n) { return (n + kRowTile - 1) / kRowTile * kRowTile; }
// Most padded rows of S slots over E experts.
inline int64_t max_padded_rows(int64_t S, int64_t E) {
    const int64_t groups = E < S ? E : S;
    return round_rows(S + groups * (kRowTile - 1));
}

struct RowPlan {
    // caller's permutation; offsets == nullptr: dense (row r is token r, weight 1)
    const int32_t* offsets = nullptr;
    const int32_t* sorted_slot = nullptr;
    int64_t T = 0, S = 0;
    int E = 1, k = 1;
    // written by launch_gather (nullptr when dense)
    int32_t* poff = nullptr;      // [E + 1] first padded row of each expert
    int32_t* uoff = nullptr;      // [E + 1] first sorted position of each expert (checked copy)
    int32_t* row_slot = nullptr;  // [padded rows] slot, or -1 (padding, dropped)
    int32_t* slot_row = nullptr;  // [S] padded row; anything for a slot without one
    int64_t max_rows = 0;         // dense: T
    int* status = nullptr;
};

// Builds the plan and copies up to two [T, K] sources into padded order (pad rows zero).
struct GatherArgs {
    RowPlan plan;
    const void* src[2] = {nullptr, nullptr};
    int64_t ld[2] = {0, 0};
    void* dst[2] = {nullptr, nullptr};
    int K = 0;
    int es = 2;  // bytes per element
    bool zero_pad = false;  // the rows are reduced over (weight gradients)
    // bf16, two sources: bias_dot[slot] = src[1] row . down_b[expert]
    const void* down_b = nullptr;  // [E, K]
    float* bias_dot = nullptr;
};
cudaError_t launch_gather_padded(const GatherArgs& a, cudaStream_t s);

// out[t] = sum over the token's slots of rows[slot_row] (+ residual[t]), slots in order.
struct SumSlotsArgs {
    RowPlan plan;
    const float* rows = nullptr;  // [padded rows, K] f32
    const void* residual = nullptr;
    int64_t ldr = 0;
    void* out = nullptr;
    int64_t ldo = 0;
    int K = 0;
    int dtype = 0;
};
cudaError_t launch_sum_slots(const SumSlotsArgs& a, cudaStream_t s);

// ------------------------------------------------------------------ matrix products
// D[m, n] = sum_r A(m, r) B(n, r).
//   kNT: A rows [m][r], B rows [n][r]   forward:         tokens x weights^T
//   kNN: A rows [m][r], B rows [r][n]   input gradient:  dz x weights
//   kTN: A rows [r][m], B rows [r][n]   weight gradient: dz^T x tokens
// Grouped (plan.offsets set): kNT and kNN have one B plane per expert (stride sb elements)
// for the rows of that expert; kTN reduces over one expert's rows into D plane e (stride so).
enum GemmKind { kNT = 0, kNN = 1, kTN = 2 };

struct GemmArgs {
    int kind = kNT;
    RowPlan plan;
    const void* a = nullptr; int64_t lda = 0;
    const void* b = nullptr; int64_t ldb = 0, sb = 0;
    // kNN: reduction indices from r_split on read b1 rows (r - r_split); kTN: D rows from
    // m_split on go to out1 rows (m - m_split); kNT: D columns from n_split on read b1's rows
    // (n - n_split) and their bias from bias1. 0: no split.
    const void* b1 = nullptr; int split = 0;
    int64_t M = 0;  // kNT / kNN: rows (dense); kTN: rows of D
    int N = 0;
    int64_t R = 0;  // reduction length (kTN: ignored when grouped, else T)
    const void* bias = nullptr; const void* bias1 = nullptr; int64_t sbias = 0;  // [N] per expert
    int act = 0;                       // enum moe_linear_activation
    const float* row_scale = nullptr;  // indexed by slot (grouped)
    const void* residual = nullptr; int64_t ldr = 0;
    void* pre = nullptr; int64_t ldp = 0;
    void* out = nullptr; int64_t ldo = 0, so = 0;
    void* out1 = nullptr;
    int dtype = MOE_DTYPE_BF16;        // a, b, bias, residual, pre
    int out_f32 = 0;                   // out is f32 instead
};
// f32: n independent products (at most kMaxSimt) in one launch; those without an output are not computed.
constexpr int kMaxSimt = 3;
cudaError_t launch_simt_gemm(const GemmArgs* a, int n, cudaStream_t s);
// bf16: one kNT product; up to three independent kNN and kTN products of one plan (those
// without an output are not computed).
cudaError_t launch_tc_gemm_nt(const GemmArgs& a, cudaStream_t s);
cudaError_t launch_tc_gemms(const GemmArgs* a, int n, cudaStream_t s);

// The forward products for a few tokens, both types.
constexpr int kSmallT = 4;
// Whether they take this form: one or two tokens, or up to four over at most 20 MB of weights, a
// gated FFN's three planes at most 48 MB (its other form is two launches of few tiles). Weights cold,
// back to back, us, this / tensor cores: 2048 x 2048 4 tokens 8.4 / 9.9, 4096 x 2048 10.9 / 11.7, 3584 x
// 3584 (26 MB) 14.3 / 12.2, 3584 x 7168 2 tokens 13.9 / 15.6, 4 tokens 21.9 / 16.0; gated FFN 4 tokens
// 2048 x 768 12.7 / 17.5, 7168 x 768 23.4 / 26.4, 3584 x 2048 (44 MB) 24.6 / 25.1, 7168 x 2048 (88 MB)
// 2 tokens 26.6 / 36, 4 tokens 57 / 36.
inline bool small_form(int64_t T, int64_t weights, bool gated, int dtype) {
    return T <= 2 || (T <= kSmallT && (dtype == MOE_DTYPE_F32 || weights <= (gated ? 24 << 20 : 10 << 20)));
}
struct SmallArgs {
    int T = 0, K = 0, N = 0;  // N: outputs (gated: units)
    int dtype = MOE_DTYPE_BF16;
    bool gated = false;
    int interleaved = 0, act = 0;  // act: enum moe_linear_activation, gated: enum moe_activation
    float limit = 0.f, alpha = 0.f;
    const void* x = nullptr; int64_t ldx = 0;
    const void *w = nullptr, *w1 = nullptr;  // w1: the up plane
    const void *bias = nullptr, *bias1 = nullptr;
    const void* residual = nullptr; int64_t ldr = 0;
    void* pre = nullptr;                     // [T, N] (gated: [T, 2N])
    void* y = nullptr; int64_t ldy = 0;
    bool prefetch = false;  // a launch of this kernel comes just before: this one starts in its tail
    int ks = 1;  // set by the launcher
};
cudaError_t launch_small(const SmallArgs& a, cudaStream_t s);

// ------------------------------------------------------------------ element-wise passes
// The gated activation of every row and its derivative.
struct GatedArgs {
    RowPlan plan;
    int I = 0;
    int interleaved = 0, act = 0;
    float limit = 0.f, alpha = 0.f;
    int dtype = MOE_DTYPE_BF16;
    // forward
    const float* gp = nullptr;  // [padded rows, 2I] f32
    void* pre = nullptr;        // [S, 2I] (may be null)
    void* h = nullptr;          // [padded rows, I]
    // backward
    const float* dh = nullptr;      // [padded rows, I] f32: dy Wd
    const float* topk_w = nullptr;  // by slot, null when dense
    void* dgu = nullptr;            // [padded rows, 2I]
    void* hw = nullptr;             // [padded rows, I]
    float* dtopk_w = nullptr;       // by slot
    const void* dyp = nullptr;      // [padded rows, K] with down bias
    const void* down_b = nullptr;   // [E, K]
    const float* bias_dot = nullptr;  // bf16: dy . down_b by slot, in place of dyp and down_b
    int K = 0;
};
// f32: on the results of launch_simt_gemm.
cudaError_t launch_gated_forward(const GatedArgs& a, cudaStream_t s);
cudaError_t launch_gated_backward(const GatedArgs& a, cudaStream_t s);
// bf16: in the epilogue of the product g = (gate/up forward; dy Wd backward), which writes
// pre and h, or dgu, hw and per row dgated_parts(plan, I, R) partial sums of dh . h.
cudaError_t launch_tc_gateup(const GemmArgs& g, const GatedArgs& ga, cudaStream_t s);
cudaError_t launch_tc_dgated(const GemmArgs& g, const GatedArgs& ga, float* partial, cudaStream_t s);
int dgated_parts(const RowPlan& p, int I, int64_t R);
// dtopk_w[slot] = the row's partial sums (+ bias_dot), from GatedArgs' plan, dtopk_w, bias_dot.
cudaError_t launch_dtopk(const GatedArgs& a, const float* partial, int parts, cudaStream_t s);

// Column sums of each expert's rows: out[e, c] = sum_r x[r, c] (* topk_w[slot of r]).
struct ColsumArgs {
    RowPlan plan;
    const void* x = nullptr; int64_t ldx = 0; int cols = 0;
    const float* row_scale = nullptr;
    void* out = nullptr; int64_t so = 0;
    void* out1 = nullptr; int split = 0;  // columns from split on go to out1
    float* partial = nullptr;             // [rows / kRowTile rounded up, cols]
    int dtype = MOE_DTYPE_BF16;
};
cudaError_t launch_colsum(const ColsumArgs (&a)[2], cudaStream_t s);  // of one plan and dtype

// dz = dy * act'(pre), rounded to the activation dtype; partial column sums of the unrounded
// dz when partial is set (act none: only the sums are taken and dz may be null).
struct DactArgs {
    int64_t T = 0;
    int N = 0, act = 0, dtype = MOE_DTYPE_BF16;
    const void* dy = nullptr; int64_t lddy = 0;
    const void* pre = nullptr;
    void* dz = nullptr;
    float* partial = nullptr;  // [dact_splits, N]
    void* db = nullptr;
};
int dact_splits(int64_t T, int N);
cudaError_t launch_dact(const DactArgs& a, cudaStream_t s);

// ------------------------------------------------------------------ norm
struct NormArgs {
    int64_t T = 0;
    int H = 0, kind = 0, dtype = MOE_DTYPE_BF16;
    float eps = 0.f;
    const void *x = nullptr, *w = nullptr, *b = nullptr, *dy = nullptr;
    int64_t ldx = 0, ldy = 0, lddy = 0, lddx = 0;
    void *y = nullptr, *dx = nullptr, *dw = nullptr, *db = nullptr;
    float* stats = nullptr;
    const float* cstats = nullptr;
    float* partial = nullptr;  // [norm_blocks, 2, H]
};
int norm_blocks(int64_t T, int H, int dtype);
cudaError_t launch_norm_forward(const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t s);

}  // namespace moe
