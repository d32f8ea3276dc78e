// train_api.cu -- the C ABI of moe_train.h: validation, workspace layout, launch order.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "train_internal.h"

using namespace moe;

namespace {

#define MOE_CHECK(expr)                          \
    do {                                         \
        const moe_status _s = (expr);            \
        if (_s != MOE_OK) return _s;             \
    } while (0)
#define MOE_CUDA(expr)                                  \
    do {                                                \
        if ((expr) != cudaSuccess) return MOE_ERR_CUDA; \
    } while (0)

constexpr int64_t kMaxRows = int64_t(1) << 30;   // slots (their padded rows fit 32 bits)
constexpr int64_t kMaxElems = int64_t(1) << 46;  // elements of any one tensor
constexpr int kMaxWidth = 1 << 28;               // columns (twice as many, and tiles of them, fit 32 bits)

constexpr int64_t kMaxTiles = int64_t(1) << 29;  // output tiles of a product (three in one launch stay below 2^31)

int esize(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// Whether the tiles of `planes` products [M, N] are few enough for the kernels' 32-bit tile numbers.
bool tiles_fit(int64_t M, int64_t N, int64_t planes, int dtype) {
    const int64_t bm = dtype == MOE_DTYPE_F32 ? 64 : 128, bn = dtype == MOE_DTYPE_F32 ? 64 : 256;
    return ((M + bm - 1) / bm) * ((N + bn - 1) / bn) * planes < kMaxTiles;
}

moe_status need(const void* p) {
    return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 ? MOE_OK : MOE_ERR_INVALID_ARGUMENT;
}
moe_status maybe(const void* p) { return p ? need(p) : MOE_OK; }
// Row stride of a [T, cols] tensor. One row has no stride to speak of, but its address
// arithmetic and tensor maps use it, so it is checked all the same.
moe_status stride(int64_t ld, int64_t cols, int dtype) {
    if (ld < cols || (ld * esize(dtype)) % 16 != 0) return MOE_ERR_INVALID_ARGUMENT;
    return ld >= (int64_t(1) << 36) ? MOE_ERR_SHAPE_OVERFLOW : MOE_OK;
}
// An output of rows against an input of rows: they may be the same tensor (`same`), or hold no
// element in common, side by side in wider rows included.
moe_status apart(const void* in, int64_t ldi, int64_t ci, const void* out, int64_t ldo, int64_t co, int64_t T, int dtype,
                 bool same) {
    if (!in || !out) return MOE_OK;
    if (same && in == out && (ldi == ldo || T == 1) && ci == co) return MOE_OK;
    const int64_t es = esize(dtype);
    const uintptr_t i0 = reinterpret_cast<uintptr_t>(in), o0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t i1 = i0 + uintptr_t(((T - 1) * ldi + ci) * es), o1 = o0 + uintptr_t(((T - 1) * ldo + co) * es);
    if (i1 <= o0 || o1 <= i0) return MOE_OK;
    if (T > 1 && ldi == ldo) {
        const int64_t ld = ldi * es, d = (int64_t(o0 - i0) % ld + ld) % ld;
        if (d >= ci * es && d + co * es <= ld) return MOE_OK;
    }
    return MOE_ERR_INVALID_ARGUMENT;
}
moe_status check_status_ptr(const int32_t* p) {
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0 ? MOE_OK : MOE_ERR_INVALID_ARGUMENT;
}

struct Carver {
    size_t off = 0;
    size_t take(int64_t bytes) {
        const size_t o = off;
        off = align256(off + size_t(bytes > 0 ? bytes : 0));
        return o;
    }
};
template <typename P> P* at(void* ws, size_t off) { return reinterpret_cast<P*>(static_cast<char*>(ws) + off); }

moe_status check_ws(const void* ws, size_t have, size_t want) {
    if (want == 0) return MOE_OK;
    MOE_CHECK(need(ws));
    return have < want ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// ------------------------------------------------------------------ linear
moe_status check_linear(const moe_linear_desc* d, int64_t T) {
    if (!d || d->in_features <= 0 || d->out_features <= 0) return MOE_ERR_INVALID_ARGUMENT;
    if (d->activation < MOE_LINEAR_NONE || d->activation > MOE_LINEAR_GELU) return MOE_ERR_INVALID_ARGUMENT;
    if (d->dtype != MOE_DTYPE_F32 && d->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
    const int q = 16 / esize(d->dtype);
    if (d->in_features % q || d->out_features % q) return MOE_ERR_INVALID_ARGUMENT;
    if (T < 0) return MOE_ERR_INVALID_ARGUMENT;
    if (d->in_features > kMaxWidth || d->out_features > kMaxWidth) return MOE_ERR_SHAPE_OVERFLOW;
    const int64_t K = d->in_features, N = d->out_features;
    if (T > kMaxRows || T * std::max(K, N) > kMaxElems || N * K > kMaxElems) return MOE_ERR_SHAPE_OVERFLOW;
    if (!tiles_fit(T, N, 1, d->dtype) || !tiles_fit(T, K, 1, d->dtype) || !tiles_fit(N, K, 1, d->dtype))
        return MOE_ERR_SHAPE_OVERFLOW;
    return MOE_OK;
}

// A forward product.
cudaError_t launch_gemm(const GemmArgs& g, cudaStream_t s) {
    return g.dtype == MOE_DTYPE_F32 ? launch_simt_gemm(&g, 1, s) : launch_tc_gemm_nt(g, s);
}

// A backward pass's independent products. Those without an output are not computed, but count in the
// choice of form, so that the others do not depend on what was asked for.
cudaError_t launch_gemms(const GemmArgs* g, int n, cudaStream_t s) {
    return g[0].dtype == MOE_DTYPE_F32 ? launch_simt_gemm(g, n, s) : launch_tc_gemms(g, n, s);
}

struct LinearWs {
    size_t dz, partial, total;
};
LinearWs linear_ws(const moe_linear_desc* d, int64_t T, bool backward) {
    LinearWs L{};
    Carver c;
    if (backward && T > 0) {
        L.dz = c.take(d->activation != MOE_LINEAR_NONE ? T * d->out_features * esize(d->dtype) : 0);
        L.partial = c.take(int64_t(dact_splits(T, d->out_features)) * d->out_features * 4);
    }
    L.total = c.off;
    return L;
}

// ------------------------------------------------------------------ ffn
struct FfnShape {
    int E, k, I, K, es, dtype;
    bool il, bias;
    int64_t T, S, rows;  // rows: padded rows at most (dense: T)
    bool dense;
};

moe_status check_ffn(const moe_config* c, int64_t T, bool dense, FfnShape* f) {
    MOE_CHECK(moe_config_validate(c));
    if (c->weight_format != MOE_DTYPE_F32 && c->weight_format != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
    if (dense && (c->num_experts != 1 || c->top_k != 1)) return MOE_ERR_INVALID_ARGUMENT;
    if (T < 0) return MOE_ERR_INVALID_ARGUMENT;
    f->E = c->num_experts;
    f->k = c->top_k;
    f->I = c->intermediate;
    f->K = expert_in(*c);
    f->dtype = c->act_dtype;
    f->es = esize(c->act_dtype);
    f->il = c->gate_up_interleaved != 0;
    f->bias = c->has_expert_bias != 0;
    f->T = T;
    f->dense = dense;
    if (f->K > kMaxWidth || f->I > kMaxWidth) return MOE_ERR_SHAPE_OVERFLOW;
    if (T > kMaxRows || T * f->k > kMaxRows) return MOE_ERR_SHAPE_OVERFLOW;
    f->S = T * f->k;
    f->rows = dense ? T : max_padded_rows(f->S, f->E);
    const int64_t K = f->K, I = f->I;  // the planes' own size: moe_config_validate
    if (f->rows * std::max(K, 2 * I) > kMaxElems) return MOE_ERR_SHAPE_OVERFLOW;
    if (!tiles_fit(f->rows, 2 * I, 1, f->dtype) || !tiles_fit(f->rows, K, 1, f->dtype) ||
        !tiles_fit(2 * I, K, f->E, f->dtype) || !tiles_fit(K, I, f->E, f->dtype))
        return MOE_ERR_SHAPE_OVERFLOW;
    return MOE_OK;
}

// The gate/up, down and bias planes the config has.
moe_status check_planes(const FfnShape& f, const void* gate, const void* up, const void* gate_up, const void* gate_b,
                        const void* up_b, const void* gate_up_b, const void* down, const void* down_b) {
    const void* want[6] = {};
    int n = 0;
    if (f.il) {
        want[n++] = gate_up;
        if (f.bias) want[n++] = gate_up_b;
    } else {
        want[n++] = gate;
        want[n++] = up;
        if (f.bias) {
            want[n++] = gate_b;
            want[n++] = up_b;
        }
    }
    want[n++] = down;
    for (int i = 0; i < n; ++i) {
        if (!want[i]) return MOE_ERR_MISSING_TENSOR;
        MOE_CHECK(need(want[i]));
    }
    if (f.bias) {
        if (!down_b) return MOE_ERR_MISSING_TENSOR;
        MOE_CHECK(need(down_b));
    }
    return MOE_OK;
}

struct FfnWs {
    size_t poff, uoff, row_slot, slot_row;
    size_t up, dyp;   // gathered rows of u and dy (routed)
    size_t gp, h;     // forward
    size_t rows_out;  // [rows, K] f32 slot rows of y or du (routed)
    size_t dh, dgu, hw, partial;
    size_t parts;     // [rows, dgated_parts] partial sums of dtopk_w (bf16, routed)
    size_t bias_dot;  // [S] dy . down_b (bf16, routed, with biases)
    size_t total;
};
// The plan's sizes; offsets only says routed or dense here.
RowPlan shape_plan(const FfnShape& f) {
    static const int32_t routed = 0;
    RowPlan p;
    p.T = f.T;
    p.S = f.S;
    p.E = f.E;
    p.k = f.k;
    p.max_rows = f.rows;
    p.offsets = f.dense ? nullptr : &routed;
    return p;
}
FfnWs ffn_ws(const FfnShape& f, bool backward) {
    FfnWs L{};
    Carver c;
    if (f.T == 0) return L;
    const bool f32 = f.dtype == MOE_DTYPE_F32;
    if (!f.dense) {
        L.poff = c.take((f.E + 1) * 4);
        L.uoff = c.take((f.E + 1) * 4);
        L.row_slot = c.take(f.rows * 4);
        L.slot_row = c.take(f.S * 4);
        L.up = c.take(f.rows * f.K * f.es);
        if (backward) L.dyp = c.take(f.rows * f.K * f.es);
        L.rows_out = c.take(f.rows * f.K * 4);
        if (backward && !f32 && f.bias) L.bias_dot = c.take(f.S * 4);
        if (backward && !f32) L.parts = c.take(f.rows * dgated_parts(shape_plan(f), f.I, f.K) * 4);
    }
    if (backward) {
        if (f32) L.dh = c.take(f.rows * f.I * 4);
        L.dgu = c.take(f.rows * 2 * f.I * f.es);
        L.hw = c.take(f.rows * f.I * f.es);
        if (f.bias)
            L.partial = c.take(round_rows(f.rows) / kRowTile * (2 * int64_t(f.I) + f.K) * 4);
    } else {
        if (f32) L.gp = c.take(f.rows * 2 * f.I * 4);
        L.h = c.take(f.rows * f.I * f.es);
    }
    L.total = c.off;
    return L;
}

RowPlan row_plan(const FfnShape& f, const int32_t* offsets, const int32_t* sorted_slot, void* ws, const FfnWs& L,
                 int32_t* status) {
    RowPlan p = shape_plan(f);
    p.status = status;
    if (!f.dense) {
        p.offsets = offsets;
        p.sorted_slot = sorted_slot;
        p.poff = at<int32_t>(ws, L.poff);
        p.uoff = at<int32_t>(ws, L.uoff);
        p.row_slot = at<int32_t>(ws, L.row_slot);
        p.slot_row = at<int32_t>(ws, L.slot_row);
    }
    return p;
}

// All three of the permutation's tensors, or none of them (dense). Without tokens the slots'
// tensors are empty and may have no address.
moe_status check_routing(const int32_t* offsets, const int32_t* sorted_slot, const float* topk_w, int64_t T,
                         bool* dense) {
    *dense = !offsets && !sorted_slot && !topk_w;
    if (*dense || T == 0) return MOE_OK;
    MOE_CHECK(need(offsets));
    MOE_CHECK(need(sorted_slot));
    return need(topk_w);
}

}  // namespace

extern "C" {

moe_status moe_linear_workspace_size(const moe_linear_desc* d, int64_t T, int32_t backward, size_t* bytes) {
    MOE_CHECK(check_linear(d, T));
    if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
    *bytes = linear_ws(d, T, backward != 0).total;
    return MOE_OK;
}

moe_status moe_linear_forward(const moe_linear_desc* d, const void* x, int64_t ldx, const void* w, const void* bias,
                              const void* residual, int64_t ldr, int64_t T, void* y, int64_t ldy, void* pre, void* ws,
                              size_t ws_bytes, int32_t* device_status, moe_stream_t stream) {
    MOE_CHECK(check_linear(d, T));
    if (T == 0) return MOE_OK;
    const int K = d->in_features, N = d->out_features;
    MOE_CHECK(need(x));
    MOE_CHECK(need(w));
    MOE_CHECK(need(y));
    MOE_CHECK(maybe(bias));
    MOE_CHECK(maybe(residual));
    MOE_CHECK(maybe(pre));
    MOE_CHECK(check_status_ptr(device_status));
    MOE_CHECK(stride(ldx, K, d->dtype));
    MOE_CHECK(stride(ldy, N, d->dtype));
    if (residual) MOE_CHECK(stride(ldr, N, d->dtype));
    MOE_CHECK(check_ws(ws, ws_bytes, linear_ws(d, T, false).total));
    MOE_CHECK(apart(x, ldx, K, y, ldy, N, T, d->dtype, false));
    MOE_CHECK(apart(residual, ldr, N, y, ldy, N, T, d->dtype, true));
    if (small_form(T, int64_t(K) * N, false, d->dtype)) {
        SmallArgs a;
        a.T = int(T); a.K = K; a.N = N; a.dtype = d->dtype; a.act = d->activation;
        a.x = x; a.ldx = ldx; a.w = w; a.bias = bias;
        a.residual = residual; a.ldr = ldr;
        a.pre = pre;
        a.y = y; a.ldy = ldy;
        MOE_CUDA(launch_small(a, (cudaStream_t)stream));
        return MOE_OK;
    }
    GemmArgs g;
    g.plan.status = device_status;
    g.kind = kNT;
    g.a = x; g.lda = ldx;
    g.b = w; g.ldb = K;
    g.M = T; g.N = N; g.R = K;
    g.bias = bias;
    g.act = d->activation;
    g.residual = residual; g.ldr = ldr;
    g.pre = pre; g.ldp = N;
    g.out = y; g.ldo = ldy;
    g.dtype = d->dtype;
    MOE_CUDA(launch_gemm(g, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_linear_backward(const moe_linear_desc* d, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                               const void* w, const void* pre, int64_t T, void* dx, int64_t lddx, void* dw, void* db,
                               void* ws, size_t ws_bytes, int32_t* device_status, moe_stream_t stream) {
    MOE_CHECK(check_linear(d, T));
    const int K = d->in_features, N = d->out_features;
    cudaStream_t s = (cudaStream_t)stream;
    MOE_CHECK(maybe(dx));
    MOE_CHECK(maybe(dw));
    MOE_CHECK(maybe(db));
    MOE_CHECK(check_status_ptr(device_status));
    if (T == 0) {
        if (dw) MOE_CUDA(cudaMemsetAsync(dw, 0, size_t(N) * K * esize(d->dtype), s));
        if (db) MOE_CUDA(cudaMemsetAsync(db, 0, size_t(N) * esize(d->dtype), s));
        return MOE_OK;
    }
    const bool act = d->activation != MOE_LINEAR_NONE;
    MOE_CHECK(need(dy));
    MOE_CHECK(stride(lddy, N, d->dtype));
    if (act && !pre) return MOE_ERR_MISSING_TENSOR;
    if (act) MOE_CHECK(need(pre));
    if (dx) {
        MOE_CHECK(need(w));
        MOE_CHECK(stride(lddx, K, d->dtype));
    }
    if (dw) {
        MOE_CHECK(need(x));
        MOE_CHECK(stride(ldx, K, d->dtype));
    }
    const LinearWs L = linear_ws(d, T, true);
    MOE_CHECK(check_ws(ws, ws_bytes, L.total));
    MOE_CHECK(apart(dy, lddy, N, dx, lddx, K, T, d->dtype, false));
    if (dw) MOE_CHECK(apart(x, ldx, K, dx, lddx, K, T, d->dtype, false));
    const void* dz = dy;
    int64_t lddz = lddy;
    if (act || db) {
        DactArgs a;
        a.T = T; a.N = N; a.act = d->activation; a.dtype = d->dtype;
        a.dy = dy; a.lddy = lddy;
        a.pre = pre;
        if (act) {
            a.dz = at<void>(ws, L.dz);
            dz = a.dz;
            lddz = N;
        }
        if (db) {
            a.partial = at<float>(ws, L.partial);
            a.db = db;
        }
        MOE_CUDA(launch_dact(a, s));
    }
    GemmArgs g[2];
    g[0].kind = kNN;
    g[0].a = dz; g[0].lda = lddz;
    g[0].b = w; g[0].ldb = K;
    g[0].M = T; g[0].N = K; g[0].R = N;
    g[0].out = dx; g[0].ldo = lddx;
    g[1].kind = kTN;
    g[1].a = dz; g[1].lda = lddz;
    g[1].b = x; g[1].ldb = ldx;
    g[1].M = N; g[1].N = K; g[1].R = T;
    g[1].out = dw; g[1].ldo = K;
    for (int i = 0; i < 2; ++i) {
        g[i].plan.status = device_status;
        g[i].dtype = d->dtype;
    }
    MOE_CUDA(launch_gemms(g, 2, s));
    return MOE_OK;
}

moe_status moe_ffn_workspace_size(const moe_config* cfg, int64_t T, int32_t backward, size_t* bytes) {
    FfnShape f;
    MOE_CHECK(check_ffn(cfg, T, false, &f));
    if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
    *bytes = ffn_ws(f, backward != 0).total;
    return MOE_OK;
}

moe_status moe_ffn_dense_workspace_size(const moe_config* cfg, int64_t T, int32_t backward, size_t* bytes) {
    FfnShape f;
    MOE_CHECK(check_ffn(cfg, T, true, &f));
    if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
    *bytes = ffn_ws(f, backward != 0).total;
    return MOE_OK;
}

moe_status moe_ffn_forward(const moe_config* cfg, const moe_weights* w, const void* u, int64_t ldu, int64_t T,
                           const int32_t* expert_offsets, const int32_t* sorted_slot, const float* topk_w,
                           const void* residual, int64_t ldr, void* y, int64_t ldy, void* pre, void* ws,
                           size_t ws_bytes, int32_t* device_status, moe_stream_t stream) {
    bool dense;
    FfnShape f;
    MOE_CHECK(check_routing(expert_offsets, sorted_slot, topk_w, T, &dense));
    MOE_CHECK(check_ffn(cfg, T, dense, &f));
    if (!w) return MOE_ERR_INVALID_ARGUMENT;
    MOE_CHECK(check_planes(f, w->gate_w, w->up_w, w->gate_up_w, w->gate_b, w->up_b, w->gate_up_b, w->down_w,
                           w->down_b));
    if (T == 0) return MOE_OK;
    MOE_CHECK(need(u));
    MOE_CHECK(need(y));
    MOE_CHECK(maybe(residual));
    MOE_CHECK(maybe(pre));
    MOE_CHECK(check_status_ptr(device_status));
    MOE_CHECK(stride(ldu, f.K, f.dtype));
    MOE_CHECK(stride(ldy, f.K, f.dtype));
    if (residual) MOE_CHECK(stride(ldr, f.K, f.dtype));
    const FfnWs L = ffn_ws(f, false);
    MOE_CHECK(check_ws(ws, ws_bytes, L.total));
    MOE_CHECK(apart(u, ldu, f.K, y, ldy, f.K, T, f.dtype, true));
    MOE_CHECK(apart(residual, ldr, f.K, y, ldy, f.K, T, f.dtype, true));
    cudaStream_t s = (cudaStream_t)stream;
    const RowPlan p = row_plan(f, expert_offsets, sorted_slot, ws, L, device_status);
    if (dense && small_form(T, 3 * int64_t(f.K) * f.I, true, f.dtype)) {
        SmallArgs a;
        a.T = int(T); a.K = f.K; a.N = f.I; a.dtype = f.dtype;
        a.gated = true; a.interleaved = f.il; a.act = cfg->activation; a.limit = cfg->swiglu_limit;
        a.alpha = cfg->swiglu_alpha;
        a.x = u; a.ldx = ldu;
        a.w = f.il ? w->gate_up_w : w->gate_w; a.w1 = w->up_w;
        if (f.bias) {
            a.bias = f.il ? w->gate_up_b : w->gate_b;
            a.bias1 = w->up_b;
        }
        a.pre = pre;
        a.y = at<void>(ws, L.h); a.ldy = f.I;
        MOE_CUDA(launch_small(a, s));
        SmallArgs o;
        o.T = int(T); o.K = f.I; o.N = f.K; o.dtype = f.dtype;
        o.x = a.y; o.ldx = f.I; o.w = w->down_w;
        o.bias = f.bias ? w->down_b : nullptr;
        o.residual = residual; o.ldr = ldr;
        o.y = y; o.ldy = ldy;
        o.prefetch = true;
        MOE_CUDA(launch_small(o, s));
        return MOE_OK;
    }
    if (!dense) {
        GatherArgs ga;
        ga.plan = p;
        ga.src[0] = u; ga.ld[0] = ldu; ga.dst[0] = at<void>(ws, L.up);
        ga.K = f.K; ga.es = f.es;
        MOE_CUDA(launch_gather_padded(ga, s));
    }
    GemmArgs g;
    g.kind = kNT;
    g.plan = p;
    g.dtype = f.dtype;
    g.a = dense ? u : at<void>(ws, L.up); g.lda = dense ? ldu : f.K;
    g.ldb = f.K; g.sb = int64_t(f.I) * f.K * (f.il ? 2 : 1);
    g.b = f.il ? w->gate_up_w : w->gate_w;
    if (!f.il) {
        g.b1 = w->up_w;
        g.split = f.I;
    }
    if (f.bias) {
        g.bias = f.il ? w->gate_up_b : w->gate_b;
        g.bias1 = f.il ? nullptr : w->up_b;
        g.sbias = int64_t(f.I) * (f.il ? 2 : 1);
    }
    g.M = f.T; g.N = 2 * f.I; g.R = f.K;
    GatedArgs ga;
    ga.plan = p;
    ga.I = f.I; ga.interleaved = f.il; ga.act = cfg->activation; ga.limit = cfg->swiglu_limit;
    ga.alpha = cfg->swiglu_alpha;
    ga.dtype = f.dtype;
    ga.pre = pre;
    ga.h = at<void>(ws, L.h);
    if (f.dtype == MOE_DTYPE_F32) {
        g.out = at<void>(ws, L.gp); g.ldo = 2 * f.I;
        ga.gp = at<float>(ws, L.gp);
        MOE_CUDA(launch_simt_gemm(&g, 1, s));
        MOE_CUDA(launch_gated_forward(ga, s));
    } else {
        MOE_CUDA(launch_tc_gateup(g, ga, s));
    }
    GemmArgs o;
    o.kind = kNT;
    o.plan = p;
    o.dtype = f.dtype;
    o.a = ga.h; o.lda = f.I;
    o.b = w->down_w; o.ldb = f.I; o.sb = int64_t(f.K) * f.I;
    o.M = f.T; o.N = f.K; o.R = f.I;
    if (f.bias) {
        o.bias = w->down_b;
        o.sbias = f.K;
    }
    if (dense) {
        o.residual = residual; o.ldr = ldr;
        o.out = y; o.ldo = ldy;
        MOE_CUDA(launch_gemm(o, s));
        return MOE_OK;
    }
    o.row_scale = topk_w;
    o.out = at<void>(ws, L.rows_out); o.ldo = f.K; o.out_f32 = 1;
    MOE_CUDA(launch_gemm(o, s));
    SumSlotsArgs sa;
    sa.plan = p;
    sa.rows = at<float>(ws, L.rows_out);
    sa.residual = residual; sa.ldr = ldr;
    sa.out = y; sa.ldo = ldy;
    sa.K = f.K;
    sa.dtype = f.dtype;
    MOE_CUDA(launch_sum_slots(sa, s));
    return MOE_OK;
}

moe_status moe_ffn_backward(const moe_config* cfg, const moe_weights* w, const void* u, int64_t ldu, int64_t T,
                            const int32_t* expert_offsets, const int32_t* sorted_slot, const float* topk_w,
                            const void* pre, const void* dy, int64_t lddy, void* du, int64_t lddu, float* dtopk_w,
                            const moe_ffn_grads* gr, void* ws, size_t ws_bytes, int32_t* device_status,
                            moe_stream_t stream) {
    bool dense;
    FfnShape f;
    MOE_CHECK(check_routing(expert_offsets, sorted_slot, topk_w, T, &dense));
    MOE_CHECK(check_ffn(cfg, T, dense, &f));
    if (!w || !gr) return MOE_ERR_INVALID_ARGUMENT;
    if (dense && dtopk_w) return MOE_ERR_INVALID_ARGUMENT;
    MOE_CHECK(check_planes(f, w->gate_w, w->up_w, w->gate_up_w, w->gate_b, w->up_b, w->gate_up_b, w->down_w,
                           w->down_b));
    MOE_CHECK(check_planes(f, gr->gate_w, gr->up_w, gr->gate_up_w, gr->gate_b, gr->up_b, gr->gate_up_b, gr->down_w,
                           gr->down_b));
    cudaStream_t s = (cudaStream_t)stream;
    const size_t plane = size_t(f.E) * f.I * f.K * f.es;
    if (T == 0) {
        if (f.il) {
            MOE_CUDA(cudaMemsetAsync(gr->gate_up_w, 0, 2 * plane, s));
            if (f.bias) MOE_CUDA(cudaMemsetAsync(gr->gate_up_b, 0, size_t(f.E) * 2 * f.I * f.es, s));
        } else {
            MOE_CUDA(cudaMemsetAsync(gr->gate_w, 0, plane, s));
            MOE_CUDA(cudaMemsetAsync(gr->up_w, 0, plane, s));
            if (f.bias) {
                MOE_CUDA(cudaMemsetAsync(gr->gate_b, 0, size_t(f.E) * f.I * f.es, s));
                MOE_CUDA(cudaMemsetAsync(gr->up_b, 0, size_t(f.E) * f.I * f.es, s));
            }
        }
        MOE_CUDA(cudaMemsetAsync(gr->down_w, 0, plane, s));
        if (f.bias) MOE_CUDA(cudaMemsetAsync(gr->down_b, 0, size_t(f.E) * f.K * f.es, s));
        return MOE_OK;
    }
    MOE_CHECK(need(u));
    MOE_CHECK(need(dy));
    MOE_CHECK(need(pre));
    MOE_CHECK(maybe(du));
    MOE_CHECK(maybe(dtopk_w));
    MOE_CHECK(check_status_ptr(device_status));
    MOE_CHECK(stride(ldu, f.K, f.dtype));
    MOE_CHECK(stride(lddy, f.K, f.dtype));
    if (du) MOE_CHECK(stride(lddu, f.K, f.dtype));
    const FfnWs L = ffn_ws(f, true);
    MOE_CHECK(check_ws(ws, ws_bytes, L.total));
    MOE_CHECK(apart(u, ldu, f.K, du, lddu, f.K, T, f.dtype, false));
    MOE_CHECK(apart(dy, lddy, f.K, du, lddu, f.K, T, f.dtype, false));
    const RowPlan p = row_plan(f, expert_offsets, sorted_slot, ws, L, device_status);
    const void *up = u, *dyp = dy;
    int64_t ldup = ldu, lddyp = lddy;
    if (!dense) {
        GatherArgs ga;
        ga.plan = p;
        ga.src[0] = u; ga.ld[0] = ldu; ga.dst[0] = at<void>(ws, L.up);
        ga.zero_pad = true;
        ga.src[1] = dy; ga.ld[1] = lddy; ga.dst[1] = at<void>(ws, L.dyp);
        ga.K = f.K; ga.es = f.es;
        if (dtopk_w && f.bias && f.dtype == MOE_DTYPE_BF16) {
            ga.down_b = w->down_b;
            ga.bias_dot = at<float>(ws, L.bias_dot);
        }
        MOE_CUDA(launch_gather_padded(ga, s));
        up = ga.dst[0];
        dyp = ga.dst[1];
        ldup = lddyp = f.K;
    }
    // dh = dy Wd
    GemmArgs g;
    g.kind = kNN;
    g.plan = p;
    g.dtype = f.dtype;
    g.a = dyp; g.lda = lddyp;
    g.b = w->down_w; g.ldb = f.I; g.sb = int64_t(f.K) * f.I;
    g.M = f.T; g.N = f.I; g.R = f.K;
    GatedArgs ga;
    ga.plan = p;
    ga.I = f.I; ga.interleaved = f.il; ga.act = cfg->activation; ga.limit = cfg->swiglu_limit;
    ga.alpha = cfg->swiglu_alpha;
    ga.dtype = f.dtype;
    ga.topk_w = topk_w;
    ga.pre = const_cast<void*>(pre);
    ga.dgu = at<void>(ws, L.dgu);
    ga.hw = at<void>(ws, L.hw);
    ga.dtopk_w = dtopk_w;
    ga.dyp = dyp;
    ga.down_b = f.bias ? w->down_b : nullptr;
    if (dtopk_w && f.bias) ga.bias_dot = at<float>(ws, L.bias_dot);
    ga.K = f.K;
    if (f.dtype == MOE_DTYPE_F32) {
        g.out = at<void>(ws, L.dh); g.ldo = f.I;
        ga.dh = at<float>(ws, L.dh);
        MOE_CUDA(launch_simt_gemm(&g, 1, s));
        MOE_CUDA(launch_gated_backward(ga, s));
    } else {
        float* parts = dtopk_w ? at<float>(ws, L.parts) : nullptr;
        MOE_CUDA(launch_tc_dgated(g, ga, parts, s));
        if (dtopk_w) MOE_CUDA(launch_dtopk(ga, parts, dgated_parts(p, f.I, f.K), s));
    }
    GemmArgs gm[3];
    int n = 0;
    {  // dWd = dy^T (w h)
        GemmArgs& t = gm[n++];
        t.kind = kTN;
        t.a = dyp; t.lda = lddyp;
        t.b = ga.hw; t.ldb = f.I;
        t.M = f.K; t.N = f.I; t.R = f.T;
        t.out = gr->down_w; t.ldo = f.I; t.so = int64_t(f.K) * f.I;
    }
    {  // [dWg; dWu] = [dg dv]^T u
        GemmArgs& t = gm[n++];
        t.kind = kTN;
        t.a = ga.dgu; t.lda = 2 * f.I;
        t.b = up; t.ldb = ldup;
        t.M = 2 * f.I; t.N = f.K; t.R = f.T;
        t.out = f.il ? gr->gate_up_w : gr->gate_w; t.ldo = f.K; t.so = int64_t(f.I) * f.K * (f.il ? 2 : 1);
        if (!f.il) {
            t.out1 = gr->up_w;
            t.split = f.I;
        }
    }
    {  // du = dg Wg + dv Wu: last, so that the sum over slots finds its rows in L2
        GemmArgs& x = gm[n++];
        x.kind = kNN;
        x.a = ga.dgu; x.lda = 2 * f.I;
        x.b = f.il ? w->gate_up_w : w->gate_w; x.ldb = f.K; x.sb = int64_t(f.I) * f.K * (f.il ? 2 : 1);
        if (!f.il) {
            x.b1 = w->up_w;
            x.split = f.I;
        }
        x.M = f.T; x.N = f.K; x.R = 2 * f.I;
        x.out = dense || !du ? du : at<void>(ws, L.rows_out); x.ldo = dense ? lddu : f.K; x.out_f32 = !dense;
    }
    for (int i = 0; i < n; ++i) {
        gm[i].plan = p;
        gm[i].dtype = f.dtype;
    }
    MOE_CUDA(launch_gemms(gm, n, s));
    if (du && !dense) {
        SumSlotsArgs sa;
        sa.plan = p;
        sa.rows = at<float>(ws, L.rows_out);
        sa.out = du; sa.ldo = lddu;
        sa.K = f.K;
        sa.dtype = f.dtype;
        MOE_CUDA(launch_sum_slots(sa, s));
    }
    if (f.bias) {
        ColsumArgs c[2];
        c[0].plan = c[1].plan = p;
        c[0].dtype = c[1].dtype = f.dtype;
        c[0].partial = at<float>(ws, L.partial);
        c[0].x = ga.dgu; c[0].ldx = 2 * f.I; c[0].cols = 2 * f.I;
        c[0].out = f.il ? gr->gate_up_b : gr->gate_b; c[0].so = int64_t(f.I) * (f.il ? 2 : 1);
        if (!f.il) {
            c[0].out1 = gr->up_b;
            c[0].split = f.I;
        }
        c[1].partial = c[0].partial + round_rows(f.rows) / kRowTile * 2 * f.I;
        c[1].x = dyp; c[1].ldx = lddyp; c[1].cols = f.K;
        c[1].row_scale = topk_w;
        c[1].out = gr->down_b; c[1].so = f.K;
        MOE_CUDA(launch_colsum(c, s));
    }
    return MOE_OK;
}

}  // extern "C"

namespace {
moe_status check_norm(const moe_norm_desc* d, int64_t T) {
    if (!d || d->width <= 0) return MOE_ERR_INVALID_ARGUMENT;
    if (d->kind != MOE_NORM_LAYER && d->kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARGUMENT;
    if (d->dtype != MOE_DTYPE_F32 && d->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(d->eps) || d->eps <= 0.f) return MOE_ERR_INVALID_ARGUMENT;
    if (d->width % (16 / esize(d->dtype))) return MOE_ERR_INVALID_ARGUMENT;
    if (T < 0) return MOE_ERR_INVALID_ARGUMENT;
    if (d->width > kMaxWidth) return MOE_ERR_SHAPE_OVERFLOW;
    if (T > kMaxRows || T * d->width > kMaxElems) return MOE_ERR_SHAPE_OVERFLOW;
    return MOE_OK;
}
size_t norm_ws(const moe_norm_desc* d, int64_t T, bool backward) {
    return backward && T > 0 ? align256(size_t(norm_blocks(T, d->width, d->dtype)) * 2 * d->width * 4) : 0;
}
}  // namespace

extern "C" {

moe_status moe_norm_workspace_size(const moe_norm_desc* d, int64_t T, int32_t backward, size_t* bytes) {
    MOE_CHECK(check_norm(d, T));
    if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
    *bytes = norm_ws(d, T, backward != 0);
    return MOE_OK;
}

moe_status moe_norm_forward(const moe_norm_desc* d, const void* x, int64_t ldx, const void* w, const void* b,
                            int64_t T, void* y, int64_t ldy, float* stats, moe_stream_t stream) {
    MOE_CHECK(check_norm(d, T));
    if (b && d->kind == MOE_NORM_RMS) return MOE_ERR_INVALID_ARGUMENT;
    if (T == 0) return MOE_OK;
    MOE_CHECK(need(x));
    MOE_CHECK(need(w));
    MOE_CHECK(maybe(b));
    MOE_CHECK(need(y));
    MOE_CHECK(maybe(stats));
    MOE_CHECK(stride(ldx, d->width, d->dtype));
    MOE_CHECK(stride(ldy, d->width, d->dtype));
    MOE_CHECK(apart(x, ldx, d->width, y, ldy, d->width, T, d->dtype, true));
    NormArgs a;
    a.T = T; a.H = d->width; a.kind = d->kind; a.dtype = d->dtype; a.eps = d->eps;
    a.x = x; a.ldx = ldx; a.w = w; a.b = b;
    a.y = y; a.ldy = ldy;
    a.stats = stats;
    MOE_CUDA(launch_norm_forward(a, (cudaStream_t)stream));
    return MOE_OK;
}

moe_status moe_norm_backward(const moe_norm_desc* d, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                             const void* w, const float* stats, int64_t T, void* dx, int64_t lddx, void* dw, void* db,
                             void* ws, size_t ws_bytes, moe_stream_t stream) {
    MOE_CHECK(check_norm(d, T));
    if (db && d->kind == MOE_NORM_RMS) return MOE_ERR_INVALID_ARGUMENT;
    MOE_CHECK(maybe(dx));
    MOE_CHECK(maybe(dw));
    MOE_CHECK(maybe(db));
    cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {
        if (dw) MOE_CUDA(cudaMemsetAsync(dw, 0, size_t(d->width) * esize(d->dtype), s));
        if (db) MOE_CUDA(cudaMemsetAsync(db, 0, size_t(d->width) * esize(d->dtype), s));
        return MOE_OK;
    }
    MOE_CHECK(need(dy));
    MOE_CHECK(need(x));
    MOE_CHECK(need(w));
    MOE_CHECK(need(stats));
    MOE_CHECK(stride(lddy, d->width, d->dtype));
    MOE_CHECK(stride(ldx, d->width, d->dtype));
    if (dx) MOE_CHECK(stride(lddx, d->width, d->dtype));
    MOE_CHECK(check_ws(ws, ws_bytes, norm_ws(d, T, true)));
    MOE_CHECK(apart(x, ldx, d->width, dx, lddx, d->width, T, d->dtype, false));
    MOE_CHECK(apart(dy, lddy, d->width, dx, lddx, d->width, T, d->dtype, false));
    NormArgs a;
    a.T = T; a.H = d->width; a.kind = d->kind; a.dtype = d->dtype; a.eps = d->eps;
    a.x = x; a.ldx = ldx; a.w = w;
    a.dy = dy; a.lddy = lddy;
    a.cstats = stats;
    a.dx = dx; a.lddx = lddx;
    a.dw = dw; a.db = db;
    a.partial = static_cast<float*>(ws);
    MOE_CUDA(launch_norm_backward(a, s));
    return MOE_OK;
}

}  // extern "C"
