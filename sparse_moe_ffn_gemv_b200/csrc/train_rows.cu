// train_rows.cu -- the padded row order of routed slots, and the row and column passes of the
// training operators: gather, per-token sum over slots, the gated activation and its
// derivative, column sums (bias gradients). All bound by HBM; every sum has a fixed order.
#include <algorithm>
#include <atomic>

#include "permute_dev.cuh"
#include "ptx.cuh"
#include "train_dev.cuh"

namespace moe {

namespace {

constexpr int kGatherThreads = 512;
constexpr int64_t kCopyBytes = 8 << 20;  // from here on copy_tokens_kernel

// Padded row of a slot, or -1 for one without (dropped): slot_row is written for slots that
// have a row only and never cleared, so what it says is checked against the row's own slot.
__device__ __forceinline__ int row_of_slot(const RowPlan& p, int slot) {
    const int r = p.slot_row[slot];
    return r >= 0 && r < p.poff[p.E] && p.row_slot[r] == slot ? r : -1;
}

// The padded order, which every block derives from the offsets itself (E <= 512: one scan in
// shared memory), so that building it needs no launch of its own; block 0 writes it down.
// Offsets that are not a rising sequence within [0, S] give an empty plan and the status.
struct PlanSmem {
    int32_t cnt[kPermE], start[kPermE], pad[kPermE + 1];
    int warp_tot[kGatherThreads / 32 + 1];
};
__device__ int build_plan(const RowPlan& p, PlanSmem& sm) {
    const int tid = threadIdx.x;
    int bad = 0;
    for (int e = tid; e < p.E; e += kGatherThreads) {
        const int lo = p.offsets[e], hi = p.offsets[e + 1];
        bad |= lo < 0 || hi < lo || hi > p.S;
        sm.start[e] = lo;
        sm.cnt[e] = hi - lo;
    }
    bad = __syncthreads_or(bad);
    for (int e = tid; e < p.E; e += kGatherThreads) {
        if (bad) sm.cnt[e] = sm.start[e] = 0;
        sm.pad[e] = (sm.cnt[e] + kRowTile - 1) / kRowTile * kRowTile;
    }
    __syncthreads();
    const int total = block_exclusive_scan<kGatherThreads>(sm.pad, p.E, sm.warp_tot);
    if (tid == 0) sm.pad[p.E] = total;
    if (blockIdx.x == 0) {
        for (int e = tid; e < p.E; e += kGatherThreads) {
            p.poff[e] = sm.pad[e];
            p.uoff[e] = sm.start[e];
        }
        if (tid == 0) {
            p.poff[p.E] = total;
            p.uoff[p.E] = sm.start[p.E - 1] + sm.cnt[p.E - 1];
            if (bad) set_status(p.status, MOE_ERR_DEVICE_CHECK);
        }
    }
    __syncthreads();
    return total;
}
// Slot of padded row r (-1: padding, or a slot id out of range), written down both ways.
__device__ __forceinline__ int plan_row(const RowPlan& p, const PlanSmem& sm, int r, int e, bool write) {
    const int i = r - sm.pad[e];
    int slot = -1;
    if (i < sm.cnt[e]) {
        slot = p.sorted_slot[sm.start[e] + i];
        if (slot < 0 || slot >= p.S) {
            if (write) set_status(p.status, MOE_ERR_DEVICE_CHECK);
            slot = -1;
        }
    }
    if (write) {
        p.row_slot[r] = slot;
        if (slot >= 0) p.slot_row[slot] = r;
    }
    return slot;
}
__device__ __forceinline__ void zero_row(const GatherArgs& a, int r, int lane) {
    const int64_t vpr = int64_t(a.K) * a.es / 16;
    for (int j = 0; j < 2; ++j)
        if (a.dst[j])
            for (int64_t c = lane; c < vpr; c += 32) static_cast<uint4*>(a.dst[j])[int64_t(r) * vpr + c] = make_uint4(0, 0, 0, 0);
}

// A slot that stands twice among the sorted ones has two rows, and slot_row names one of them. The
// other is dropped: whether row r, of that slot, is one.
__device__ __forceinline__ bool is_repeat(const RowPlan& p, int r, int slot) { return slot >= 0 && p.slot_row[slot] != r; }

// Few rows: the plan and the copies in one launch, a warp per padded row. Padding is zeroed as
// far as a reduction over the expert's rows reads; rows of dropped slots are zeros too.
__global__ void __launch_bounds__(kGatherThreads) gather_padded_kernel(const GatherArgs a) {
    __shared__ PlanSmem sm;
    pdl_begin();
    const RowPlan& p = a.plan;
    const int total = build_plan(p, sm);
    const int lane = threadIdx.x & 31;
    const int64_t vpr = int64_t(a.K) * a.es / 16;
    const int warps = gridDim.x * (kGatherThreads / 32);
    for (int r = blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5); r < total; r += warps) {
        const int e = expert_of_row(sm.pad, p.E, r);
        const int slot = plan_row(p, sm, r, e, lane == 0);
        if (slot < 0) {
            const int i = r - sm.pad[e];
            if (i < sm.cnt[e] || (a.zero_pad && i < (sm.cnt[e] + kRowPad - 1) / kRowPad * kRowPad)) zero_row(a, r, lane);
            continue;
        }
        const int64_t t = slot / p.k;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!a.src[j]) continue;
            const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(a.src[j]) + t * a.ld[j] * a.es);
            uint4* d = static_cast<uint4*>(a.dst[j]) + int64_t(r) * vpr;
            int64_t c = lane;
            for (; c + 96 < vpr; c += 128) {  // four vectors in flight per lane
                const uint4 v0 = s[c], v1 = s[c + 32], v2 = s[c + 64], v3 = s[c + 96];
                d[c] = v0; d[c + 32] = v1; d[c + 64] = v2; d[c + 96] = v3;
            }
            for (; c < vpr; c += 32) d[c] = s[c];
        }
    }
}

// Many rows: the plan, a thread per padded row; copy_tokens_kernel does the rest.
__global__ void __launch_bounds__(kGatherThreads) plan_rows_kernel(const GatherArgs a) {
    __shared__ PlanSmem sm;
    pdl_begin();
    const RowPlan& p = a.plan;
    const int total = build_plan(p, sm);
    for (int r = blockIdx.x * kGatherThreads + threadIdx.x; r < total; r += gridDim.x * kGatherThreads)
        plan_row(p, sm, r, expert_of_row(sm.pad, p.E, r), true);
}

// Token by token: a token's rows of the sources (a piece of up to kPiece bytes each) come to
// shared memory once and go out to every row of its k slots, by bulk copies that one lane
// issues, so that no row is read more than once and no thread waits for a load or a store of
// its own (a warp copying one row at a time moved 3.8 TB/s). With a down bias, dy . down_b[e] of
// every slot is taken from the rows in passing.
constexpr int kPiece = 8192;
constexpr int kCopyWarps = 8;
__global__ void __launch_bounds__(kCopyWarps * 32) copy_tokens_kernel(const GatherArgs a) {
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ uint64_t full[kCopyWarps];
    __shared__ int32_t pad[kPermE + 1];
    const RowPlan& p = a.plan;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row_bytes = int64_t(a.K) * a.es;
    const int piece = int(min(int64_t(kPiece), row_bytes));
    const int ns = a.src[1] ? 2 : 1;
    uint8_t* buf = sm + warp * ns * piece;
    if (lane == 0) mbar_init(&full[warp], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_begin();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) pad[e] = p.poff[e];
    __syncthreads();
    const uint64_t pol = policy_evict_first();
    uint32_t phase = 0;
    for (int64_t t = int64_t(blockIdx.x) * kCopyWarps + warp; t < p.T; t += int64_t(gridDim.x) * kCopyWarps) {
        float dot[kMaxTopK];
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) dot[j] = 0.0f;
        const int r = lane < p.k ? row_of_slot(p, int(t) * p.k + lane) : -1;  // of slot `lane`
        for (int64_t at = 0; at < row_bytes; at += piece) {
            const uint32_t n = uint32_t(min(int64_t(piece), row_bytes - at));
            if (lane == 0) {
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the buffers are free
                mbar_expect_tx(&full[warp], ns * n);
                for (int i = 0; i < ns; ++i)
                    bulk_g2s(buf + i * piece, static_cast<const char*>(a.src[i]) + t * a.ld[i] * a.es + at, n, &full[warp], pol);
            }
            __syncwarp();
            if (!mbar_try(&full[warp], phase) && !mbar_wait(&full[warp], phase, gtimer() + 2000000000ull)) {
                set_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
                mbar_wait(&full[warp], phase, gtimer() + 2000000000ull);  // its copies may still land
                if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                return;
            }
            phase ^= 1u;
            for (int j = 0; j < p.k; ++j) {
                const int row = __shfl_sync(0xffffffffu, r, j);
                if (row < 0) continue;
                if (lane == 0)
                    for (int i = 0; i < ns; ++i)
                        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                         static_cast<char*>(a.dst[i]) + row * row_bytes + at),
                                     "r"(su32(buf + i * piece)), "r"(n)
                                     : "memory");
            }
            if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            if (a.down_b) {  // bf16 only
                for (int j = 0; j < p.k; ++j) {
                    const int row = __shfl_sync(0xffffffffu, r, j);
                    if (row < 0) continue;
                    const int e = expert_of_row(pad, p.E, row);
                    const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(a.down_b) + int64_t(e) * a.K + at / 2;
                    float acc = 0.0f;
                    for (uint32_t c = lane * 8; c < n / 2; c += 256) {
                        float x[8], y[8];
                        load_vec(reinterpret_cast<const __nv_bfloat16*>(buf + piece) + c, x);
                        load_vec(b + c, y);
#pragma unroll
                        for (int q = 0; q < 8; ++q) acc = fmaf(x[q], y[q], acc);
                    }
#pragma unroll
                    for (int q = 0; q < kMaxTopK; ++q)
                        if (q == j) dot[q] += acc;
                }
                __syncwarp();  // the buffers may be refilled
            }
        }
        if (a.down_b) {
#pragma unroll
            for (int j = 0; j < kMaxTopK; ++j) {
                if (j >= p.k) break;
                const float v = warp_sum(dot[j]);
                if (lane == 0) a.bias_dot[t * p.k + j] = v;
            }
        }
    }
    // rows that no token names: padding as far as a reduction reads, dropped slots, and the second
    // row of a slot that stands twice (of no slot from here on) are zeros. Neighbouring rows go to
    // different warps, since padding stands together.
    const int total = pad[p.E], warps = gridDim.x * kCopyWarps;
    for (int r0 = blockIdx.x * kCopyWarps + warp; r0 < total; r0 += 32 * warps) {
        const int64_t rl = r0 + int64_t(lane) * warps;
        bool zero = false;
        if (rl < total) {
            const int r = int(rl), slot = p.row_slot[r];
            if (slot < 0) {
                const int e = expert_of_row(pad, p.E, r), i = r - pad[e], cnt = p.uoff[e + 1] - p.uoff[e];
                zero = i < cnt || (a.zero_pad && i < (cnt + kRowPad - 1) / kRowPad * kRowPad);
            } else if (is_repeat(p, r, slot)) {
                p.row_slot[r] = -1;
                set_status(p.status, MOE_ERR_DEVICE_CHECK);
                zero = true;
            }
        }
        for (unsigned m = __ballot_sync(0xffffffffu, zero); m; m &= m - 1) zero_row(a, r0 + (__ffs(m) - 1) * warps, lane);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Each token's slots' rows added in slot order in f32. (gather_padded_kernel cannot see a slot that
// stands twice, since its blocks plan side by side: it shows here.)
template <typename T>
__global__ void __launch_bounds__(256) sum_slots_kernel(const SumSlotsArgs a) {
    pdl_begin();
    for (int r = blockIdx.x * 256 + threadIdx.x; r < a.plan.poff[a.plan.E]; r += gridDim.x * 256)
        if (is_repeat(a.plan, r, a.plan.row_slot[r])) set_status(a.plan.status, MOE_ERR_DEVICE_CHECK);
    constexpr int V = Vec<T>::N;
    const int vpr = a.K / V;
    const int64_t n = a.plan.T * vpr;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t t = i / vpr;
        const int c = int(i - t * vpr) * V;
        float acc[V] = {};
        for (int j = 0; j < a.plan.k; ++j) {
            const int r = row_of_slot(a.plan, int(t) * a.plan.k + j);
            if (r < 0) continue;
            float f[V];
#pragma unroll
            for (int q = 0; q < V; q += 4) {
                const float4 v = *reinterpret_cast<const float4*>(a.rows + int64_t(r) * a.K + c + q);
                f[q] = v.x; f[q + 1] = v.y; f[q + 2] = v.z; f[q + 3] = v.w;
            }
#pragma unroll
            for (int q = 0; q < V; ++q) acc[q] += f[q];
        }
        if (a.residual) {
            float f[V];
            load_vec(static_cast<const T*>(a.residual) + t * a.ldr + c, f);
#pragma unroll
            for (int q = 0; q < V; ++q) acc[q] += f[q];
        }
        store_vec(static_cast<T*>(a.out) + t * a.ldo + c, acc);
    }
}

// Rows of the plan: how many, and per row its slot and its row in the caller's sorted order
// (-1 for padding).
struct RowRef {
    int e;
    int64_t pos;  // caller's sorted position, or -1
    int slot;
};
__device__ __forceinline__ int64_t plan_rows(const RowPlan& p) { return p.offsets ? p.poff[p.E] : p.T; }
__device__ __forceinline__ RowRef row_ref(const RowPlan& p, int64_t r) {
    RowRef o;
    if (!p.offsets) {
        o.e = 0;
        o.pos = r;
        o.slot = int(r);
        return o;
    }
    o.slot = p.row_slot[r];
    o.e = expert_of_row(p.poff, p.E, int(r));
    o.pos = o.slot < 0 ? -1 : int64_t(p.uoff[o.e]) + (r - p.poff[o.e]);
    return o;
}

// One warp per row; gate and up of unit i. (f32; bf16 has both passes in its products' epilogues.)
__global__ void __launch_bounds__(256) gated_forward_kernel(const GatedArgs a) {
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int64_t rows = plan_rows(a.plan), warps = int64_t(gridDim.x) * 8;
    for (int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); r < rows; r += warps) {
        const RowRef o = row_ref(a.plan, r);
        const float* gp = a.gp + r * 2 * a.I;
        float* h = static_cast<float*>(a.h) + r * a.I;
        float* pre = a.pre && o.pos >= 0 ? static_cast<float*>(a.pre) + o.pos * 2 * a.I : nullptr;
        for (int i = lane; i < a.I; i += 32) {
            const int cg = a.interleaved ? 2 * i : i, cv = a.interleaved ? 2 * i + 1 : a.I + i;
            const float g = gp[cg], v = gp[cv];
            h[i] = gated_h<false>(a.act, g, v, a.limit, a.alpha);
            if (pre) {
                pre[cg] = g;
                pre[cv] = v;
            }
        }
    }
}

__global__ void __launch_bounds__(256) gated_backward_kernel(const GatedArgs a) {
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int64_t rows = plan_rows(a.plan), warps = int64_t(gridDim.x) * 8;
    for (int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); r < rows; r += warps) {
        const RowRef o = row_ref(a.plan, r);
        float* dgu = static_cast<float*>(a.dgu) + r * 2 * a.I;
        float* hw = static_cast<float*>(a.hw) + r * a.I;
        const float* pre = static_cast<const float*>(a.pre) + o.pos * 2 * a.I;
        const float wt = a.topk_w && o.slot >= 0 ? a.topk_w[o.slot] : 1.0f;
        float dw = 0.0f;
        for (int i = lane; i < a.I; i += 32) {
            const int cg = a.interleaved ? 2 * i : i, cv = a.interleaved ? 2 * i + 1 : a.I + i;
            float dg = 0.f, dv = 0.f, hh = 0.f;
            if (o.pos >= 0) {
                float hg, hv;
                gated_grad(a.act, pre[cg], pre[cv], a.limit, a.alpha, hh, hg, hv);
                const float d = a.dh[r * a.I + i];
                dw += d * hh;
                dg = d * wt * hg;
                dv = d * wt * hv;
                hh *= wt;
            }
            dgu[cg] = dg;
            dgu[cv] = dv;
            hw[i] = hh;
        }
        if (!a.dtopk_w || o.slot < 0 || !a.plan.offsets) continue;
        if (a.down_b)
            for (int c = lane; c < a.K; c += 32)
                dw += static_cast<const float*>(a.dyp)[r * a.K + c] *
                      static_cast<const float*>(a.down_b)[int64_t(o.e) * a.K + c];
        dw = warp_sum(dw);
        if (lane == 0) a.dtopk_w[o.slot] = dw;
    }
    if (a.dtopk_w && a.plan.offsets)  // slots without a row
        for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < a.plan.S; i += int64_t(gridDim.x) * 256)
            if (row_of_slot(a.plan, int(i)) < 0) a.dtopk_w[i] = 0.0f;
}

// One thread per slot: its row's partial sums in order, plus dy . down_b with a down bias.
__global__ void __launch_bounds__(256) dtopk_kernel(const GatedArgs a, const float* partial, int parts) {
    pdl_begin();
    for (int64_t slot = int64_t(blockIdx.x) * 256 + threadIdx.x; slot < a.plan.S; slot += int64_t(gridDim.x) * 256) {
        const int64_t r = row_of_slot(a.plan, int(slot));
        float dw = 0.0f;
        if (r >= 0) {
            if (a.bias_dot) dw = a.bias_dot[slot];
#pragma unroll 8
            for (int i = 0; i < parts; ++i) dw += partial[r * parts + i];
        }
        a.dtopk_w[slot] = dw;
    }
}

// Column sums, first pass: a block sums kRowTile rows (which belong to one expert) of 64
// 16-byte column vectors; each thread one vector and every 4th row, 8 rows' loads in flight.
constexpr int kColVecs = 64, kColRows = 4, kColDeep = 8;
template <typename T>
__global__ void __launch_bounds__(kColVecs * kColRows) colsum_kernel(const ColsumArgs a0, const ColsumArgs a1, int blocks0,
                                                                     int blocks) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    __shared__ float sm[kColRows][kColVecs][V + 1];
    const RowPlan& p = a0.plan;
    const int64_t b = int64_t(blockIdx.x) * kRowTile;
    int64_t end = p.T;
    if (p.offsets) {
        if (b >= p.poff[p.E]) return;
        const int e = expert_of_row(p.poff, p.E, int(b));
        end = p.poff[e] + (p.uoff[e + 1] - p.uoff[e]);
    }
    end = min(end, b + kRowTile);
    const int ry = threadIdx.x / kColVecs;
    for (int cb = blockIdx.y; cb < blocks; cb += gridDim.y) {  // one, up to 65535 column blocks
        const bool second = cb >= blocks0;
        const ColsumArgs& a = second ? a1 : a0;
        const int c = ((cb - (second ? blocks0 : 0)) * kColVecs + threadIdx.x % kColVecs) * V;
        float acc[V] = {};
        if (c < a.cols) {
            for (int64_t r = b + ry; r < end; r += kColDeep * kColRows) {
                uint4 f[kColDeep];
                float sc[kColDeep];
#pragma unroll
                for (int u = 0; u < kColDeep; ++u) {
                    const int64_t ru = r + u * kColRows;
                    f[u] = make_uint4(0, 0, 0, 0);
                    sc[u] = 1.0f;
                    if (ru >= end) continue;
                    f[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + ru * a.ldx + c);
                    if (a.row_scale) {
                        const int slot = p.row_slot[ru];
                        sc[u] = slot < 0 ? 0.0f : a.row_scale[slot];
                    }
                }
#pragma unroll
                for (int u = 0; u < kColDeep; ++u) {
                    float v[V];
                    unpack_vec<T>(f[u], v);
#pragma unroll
                    for (int q = 0; q < V; ++q) acc[q] = fmaf(v[q], sc[u], acc[q]);
                }
            }
        }
        __syncthreads();  // the column block before has been read
#pragma unroll
        for (int q = 0; q < V; ++q) sm[ry][threadIdx.x % kColVecs][q] = acc[q];
        __syncthreads();
        if (ry == 0 && c < a.cols) {
            float* o = a.partial + int64_t(blockIdx.x) * a.cols + c;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                float s = 0.f;
#pragma unroll
                for (int y = 0; y < kColRows; ++y) s += sm[y][threadIdx.x][q];
                o[q] = s;
            }
        }
    }
}

// Second pass, 32 columns of one expert per block: 8 threads per column each add every 8th
// partial row of the expert, then those 8 in order; rounded once. Without a plan (dense): the
// `parts` rows of one matrix.
template <typename T>
__global__ void __launch_bounds__(256) colsum_finish_kernel(const ColsumArgs a0, const ColsumArgs a1, int blocks0, int parts) {
    pdl_begin();
    __shared__ float sm[8][33];
    const int e = blockIdx.y;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const bool second = int(blockIdx.x) >= blocks0;
    const ColsumArgs& a = second ? a1 : a0;
    const int c = (blockIdx.x - (second ? blocks0 : 0)) * 32 + x;
    int64_t p0 = 0, p1 = parts;
    if (a.plan.offsets) {
        p0 = a.plan.poff[e] / kRowTile;
        p1 = a.plan.poff[e + 1] / kRowTile;
    }
    float s = 0.f;
    if (c < a.cols)
#pragma unroll 4
        for (int64_t z = p0 + y; z < p1; z += 8) s += a.partial[z * a.cols + c];
    sm[y][x] = s;
    __syncthreads();
    if (y != 0 || c >= a.cols) return;
    s = sm[0][x];
#pragma unroll
    for (int j = 1; j < 8; ++j) s += sm[j][x];
    T* o = a.split && c >= a.split ? static_cast<T*>(a.out1) + e * a.so + (c - a.split)
                                   : static_cast<T*>(a.out) + e * a.so + c;
    *o = from_f<T>(s);
}

// dz of a block of rows, and its column sums: two rows of loads in flight per thread, four
// blocks per SM.
template <typename T>
__global__ void __launch_bounds__(kColVecs * kColRows, 4) dact_kernel(const DactArgs a, int splits) {
    pdl_begin();
    constexpr int V = Vec<T>::N;
    constexpr bool FAST = V == 8;
    const int64_t per = (a.T + splits - 1) / splits;
    const int64_t b = blockIdx.y * per, end = min(a.T, b + per);
    const int c = (blockIdx.x * kColVecs + threadIdx.x % kColVecs) * V;
    const int ry = threadIdx.x / kColVecs;
    float acc[V] = {};
    if (c < a.N) {
        for (int64_t r = b + ry; r < end; r += 2 * kColRows) {
            uint4 dv[2], zv[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t ru = r + u * kColRows;
                dv[u] = zv[u] = make_uint4(0, 0, 0, 0);
                if (ru >= end) continue;
                dv[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.dy) + ru * a.lddy + c);
                if (a.act != MOE_LINEAR_NONE)
                    zv[u] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.pre) + ru * a.N + c);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t ru = r + u * kColRows;
                float f[V];
                unpack_vec<T>(dv[u], f);
                if (a.act != MOE_LINEAR_NONE && ru < end) {
                    float z[V];
                    unpack_vec<T>(zv[u], z);
#pragma unroll
                    for (int q = 0; q < V; ++q) f[q] *= linear_dact<FAST>(a.act, z[q]);
                    store_vec(static_cast<T*>(a.dz) + ru * a.N + c, f);
                }
#pragma unroll
                for (int q = 0; q < V; ++q) acc[q] += f[q];
            }
        }
    }
    if (!a.partial) return;
    __shared__ float sm[kColRows][kColVecs][V + 1];
#pragma unroll
    for (int q = 0; q < V; ++q) sm[ry][threadIdx.x % kColVecs][q] = acc[q];
    __syncthreads();
    if (ry == 0 && c < a.N) {
        float* o = a.partial + int64_t(blockIdx.y) * a.N + c;
#pragma unroll
        for (int q = 0; q < V; ++q) {
            float s = 0.f;
#pragma unroll
            for (int y = 0; y < kColRows; ++y) s += sm[y][threadIdx.x][q];
            o[q] = s;
        }
    }
}

unsigned grid_for(int64_t items, int64_t per_block, int64_t most) {
    return unsigned(std::max<int64_t>(1, std::min(most, (items + per_block - 1) / per_block)));
}

}  // namespace

cudaError_t launch_gather_padded(const GatherArgs& a, cudaStream_t s) {
    const unsigned grid = grid_for(a.plan.max_rows, kGatherThreads / 32, 148 * 4);
    // few rows: one launch that copies as it plans; else (and for the bias products) two
    if (!a.down_b && a.plan.S * a.K * a.es < kCopyBytes) {
        return launch_chained(gather_padded_kernel, grid, kGatherThreads, 0, s, a);
    }
    MOE_LAUNCH(launch_chained(plan_rows_kernel, grid_for(a.plan.max_rows, kGatherThreads, 148 * 2), kGatherThreads, 0, s, a));
    const int64_t row = int64_t(a.K) * a.es;
    const int smem = int(std::min<int64_t>(kPiece, row)) * (a.src[1] ? 2 : 1) * kCopyWarps;
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(allowed.load() & bit)) {
        e = cudaFuncSetAttribute(copy_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kPiece * kCopyWarps);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit);
    }
    copy_tokens_kernel<<<grid_for(a.plan.T, kCopyWarps, 148 * std::max(1, std::min(8, 200 * 1024 / smem))), kCopyWarps * 32,
                         smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_sum_slots(const SumSlotsArgs& a, cudaStream_t s) {
    const int V = a.dtype == MOE_DTYPE_F32 ? 4 : 8;
    const unsigned grid = grid_for(a.plan.T * (a.K / V), 256, 148 * 16);
    if (a.dtype == MOE_DTYPE_F32) return launch_spread(sum_slots_kernel<float>, grid, 256, s, a);
    return launch_spread(sum_slots_kernel<__nv_bfloat16>, grid, 256, s, a);
}

cudaError_t launch_gated_forward(const GatedArgs& a, cudaStream_t s) {
    return launch_chained(gated_forward_kernel, grid_for(a.plan.max_rows, 8, 148 * 8), 256, 0, s, a);
}

cudaError_t launch_gated_backward(const GatedArgs& a, cudaStream_t s) {
    return launch_chained(gated_backward_kernel, grid_for(a.plan.max_rows, 8, 148 * 8), 256, 0, s, a);
}

cudaError_t launch_dtopk(const GatedArgs& a, const float* partial, int parts, cudaStream_t s) {
    dtopk_kernel<<<grid_for(a.plan.S, 256, 148 * 8), 256, 0, s>>>(a, partial, parts);
    return cudaGetLastError();
}

cudaError_t launch_colsum(const ColsumArgs (&a)[2], cudaStream_t s) {
    const int V = a[0].dtype == MOE_DTYPE_F32 ? 4 : 8, per = kColVecs * V;
    const int64_t tiles = (a[0].plan.max_rows + kRowTile - 1) / kRowTile;
    const int c0 = (a[0].cols + per - 1) / per, c1 = (a[1].cols + per - 1) / per;
    const int f0 = (a[0].cols + 31) / 32, f1 = (a[1].cols + 31) / 32;
    const dim3 grid(unsigned(tiles), std::min(c0 + c1, 65535)), fin(f0 + f1, a[0].plan.E);
    if (a[0].dtype == MOE_DTYPE_F32) {
        MOE_LAUNCH(launch_spread(colsum_kernel<float>, grid, kColVecs * kColRows, s, a[0], a[1], c0, c0 + c1));
        MOE_LAUNCH(launch_chained(colsum_finish_kernel<float>, fin, 256, 0, s, a[0], a[1], f0, int(tiles)));
    } else {
        MOE_LAUNCH(launch_spread(colsum_kernel<__nv_bfloat16>, grid, kColVecs * kColRows, s, a[0], a[1], c0, c0 + c1));
        MOE_LAUNCH(launch_chained(colsum_finish_kernel<__nv_bfloat16>, fin, 256, 0, s, a[0], a[1], f0, int(tiles)));
    }
    return cudaSuccess;
}

int dact_splits(int64_t T, int N) {
    const int64_t cb = (N + 511) / 512;
    return int(std::max<int64_t>(1, std::min<int64_t>(592 / cb, T / 16)));
}

cudaError_t launch_dact(const DactArgs& a, cudaStream_t s) {
    const int V = a.dtype == MOE_DTYPE_F32 ? 4 : 8;
    const int splits = dact_splits(a.T, a.N);
    const dim3 grid((a.N / V + kColVecs - 1) / kColVecs, splits);
    if (a.dtype == MOE_DTYPE_F32) MOE_LAUNCH(launch_chained(dact_kernel<float>, grid, kColVecs * kColRows, 0, s, a, splits));
    else MOE_LAUNCH(launch_chained(dact_kernel<__nv_bfloat16>, grid, kColVecs * kColRows, 0, s, a, splits));
    if (a.partial) {
        ColsumArgs c;
        c.cols = a.N;
        c.out = a.db;
        c.partial = a.partial;
        const unsigned fin = (a.N + 31) / 32;
        if (a.dtype == MOE_DTYPE_F32) MOE_LAUNCH(launch_chained(colsum_finish_kernel<float>, fin, 256, 0, s, c, c, fin, splits));
        else MOE_LAUNCH(launch_chained(colsum_finish_kernel<__nv_bfloat16>, fin, 256, 0, s, c, c, fin, splits));
    }
    return cudaSuccess;
}

}  // namespace moe
