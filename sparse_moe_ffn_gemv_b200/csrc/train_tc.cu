// train_tc.cu -- bf16 matrix products of the training operators on the 5th-generation tensor
// cores (tcgen05, accumulators in TMEM), fed by TMA, with the element-wise work of each
// product in its epilogue.
//
//   D[m, n] = sum_r A(m, r) B(n, r)       f32 accumulation
//   kNT  A [m][r], B [n][r]  both operands with the reduction contiguous (K-major)
//   kNN  A [m][r], B [r][n]  B with n contiguous (MN-major): dz times a weight plane
//   kTN  A [r][m], B [r][n]  both MN-major: dz^T times the tokens, reduced over an expert's rows
//   kMix the independent kNN and kTN products of a small backward pass in one launch (large ones
//        run one after the other: together they measured no faster)
//
// No operand is transposed in memory: the matrix instructions read either order from shared
// memory, and TMA brings either as boxes of one or two 64-column blocks (MN-major, 64 rows) or
// 64 x 128 (K-major) with the 128-byte swizzle. Tiles are 128 x 256 on one CTA, or 256 x 256 on a
// pair of CTAs (cta_group::2: each CTA loads half of both operands, which halves the operand
// traffic per product; one CTA's tile needs 96 bytes per cycle of L2 reads to keep its tensor core
// busy, a pair's 64), or 512 x 256 on a pair (48 bytes) for long dense reductions.
//
// One persistent CTA (pair) per SM (pair):
//   warp 0      TMA producer into a ring of 64-deep reduction blocks
//   warp 1      MMA issuer (one thread; of a pair, the leader's)
//   warps 2..9  epilogue, two accumulator sets in TMEM so that it overlaps the next tile's
//               products: one accumulator row per lane, 32 columns at a time, results turned
//               through 2 KB of shared memory per warp so that global rows are written and
//               read in whole 32-byte sectors
// The gated derivative's epilogue is at the 168 registers that 320 threads can have and spills: 36
// bytes stored, 56 loaded per thread (interleaved planes 8 and 8); the split forms, whose CTAs run one
// tile each, 204 and 152.
// Every wait gives up after 2 s, records MOE_ERR_DEVICE_TIMEOUT, lets its own copies and
// products finish and returns; TMEM is always freed.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "ptx.cuh"
#include "train_dev.cuh"

namespace moe {

namespace {

constexpr int kBR = 64;        // reduction block: 128 bytes of bf16, one swizzle atom
constexpr int kCols = 256;     // columns of a tile (N of the matrix instruction)
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxE = 512;
constexpr int kABytes = 128 * kBR * 2;  // one 128-row operand tile
constexpr uint64_t kWaitNs = 2000000000ull;

constexpr int kMix = 3;  // besides enum GemmKind
constexpr int kMaxMix = 3;
// kGateUpI, kDGatedI: alternating gate / up columns.
// kStoreBulk: kTN on pairs, D leaves by TMA.
// kStoreTall: pairs on tiles of 512 rows.
enum Epi { kStore = 0, kGateUp = 1, kGateUpI = 2, kDGated = 3, kDGatedI = 4, kStoreBulk = 5, kStoreTall = 6 };

// Division by a launch constant: n / d = umulhi(n, m) >> s for 0 <= n < 2^31 (m = ceil(2^(32+s) / d)
// with 2^s < d <= 2^(s+1)), two instructions in place of a divide in every role's tile walk.
struct FastDiv {
    uint32_t d, m, s;
    __device__ __forceinline__ int operator()(int n) const {
        return d == 1 ? n : int(__umulhi(uint32_t(n), m) >> s);
    }
};
FastDiv fast_div(int64_t d) {
    FastDiv f{uint32_t(d), 0, 0};
    if (d <= 1) return f;
    uint32_t lg = 0;  // ceil(log2 d)
    while ((int64_t(1) << lg) < d) ++lg;
    f.s = lg - 1;
    f.m = uint32_t(((uint64_t(1) << (32 + f.s)) + d - 1) / d);
    return f;
}

struct TcTrain {
    CUtensorMap a, b0, b1;
    CUtensorMap o0, o1;     // kStoreBulk: the planes of D
    FastDiv d_tile, d_m, d_band, d_width, d_tail;  // see tile_of
    int tn;                 // kMix: a kTN product
    int bulk_out, tall;     // host: kStoreBulk, kStoreTall
    int wide_a, wide_b;     // MN-major operand in boxes of two 64-column blocks (see map_mn)
    int splits;             // CTAs of a cluster that share a tile's reduction (SPLIT)
    // rows
    const int32_t *offsets, *poff, *uoff, *row_slot;  // grouped (offsets != null)
    int E;
    int64_t rows;           // dense: rows of A (kNT, kNN) or reduction rows (kTN)
    // tile grid: rows of D in row tiles (kTN: of `halves` planes of `mrows` rows each), n_blocks
    int64_t mrows;
    int halves, m_blocks, n_blocks, band;
    int N;                  // columns of D (kGateUp: units)
    int nk, nk_half;        // reduction blocks (kNT, kNN) and of one half (kNN split)
    int b_split;            // kNN: the second half reads b1
    // epilogue
    const __nv_bfloat16 *bias0, *bias1;
    int64_t sbias;
    int act;
    const float* row_scale;
    const __nv_bfloat16* residual;
    int64_t ldr;
    __nv_bfloat16* pre;     // kStore: z; kGateUp: out; kDGated: in
    int64_t ldp;
    void *out, *out1;
    int64_t ldo, so;
    int out_f32;
    float limit, alpha, cexp;
    __nv_bfloat16 *dgu, *hw;
    float* partial;         // kDGated: [rows, parts]
    int parts;
    int* status;
};

template <int NP> struct TcArgs {
    TcTrain p[NP];  // one plan and status for all
    int n;
};

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand descriptors, 128-byte swizzle. K-major: 8-row groups 1024 B apart.
// MN-major: 64-element blocks of m (n) 8192 B apart, groups of 8 reduction rows 1024 B apart.
template <bool MN>
__device__ __forceinline__ uint64_t operand(uint32_t saddr) {
    const uint64_t lbo = MN ? 8192 >> 4 : 1, sbo = 1024 >> 4;
    return uint64_t((saddr & 0x3FFFFu) >> 4) | (lbo << 16) | (sbo << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Bytes from one 16-deep reduction step to the next within a block.
template <bool MN> constexpr uint32_t kStep = MN ? 16 * 128 : 32;

__host__ __device__ constexpr uint32_t idesc(bool a_mn, bool b_mn, int m, int n) {  // bf16 x bf16 -> f32
    return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
           (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t acc) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(desc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(desc), "r"(acc)
            : "memory");
}
// Arrive on the barrier (of both CTAs of a pair) once the products issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                su32(bar)),
            "h"(uint16_t(3))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(bar))
                     : "memory");
}
// Arrive on the leader's barrier. CTA scope: what is handed over is TMEM, ordered by the tcgen05
// fence before it; a release at cluster scope would first wait for the warp's global stores
// (a third of the weight gradients' epilogue went there).
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(bar, 0)) : "memory");
}
// 32 accumulator columns of this lane's row; valid after tmem_wait.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Bounded wait; the clock starts when the wait does, so that a long launch is no timeout. The
// thread sleeps in the test (it wakes when the phase completes): under the power cap polling
// costs clocks, 8192^3 took 10% longer with the products' issuer spinning.
__device__ __forceinline__ bool wait_bar(uint64_t* b, uint32_t parity) {
    if (mbar_try_sleep(b, parity, 20000u)) return true;
    const uint64_t deadline = gtimer() + kWaitNs;
    while (!mbar_try_sleep(b, parity, 20000u))
        if (gtimer() > deadline) return false;
    return true;
}

// ------------------------------------------------------------------ 64-byte row segments
// A warp's 32 rows of 64 bytes: lane r holds row r (four 16-byte pieces). In shared memory
// piece c of row r sits at place c ^ (r / 2 % 4) of its row, so that neither side of the turn
// has bank conflicts.
__device__ __forceinline__ uint32_t seg(int r, int c) { return uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

// Writes rows [0, rows) of the segment, its first `bytes` bytes (a multiple of 16).
__device__ __forceinline__ void store_rows(uint8_t* sm, int lane, const uint4 (&v)[4], void* base, int64_t ld_bytes,
                                           int rows, int bytes) {
#pragma unroll
    for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(sm + seg(lane, c)) = v[c];
    __syncwarp();
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        const uint4 x = *reinterpret_cast<const uint4*>(sm + seg(r, c));
        if (r < rows && c * 16 < bytes) *reinterpret_cast<uint4*>(static_cast<char*>(base) + r * ld_bytes + c * 16) = x;
    }
    __syncwarp();
}
// Rows of 128 bytes in the same 2 KB, 16 rows at a time (piece c of row r at c ^ (r % 8)): whole
// cache lines, half the write requests.
__device__ __forceinline__ void store_lines(uint8_t* sm, int lane, const uint4 (&lo)[4], const uint4 (&hi)[4], void* base,
                                            int64_t ld_bytes, int rows, int bytes) {
    const int c = lane & 7;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if ((lane >> 4) == h) {
            const int r = lane & 15;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                *reinterpret_cast<uint4*>(sm + r * 128 + ((i ^ (r & 7)) << 4)) = lo[i];
                *reinterpret_cast<uint4*>(sm + r * 128 + (((4 + i) ^ (r & 7)) << 4)) = hi[i];
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 4 + (lane >> 3);
            const uint4 x = *reinterpret_cast<const uint4*>(sm + r * 128 + ((c ^ (r & 7)) << 4));
            if (h * 16 + r < rows && c * 16 < bytes)
                *reinterpret_cast<uint4*>(static_cast<char*>(base) + (h * 16 + r) * ld_bytes + c * 16) = x;
        }
        __syncwarp();
    }
}
// Reading them: fetch issues the loads (rows and bytes past the limits give zeros), turn hands
// each lane its row.
__device__ __forceinline__ void fetch_rows(int lane, uint4 (&x)[4], const void* base, int64_t ld_bytes, int rows,
                                           int bytes) {
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        x[i] = make_uint4(0, 0, 0, 0);
        if (r < rows && c * 16 < bytes)
            x[i] = *reinterpret_cast<const uint4*>(static_cast<const char*>(base) + r * ld_bytes + c * 16);
    }
}
__device__ __forceinline__ void turn_rows(uint8_t* sm, int lane, uint4 (&x)[4]) {
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(sm + seg(i * 8 + (lane >> 2), c)) = x[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(sm + seg(lane, i));
    __syncwarp();
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void pack_row(const float (&f)[32], uint4 (&v)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        v[c] = make_uint4(pack2(f[8 * c], f[8 * c + 1]), pack2(f[8 * c + 2], f[8 * c + 3]),
                          pack2(f[8 * c + 4], f[8 * c + 5]), pack2(f[8 * c + 6], f[8 * c + 7]));
}
__device__ __forceinline__ void unpack_row(const uint4 (&v)[4], float (&f)[32]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float t[8];
        unpack8(v[c], t);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[8 * c + j] = t[j];
    }
}
// 32 bias values from column c on, columns past `limit` zero (limit and c multiples of 8).
__device__ __forceinline__ void add_bias(const __nv_bfloat16* b, int c, int limit, float (&f)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (c + 8 * q >= limit) break;
        float t[8];
        unpack8(*reinterpret_cast<const uint4*>(b + c + 8 * q), t);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[8 * q + j] += t[j];
    }
}

// ------------------------------------------------------------------ tiles
struct Tile {
    int e;          // expert, or 0
    int half;       // kTN: plane of D
    int64_t row0;   // first row of D in A's row space (kTN: in the plane)
    int limit;      // rows of D to write (grouped: up to the next reduction block of kTN)
    int nvalid;     // of those, rows that hold slots
    int n0;         // first column
    int nk;         // reduction blocks
    int last;       // 16-deep steps of the last one
    int64_t r0;     // kTN: first reduction row
    int64_t pos0;   // first row in the caller's sorted order
};

struct Tables {
    int poff[kMaxE + 1], ts[kMaxE + 1], uoff[kMaxE + 1];
};

template <int KIND, int EPI, bool PAIR>
struct Shape {
    // Tall: each CTA holds two 128-row halves of A against one half of B, 48 KB of operands per
    // 1024 cycles of products in place of 32 KB per 512 (a CTA's copies bring about 64 bytes per
    // cycle, so that the shorter tile has none to spare). Both accumulator sets belong to one
    // tile: the epilogue of a half runs beside the next tile's products on the other.
    static constexpr bool TALL = EPI == kStoreTall;
    static constexpr int MH = TALL ? 2 : 1;             // 128-row halves per CTA
    static constexpr int BM = (PAIR ? 256 : 128) * MH;
    static constexpr bool BMN = KIND != kNT;
    static constexpr int NP = KIND == kMix ? kMaxMix : 1;
    static constexpr int B_BYTES = PAIR ? kABytes : 2 * kABytes;
    static constexpr int A_BYTES = MH * kABytes;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    // Short reductions on pairs (an expert's few rows): a tile of D leaves through shared memory by
    // TMA, 8 KB per epilogue warp, for which two stages of the ring go. The warps' own stores made
    // the epilogue 3.7 k cycles per tile, more than the products of 170 rows (256 experts of 2048 x
    // 768, 4096 tokens: both weight gradients 585 -> 523 us); with long reductions the two stages
    // are worth more (8192^3 764 us with them, 809 without).
    static constexpr bool TMA_OUT = EPI == kStoreBulk;
    static constexpr int STAGES = PAIR && !TMA_OUT && !TALL ? 6 : 4;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int STG_WARP = TMA_OUT ? 8192 : 2048;
    static constexpr int STG = kEpiWarps * STG_WARP;
    static constexpr int SMEM = RING + STG + 256 + int(sizeof(Tables)) + 1024;
    static constexpr bool GATEUP = EPI == kGateUp || EPI == kGateUpI, DGATED = EPI == kDGated || EPI == kDGatedI;
    static constexpr bool IL = EPI == kGateUpI || EPI == kDGatedI;
    static constexpr int UNITS = GATEUP ? 128 : kCols;  // columns (units) a tile covers
    static_assert(SMEM <= 232448, "dynamic shared memory per block");
};

template <int KIND, int EPI, bool PAIR>
__device__ __forceinline__ Tile tile_of(const TcTrain& P, const Tables& tb, int idx) {
    using S = Shape<KIND, EPI, PAIR>;
    Tile t;
    t.half = 0;
    t.e = 0;
    t.r0 = t.pos0 = 0;
    t.last = kBR / 16;
    if (KIND == kTN || (KIND == kMix && P.tn)) {
        // expert by expert; within one (dense: within a band of column blocks), the row blocks
        // of a column block in turn
        t.e = P.d_tile(idx);
        const int l = idx - t.e * int(P.d_tile.d);
        int mb, nb;
        const int b = P.d_band(l), w = l - b * int(P.d_band.d), c0 = b * P.band;
        if (P.n_blocks - c0 >= P.band) {
            mb = P.d_width(w);
            nb = c0 + w - mb * P.band;
        } else {
            mb = P.d_tail(w);
            nb = c0 + w - mb * int(P.d_tail.d);
        }
        t.half = P.d_m(mb);
        t.row0 = int64_t(mb - t.half * P.m_blocks) * S::BM;
        t.limit = int(min(int64_t(S::BM), P.mrows - t.row0));
        t.nvalid = t.limit;
        t.n0 = nb * kCols;
        int64_t n = P.rows;
        if (P.offsets) {
            t.r0 = tb.poff[t.e];
            n = tb.uoff[t.e + 1] - tb.uoff[t.e];
        }
        t.nk = int((n + kBR - 1) / kBR);
        // rows past the last 16-deep step with a row are not zeroed, and belong to no product
        if (P.offsets && t.nk > 0) t.last = int((n - int64_t(t.nk - 1) * kBR + 15) / 16);
        return t;
    }
    t.nk = P.nk;
    if (!P.offsets) {  // bands of row tiles, every column block in turn
        const int b = P.d_band(idx), w = idx - b * int(P.d_band.d), r0 = b * P.band;
        int nb, mt;
        if (P.m_blocks - r0 >= P.band) {
            nb = P.d_width(w);
            mt = r0 + w - nb * P.band;
        } else {
            nb = P.d_tail(w);
            mt = r0 + w - nb * int(P.d_tail.d);
        }
        t.row0 = int64_t(mt) * S::BM;
        t.n0 = nb * S::UNITS;
        t.limit = int(min(int64_t(S::BM), P.rows - t.row0));
        t.nvalid = t.limit;
        t.pos0 = t.row0;
        return t;
    }
    int lo = 0, hi = P.E - 1;  // largest e whose tiles start at or before idx
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tb.ts[mid] * P.n_blocks <= idx) lo = mid;
        else hi = mid - 1;
    }
    const int nt = tb.ts[lo + 1] - tb.ts[lo];
    const int l = idx - tb.ts[lo] * P.n_blocks;
    const int nb = nt == 1 ? l : l / nt, mt = l - nb * nt;
    t.e = lo;
    t.row0 = tb.poff[lo] + int64_t(mt) * S::BM;
    t.n0 = nb * S::UNITS;
    const int left = tb.uoff[lo + 1] - tb.uoff[lo] - mt * S::BM;
    t.limit = max(0, min(S::BM, (left + kRowPad - 1) / kRowPad * kRowPad));
    t.nvalid = max(0, min(S::BM, left));
    t.pos0 = tb.uoff[lo] + int64_t(mt) * S::BM;
    return t;
}

// TMA loads, completing on this CTA's barrier or (PAIR) on the leader's at its cluster address.
// No L2 policy: createpolicy's evict_normal marks lines for demotion once hit, which had the
// tiles of a band read 1.5 GB from HBM where 0.9 GB do (8192^3).
template <bool PAIR>
__device__ __forceinline__ void load3(void* dst, const CUtensorMap* m, uint64_t* bar, uint32_t bar_c, int c0, int c1,
                                      int c2) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(su32(dst)),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_c), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(su32(dst)),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(su32(bar)), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void load4(void* dst, const CUtensorMap* m, uint64_t* bar, uint32_t bar_c, int c0, int c1,
                                      int c2, int c3) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(su32(dst)),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_c), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(su32(dst)),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(su32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
            : "memory");
}

// An MN-major operand tile of BYTES: columns from col on, 64 reduction rows from r on, of plane e.
// `boxes`: 64-column boxes that are wanted (narrow maps), or 128-column ones (wide).
template <bool PAIR, int BYTES>
__device__ __forceinline__ void load_mn(uint8_t* dst, const CUtensorMap* m, int wide, int boxes, uint64_t* bar, uint32_t bar_c,
                                        int col, int r, int e) {
    if (wide) {
#pragma unroll
        for (int j = 0; j < BYTES / 16384; ++j)
            if (j < boxes) load4<PAIR>(dst + j * 16384, m, bar, bar_c, 0, r, col / 64 + 2 * j, e);
    } else {
#pragma unroll
        for (int j = 0; j < BYTES / 8192; ++j)
            if (j < boxes) load4<PAIR>(dst + j * 8192, m, bar, bar_c, col + 64 * j, r, 0, e);
    }
}

// SPLIT: the CTAs of a cluster share one tile, each a part of its reduction; their accumulators
// meet in shared memory, where each CTA adds up a part of the columns (in rank order) and runs
// the epilogue on it. For problems of fewer tiles than SMs.
template <int KIND, int EPI, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) tc_train_kernel(const __grid_constant__ TcArgs<Shape<KIND, EPI, PAIR>::NP> A) {
    static_assert(!(PAIR && SPLIT), "one or the other");
    using S = Shape<KIND, EPI, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stg = smem + S::RING;
    uint64_t* full = reinterpret_cast<uint64_t*>(stg + S::STG);
    uint64_t* empty = full + S::STAGES;
    uint64_t* acc_full = empty + S::STAGES;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    Tables& tb = *reinterpret_cast<Tables*>(stg + S::STG + 256);

    const TcTrain& P = A.p[0];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = PAIR ? cluster_rank() : 0u;
    const int srank = SPLIT ? int(cluster_rank()) : 0, splits = SPLIT ? P.splits : 1;
    const int tile0 = PAIR ? int(blockIdx.x >> 1) : SPLIT ? int(blockIdx.x) / splits : int(blockIdx.x);
    const int tstep = PAIR ? int(gridDim.x >> 1) : SPLIT ? 1 << 30 : int(gridDim.x);
    // this CTA's reduction blocks of a tile
    auto kb_begin = [&](const Tile& t) { return SPLIT ? t.nk * srank / splits : 0; };
    auto kb_end = [&](const Tile& t) { return SPLIT ? t.nk * (srank + 1) / splits : t.nk; };
    if (warp == 1 && lane == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], (PAIR ? 2 : 1) * kEpiWarps);
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    // no TMEM before the wait, no leave for the next launch before TMEM is had: neither side can hold
    // what the other waits for
    wait_before();
    if (warp == 0) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(tmem_slot)));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(tmem_slot)));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    if (P.offsets) {
        for (int e = threadIdx.x; e <= P.E; e += kThreads) {
            tb.poff[e] = P.poff[e];
            tb.uoff[e] = P.uoff[e];
        }
        __syncthreads();
        if (warp == 2) {  // row tiles of each expert, summed up (16 experts per lane)
            int n = 0;
            for (int i = 0; i < kMaxE / 32; ++i) {
                const int e = lane * (kMaxE / 32) + i;
                if (e < P.E) n += (tb.poff[e + 1] - tb.poff[e] + S::BM - 1) / S::BM;
            }
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            int run = incl - n;
            for (int i = 0; i < kMaxE / 32; ++i) {
                const int e = lane * (kMaxE / 32) + i;
                if (e < P.E) {
                    tb.ts[e] = run;
                    run += (tb.poff[e + 1] - tb.poff[e] + S::BM - 1) / S::BM;
                    if (e == P.E - 1) tb.ts[P.E] = run;
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    fence_after();
    launch_next();
    const uint32_t tmem = *tmem_slot;
    // tiles of the problems one after the other
    auto tiles_of = [&](const TcTrain& p) {
        if (KIND == kTN || (KIND == kMix && p.tn)) return p.E * p.m_blocks * p.halves * p.n_blocks;
        return (p.offsets ? tb.ts[p.E] : p.m_blocks) * p.n_blocks;
    };
    int ends[S::NP];
    ends[0] = tiles_of(A.p[0]);
#pragma unroll
    for (int i = 1; i < S::NP; ++i) ends[i] = ends[i - 1] + (i < A.n ? tiles_of(A.p[i]) : 0);
    const int total = ends[S::NP - 1];
    auto problem = [&](int idx, int& local) -> const TcTrain& {
        int i = 0;
        local = idx;
#pragma unroll
        for (int j = 1; j < S::NP; ++j)
            if (idx >= ends[j - 1]) {
                i = j;
                local = idx - ends[j - 1];
            }
        return A.p[S::NP == 1 ? 0 : i];
    };
    bool gave_up = false;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, armed = 0, last = 0;
            for (int idx = tile0; idx < total && !gave_up; idx += tstep) {
                int local;
                const TcTrain& P = problem(idx, local);
                const bool tn = KIND == kTN || (KIND == kMix && P.tn);
                const Tile t = tile_of<KIND, EPI, PAIR>(P, tb, local);
                const int arow = int(t.row0) + 128 * int(crank);
                // boxes of operand B that hold columns of D (the others' products are not taken)
                const int box = !S::BMN || P.wide_b ? 128 : 64;
                const int boxes = PAIR || S::GATEUP ? S::B_BYTES / (box * kBR * 2) : (min(kCols, P.N - t.n0) + box - 1) / box;
                const uint32_t bytes = (PAIR ? 2 : 1) * (S::A_BYTES + boxes * box * kBR * 2);
                const int kend = kb_end(t);
                for (int kb = kb_begin(t); kb < kend; ++kb) {
                    if (!wait_bar(&empty[stage], phase ^ 1u)) {
                        gave_up = true;
                        break;
                    }
                    uint8_t* sa = smem + stage * S::STAGE;
                    uint8_t* sb = sa + S::A_BYTES;
                    const uint32_t fb = PAIR ? mapa_shared(&full[stage], 0) : 0u;
                    if (crank == 0) mbar_expect_tx(&full[stage], bytes);
                    const int half = S::BMN && !tn && kb >= P.nk_half ? 1 : 0;
                    const int kc = (kb - half * P.nk_half) * kBR;
                    if (tn) {
                        const int r = int(t.r0) + kb * kBR;
#pragma unroll
                        for (int h = 0; h < S::MH; ++h)
                            load_mn<PAIR, kABytes>(sa + h * kABytes, &P.a, P.wide_a, 2, &full[stage], fb, arow + 256 * h, r, t.half);
                        load_mn<PAIR, S::B_BYTES>(sb, &P.b0, P.wide_b, boxes, &full[stage], fb, t.n0 + 128 * int(crank), r, 0);
                    } else {
#pragma unroll
                        for (int h = 0; h < S::MH; ++h)
                            load3<PAIR>(sa + h * kABytes, &P.a, &full[stage], fb, kc, half, arow + 256 * h);
                        if constexpr (S::BMN) {
                            load_mn<PAIR, S::B_BYTES>(sb, half && P.b_split ? &P.b1 : &P.b0, P.wide_b, boxes, &full[stage], fb,
                                                      t.n0 + 128 * int(crank), kc, t.e);
                        } else if constexpr (S::GATEUP) {
                            // gate rows, then up rows; of a pair, CTA 0 gate and CTA 1 up
                            if constexpr (PAIR) {
                                if (S::IL) load4<PAIR>(sb, &P.b0, &full[stage], fb, kc, int(crank), t.n0, t.e);
                                else load4<PAIR>(sb, crank ? &P.b1 : &P.b0, &full[stage], fb, kc, 0, t.n0, t.e);
                            } else {
                                load4<PAIR>(sb, &P.b0, &full[stage], fb, kc, 0, t.n0, t.e);
                                if (S::IL) load4<PAIR>(sb + kABytes, &P.b0, &full[stage], fb, kc, 1, t.n0, t.e);
                                else load4<PAIR>(sb + kABytes, &P.b1, &full[stage], fb, kc, 0, t.n0, t.e);
                            }
                        } else {
                            const int nb = t.n0 + 128 * int(crank);
#pragma unroll
                            for (int j = 0; j < S::B_BYTES / kABytes; ++j)
                                if (j < boxes) load4<PAIR>(sb + j * kABytes, &P.b0, &full[stage], fb, kc, 0, nb + 128 * j, t.e);
                        }
                    }
                    armed |= 1u << stage;
                    last = (last & ~(1u << stage)) | (phase << stage);
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every copy has landed (of a pair: and been read) before this CTA may leave
            for (int s = 0; s < S::STAGES; ++s)
                if ((armed >> s) & 1u) wait_bar(PAIR ? &empty[s] : &full[s], (last >> s) & 1u);
            if (gave_up) set_status(P.status, MOE_ERR_DEVICE_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && crank == 0) {
            // -------------------------------------------------------- MMA issuer
            uint32_t stage = 0, phase = 0, it = 0;
            for (int idx = tile0; idx < total && !gave_up; idx += tstep) {
                int local;
                const TcTrain& P = problem(idx, local);
                const bool tn = KIND == kTN || (KIND == kMix && P.tn);
                const Tile t = tile_of<KIND, EPI, PAIR>(P, tb, local);
                const int kbeg = kb_begin(t), kend = kb_end(t);
                if (kbeg == kend) continue;
                // accumulator set (tall: of the first half) and its phase
                const uint32_t ab = S::TALL ? 0u : it & 1u, ph = S::TALL ? it & 1u : (it >> 1) & 1u;
                ++it;
                if (!wait_bar(&acc_empty[ab], ph ^ 1u)) {
                    gave_up = true;
                    break;
                }
                fence_after();
                const uint32_t d0 = tmem + ab * kCols;
                const uint32_t desc = idesc(tn, S::BMN, S::TALL ? 256 : S::BM,
                                            PAIR || S::GATEUP ? kCols : (min(kCols, P.N - t.n0) + 15) / 16 * 16);
                // the four (or last) 16-deep steps of one block for half h
                auto block = [&](uint32_t st, int kb, int h) {
                    const uint32_t sa = su32(smem + st * S::STAGE) + h * kABytes;
                    const uint32_t sb = su32(smem + st * S::STAGE) + S::A_BYTES;
                    auto products = [&](auto a_mn) {
                        constexpr bool AMN = decltype(a_mn)::value;
                        auto step = [&](int k) {
                            mma<PAIR>(d0 + h * kCols, operand<AMN>(sa + k * kStep<AMN>),
                                      operand<S::BMN>(sb + k * kStep<S::BMN>), desc, kb > kbeg || k > 0 ? 1u : 0u);
                        };
                        if (AMN && t.last < kBR / 16 && kb == t.nk - 1) {
                            for (int k = 0; k < t.last; ++k) step(k);
                        } else {
#pragma unroll
                            for (int k = 0; k < kBR / 16; ++k) step(k);
                        }
                    };
                    if (tn) products(std::true_type{});
                    else products(std::false_type{});
                };
                int kb = kbeg;
                if constexpr (S::TALL) {
                    // the first ring's worth of blocks on the first half before any on the second,
                    // whose accumulators the epilogue of the tile before still reads
                    const int head = min(kend, kbeg + S::STAGES);
                    uint32_t st = stage, sp = phase;
                    for (; kb < head; ++kb) {
                        if (!wait_bar(&full[st], sp)) {
                            gave_up = true;
                            break;
                        }
                        fence_after();
                        block(st, kb, 0);
                        if (++st == S::STAGES) {
                            st = 0;
                            sp ^= 1u;
                        }
                    }
                    if (gave_up) break;
                    if (head == kend) commit<PAIR>(&acc_full[0]);
                    if (!wait_bar(&acc_empty[1], ph ^ 1u)) {
                        gave_up = true;
                        break;
                    }
                    fence_after();
                    for (kb = kbeg; kb < head; ++kb) {
                        block(stage, kb, 1);
                        commit<PAIR>(&empty[stage]);
                        if (++stage == S::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (head == kend) {
                        commit<PAIR>(&acc_full[1]);
                        continue;
                    }
                }
                for (; kb < kend; ++kb) {
                    if (!wait_bar(&full[stage], phase)) {
                        gave_up = true;
                        break;
                    }
                    fence_after();
                    block(stage, kb, 0);
                    if constexpr (S::TALL) {
                        if (kb == kend - 1) commit<PAIR>(&acc_full[0]);
                        block(stage, kb, 1);
                    }
                    commit<PAIR>(&empty[stage]);
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (gave_up) break;
                commit<PAIR>(&acc_full[S::TALL ? 1 : ab]);
            }
            commit<PAIR>(drain);
            wait_bar(drain, 0);
            if (gave_up) set_status(P.status, MOE_ERR_DEVICE_TIMEOUT);
        }
        __syncwarp();
    }
    // ---------------------------------------------------------------- epilogue
    if constexpr (SPLIT) {
        // this CTA's part of the sums into shared memory (the ring: its products are done), 16
        // bytes of four columns per row, rows adjacent
        if (warp >= 2 && tile0 < total) {
            int local;
            const TcTrain& P = problem(tile0, local);
            const bool tn = KIND == kTN || (KIND == kMix && P.tn);
            const Tile t = tile_of<KIND, EPI, PAIR>(P, tb, local);
            const bool any = kb_begin(t) < kb_end(t);
            bool ok = true;
            if (any) {
                ok = wait_bar(&acc_full[0], 0);
                if (!ok) set_status(P.status, MOE_ERR_DEVICE_TIMEOUT);
                fence_after();
            }
            const int q = warp & 3, ch = (warp - 2) >> 2;
            if (q * 32 >= (tn ? t.limit : t.nvalid)) ok = false;  // rows that nobody reads
#pragma unroll 1
            for (int c = 4 * ch; ok && c < 4 * ch + 4; ++c) {
                uint32_t r[32];
                if (any) {
                    tmem_load(tmem + (uint32_t(q * 32) << 16) + 32 * c, r);
                    tmem_wait(r);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(smem + ((c * 8 + j) * 128 + q * 32 + lane) * 16) =
                        make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            }
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp >= 2) {
        const int q = warp & 3;                    // TMEM lane quarter of this warp
        const int ch = (warp - 2) >> 2;            // column half
        uint8_t* sm = stg + (warp - 2) * S::STG_WARP;
        uint32_t it = 0;
        // the warp's 32-column chunks of a tile (kGateUp: of its 128 units)
        constexpr int kChunks = S::GATEUP ? 4 : 8;
        int c0 = ch * (kChunks / 2), c1 = c0 + kChunks / 2;
        if constexpr (SPLIT) {
            const int n = kChunks / splits, half = (n + 1) / 2;
            c0 = srank * n + ch * half;
            c1 = min(c0 + half, (srank + 1) * n);
        }
        // kDGated: pre-activations of the next 32 columns (gate, up), one chunk ahead
        uint4 x0[4], x1[4];
        auto fetch_pre = [&](const Tile& t, int wrow, int c, int vrows) {
            const int col = t.n0 + 32 * c;
            const int bytes = (P.N - col) * 2;
            const __nv_bfloat16* pr = P.pre + (t.pos0 + wrow) * P.ldp;
            if constexpr (S::IL) {
                fetch_rows(lane, x0, pr + 2 * col, P.ldp * 2, vrows, 2 * bytes);
                fetch_rows(lane, x1, pr + 2 * col + 32, P.ldp * 2, vrows, 2 * bytes - 64);
            } else {
                fetch_rows(lane, x0, pr + col, P.ldp * 2, vrows, bytes);
                fetch_rows(lane, x1, pr + P.N + col, P.ldp * 2, vrows, bytes);
            }
        };
        auto epilogue = [&](int idx, int h) -> bool {
            const int wrow = 256 * h + int(crank) * 128 + q * 32;  // first tile row of the warp
            int local;
            const TcTrain& P = problem(idx, local);
            const bool tn = KIND == kTN || (KIND == kMix && P.tn);
            const Tile t = tile_of<KIND, EPI, PAIR>(P, tb, local);
            const int rows = min(32, t.limit - wrow);     // may be negative
            const int vrows = min(32, t.nvalid - wrow);
            const int64_t row = t.row0 + wrow;            // the warp's first row
            const uint32_t ab = S::TALL ? uint32_t(h) : it & 1u, ph = S::TALL ? it & 1u : (it >> 1) & 1u;
            float rs = 1.0f;
            if (!tn && P.offsets && P.row_scale && lane < vrows) {
                const int slot = P.row_slot[row + lane];
                rs = slot < 0 ? 0.0f : P.row_scale[slot];
            }
            if constexpr (S::DGATED)
                if (c0 < c1) fetch_pre(t, wrow, c0, vrows);
            if (!SPLIT && t.nk > 0) {
                if (h == S::MH - 1) ++it;
                const int ok = lane == 0 ? int(wait_bar(&acc_full[ab], ph)) : 0;  // one lane waits
                if (!__shfl_sync(0xffffffffu, ok, 0)) {
                    if (lane == 0) set_status(P.status, MOE_ERR_DEVICE_TIMEOUT);
                    return false;
                }
                fence_after();
            }
            const uint32_t tacc = tmem + (uint32_t(q * 32) << 16) + ab * kCols;
            // accumulator columns 32 c .. 32 c + 31 of this lane's row
            auto acc = [&](int c, uint32_t (&r)[32]) {
                if constexpr (SPLIT) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                    if ((tn ? rows : vrows) <= 0) return;
                    // the ranks' sums in rank order, the next rank's loads under way meanwhile
                    const uint32_t own = su32(smem + (c * 8 * 128 + q * 32 + lane) * 16);
                    float4 v[2][8];
                    auto issue = [&](int p, float4 (&x)[8]) {
                        uint32_t at;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(own), "r"(p));
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                         : "=f"(x[j].x), "=f"(x[j].y), "=f"(x[j].z), "=f"(x[j].w)
                                         : "r"(at + j * 2048)
                                         : "memory");
                    };
                    auto add = [&](const float4 (&x)[8]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) + x[j].x);
                            r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) + x[j].y);
                            r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) + x[j].z);
                            r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) + x[j].w);
                        }
                    };
                    issue(0, v[0]);
#pragma unroll 1
                    for (int p = 0; p < splits; p += 2) {  // splits is even
                        issue(p + 1, v[1]);
                        add(v[0]);
                        if (p + 2 < splits) issue(p + 2, v[0]);
                        add(v[1]);
                    }
                } else {
                    tmem_load(tacc + 32 * c, r);
                    tmem_wait(r);
                }
            };
            auto release = [&]() {  // this warp has read its part of the accumulators
                if constexpr (SPLIT) return;
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) arrive_leader(&acc_empty[ab]);
                    else mbar_arrive(&acc_empty[ab]);
                }
            };
            if constexpr (S::GATEUP) {
                // gate of the tile's 128 units in columns 0..127, up in 128..255
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    uint32_t gr[32], vr[32];
                    acc(c, gr);
                    acc(4 + c, vr);
                    if (c == c1 - 1) release();
                    const int u0 = t.n0 + 32 * c;
                    if (u0 >= P.N || vrows <= 0) continue;
                    float g[32], v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        g[j] = __uint_as_float(gr[j]);
                        v[j] = __uint_as_float(vr[j]);
                    }
                    if (P.bias0) {
                        if constexpr (S::IL) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                float z[32] = {};
                                add_bias(P.bias0 + t.e * P.sbias, 2 * u0 + 32 * b, 2 * P.N, z);
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    g[16 * b + j] += z[2 * j];
                                    v[16 * b + j] += z[2 * j + 1];
                                }
                            }
                        } else {
                            add_bias(P.bias0 + t.e * P.sbias, u0, P.N, g);
                            add_bias(P.bias1 + t.e * P.sbias, u0, P.N, v);
                        }
                    }
                    const int bytes = (P.N - u0) * 2;  // of a row of units from u0 on
                    uint4 w[4];
                    if (P.pre) {
                        __nv_bfloat16* pr = P.pre + (t.pos0 + wrow) * P.ldp;
                        if constexpr (S::IL) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int j = 16 * b + 4 * i;
                                    w[i] = make_uint4(pack2(g[j], v[j]), pack2(g[j + 1], v[j + 1]),
                                                      pack2(g[j + 2], v[j + 2]), pack2(g[j + 3], v[j + 3]));
                                }
                                store_rows(sm, lane, w, pr + 2 * u0 + 32 * b, P.ldp * 2, vrows, 2 * bytes - 64 * b);
                            }
                        } else {
                            pack_row(g, w);
                            store_rows(sm, lane, w, pr + u0, P.ldp * 2, vrows, bytes);
                            pack_row(v, w);
                            store_rows(sm, lane, w, pr + P.N + u0, P.ldp * 2, vrows, bytes);
                        }
                    }
                    auto units = [&](auto clamped) {
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float2 h = gated_h2<decltype(clamped)::value>(make_float2(g[j], g[j + 1]),
                                                                                make_float2(v[j], v[j + 1]), P.limit, P.cexp);
                            g[j] = h.x;
                            g[j + 1] = h.y;
                        }
                    };
                    if (P.act == MOE_ACT_SWIGLU) units(std::false_type{});
                    else units(std::true_type{});
                    pack_row(g, w);
                    store_rows(sm, lane, w, static_cast<__nv_bfloat16*>(P.out) + row * P.ldo + u0, P.ldo * 2, vrows, bytes);
                }
            } else if constexpr (S::DGATED) {
                float2 dw = make_float2(0.0f, 0.0f);
                const bool valid = lane < vrows;
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    const int col = t.n0 + 32 * c;
                    const int bytes = (P.N - col) * 2;
                    turn_rows(sm, lane, x0);
                    turn_rows(sm, lane, x1);
                    const uint32_t a0[16] = {x0[0].x, x0[0].y, x0[0].z, x0[0].w, x0[1].x, x0[1].y, x0[1].z, x0[1].w,
                                             x0[2].x, x0[2].y, x0[2].z, x0[2].w, x0[3].x, x0[3].y, x0[3].z, x0[3].w};
                    const uint32_t a1[16] = {x1[0].x, x1[0].y, x1[0].z, x1[0].w, x1[1].x, x1[1].y, x1[1].z, x1[1].w,
                                             x1[2].x, x1[2].y, x1[2].z, x1[2].w, x1[3].x, x1[3].y, x1[3].z, x1[3].w};
                    if (c + 1 < c1) fetch_pre(t, wrow, c + 1, vrows);
                    uint32_t dr[32];
                    acc(c, dr);
                    if (c == c1 - 1) release();
                    if (bytes <= 0 || rows <= 0) continue;
                    uint32_t o0[16], o1[16], oh[16];  // dg and dv (or alternating), w h
                    auto units = [&](auto clamped, auto whole) {
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float2 g, v, h, hg, hv;
                            if constexpr (S::IL) {
                                const uint32_t xa = j < 16 ? a0[j % 16] : a1[j % 16], xb = j < 16 ? a0[j % 16 + 1] : a1[j % 16 + 1];
                                g = make_float2(bf16lo(xa), bf16lo(xb));
                                v = make_float2(bf16hi(xa), bf16hi(xb));
                            } else {
                                g = make_float2(bf16lo(a0[j / 2]), bf16hi(a0[j / 2]));
                                v = make_float2(bf16lo(a1[j / 2]), bf16hi(a1[j / 2]));
                            }
                            gated_grad2<decltype(clamped)::value>(g, v, P.limit, P.alpha, P.cexp, h, hg, hv);
                            const float2 d = make_float2(__uint_as_float(dr[j]), __uint_as_float(dr[j + 1]));
                            // columns past N hold no unit
                            if (decltype(whole)::value || 8 * (j / 8) * 2 < bytes) dw = fma2(d, h, dw);
                            const float2 dr2 = mul2(d, make_float2(rs, rs));
                            const float2 dg = mul2(dr2, hg), dv = mul2(dr2, hv);
                            h = mul2(h, make_float2(rs, rs));
                            if constexpr (S::IL) {
                                (j < 16 ? o0[j % 16] : o1[j % 16]) = pack2(dg.x, dv.x);
                                (j < 16 ? o0[j % 16 + 1] : o1[j % 16 + 1]) = pack2(dg.y, dv.y);
                            } else {
                                o0[j / 2] = pack2(dg.x, dg.y);
                                o1[j / 2] = pack2(dv.x, dv.y);
                            }
                            oh[j / 2] = pack2(h.x, h.y);
                        }
                    };
                    auto either = [&](auto whole) {
                        if (P.act == MOE_ACT_SWIGLU) units(std::false_type{}, whole);
                        else units(std::true_type{}, whole);
                    };
                    if (bytes >= 64) either(std::true_type{});
                    else either(std::false_type{});
                    if (vrows < 32 && !valid) {  // rows without a slot are zeros: the weight gradients reduce over them
#pragma unroll
                        for (int j = 0; j < 16; ++j) o0[j] = o1[j] = oh[j] = 0;
                    }
                    __nv_bfloat16* o = P.dgu + row * 2 * P.N;
                    const int64_t ldb = int64_t(P.N) * 4;
                    auto put = [&](const uint32_t (&r)[16], void* at, int64_t ld, int n) {
                        const uint4 w[4] = {make_uint4(r[0], r[1], r[2], r[3]), make_uint4(r[4], r[5], r[6], r[7]),
                                            make_uint4(r[8], r[9], r[10], r[11]), make_uint4(r[12], r[13], r[14], r[15])};
                        store_rows(sm, lane, w, at, ld, rows, n);
                    };
                    if constexpr (S::IL) {
                        put(o0, o + 2 * col, ldb, 2 * bytes);
                        put(o1, o + 2 * col + 32, ldb, 2 * bytes - 64);
                    } else {
                        put(o0, o + col, ldb, bytes);
                        put(o1, o + P.N + col, ldb, bytes);
                    }
                    put(oh, P.hw + row * P.N + col, int64_t(P.N) * 2, bytes);
                }
                if (P.partial && valid) P.partial[(row + lane) * P.parts + ((t.n0 / kCols) * splits + srank) * 2 + ch] = dw.x + dw.y;
            } else if (tn) {
                if constexpr (S::TMA_OUT) {
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the tile before
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 w[4];
                        float f[32];
                        if (t.nk > 0) {
                            uint32_t dr[32];
                            acc(4 * ch + c, dr);
#pragma unroll
                            for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(dr[j]);
                        } else {  // an expert without rows: its gradient is zero
#pragma unroll
                            for (int j = 0; j < 32; ++j) f[j] = 0.0f;
                        }
                        if (c == 3 && t.nk > 0) release();
                        pack_row(f, w);
                        // two boxes of 64 columns, 128-byte swizzle
                        uint8_t* box = sm + (c >> 1) * 4096 + lane * 128;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4*>(box + ((((c & 1) * 4 + j) ^ (lane & 7)) << 4)) = w[j];
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0 && rows > 0) {
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int col = t.n0 + 128 * ch + 64 * b;
                            if (col < P.N)
                                asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                                                 reinterpret_cast<uint64_t>(t.half ? &P.o1 : &P.o0)),
                                             "r"(col), "r"(int(row)), "r"(t.e), "r"(su32(sm + b * 4096))
                                             : "memory");
                        }
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    return true;
                }
                __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(t.half ? P.out1 : P.out) + t.e * P.so + row * P.ldo;
                if constexpr (SPLIT) {
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        uint32_t dr[32];
                        acc(c, dr);
                        float f[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(dr[j]);
                        uint4 w[4];
                        pack_row(f, w);
                        const int col = t.n0 + 32 * c;
                        store_rows(sm, lane, w, ob + col, P.ldo * 2, rows, (P.N - col) * 2);
                    }
                } else {
                // everything out of TMEM first: the next products need not wait for the stores
                uint4 w[4][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float f[32];
                    if (t.nk > 0) {
                        uint32_t dr[32];
                        acc(4 * ch + c, dr);
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(dr[j]);
                    } else {  // an expert without rows: its gradient is zero
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = 0.0f;
                    }
                    pack_row(f, w[c]);
                }
                if (t.nk > 0) release();
                if (rows <= 0) return true;
#pragma unroll
                for (int c = 0; c < 4; c += 2) {
                    const int col = t.n0 + 128 * ch + 32 * c;
                    store_lines(sm, lane, w[c], w[c + 1], ob + col, P.ldo * 2, rows, (P.N - col) * 2);
                }
                }
            } else {
                char* ob = static_cast<char*>(P.out) + row * P.ldo * (P.out_f32 ? 4 : 2);
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    const int col = t.n0 + 32 * c;
                    uint32_t dr[32];
                    acc(c, dr);
                    if (c == c1 - 1) release();
                    float f[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(dr[j]);
                    const int bytes = (P.N - col) * 2;
                    if (bytes <= 0 || vrows <= 0) continue;
                    uint4 w[4];
                    if (P.bias0) add_bias(P.bias0 + t.e * P.sbias, col, P.N, f);
                    if (P.pre) {
                        pack_row(f, w);
                        store_rows(sm, lane, w, P.pre + row * P.ldp + col, P.ldp * 2, vrows, bytes);
                    }
                    // a loop per activation: its 32 chains run side by side (chosen inside, GELU added 8 us
                    // to a launch of few tiles, 128 tokens 512 -> 2048 9.0 -> 17.1 us)
                    if (P.act == MOE_LINEAR_GELU) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = linear_act<true>(MOE_LINEAR_GELU, f[j]);
                    } else if (P.act == MOE_LINEAR_SILU) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] = linear_act<true>(MOE_LINEAR_SILU, f[j]);
                    }
                    if (P.row_scale) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] *= rs;
                    }
                    if (P.residual) {
                        float z[32];
                        fetch_rows(lane, w, P.residual + row * P.ldr + col, P.ldr * 2, vrows, bytes);
                        turn_rows(sm, lane, w);
                        unpack_row(w, z);
#pragma unroll
                        for (int j = 0; j < 32; ++j) f[j] += z[j];
                    }
                    if (P.out_f32) {
                        uint4 hi[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            w[p] = make_uint4(__float_as_uint(f[4 * p]), __float_as_uint(f[4 * p + 1]),
                                              __float_as_uint(f[4 * p + 2]), __float_as_uint(f[4 * p + 3]));
                            hi[p] = make_uint4(__float_as_uint(f[16 + 4 * p]), __float_as_uint(f[16 + 4 * p + 1]),
                                               __float_as_uint(f[16 + 4 * p + 2]), __float_as_uint(f[16 + 4 * p + 3]));
                        }
                        store_lines(sm, lane, w, hi, ob + col * 4, P.ldo * 4, vrows, 2 * bytes);
                    } else {
                        pack_row(f, w);
                        store_rows(sm, lane, w, ob + col * 2, P.ldo * 2, vrows, bytes);
                    }
                }
            }
            return true;
        };
        if constexpr (SPLIT) {
            if (tile0 < total) epilogue(tile0, 0);
        } else {
            for (int idx = tile0; idx < total; idx += tstep) {
                bool ok = true;
#pragma unroll 1
                for (int h = 0; h < S::MH && ok; ++h) ok = epilogue(idx, h);
                if (!ok) break;
            }
        }
        if constexpr (S::TMA_OUT)
            if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    if constexpr (PAIR || SPLIT) cluster_sync();  // no CTA leaves while another reads its shared memory
    if (warp == 0) {
        fence_after();
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// ------------------------------------------------------------------ host side
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// bf16 tensor map, innermost dimension first; ld[i]: elements between indices of dimension i + 1.
bool encode(CUtensorMap* m, const void* base, int rank, const int64_t* dims, const int64_t* ld, const int* box) {
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[4], st[3];
    cuuint32_t b[4], es[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = cuuint64_t(dims[i]);
        b[i] = cuuint32_t(box[i]);
        if (i < rank - 1) st[i] = cuuint64_t(ld[i]) * 2;
    }
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(base), d, st, b, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of a B200 (the library's only target), asked once.
int sms() {
    static const int n = [] {
        int dev = 0, v = 148;
        if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        return v;
    }();
    return n;
}

// Allows a kernel its shared memory, once per device.
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return err;
    done.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}

template <int KIND, int EPI, bool PAIR, bool SPLIT>
cudaError_t launch_t(const TcTrain* P, int np, int64_t max_tiles, cudaStream_t s) {
    using S = Shape<KIND, EPI, PAIR>;
    TcArgs<S::NP> args;
    for (int i = 0; i < S::NP; ++i) args.p[i] = P[std::min(i, np - 1)];
    args.n = np;
    auto kern = tc_train_kernel<KIND, EPI, PAIR, SPLIT>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_smem(kern, S::SMEM, allowed);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : SPLIT ? P->splits : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // Not chained: experts' tiles on single CTAs over more than one round. Their blocks' places, which
    // share operands by neighbourhood, would be those of the tail before (gate/up after the row copy
    // 338 -> 344 us, down after gate/up 200 -> 218 us; on pairs 527 -> 516 us).
    cfg.numAttrs = PAIR || SPLIT || !P->offsets || max_tiles <= sms() ? 2 : 0;
    if (SPLIT) {
        cfg.gridDim = dim3(unsigned(max_tiles) * P->splits);
        if ((err = cudaLaunchKernelEx(&cfg, kern, args)) != cudaSuccess) return err;
        return cudaGetLastError();
    }
    int most = sms();
    if (PAIR) {  // pairs that can be resident at once (an odd SM of a GPC stays out)
        static std::atomic<int> fits{0};
        int resident = fits.load();
        if (resident == 0) {
            cfg.gridDim = dim3(2 * (most / 2));
            if ((err = cudaOccupancyMaxActiveClusters(&resident, kern, &cfg)) != cudaSuccess) return err;
            if (resident <= 0) return cudaErrorInvalidConfiguration;
            fits.store(resident);
        }
        most = std::min(resident, most / 2);
    }
    const int n = int(std::min<int64_t>(max_tiles, most));
    if (n <= 0) return cudaSuccess;
    cfg.gridDim = dim3(PAIR ? 2 * n : n);
    if ((err = cudaLaunchKernelEx(&cfg, kern, args)) != cudaSuccess) return err;
    return cudaGetLastError();
}

// The forms of a product: split, pairs (tall where P says so), or one CTA per tile.
template <int KIND, int EPI>
cudaError_t launch(const TcTrain& P, bool pair, int64_t max_tiles, cudaStream_t s) {
    if constexpr (EPI == kStore)
        if (P.tall) return launch_t<KIND, kStoreTall, true, false>(&P, 1, max_tiles, s);
    if (P.splits > 1) return launch_t<KIND, EPI, false, true>(&P, 1, max_tiles, s);
    return pair ? launch_t<KIND, EPI, true, false>(&P, 1, max_tiles, s)
                : launch_t<KIND, EPI, false, false>(&P, 1, max_tiles, s);
}

int64_t blocks_of(int64_t n, int64_t b) { return (n + b - 1) / b; }

TcTrain base_of(const RowPlan& p) {
    TcTrain P;
    memset(&P, 0, sizeof(P));
    P.offsets = p.offsets;
    P.poff = p.poff;
    P.uoff = p.uoff;
    P.row_slot = p.row_slot;
    P.E = p.E;
    P.rows = p.T;
    P.halves = 1;
    P.status = p.status;
    P.splits = 1;
    return P;
}

// A as [rows][halves][cols of a half], K-major boxes of 64 columns x 128 rows.
bool map_a_k(CUtensorMap* m, const void* a, int64_t rows, int64_t ld, int64_t cols, int halves) {
    const int64_t d[3] = {cols, halves, rows}, st[2] = {halves > 1 ? cols : ld, ld};
    const int box[3] = {64, 1, 128};
    return encode(m, a, 3, d, st, box);
}
// MN-major operand of planes [E][r][n]: 64 x 64 boxes, whose inner row is one 128-byte swizzle
// row. Where n is a multiple of 64 the columns are a dimension of blocks of their own, and one
// copy brings two blocks: the producer's one thread issues a copy in about 100 cycles, and with
// four per 512-cycle reduction block it starved the products (32 experts of 2880 x 2880: 8.3
// blocks took 6.9 k cycles).
bool map_mn(CUtensorMap* m, int& wide, const void* b, int64_t E, int64_t r, int64_t n, int64_t ld, int64_t plane) {
    wide = n % 64 == 0;
    const int64_t d[4] = {wide ? 64 : n, r, wide ? n / 64 : 1, E}, st[3] = {ld, 64, plane};
    const int box[4] = {64, 64, wide ? 2 : 1, 1};
    return encode(m, b, 4, d, st, box);
}
// Weight planes [E][rows][halves][K] as the K-major B operand.
bool map_b_k(CUtensorMap* m, const void* b, int64_t E, int64_t rows, int halves, int64_t K) {
    const int64_t d[4] = {K, halves, rows, E}, st[3] = {K, halves * K, rows * halves * K};
    const int box[4] = {64, 1, 128, 1};
    return encode(m, b, 4, d, st, box);
}
// Planes [E][rows][n] of a weight gradient, written in boxes of 64 columns x 32 rows.
bool map_out(CUtensorMap* m, const void* o, int64_t E, int64_t rows, int64_t n, int64_t ld, int64_t plane) {
    const int64_t d[3] = {n, rows, E}, st[2] = {ld, E > 1 ? plane : rows * ld};
    const int box[3] = {64, 32, 1};
    return encode(m, o, 3, d, st, box);
}

// 512-row tiles where their rounds over the GPU's pairs cost less, and the reduction is long: a
// round of them takes about 1.94 rounds of 256-row tiles over 8192 (8192^3: 7 of 101 us against 14
// of 52), 2.1 over 4096 (their epilogue hides less), and their number divides worse.
bool use_tall(int64_t rows, int64_t halves, int64_t n_blocks, int64_t nk) {
    const int64_t pairs = sms() / 2;
    const int64_t tall = blocks_of(blocks_of(rows, 512) * halves * n_blocks, pairs);
    const int64_t flat = blocks_of(blocks_of(rows, 256) * halves * n_blocks, pairs);
    return nk >= 96 && 97 * tall < 50 * flat;
}

// 256-row tiles on CTA pairs where they fill the GPU about as well as 128-row tiles.
bool use_pair(const RowPlan& p, int64_t rows, int64_t n_blocks) {
    if (p.offsets) return p.S >= 384 * int64_t(p.E);
    return blocks_of(rows, 256) * n_blocks >= sms() / 2;
}

// Clusters of 2, 4 or 8 CTAs of the split kernels that the GPU holds at once (a GPC's SMs do not
// divide into eights: 16 clusters of 8 took two rounds, 2048 x 64 over 8192 34 us). Every split
// kernel has the same block and the same shared memory.
int clusters_of(int s) {
    static std::atomic<int> fits[4];
    std::atomic<int>& f = fits[s == 2 ? 0 : s == 4 ? 1 : 2];
    int n = f.load();
    if (n > 0) return n;
    using S = Shape<kNT, kStore, false>;
    auto kern = tc_train_kernel<kNT, kStore, false, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.gridDim = dim3(sms() / s * s);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static std::atomic<uint64_t> allowed{0};
    if (allow_smem(kern, S::SMEM, allowed) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        n = 1;
    }
    f.store(n);
    return n;
}

// What a tile of nk reduction blocks takes when s CTAs share it, in 10 ns: a block 0.39 us with its
// weights coming from HBM, the clusters' meeting 0.6 us + 0.2 to 1 us per CTA by the tile's rows
// (measured whole / by 2 / 4 / 8, us: 16 rows, 16 blocks 11.6 / 9.8 / 8.2 / 8.9, 32 blocks 16.0 /
// 12.2 / 9.6 / 9.8; 64 rows, 16 blocks 11.9 / 10.3 / 9.2 / 10.4; 128 rows, 8 blocks 9.2 / 10.0 / 10.7 /
// 13.7, 16 blocks 12.6 / 11.8 / 11.8 / 14.9, 32 blocks 16.9 / 14.2 / 13.3 / 15.7).
int64_t split_cost(int64_t nk, int s, int64_t rows) {
    return 39 * ((nk + s - 1) / s) + (s > 1 ? 60 + (rows <= 32 ? 20 : rows <= 64 ? 40 : 100) * s : 0);
}
// CTAs per tile (1, 2, 4, 8; at most `most`, what the columns divide into): as many as pay and
// the SMs hold at once.
int splits_of(int64_t tiles, int64_t nk, int most, int64_t rows) {
    int best = 1;
    for (int s = 2; s <= most; s *= 2)
        if (split_cost(nk, s, rows) < split_cost(nk, best, rows) && tiles <= clusters_of(s)) best = s;
    return best;
}

// Rows of a tile, about.
int64_t row_hint(const RowPlan& p, int64_t rows) { return p.offsets ? (p.S + p.E - 1) / p.E : rows; }

// Bands of P.band of `n` blocks, with `other` blocks of the other kind in turn in each.
void set_bands(TcTrain& P, int n, int other) {
    P.d_band = fast_div(int64_t(P.band) * other);
    P.d_width = fast_div(P.band);
    P.d_tail = fast_div(std::max(1, n % P.band));
}

// Blocks of a band: with every block of the other kind they should fill the GPU, and where
// those are many, the tiles running together should be about square, so that they share both
// operands in L2.
int band_of(int n, int other, int conc) {
    int b = std::max(1, conc / std::max(1, other));
    while (b * b < conc) ++b;
    return std::min(n, b);
}

// Row tiles at most, and the dense problem's bands.
int64_t row_grid(TcTrain& P, const RowPlan& p, bool pair) {
    const int BM = P.tall ? 512 : pair ? 256 : 128;
    P.m_blocks = int(p.offsets ? blocks_of(p.max_rows, BM) + (pair ? std::min<int64_t>(p.E, p.S) : 0)
                               : blocks_of(p.T, BM));
    const int conc = pair ? sms() / 2 : sms();
    P.band = band_of(P.m_blocks, P.n_blocks, conc);
    set_bands(P, P.m_blocks, P.n_blocks);
    return int64_t(P.m_blocks) * P.n_blocks;
}

}  // namespace

namespace {

// A problem's launch parameters (without an output: no tensor maps), whether it runs on CTA pairs,
// and its tiles at most.
bool set_up(const GemmArgs& a, TcTrain& P, bool& pair, int64_t& tiles) {
    P = base_of(a.plan);
    const bool grouped = a.plan.offsets != nullptr;
    P.N = a.N;
    P.n_blocks = int(blocks_of(a.N, kCols));
    P.out = a.out;
    P.out1 = a.out1;
    P.ldo = a.ldo;
    P.so = a.so;
    if (a.kind == kTN) {
        P.tn = 1;
        P.halves = a.split ? 2 : 1;
        P.mrows = a.M / P.halves;
        const int64_t rows = grouped ? a.plan.max_rows : a.R;
        P.rows = a.R;
        P.E = grouped ? a.plan.E : 1;
        const int64_t tiles256 = blocks_of(P.mrows, 256) * P.halves * P.n_blocks * P.E;
        pair = tiles256 >= sms() / 2;
        P.tall = pair && !grouped && use_tall(P.mrows, P.halves, P.n_blocks, blocks_of(a.R, kBR));
        P.m_blocks = int(blocks_of(P.mrows, P.tall ? 512 : pair ? 256 : 128));
        // an expert's tiles: one column block at a time; dense: as many as fill the GPU with every row block
        P.band = grouped ? 1 : band_of(P.n_blocks, P.m_blocks * P.halves, pair ? sms() / 2 : sms());
        set_bands(P, P.n_blocks, P.m_blocks * P.halves);
        P.d_tile = fast_div(int64_t(P.m_blocks) * P.halves * P.n_blocks);
        P.d_m = fast_div(P.m_blocks);
        tiles = int64_t(P.E) * P.m_blocks * P.halves * P.n_blocks;
        P.nk = int(blocks_of(a.R, kBR));
        if (!pair && !grouped) P.splits = splits_of(tiles, P.nk, 8, P.mrows);
        if (!a.out) return true;
        P.bulk_out = pair && (grouped ? a.plan.S / a.plan.E : a.R) < 16 * kBR;
        if (P.bulk_out && (!map_out(&P.o0, a.out, P.E, P.mrows, a.N, a.ldo, a.so) ||
                     (P.halves > 1 && !map_out(&P.o1, a.out1, P.E, P.mrows, a.N, a.ldo, a.so))))
            return false;
        return map_mn(&P.a, P.wide_a, a.a, P.halves, rows, P.mrows, a.lda, P.halves > 1 ? P.mrows : rows * a.lda) &&
               map_mn(&P.b0, P.wide_b, a.b, 1, rows, a.N, a.ldb, rows * a.ldb);
    }
    pair = use_pair(a.plan, a.M, P.n_blocks);
    const int64_t rows = grouped ? a.plan.max_rows : a.M;
    if (!grouped) P.rows = a.M;
    RowPlan rp = a.plan;
    rp.T = a.M;
    P.tall = pair && !grouped && use_tall(a.M, 1, P.n_blocks, blocks_of(a.R, kBR));
    tiles = row_grid(P, rp, pair);
    P.bias0 = static_cast<const __nv_bfloat16*>(a.bias);
    P.sbias = a.sbias;
    P.act = a.act;
    P.row_scale = a.row_scale;
    P.residual = static_cast<const __nv_bfloat16*>(a.residual);
    P.ldr = a.ldr;
    P.pre = static_cast<__nv_bfloat16*>(a.pre);
    P.ldp = a.ldp;
    P.out_f32 = a.out_f32;
    const int64_t E = grouped ? a.plan.E : 1;
    const int halves = a.kind == kNN && a.split ? 2 : 1;
    const int64_t R = a.R / halves;
    P.nk_half = int(blocks_of(R, kBR));
    P.nk = P.nk_half * halves;
    P.b_split = halves > 1;
    if (!pair) P.splits = splits_of(tiles, P.nk, 8, row_hint(a.plan, a.M));
    if (!a.out) return true;
    if (!map_a_k(&P.a, a.a, rows, a.lda, R, halves)) return false;
    if (a.kind == kNT) return map_b_k(&P.b0, a.b, E, a.N, 1, R);
    return map_mn(&P.b0, P.wide_b, a.b, E, R, a.N, a.ldb, R * a.ldb) &&
           (halves == 1 || map_mn(&P.b1, P.wide_b, a.b1, E, R, a.N, a.ldb, R * a.ldb));
}

}  // namespace

cudaError_t launch_tc_gemm_nt(const GemmArgs& a, cudaStream_t s) {
    TcTrain P;
    bool pair;
    int64_t tiles;
    if (!set_up(a, P, pair, tiles)) return cudaErrorInvalidValue;
    return launch<kNT, kStore>(P, pair, tiles, s);
}

cudaError_t launch_tc_gemms(const GemmArgs* a, int n, cudaStream_t s) {
    TcTrain P[kMaxMix];
    bool pair[kMaxMix];
    int64_t tiles[kMaxMix];
    if (n > kMaxMix) return cudaErrorInvalidValue;
    for (int i = 0; i < n; ++i)
        if (!set_up(a[i], P[i], pair[i], tiles[i])) return cudaErrorInvalidValue;
    // together no more tiles than SMs: one launch, split by the longest reduction, unless one after
    // the other each is split better and that is worth the launches (7508 tokens 400 -> 1864 60 us
    // together, 44 apart). Gradients that were not asked for count here too, so that the others do
    // not depend on them.
    int64_t sum = 0, nk = 0, rows = 0, apart = 0;
    bool any_pair = false;
    for (int i = 0; i < n; ++i) {
        const int64_t r = P[i].tn ? P[i].mrows : row_hint(a[i].plan, a[i].M);
        sum += tiles[i];
        nk = std::max<int64_t>(nk, P[i].nk);
        rows = std::max(rows, r);
        apart += split_cost(P[i].nk, P[i].splits, r) + 250;
        any_pair = any_pair || pair[i];
    }
    const int splits = splits_of(sum, nk, 8, rows);
    if (n > 1 && !any_pair && sum <= sms() && split_cost(nk, splits, rows) + 250 <= apart) {
        int m = 0;
        sum = 0;
        for (int i = 0; i < n; ++i) {
            if (!a[i].out) continue;
            P[m] = P[i];
            P[m++].splits = splits;
            sum += tiles[i];
        }
        if (m == 0) return cudaSuccess;
        n = m;
        return splits > 1 ? launch_t<kMix, kStore, false, true>(P, n, sum, s)
                          : launch_t<kMix, kStore, false, false>(P, n, sum, s);
    }
    for (int i = 0; i < n; ++i) {
        if (!a[i].out) continue;
        const cudaError_t e = P[i].bulk_out ? launch_t<kTN, kStoreBulk, true, false>(&P[i], 1, tiles[i], s)
                              : P[i].tn     ? launch<kTN, kStore>(P[i], pair[i], tiles[i], s)
                                            : launch<kNN, kStore>(P[i], pair[i], tiles[i], s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_tc_gateup(const GemmArgs& g, const GatedArgs& ga, cudaStream_t s) {
    TcTrain P = base_of(g.plan);
    const bool grouped = g.plan.offsets != nullptr;
    P.N = ga.I;
    P.n_blocks = int(blocks_of(ga.I, 128));
    const bool pair = use_pair(g.plan, g.plan.T, P.n_blocks);
    const int64_t tiles = row_grid(P, g.plan, pair);
    const int64_t rows = grouped ? g.plan.max_rows : g.plan.T, E = grouped ? g.plan.E : 1;
    P.nk = P.nk_half = int(blocks_of(g.R, kBR));
    if (!pair) P.splits = splits_of(tiles, P.nk, 4, row_hint(g.plan, g.plan.T));
    P.bias0 = static_cast<const __nv_bfloat16*>(g.bias);
    P.bias1 = static_cast<const __nv_bfloat16*>(g.bias1);
    P.sbias = g.sbias;
    P.act = ga.act;
    P.limit = ga.limit;
    P.alpha = ga.alpha;
    P.cexp = -1.44269504f * (ga.act == MOE_ACT_SWIGLU ? 1.0f : ga.alpha);  // exp as a power of two
    P.pre = static_cast<__nv_bfloat16*>(ga.pre);
    P.ldp = 2 * ga.I;
    P.out = ga.h;
    P.ldo = ga.I;
    if (!map_a_k(&P.a, g.a, rows, g.lda, g.R, 1) || !map_b_k(&P.b0, g.b, E, ga.I, ga.interleaved ? 2 : 1, g.R))
        return cudaErrorInvalidValue;
    if (!ga.interleaved && !map_b_k(&P.b1, g.b1, E, ga.I, 1, g.R)) return cudaErrorInvalidValue;
    if (ga.interleaved) return launch<kNT, kGateUpI>(P, pair, tiles, s);
    return launch<kNT, kGateUp>(P, pair, tiles, s);
}

int dgated_parts(const RowPlan& p, int I, int64_t R) {
    TcTrain P = base_of(p);
    P.n_blocks = int(blocks_of(I, kCols));
    const bool pair = use_pair(p, p.T, P.n_blocks);
    const int64_t tiles = row_grid(P, p, pair);
    return 2 * P.n_blocks * (pair ? 1 : splits_of(tiles, blocks_of(R, kBR), 8, row_hint(p, p.T)));
}

cudaError_t launch_tc_dgated(const GemmArgs& g, const GatedArgs& ga, float* partial, cudaStream_t s) {
    TcTrain P = base_of(g.plan);
    const bool grouped = g.plan.offsets != nullptr;
    P.N = ga.I;
    P.n_blocks = int(blocks_of(ga.I, kCols));
    const bool pair = use_pair(g.plan, g.plan.T, P.n_blocks);
    const int64_t tiles = row_grid(P, g.plan, pair);
    const int64_t rows = grouped ? g.plan.max_rows : g.plan.T, E = grouped ? g.plan.E : 1;
    P.nk = P.nk_half = int(blocks_of(g.R, kBR));
    if (!pair) P.splits = splits_of(tiles, P.nk, 8, row_hint(g.plan, g.plan.T));
    P.act = ga.act;
    P.limit = ga.limit;
    P.alpha = ga.alpha;
    P.cexp = -1.44269504f * (ga.act == MOE_ACT_SWIGLU ? 1.0f : ga.alpha);  // exp as a power of two
    P.row_scale = ga.topk_w;
    P.pre = static_cast<__nv_bfloat16*>(ga.pre);
    P.ldp = 2 * ga.I;
    P.dgu = static_cast<__nv_bfloat16*>(ga.dgu);
    P.hw = static_cast<__nv_bfloat16*>(ga.hw);
    P.partial = partial;
    P.parts = dgated_parts(g.plan, ga.I, g.R);
    if (!map_a_k(&P.a, g.a, rows, g.lda, g.R, 1) || !map_mn(&P.b0, P.wide_b, g.b, E, g.R, ga.I, g.ldb, g.sb))
        return cudaErrorInvalidValue;
    if (ga.interleaved) return launch<kNN, kDGatedI>(P, pair, tiles, s);
    return launch<kNN, kDGated>(P, pair, tiles, s);
}

}  // namespace moe
