// Matrix products grouped by expert over ragged row ranges (tcgen05), for use next to the
// fused FFN: the plain product and its two gradients over bf16 operands, and the product of
// E4M3 operands with one fp32 scale per 128 of the reduction dimension on both sides.
//
// With rows r of expert e in [offsets[e], offsets[e+1]):
//   forward  y[r, n]     = sum_k x[r, k] w[e, n, k]
//   dgrad    dx[r, k]    = sum_n dy[r, n] w[e, n, k]
//   wgrad    dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]
//   fp8      y[r, n]     = sum_b (sum_{k in b} xq[r, k] wq[e, n, k]) xs[r, b] ws[e, n, b]
//
// All four are one tile product D[m, j] = sum_c A[m, c] B[j, c] whose m runs along the
// contiguous dimension of the output, so a warp's 32 TMEM lanes store 32 neighbouring
// elements of one output row:
//             m   j     c     A                        B
//   forward   n   row   k     w rows (c contiguous)    x rows (c contiguous)
//   dgrad     k   row   n     w read along k (m cont.) dy rows (c contiguous)
//   wgrad     k   n     row   x rows (m contiguous)    dy rows (j contiguous)
// Operands whose reduction dimension is contiguous in memory are K-major shared-memory
// tiles, the others MN-major ones (the tensor core transposes while it reads); both arrive
// by TMA in the 128-byte swizzle, and nothing is transposed or copied beforehand.
#include "common.cuh"
#include "internal.h"
#include <type_traits>

namespace moe {

constexpr int kGemmFwd = 0, kGemmDgrad = 1, kGemmWgrad = 2, kGemmFp8 = 3;

// Warps 0-3: TMA, MMA, scales, tail rows; from 4 on the epilogue: 16 warps for large bf16 tiles
// (it stores once per tile, and many warps hide each other's latencies), 12 for large fp8 ones
// (their sums stay in registers from K block to K block; 8 or 16 warps took 6% and 50% longer),
// 8 for small tiles.
__host__ __device__ constexpr int gemm_epi_warps(bool fp8, int BN) { return BN <= 64 ? 8 : fp8 ? 12 : 16; }
// CTAs per SM: two for the smallest tiles, so that one of them, or the next kernel's, sets up and
// loads while the other computes or stores.
__host__ __device__ constexpr int gemm_ctas(int BN) { return BN <= 32 ? 2 : 1; }
__host__ __device__ constexpr int gemm_threads(bool fp8, int BN) { return 128 + 32 * gemm_epi_warps(fp8, BN); }
constexpr int kGemmABytes = 128 * 128;     // one CTA's A tile of a stage: 128 m x 128 bytes
constexpr int kGemmBoxRows = 32;           // rows of B in a small TMA box (K-major B)
__host__ __device__ constexpr int gemm_big_box(int rows) { return rows > 128 ? 128 : rows; }   // ... in a large one
constexpr int kGemmMaxStages = 10;
constexpr int kGemmXsSlots = 2;            // ring of scales (fp8), four K blocks each

struct GemmParams {
    const int32_t *offsets;   // [E+1]; null: one expert with all rows
    int E, n_rows;
    int M;                    // extent of m (columns of the output)
    int J;                    // wgrad: extent of j (rows of one expert's output)
    int C;                    // extent of c (unused by wgrad: the expert's rows)
    int m_tiles, j_tiles;     // tiles along m; wgrad: along j
    int stages;               // shared-memory ring depth
    int part;                 // K blocks that the tensor core sums by itself (fp8: 1)
    void *out;
    int64_t ldo, out_estride; // elements; out_estride: wgrad
    int out_fp32, accumulate;
    int quads;                // fp8: weight rows in the lane order that gives a thread four neighbours
    int vec;                  // fp8: results may be stored four at a time
    const float *xs, *ws;     // fp8 scales: [n_rows][xs_ld], [E][M][ws_ld]
    int64_t xs_ld, ws_ld, ws_estride;
};

struct alignas(16) GemmSmem {
    uint64_t full[kGemmMaxStages];    // operands of a stage landed (and tail rows cleared)
    uint64_t empty[kGemmMaxStages];   // the stage's MMAs have read them
    uint64_t tail[kGemmMaxStages];    // wgrad: a stage with rows to clear landed in this CTA
    uint64_t tailpeer[kGemmMaxStages];   // and the pair's other CTA has cleared its own
    uint64_t accfull[4], accempty[4];
    uint64_t scfull[kGemmXsSlots], scempty[kGemmXsSlots];
    uint32_t tmem_base;
    int abort_flag;
    int total_items;
};

// Behind it: each expert's first row and rows (int2) and its first row tile (int, one more), for
// E experts where shared memory is short, else for kMaxExperts (a fixed place, which saves the
// epilogue registers); and, for fp8, kGemmXsSlots times four K blocks' scales of the tile's rows
// ([BN]) and of the CTA's weight rows ([128]).
template <int BN>
__host__ __device__ constexpr int gemm_table(int E) { return BN <= 32 ? E : kMaxExperts; }
template <int BN>
__host__ __device__ constexpr int gemm_tables_bytes(int E) { return ((gemm_table<BN>(E) + 1) * 12 + 15) & ~15; }
template <bool FP8, int BN>
__host__ __device__ constexpr int gemm_smem_bytes(int E) {
    return (int)sizeof(GemmSmem) + gemm_tables_bytes<BN>(E) + (FP8 ? kGemmXsSlots * 4 * (BN + 128) * 4 : 0);
}
__device__ __forceinline__ const int2 *gemm_ranges(const GemmSmem &sm) { return reinterpret_cast<const int2 *>(&sm + 1); }
template <int BN>
__device__ __forceinline__ const int *gemm_tile_starts(const GemmSmem &sm, const GemmParams &p) {
    return reinterpret_cast<const int *>(gemm_ranges(sm) + gemm_table<BN>(p.E));
}

struct GemmItem {
    int e, m0;      // expert, first m of the CTA group's tile
    int row0;       // first row of x or dy (wgrad: first row of the expert)
    int valid;      // rows of the tile (wgrad: rows of the expert)
    int j0, nt;     // first j of the output tile; MMA N
    int kblocks;
};

// Row range of expert e, kept inside the n_rows rows whatever the offsets hold.
__device__ __forceinline__ void gemm_range(const GemmParams &p, int e, int &beg, int &n) {
    if (!p.offsets) {
        beg = 0;
        n = p.n_rows;
        return;
    }
    const int a = p.offsets[e], b = p.offsets[e + 1];
    beg = min(max(a, 0), p.n_rows);
    const int end = min(max(b, 0), p.n_rows);
    n = max(end - beg, 0);
    if (a < 0 || b > p.n_rows || b < a) flag_error(2);
}

// An expert's n rows are cut into ceil(n / BN) tiles of equal size, rounded up to the step of
// the MMA's N, so 260 rows cost two tiles of about 130, not one of 256 and one of 4.
template <int CG, int BN>
__device__ __forceinline__ int gemm_tile_rows(int n) {
    const int t = (n + BN - 1) / BN;
    const int r = (n + t - 1) / t;
    constexpr int G = 16 * CG;
    return (r + G - 1) / G * G;
}

// Tile i of an expert's jt by p.m_tiles: along m first; with STRIPS in strips of kGemmStrip m
// tiles, so that the tiles at work at a time form a compact block, which reads each operand
// from HBM a few times only when they do not fit in L2.
constexpr int kGemmStrip = 16;
template <bool STRIPS>
__device__ __forceinline__ void gemm_order(const GemmParams &p, int i, int jt, int &m, int &j) {
    int width = p.m_tiles, m0 = 0;
    if (STRIPS) {
        m0 = i / (kGemmStrip * jt) * kGemmStrip;
        i -= m0 * jt;
        width = min(kGemmStrip, p.m_tiles - m0);
    }
    j = i / width;
    m = m0 + i - j * width;
}

template <int MODE, int CG, int BN, bool STRIPS>
__device__ __forceinline__ GemmItem gemm_item(const GemmSmem &sm, const GemmParams &p, int item) {
    const int2 *range = gemm_ranges(sm);
    const int *tile_start = gemm_tile_starts<BN>(sm, p);
    constexpr int G = 16 * CG;
    GemmItem it;
    int m, j;
    if (MODE == kGemmWgrad) {
        const int tiles = p.m_tiles * p.j_tiles;
        it.e = item / tiles;
        gemm_order<STRIPS>(p, item - it.e * tiles, p.j_tiles, m, j);
        it.m0 = m * (128 * CG);
        it.j0 = j * BN;
        it.row0 = range[it.e].x;
        it.valid = range[it.e].y;
        it.nt = min(BN, (p.J - it.j0 + G - 1) / G * G);
        it.kblocks = (it.valid + 63) / 64;
        return it;
    }
    const int rt = item / p.m_tiles;
    int lo = 0, hi = p.E - 1;   // expert with tile_start[e] <= rt < tile_start[e+1]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tile_start[mid] <= rt) lo = mid; else hi = mid - 1;
    }
    it.e = lo;
    const int beg = range[lo].x, n = range[lo].y, t0 = tile_start[lo];
    if (STRIPS) {
        gemm_order<true>(p, item - t0 * p.m_tiles, tile_start[lo + 1] - t0, m, j);
    } else {
        j = rt - t0;
        m = item - rt * p.m_tiles;
    }
    it.m0 = m * (128 * CG);
    const int tr = gemm_tile_rows<CG, BN>(n);
    it.row0 = beg + j * tr;
    it.valid = min(tr, n - j * tr);
    it.j0 = it.row0;
    it.nt = (it.valid + G - 1) / G * G;
    constexpr int CB = MODE == kGemmFp8 ? 128 : 64;
    it.kblocks = (p.C + CB - 1) / CB;
    return it;
}

// ------------------------------------------------------------------ PTX of this file

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t mapa_u32(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Arrival on a barrier of any CTA of the cluster, by its shared::cluster address. Cluster
// scope is for arrivals that publish shared-memory writes; it costs about a microsecond when
// copies are in flight, so the ones that only free TMEM (read with tcgen05.wait::ld) go
// without.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// ... by the warp's lane 0, without a branch.
__device__ __forceinline__ void mbar_arrive_remote_lane0(uint32_t addr) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(addr),
                 "r"(threadIdx.x & 31)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// mbar_wait of common.cuh whose first polls (each suspends the thread for a while) go without
// the load of the limit, which takes longer than most of these waits. CLUSTER: cluster scope,
// for what mbar_arrive_cluster publishes.
template <bool CLUSTER = false>
__device__ __forceinline__ bool gemm_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    auto poll = [&] {
        if (!CLUSTER) return mbar_try_wait(bar, parity);
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        return ok != 0;
    };
    for (int i = 0; i < 32; ++i)
        if (poll()) return true;
    const uint64_t t0 = globaltimer();
    const uint64_t limit = *reinterpret_cast<volatile uint64_t *>(&g_wait_limit_ns);
    while (true) {
        if (poll()) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > limit) {
            *abort_flag = 1;
            flag_error(1);
            return false;
        }
    }
}

// A whole warp's wait: one answer for all lanes (no divergence, and the same where some lanes
// gave up).
__device__ __forceinline__ bool gemm_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, gemm_wait(bar, parity, abort_flag));
}

// TMA boxes into this CTA's shared memory; `bar` is a shared::cluster address, the pair
// leader's barrier for CTA pairs.
template <int CG>
__device__ __forceinline__ void gemm_tma_2d(void *dst, const CUtensorMap *m, uint32_t bar, int c0, int c1) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void gemm_tma_3d(void *dst, const CUtensorMap *m, uint32_t bar, int c0, int c1, int c2) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

// Groups of 32 rows, row 4 a + b of a group in place 8 b + a: dimensions (c, a, b, group, expert).
template <int CG>
__device__ __forceinline__ void gemm_tma_5d(void *dst, const CUtensorMap *m, uint32_t bar, int c0, int g, int e) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(c0), "r"(0), "r"(g), "r"(e)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
            "l"(m), "r"(bar), "r"(c0), "r"(0), "r"(g), "r"(e)
            : "memory");
}

template <int CG, bool FP8>
__device__ __forceinline__ void gemm_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (CG == 1 && !FP8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else if (!FP8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// Arrive on `bar` (both CTAs' copies for a pair) once this thread's MMAs so far are done.
template <int CG>
__device__ __forceinline__ void gemm_commit(uint64_t *bar) {
    if (CG == 1)
        mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void gemm_tmem_alloc(uint32_t *dst, uint32_t cols) {
    if (CG == 1) {
        tmem_alloc(dst, cols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void gemm_tmem_dealloc(uint32_t t, uint32_t cols) {
    if (CG == 1)
        tmem_dealloc(t, cols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
}

// Pairs of fp32 in one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 16 lanes x 32 columns of an accumulator in the layout of matrix fragments: register 2k + i of
// thread T is lane T/4 + 8i, column 4k + T%4. (Loads of 32 such columns for two warps a quarter
// take 1.15 times as long as with a lane per thread; the wider fragments of 16x256b, 1.7 times.)
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// tcgen05.wait::ld that the loaded registers pass through, so that no use of them can be
// scheduled before it.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// Shared-memory descriptor of an MN-major tile in the 128-byte swizzle: 64 elements of the
// m (or j) dimension per 128-byte row, one row per c, 8-row groups 1024 bytes apart; the
// next 64 elements of m are a whole box of 64 rows (8192 bytes) further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFF) >> 4);
    d |= (uint64_t)(8192 >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// One element of the result. The stores stay in program order (volatile), so that the compiler
// does not hold many addresses and converted values at once and spill.
template <bool F32>
__device__ __forceinline__ void gemm_store(const GemmParams &p, int64_t at, float v, bool on) {
    if (F32) {
        float *d = reinterpret_cast<float *>(p.out) + at;
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.f32 [%0], %1;\n\t}" ::"l"(d), "f"(v),
                     "r"((uint32_t)on)
                     : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b16 h;\n\tsetp.ne.u32 p, %2, 0;\n\tcvt.rn.bf16.f32 h, %1;\n\t"
            "@p st.global.b16 [%0], h;\n\t}" ::"l"(reinterpret_cast<__nv_bfloat16 *>(p.out) + at),
            "f"(v), "r"((uint32_t)on)
            : "memory");
    }
}

// Four neighbouring elements at an aligned address.
template <bool F32>
__device__ __forceinline__ void gemm_store4(const GemmParams &p, int64_t at, const float (&v)[4], bool on) {
    if (F32)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p st.global.v4.f32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(
                         reinterpret_cast<float *>(p.out) + at),
                     "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"((uint32_t)on)
                     : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b32 a, b;\n\tsetp.ne.u32 p, %5, 0;\n\tcvt.rn.bf16x2.f32 a, %2, %1;\n\t"
            "cvt.rn.bf16x2.f32 b, %4, %3;\n\t@p st.global.v2.b32 [%0], {a, b};\n\t}" ::"l"(
                reinterpret_cast<__nv_bfloat16 *>(p.out) + at),
            "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"((uint32_t)on)
            : "memory");
}

// Adds ACT units (16 columns each, 16 G apart) of an accumulator at TMEM address t to the sums.
template <int NU, int ACT, int G>
__device__ __forceinline__ void gemm_add_part(float (&acc)[NU][16], uint32_t t) {
#pragma unroll
    for (int i = 0; i < ACT; ++i) {
        uint32_t v[16];
        tmem_ld16(t + i * (16 * G), v);
        tmem_wait_ld16(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] += __uint_as_float(v[j]);
    }
}

// wgrad, whose time goes with its stores: writes a lane's sums, NU units of 16 columns, 16 G apart, from
// element o on; columns from lim on (unit and column counted from the tile's first) do not exist. One
// address that moves from row to row and, in whole tiles, no condition per element: 391 -> 364 us for
// 128 experts' gradients of 1536 x 2048 in 32 bits from 32768 rows. (The other products, which store
// less, were 1 to 2% slower with it.)
template <bool F32, int NU, int G>
__device__ __forceinline__ void gemm_store_rows(const GemmParams &p, int64_t o, float (&acc)[NU][16], int g, int lim) {
    constexpr int esz = F32 ? 4 : 2;
    const uint64_t row = (uint64_t)p.ldo * esz;
    uint64_t at = reinterpret_cast<uint64_t>(p.out) + (uint64_t)o * esz;
    if (F32 && p.accumulate) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if ((i * G + g) * 16 + j < lim) acc[i][j] += *reinterpret_cast<const float *>(at + (i * G * 16 + j) * row);
        }
    }
    auto put = [&](float v) {
        if constexpr (F32) __stcs(reinterpret_cast<float *>(at), v);
        else *reinterpret_cast<__nv_bfloat16 *>(at) = __float2bfloat16_rn(v);
    };
    const bool whole = __all_sync(0xffffffffu, lim >= 16 * G * NU);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        if (whole != (part == 0)) continue;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
#pragma unroll
            for (int j = 0; j < 16; ++j, at += row)
                if (part == 0 || (i * G + g) * 16 + j < lim) put(acc[i][j]);
            at += row * (16 * (G - 1));
        }
    }
}

// fp8: adds ACT groups (32 columns each, 32 G apart) of an accumulator, times the columns' scales
// xs and the four lanes' scales w (pairs of lanes 8 apart), to the sums. In the fragment layout a
// thread needs a quarter of the columns' scales; with a lane's whole row per thread the copies
// of them filled the path from shared memory (128 bytes a clock) for longer than the arithmetic
// takes, two operations an element (384 clocks a block of 192 columns).
template <int NG, int ACT, int G, typename F>
__device__ __forceinline__ void gemm_add_scaled(float (&acc)[NG][2][16], uint32_t t, const float *xs, const uint64_t (&w)[2],
                                                F &&release) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < ACT; ++i) {
        uint32_t v[16];
        tmem_ld_16x32(t + i * (32 * G), v);
        // the scales of a thread's eight columns 4k + T%4 lie next to each other
        const float4 *xs4 = reinterpret_cast<const float4 *>(xs + i * (32 * G) + 8 * (lane & 3));
        const float4 fa = xs4[0], fb = xs4[1];
        const float f[8] = {fa.x, fa.y, fa.z, fa.w, fb.x, fb.y, fb.z, fb.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h) tmem_ld_16x32(t + i * (32 * G) + (16u << 16), v);
            tmem_wait_ld16(v);
            if (i == ACT - 1 && h == 1) release();
#pragma unroll
            for (int k = 0; k < 8; ++k) {   // (sums kept as pairs made the compiler move and spill them: 15% slower)
                uint64_t a = pack2(acc[i][h][2 * k], acc[i][h][2 * k + 1]);
                a = fma2(mul2(pack2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), pack2(f[k], f[k])), w[h], a);
                unpack2(a, acc[i][h][2 * k], acc[i][h][2 * k + 1]);
            }
        }
    }
}

// ------------------------------------------------------------------ kernel

template <int MODE, int CG, int BN, bool STRIPS>
__device__ __forceinline__ void gemm_body(const CUtensorMap &amap, const CUtensorMap &bmap, const CUtensorMap &bbig,
                                          const GemmParams &p) {
    constexpr bool FP8 = MODE == kGemmFp8;
    constexpr bool A_MN = MODE == kGemmDgrad || MODE == kGemmWgrad, B_MN = MODE == kGemmWgrad;
    constexpr int EPI = gemm_epi_warps(FP8, BN);
    constexpr int BROWS = BN / CG;                       // j's of B that this CTA holds
    constexpr int BIG = gemm_big_box(BROWS);
    constexpr int STAGE = kGemmABytes + BROWS * 128;
    constexpr int CB = FP8 ? 128 : 64;                   // c's per stage
    constexpr int NACC = BN <= 128 ? 4 : 2;              // accumulators
    constexpr uint32_t TMEM_COLS = BN <= 32 ? 128 : BN <= 64 ? 256 : 512;   // a power of two with room for them
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int ns = p.stages;
    GemmSmem &sm = *reinterpret_cast<GemmSmem *>(ring + ns * STAGE);
    float *xs_s = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(&sm + 1) + gemm_tables_bytes<BN>(p.E));
    float *ws_s = xs_s + kGemmXsSlots * 4 * BN;
    volatile int *abort_flag = &sm.abort_flag;
    const int warp = warp_id(), lane = lane_id();
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int first = CG == 2 ? blockIdx.x / 2 : blockIdx.x, step = CG == 2 ? gridDim.x / 2 : gridDim.x;

    // what needs none of the previous kernel's results comes before the wait for it
    if (threadIdx.x == 0) {
        for (int s = 0; s < ns; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
            mbar_init(&sm.tail[s], 1);
            mbar_init(&sm.tailpeer[s], 1);
        }
        for (int b = 0; b < NACC; ++b) {
            mbar_init(&sm.accfull[b], 1);
            mbar_init(&sm.accempty[b], CG * EPI);
        }
        for (int s = 0; s < kGemmXsSlots; ++s) {
            mbar_init(&sm.scfull[s], 2);
            mbar_init(&sm.scempty[s], EPI);
        }
        sm.abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&amap);
        tma_prefetch_desc(&bmap);
        if (MODE != kGemmWgrad && BIG > kGemmBoxRows) tma_prefetch_desc(&bbig);
    }
    pdl_wait();
    int2 *range = const_cast<int2 *>(gemm_ranges(sm));
    int *tile_start = const_cast<int *>(gemm_tile_starts<BN>(sm, p));
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int beg, n;
        gemm_range(p, e, beg, n);
        range[e] = make_int2(beg, n);
    }
    __syncthreads();
    // TMEM between the wait and the release: a kernel that holds some while it waits for another one
    // that has yet to allocate its own on the same SM would never end
    if (warp == 2) gemm_tmem_alloc<CG>(&sm.tmem_base, TMEM_COLS);
    if (warp == 3) {   // first row tile of each expert
        int run = 0;
        if (lane == 0) tile_start[0] = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int incl = e < p.E ? (range[e].y + BN - 1) / BN : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
            }
            if (e < p.E) tile_start[e + 1] = run + incl;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) sm.total_items = MODE == kGemmWgrad ? p.E * p.j_tiles * p.m_tiles : run * p.m_tiles;
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) pdl_release();
    if (CG == 2) cluster_sync_all();   // the peer's barriers exist before anything arrives on them
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const int total = sm.total_items;
    if (warp == 0) {
        // =================================================== producer (one thread)
        if (lane == 0) {
            const uint32_t lead_full0 = CG == 2 ? mapa_u32(smem_u32(&sm.full[0]), 0) : smem_u32(&sm.full[0]);
            int s = 0, kc = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int item = first; item < total && ok; item += step) {
                const GemmItem it = gemm_item<MODE, CG, BN, STRIPS>(sm, p, item);
                const int bj0 = it.j0 + (int)rank * (it.nt / CG);          // this CTA's share of B
                // K-major B in boxes of BIG rows, a rest of up to BIG - 64 rows in boxes of 32: each
                // box takes time to issue (4 KB boxes only: a quarter off the rate; three of them
                // for 96 rows instead of one of 128: 258 against 242 us for E = 8, 1025 rows each,
                // K = N = 4096), and a box takes no more than 63 rows too many
                const int share = it.nt / CG;
                const int big = BIG > kGemmBoxRows ? (share + 63) / BIG : 0;
                const int small = big * BIG >= share ? 0 : (share - big * BIG + kGemmBoxRows - 1) / kGemmBoxRows;
                const int chunks = (share + 63) / 64;
                const uint32_t bytes = kGemmABytes + (B_MN ? chunks * 8192 : (big * BIG + small * kGemmBoxRows) * 128);
                const int m0 = it.m0 + (int)rank * 128;
                for (int kb = 0; kb < it.kblocks; ++kb) {
                    if (!gemm_wait(&sm.empty[s], ph ^ 1, abort_flag)) { ok = false; break; }
                    uint32_t bar = lead_full0 + 8 * s;
                    if (MODE == kGemmWgrad && kb == it.kblocks - 1 && (it.valid & 15)) {
                        bar = smem_u32(&sm.tail[s]);   // rows to clear: this CTA's warp 3 goes first
                        mbar_expect_tx(&sm.tail[s], bytes);
                    } else if (rank == 0) {
                        mbar_expect_tx(&sm.full[s], CG * bytes);   // both CTAs' copies arrive here
                    }
                    uint8_t *a = ring + s * STAGE, *b = a + kGemmABytes;
                    const int c0 = kb * CB;
                    if (MODE == kGemmWgrad) {
                        const int r0 = it.row0 + c0;
                        gemm_tma_2d<CG>(a, &amap, bar, m0, r0);
                        gemm_tma_2d<CG>(a + 8192, &amap, bar, m0 + 64, r0);
                        for (int i = 0; i < chunks; ++i) gemm_tma_2d<CG>(b + i * 8192, &bmap, bar, bj0 + i * 64, r0);
                    } else {
                        if (A_MN) {
                            gemm_tma_3d<CG>(a, &amap, bar, m0, c0, it.e);
                            gemm_tma_3d<CG>(a + 8192, &amap, bar, m0 + 64, c0, it.e);
                        } else if (FP8 && p.quads) {
                            gemm_tma_5d<CG>(a, &amap, bar, c0, m0 / 32, it.e);
                        } else {
                            gemm_tma_3d<CG>(a, &amap, bar, c0, m0, it.e);
                        }
                        for (int i = 0; i < big; ++i) gemm_tma_2d<CG>(b + i * BIG * 128, &bbig, bar, c0, bj0 + i * BIG);
                        for (int i = 0; i < small; ++i)
                            gemm_tma_2d<CG>(b + (big * BIG + i * kGemmBoxRows) * 128, &bmap, bar, c0,
                                            bj0 + big * BIG + i * kGemmBoxRows);
                    }
                    ++kc;
                    if (++s == ns) { s = 0; ph ^= 1; }
                }
            }
            // stay until the MMAs have released every stage, so that no copy and no arrival
            // is on its way into this CTA's shared memory when it ends
            for (int j = kc > ns ? kc - ns : 0; j < kc; ++j) {
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(&sm.empty[j % ns], (j / ns) & 1)) {
                    if (*abort_flag || globaltimer() - t0 > kWaitLimitNs) { flag_error(1); break; }
                }
            }
        }
    } else if (warp == 1) {
        // =================================================== MMA issuer (the leader's)
        // The whole warp runs the loop, so that descriptors and barrier addresses are uniform
        // values, and one elected thread issues: with the loop inside that thread each block
        // took some 400 cycles to issue, more than its MMAs take to run.
        if (rank == 0) {
            constexpr uint32_t idesc0 = (1u << 4) | (FP8 ? 0u : (1u << 7) | (1u << 10)) | (A_MN ? 1u << 15 : 0u) |
                                        (B_MN ? 1u << 16 : 0u) | ((uint32_t)(128 * CG >> 4) << 24);
            constexpr uint64_t AK = A_MN ? 128 : 2, BK = B_MN ? 128 : 2;   // 16 (fp8: 32) c's further
            const bool issues = elect_one();
            const int part = FP8 ? 1 : p.part;
            const uint32_t ring0 = smem_u32(ring);
            const uint64_t ad0 = A_MN ? smem_desc_mn_sw128(ring0) : smem_desc_sw128(ring0);
            const uint64_t bd0 = B_MN ? smem_desc_mn_sw128(ring0 + kGemmABytes) : smem_desc_sw128(ring0 + kGemmABytes);
            int s = 0, u = 0;   // u: accumulator uses so far
            uint32_t ph = 0;
            bool ok = true;
            for (int item = first; item < total && ok; item += step) {
                const GemmItem it = gemm_item<MODE, CG, BN, STRIPS>(sm, p, item);
                const uint32_t idesc = idesc0 | ((uint32_t)(it.nt >> 3) << 17);
                int left = 0;   // blocks that this accumulator still takes
                for (int kb = 0; kb < it.kblocks; ++kb) {
                    const bool fresh = left == 0;
                    if (fresh) {
                        left = min(part, it.kblocks - kb);
                        if (!gemm_wait_warp(&sm.accempty[u % NACC], ((u / NACC) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    }
                    if (!gemm_wait_warp(&sm.full[s], ph, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d = tmem + (u % NACC) * BN;
                    const uint64_t ad = ad0 + (uint32_t)(s * (STAGE / 16)), bd = bd0 + (uint32_t)(s * (STAGE / 16));
                    const bool last = --left == 0;
                    if (issues) {
                        if (MODE == kGemmWgrad && it.valid - kb * 64 < 49) {   // the steps with rows of the expert
                            for (int i = 0; i < (it.valid - kb * 64 + 15) / 16; ++i)
                                gemm_mma<CG, FP8>(d, ad + AK * i, bd + BK * i, idesc, !(fresh && i == 0));
                        } else {
                            gemm_mma<CG, FP8>(d, ad, bd, idesc, !fresh);
                            gemm_mma<CG, FP8>(d, ad + AK, bd + BK, idesc, 1);
                            gemm_mma<CG, FP8>(d, ad + 2 * AK, bd + 2 * BK, idesc, 1);
                            gemm_mma<CG, FP8>(d, ad + 3 * AK, bd + 3 * BK, idesc, 1);
                        }
                        gemm_commit<CG>(&sm.empty[s]);
                        if (last) gemm_commit<CG>(&sm.accfull[u % NACC]);
                    }
                    __syncwarp();
                    if (last) ++u;
                    if (++s == ns) { s = 0; ph ^= 1; }
                }
            }
        }
    } else if (FP8 && (warp == 2 || warp == 3)) {
        // =================================================== scales (fp8)
        // The scales of the tile's rows and of the CTA's 128 weight rows, four K blocks at a time
        // (one 16-byte load a row where the arrays allow it: a 4-byte copy a row and block kept
        // the L1 busy for longer than the block's MMAs), transposed on the way into the slots of
        // four. The next four are loaded before this warp waits for a slot.
        constexpr int R = (BN + 128 + 63) / 64;   // per lane of the two warps, counting rows of x, then of w
        const bool vec = p.xs_ld % 4 == 0 && p.ws_estride % 4 == 0 &&
                         ((reinterpret_cast<uintptr_t>(p.xs) | reinterpret_cast<uintptr_t>(p.ws)) & 15) == 0;
        int x = 0;   // slots filled so far
        bool ok = true;
        for (int item = first; item < total && ok; item += step) {
            const GemmItem it = gemm_item<MODE, CG, BN, STRIPS>(sm, p, item);
            const int r0 = (warp - 2) * 32 + lane, mbase = it.m0 + (int)rank * 128;
            float4 nx[R];
            auto load = [&](int kb) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int r = r0 + 64 * i, w = r - BN;
                    nx[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (!(w < 0 ? r < it.valid : w < 128 && mbase + w < p.M) || kb >= it.kblocks) continue;
                    const float *src = w < 0 ? p.xs + (int64_t)(it.row0 + r) * p.xs_ld + kb
                                             : p.ws + (int64_t)it.e * p.ws_estride + (int64_t)(mbase + w) * p.ws_ld + kb;
                    if (vec) {
                        nx[i] = __ldg(reinterpret_cast<const float4 *>(src));
                    } else {
                        nx[i].x = src[0];
                        if (kb + 1 < it.kblocks) nx[i].y = src[1];
                        if (kb + 2 < it.kblocks) nx[i].z = src[2];
                        if (kb + 3 < it.kblocks) nx[i].w = src[3];
                    }
                }
            };
            load(0);
            for (int kb = 0; kb < it.kblocks && ok; kb += 4) {
                float4 cur[R];
#pragma unroll
                for (int i = 0; i < R; ++i) cur[i] = nx[i];
                load(kb + 4);
                const int slot = x % kGemmXsSlots;
                if (!gemm_wait_warp(&sm.scempty[slot], ((x / kGemmXsSlots) & 1) ^ 1, abort_flag)) { ok = false; break; }
                ++x;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const int r = r0 + 64 * i, w = r - BN;
                        const float v = b == 0 ? cur[i].x : b == 1 ? cur[i].y : b == 2 ? cur[i].z : cur[i].w;
                        if (w < 0) xs_s[(slot * 4 + b) * BN + ((r & ~31) | (r & 3) << 3 | (r >> 2 & 7))] = v;   // as gemm_add_scaled reads it
                        else if (w < 128) ws_s[(slot * 4 + b) * 128 + w] = v;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.scfull[slot]);
            }
        }
    } else if (warp < 4) {
        // =================================================== wgrad (warp 3): rows behind the expert's last
        // The last block of an expert holds rows of the next one; the up to 15 of them that
        // the last MMA step would read are cleared in both operands (0 * inf is not 0).
        if (MODE == kGemmWgrad && warp == 3) {
            int s = 0;
            uint32_t tph = 0;   // bit s: parity of tail[s]
            bool ok = true;
            for (int item = first; item < total && ok; item += step) {
                const GemmItem it = gemm_item<MODE, CG, BN, STRIPS>(sm, p, item);
                if (!it.kblocks) continue;
                s = (s + it.kblocks - 1) % ns;   // the stage of the last block
                if (it.valid & 15) {
                    if (!gemm_wait_warp(&sm.tail[s], (tph >> s) & 1, abort_flag)) { ok = false; break; }
                    tph ^= 1u << s;
                    uint8_t *a = ring + s * STAGE;
                    const int r0 = it.valid & 63, r1 = (r0 + 15) & ~15;
                    const int chunks = 2 + (it.nt / CG + 63) / 64;   // A's two, then B's
                    for (int r = r0 + (lane >> 3); r < r1; r += 4)
                        for (int c = 0; c < chunks; ++c)
                            *reinterpret_cast<uint4 *>(a + c * 8192 + r * 128 + (lane & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (CG == 2 && rank == 1) {
                        if (lane == 0) mbar_arrive_cluster(mapa_u32(smem_u32(&sm.tailpeer[s]), 0));
                    } else {
                        if (CG == 2 && !__all_sync(0xffffffffu, gemm_wait<true>(&sm.tailpeer[s], ((tph >> s) & 1) ^ 1, abort_flag))) { ok = false; break; }
                        if (lane == 0) mbar_arrive(&sm.full[s]);
                    }
                }
                s = s + 1 == ns ? 0 : s + 1;
            }
        }
    } else {
        // =================================================== epilogue
        // Warp quarter q owns TMEM lanes 32q..32q+31; the quarter's G warps take turns on groups
        // of columns.
        constexpr int G = EPI / 4;
        const int q = warp & 3, g = (warp - 4) >> 2;
        const uint32_t lead_empty0 = CG == 2 ? mapa_u32(smem_u32(&sm.accempty[0]), 0) : smem_u32(&sm.accempty[0]);
        int u = 0;   // accumulators used so far
        bool ok = true;
        if constexpr (FP8) {
            constexpr int NG = (BN / 32 + G - 1) / G;   // groups of 32 columns per warp
            // the thread's four rows of a quarter: r0, r0 + dr, ...
            const int r0 = p.quads ? lane & ~3 : lane >> 2, dr = p.quads ? 1 : 8;
            int x = 0;                                  // slots of scales used so far
            for (int item = first; item < total && ok; item += step) {
                const GemmItem it = gemm_item<MODE, CG, BN, STRIPS>(sm, p, item);
                const int groups = ((it.nt + 31) / 32 + G - 1 - g) / G;
                float acc[NG][2][16];   // [h]: lanes 16 h + ...
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[i][j >> 4][j & 15] = 0.0f;
                for (int kb = 0; kb < it.kblocks; ++kb, ++u) {
                    const int slot = x % kGemmXsSlots;
                    if ((kb & 3) == 0 && !gemm_wait_warp(&sm.scfull[slot], (x / kGemmXsSlots) & 1, abort_flag)) { ok = false; break; }
                    if (!gemm_wait_warp(&sm.accfull[u % NACC], (u / NACC) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (u % NACC) * BN + g * 32;
                    const float *xs = xs_s + (slot * 4 + (kb & 3)) * BN + g * 32;
                    const float *ws = ws_s + (slot * 4 + (kb & 3)) * 128 + q * 32 + r0;
                    const uint64_t w[2] = {pack2(ws[0], ws[dr]), pack2(ws[2 * dr], ws[3 * dr])};
                    // all of a warp's groups, or half of them: a condition per group would cost a
                    // select per sum
                    auto release = [&] {   // the accumulator is read
                        tc_fence_before();
                        __syncwarp();
                        if (CG == 2) mbar_arrive_remote_lane0(lead_empty0 + 8 * (u % NACC));
                        else if (lane == 0) mbar_arrive(&sm.accempty[u % NACC]);
                    };
                    if (2 * groups > NG) gemm_add_scaled<NG, NG, G>(acc, t, xs, w, release);
                    else if (groups > 0) gemm_add_scaled<NG, (NG + 1) / 2, G>(acc, t, xs, w, release);
                    else release();
                    const bool sc_done = (kb & 3) == 3 || kb + 1 == it.kblocks;
                    if (sc_done) {
                        if (lane == 0) mbar_arrive(&sm.scempty[slot]);
                        ++x;
                    }
                }
                if (!ok) break;
                const int m = it.m0 + (int)rank * 128 + q * 32 + r0, j = g * 32 + (lane & 3);
                const int64_t o = (int64_t)(it.j0 + j) * p.ldo + m;
                auto store = [&](auto f32) {
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int col = i * (32 * G) + 4 * k;   // j columns further for this thread
                            const int64_t at = o + (int64_t)col * p.ldo;
                            const float v[4] = {acc[i][0][2 * k], acc[i][0][2 * k + 1], acc[i][1][2 * k], acc[i][1][2 * k + 1]};
                            if (p.vec) {
                                gemm_store4<f32.value>(p, at, v, m < p.M && j + col < it.valid);
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    gemm_store<f32.value>(p, at + e * dr, v[e], m + e * dr < p.M && j + col < it.valid);
                            }
                        }
                    }
                };
                if (p.out_fp32) store(std::true_type{});
                else store(std::false_type{});
            }
        } else {
            constexpr int NU = BN / (16 * G);   // units of 16 columns per warp
            const int part = p.part;
            for (int item = first; item < total && ok; item += step) {
                const GemmItem it = gemm_item<MODE, CG, BN, STRIPS>(sm, p, item);
                if (MODE == kGemmWgrad && p.accumulate && !it.kblocks) continue;   // nothing to add: dw is not touched
                const int m = it.m0 + (int)rank * 128 + q * 32 + lane;
                const int jn = MODE == kGemmWgrad ? min(it.nt, p.J - it.j0) : it.valid;   // columns to store
                const int units = (it.nt / 16 + G - 1 - g) / G;
                float acc[NU][16];
#pragma unroll
                for (int i = 0; i < NU; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[i][j] = 0.0f;
                for (int kb = 0; kb < it.kblocks; kb += part, ++u) {
                    if (!gemm_wait_warp(&sm.accfull[u % NACC], (u / NACC) & 1, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (u % NACC) * BN + g * 16;
                    if (2 * units > NU) gemm_add_part<NU, NU, G>(acc, t);
                    else if (units > 0) gemm_add_part<NU, (NU + 1) / 2, G>(acc, t);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 2) mbar_arrive_remote(lead_empty0 + 8 * (u % NACC));
                        else mbar_arrive(&sm.accempty[u % NACC]);
                    }
                }
                if (!ok) break;
                int64_t o = (int64_t)(it.j0 + g * 16) * p.ldo + m;
                const int lim = m < p.M ? jn : 0;
                if constexpr (MODE == kGemmWgrad) {
                    o += (int64_t)it.e * p.out_estride;
                    if (p.out_fp32) gemm_store_rows<true, NU, G>(p, o, acc, g, lim);
                    else gemm_store_rows<false, NU, G>(p, o, acc, g, lim);
                    continue;
                }
                auto store = [&](auto f32) {
#pragma unroll
                    for (int i = 0; i < NU; ++i) {
#pragma unroll
                        for (int j = 0; j < 16; ++j, o += p.ldo) {
                            gemm_store<f32.value>(p, o, acc[i][j], (i * G + g) * 16 + j < lim);
                        }
                        o += 16 * (G - 1) * p.ldo;
                    }
                };
                if (p.out_fp32) store(std::true_type{});
                else store(std::false_type{});
            }
        }
    }
    // ---- the accumulators are read, no copy or arrival is in flight: release TMEM
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (sm.abort_flag) {   // a wait gave up: let whatever was in flight land first
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
    }
    if (CG == 2) cluster_sync_all();
    tc_fence_after();
    if (warp == 2) gemm_tmem_dealloc<CG>(tmem, TMEM_COLS);
}

// The fp8 kernel reads its parameters where the launch put them, the others a copy: either way the
// other one's registers come out worse (32768 rows over 128 experts of 2048 x 1536: fp8 229 against
// 217 us, bf16 251 against 246).
template <int MODE, int CG, int BN, bool STRIPS>
__global__ void __launch_bounds__(gemm_threads(false, BN), gemm_ctas(BN))
gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
            const __grid_constant__ CUtensorMap bbig, GemmParams p) {
    gemm_body<MODE, CG, BN, STRIPS>(amap, bmap, bbig, p);
}
template <int CG, int BN, bool STRIPS>
__global__ void __launch_bounds__(gemm_threads(true, BN), gemm_ctas(BN))
gemm_fp8_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                const __grid_constant__ CUtensorMap bbig, const __grid_constant__ GemmParams p) {
    gemm_body<kGemmFp8, CG, BN, STRIPS>(amap, bmap, bbig, p);
}

// ------------------------------------------------------------------ launch

// 2D map of a row-major matrix [rows][cols] with `ld` elements per row.
static moe_status gemm_map2(CUtensorMap *m, int esz, const void *base, int64_t rows, int64_t cols, int64_t ld,
                            int box_cols, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)std::max<int64_t>(rows, 1)};
    const uint64_t strides[1] = {(uint64_t)(ld * esz)};
    const uint32_t box[2] = {(uint32_t)box_cols, (uint32_t)box_rows};
    return make_tmap(m, esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

static moe_status gemm_map3(CUtensorMap *m, int esz, const void *base, int64_t E, int64_t rows, int64_t cols,
                            int64_t ld, int64_t estride, int box_cols, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)E};
    const uint64_t strides[2] = {(uint64_t)(ld * esz), (uint64_t)(estride * esz)};
    const uint32_t box[3] = {(uint32_t)box_cols, (uint32_t)box_rows, 1};
    return make_tmap(m, esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// One-byte weights [E][rows][cols] for gemm_tma_5d: 128 rows by 128 columns a box.
static moe_status gemm_map_quads(CUtensorMap *m, const void *base, int64_t E, int64_t rows, int64_t cols, int64_t ld,
                                 int64_t estride) {
    const uint64_t dims[5] = {(uint64_t)cols, 8, 4, (uint64_t)(rows / 32), (uint64_t)E};
    const uint64_t strides[4] = {(uint64_t)(4 * ld), (uint64_t)ld, (uint64_t)(32 * ld), (uint64_t)estride};
    const uint32_t box[5] = {128, 8, 4, 4, 1};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// One configuration: CG CTAs per tile (128 m's each), tiles of up to BN j's.
template <int MODE, int CG, int BN, bool STRIPS = false>
static moe_status gemm_launch(const GemmArgs &a, int nsm, cudaStream_t st) {
    constexpr bool FP8 = MODE == kGemmFp8;
    constexpr int STAGE = kGemmABytes + BN / CG * 128, BIG = gemm_big_box(BN / CG);
    constexpr int kSmemMax = gemm_ctas(BN) == 2 ? 113 * 1024 : 227 * 1024, esz = FP8 ? 1 : 2, cb = 128 / esz;
    const int N = a.N, K = a.K;
    CUtensorMap am, bm, bbig;
    GemmParams p;
    memset(&p, 0, sizeof(p));
    p.offsets = a.offsets;
    p.E = a.E;
    p.n_rows = a.n_rows;
    p.out = a.out;
    p.ldo = a.ldo;
    p.out_fp32 = a.out_fp32;
    moe_status r;
    int64_t tiles = (int64_t)a.n_rows / BN + std::min(a.n_rows, a.E);   // most row tiles that the rows can make
    if (MODE == kGemmWgrad) {
        if ((r = gemm_map2(&am, 2, a.w, a.n_rows, K, a.ldw, 64, 64)) != MOE_OK) return r;
        if ((r = gemm_map2(&bm, 2, a.x, a.n_rows, N, a.ldx, 64, 64)) != MOE_OK) return r;
        bbig = bm;   // not used
        p.M = K;
        p.J = N;
        p.j_tiles = (N + BN - 1) / BN;
        p.out_estride = a.out_estride;
        p.accumulate = a.accumulate;
        tiles = (int64_t)a.E * p.j_tiles;
    } else {
        const bool dgrad = MODE == kGemmDgrad;
        p.M = dgrad ? K : N;
        p.C = dgrad ? N : K;
        // fp8 weights of whole groups of 32 rows arrive in an order that gives each epilogue thread
        // four neighbouring rows, so that it stores 8 or 16 bytes at a time
        p.quads = FP8 && N % 32 == 0;
        const int osz = a.out_fp32 ? 4 : 2;
        p.vec = p.quads && a.ldo % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % (4 * osz) == 0;
        r = p.quads ? gemm_map_quads(&am, a.w, a.E, N, K, a.ldw, a.w_estride)
                    : gemm_map3(&am, esz, a.w, a.E, N, K, a.ldw, a.w_estride, cb, dgrad ? 64 : 128);
        if (r != MOE_OK) return r;
        if ((r = gemm_map2(&bm, esz, a.x, a.n_rows, p.C, a.ldx, cb, kGemmBoxRows)) != MOE_OK) return r;
        if ((r = gemm_map2(&bbig, esz, a.x, a.n_rows, p.C, a.ldx, cb, BIG)) != MOE_OK) return r;
        p.xs = a.xs;
        p.ws = a.ws;
        p.xs_ld = p.ws_ld = (K + 127) / 128;
        p.ws_estride = a.ws_estride;
    }
    p.stages = std::min<int>(kGemmMaxStages, (kSmemMax - 1024 - gemm_smem_bytes<FP8, BN>(a.E)) / STAGE);
    p.m_tiles = (p.M + 128 * CG - 1) / (128 * CG);
    // The tensor core truncates as it adds, an error that grows with the length of the sum: fp32
    // results add up parts of 512 in rounded fp32 (K = 4096: 4.4e-6 off in the 2-norm without, 4.8e-7
    // with; operands of one sign 1.1e-5 and 7e-7), bf16 ones, whose rounding is up to 2^-8, parts of
    // 8192 (about 9e-6; of one sign 4e-5 too small). It also bounds what the epilogue waits for at a
    // time, whatever K or an expert's rows.
    p.part = p.out_fp32 ? 8 : 128;
    const size_t smem = (size_t)p.stages * STAGE + gemm_smem_bytes<FP8, BN>(a.E) + 1024;
    constexpr auto kern = [] {
        if constexpr (FP8) return gemm_fp8_kernel<CG, BN, STRIPS>;
        else return gemm_kernel<MODE, CG, BN, STRIPS>;
    }();
    cudaError_t e = ensure_max_smem<kern>((int)smem);
    if (e != cudaSuccess) return set_cuda_error(e, "grouped product shared memory");
    const int64_t groups = std::max<int64_t>(1, std::min<int64_t>(tiles * p.m_tiles, gemm_ctas(BN) * nsm / CG));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups * CG));
    cfg.blockDim = dim3(gemm_threads(FP8, BN));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    count_launch();
    e = cudaLaunchKernelEx(&cfg, kern, am, bm, bbig, p);
    return e == cudaSuccess ? MOE_OK : set_cuda_error(e, "grouped product launch");
}

// Rounds over the SMs that tiles of BN rows take. The row ranges are on the device, so the tiles are
// estimated: half a tile per expert more than its rows fill, and one at least.
static double gemm_rounds(const GemmArgs &a, int M, int nsm, int CG, int BN) {
    const double e = std::max(1, std::min(a.E, a.n_rows));
    const double tiles = e * std::max(1.0, a.n_rows / (e * BN) + 0.5);
    return tiles * ((M + 128 * CG - 1) / (128 * CG)) / (gemm_ctas(BN) * nsm / CG);
}
// Their time where a whole round takes `round`: the mean of 10% fewer and 15% more tiles' rounds.
static double gemm_time(double rounds, double round) {
    return 0.5 * (std::ceil(0.9 * rounds) + std::ceil(1.15 * rounds)) * round;
}

// Up to 8 rounds of pairs, the tile that needs the least time in whole rounds. A round's time, in that
// of pairs, was measured at K = 2048 (tiles of 32, 64, 128 rows and pairs: 10.3, 11, 12 and 15 us;
// fp8 11.2, 7.5, 11.6 and 14; with one CTA an SM at most, fp8 tiles of 32 are the quickest of all).
// Against a choice by the mean of an expert's rows alone (up to 24, 48 or more): 9% less on average over
// 693 sizes, 2% above the best tile of each; 8 experts of 64 rows, K = 2048, N = 512: 18.0 -> 13.5 us;
// N = 2048: 18.7 -> 16.7; 40 experts of 32 rows, N = 512: 24.5 -> 17.7.
// Beyond, reading the weights bounds the products of few rows, and a tile should hold an expert's
// rows so that they are read once: tiles of 32 or 64 rows where experts have up to 24 or 48 (fp8: 80)
// on average (128 experts, N = K = 2048, 64 rows: 208 us with tiles of 64, 194 with pairs; fp8 140 and 144).
// Weight gradients, whose tiles are known, take whole rounds too; a round of 64 and of 128 columns takes
// 0.52 and 0.55 of a round of pairs where its time goes with what it stores, 0.7 and 0.8 where it goes with
// the sums (512 rows an expert and more): 11% less time than with pairs alone over 198 sizes (32-bit
// results, K = N = 512: 8 experts of 16 rows 9.1 -> 5.6 us, of 1000 rows 19.3 -> 15.5).
// More than kGemmStrip tiles of 256 m's (M > 4096): in strips (8192^3: 715 against 775 us; with
// fewer, where they would only change the order within an expert, the kernels without the
// divisions are 1 to 2% faster).
template <int MODE, int BN>
static moe_status gemm_pick(const GemmArgs &a, int nsm, cudaStream_t st) {
    const int M = MODE == kGemmWgrad || MODE == kGemmDgrad ? a.K : a.N;
    if constexpr (MODE != kGemmWgrad) {
        constexpr bool FP8 = MODE == kGemmFp8;
        const double pairs = gemm_time(gemm_rounds(a, M, nsm, 2, BN), 1.0);
        int bn = a.n_rows <= 24 * (int64_t)a.E ? 32 : a.n_rows <= (FP8 ? 80 : 48) * (int64_t)a.E ? 64 : BN;
        if (pairs <= 8) {
            const double rounds = gemm_rounds(a, M, nsm, 1, 32);
            const double t32 = FP8 && rounds <= 0.5 ? 0.58 : gemm_time(rounds, FP8 ? 0.85 : 0.69);
            const double t64 = gemm_time(gemm_rounds(a, M, nsm, 1, 64), FP8 ? 0.6 : 0.75);
            const double t128 = gemm_time(gemm_rounds(a, M, nsm, 1, 128), 0.85);
            const double least = std::min(std::min(t32, t64), std::min(t128, pairs));
            bn = least == t32 ? 32 : least == t64 ? 64 : least == t128 ? 128 : BN;
        }
        if (bn == 32) return gemm_launch<MODE, 1, 32>(a, nsm, st);
        if (bn == 64) return gemm_launch<MODE, 1, 64>(a, nsm, st);
        if (bn == 128) return gemm_launch<MODE, 1, 128>(a, nsm, st);
    } else {
        auto rounds = [&](int CG, int bn) {
            return std::ceil((double)a.E * ((a.N + bn - 1) / bn) * ((a.K + 128 * CG - 1) / (128 * CG)) / (nsm / CG));
        };
        const bool few = a.n_rows <= 512 * (int64_t)a.E;
        const double pairs = rounds(2, BN), t64 = rounds(1, 64) * (few ? 0.52 : 0.7), t128 = rounds(1, 128) * (few ? 0.55 : 0.8);
        if (pairs <= 8 && t64 <= std::min(t128, pairs)) return gemm_launch<MODE, 1, 64>(a, nsm, st);
        if (pairs <= 8 && t128 <= pairs) return gemm_launch<MODE, 1, 128>(a, nsm, st);
    }
    if (M > kGemmStrip * 256) return gemm_launch<MODE, 2, BN, true>(a, nsm, st);
    return gemm_launch<MODE, 2, BN>(a, nsm, st);
}

moe_status launch_grouped_gemm(const GemmArgs &a, int nsm, cudaStream_t st) {
    switch (a.op) {
        case kGemmOpForward: return gemm_pick<kGemmFwd, 256>(a, nsm, st);
        case kGemmOpDgrad: return gemm_pick<kGemmDgrad, 256>(a, nsm, st);
        case kGemmOpWgrad: return gemm_pick<kGemmWgrad, 256>(a, nsm, st);
        default: return gemm_pick<kGemmFp8, 192>(a, nsm, st);
    }
}

// ------------------------------------------------------------------ FP8 quantiser
// Bound by memory (3.03 bytes an element, 5.03 with SwiGLU) once the arithmetic per element is
// short: 16 elements a lane, so that a block's scale and addresses are worked out by 8 lanes
// and not by 16, maxima on pairs of bf16 and quotients by a reciprocal. Scales and codes are
// those of correctly rounded fp32 divisions of the values bit for bit; with SwiGLU the values
// themselves go through expf and an approximate division, a few units in the last place off
// (more for gates below -87, where exp(gate) is below fp32's normal numbers).

constexpr int kQuantAhead = 2;   // blocks of a lane group whose loads are under way at a time

// RN(v / s) from r = RN(1 / s): Markstein's method (IBM J. Res. Dev. 34, 1990), exact while
// nothing over- or underflows on the way. The remainder is taken with its sign turned, so that
// the quotient of -0 is -0: v - q s would be +0 there, and +0 + -0 is +0.
__device__ __forceinline__ float quotient(float v, float s, float r) {
    const float q = __fmul_rn(v, r);
    return __fmaf_rn(-__fmaf_rn(q, s, -v), r, q);
}

__device__ __forceinline__ uint32_t e4m3x4_code(float a, float b, float c, float d) {
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// v / (1 + exp(-v)), with exp(-|v|) <= 1 so that nothing overflows and the divisor is in [1, 2].
__device__ __forceinline__ float silu(float v) {
    const float e = expf(-fabsf(v));
    return __fdividef(v >= 0.0f ? v : v * e, 1.0f + e);
}

// Eight lanes have a block of 128, 16 elements each; the next block of a lane group is drow rows
// and dkb blocks further.
template <bool SWIGLU>
__global__ void __launch_bounds__(256) quantize_fp8_kernel(const __nv_bfloat16 *x, int64_t ldx, int rows, int K, int KB,
                                                           int drow, int dkb, uint8_t *codes, int64_t ldc, float *scale) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_release();
    const int l8 = threadIdx.x & 7;
    const int64_t first = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
    int64_t row = first / KB;
    int kb = (int)(first - row * KB);
    // a warp's lane groups leave the loop together (the shuffles name 32 lanes)
    while (__any_sync(0xffffffffu, row < rows)) {
        uint32_t a[kQuantAhead][8], b[SWIGLU ? kQuantAhead : 1][8];
        int64_t at[kQuantAhead];
        int c[kQuantAhead];
#pragma unroll
        for (int u = 0; u < kQuantAhead; ++u) {
            at[u] = row;
            c[u] = kb;
            const bool in = row < rows && kb * 128 + l8 * 16 < K;   // K is a multiple of 16
            const __nv_bfloat16 *src = x + row * ldx + kb * 128 + l8 * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 v = in ? __ldcs(reinterpret_cast<const uint4 *>(src) + h) : make_uint4(0u, 0u, 0u, 0u);
                a[u][4 * h] = v.x;
                a[u][4 * h + 1] = v.y;
                a[u][4 * h + 2] = v.z;
                a[u][4 * h + 3] = v.w;
                if (SWIGLU) {
                    const uint4 g = in ? __ldcs(reinterpret_cast<const uint4 *>(src + K) + h) : make_uint4(0u, 0u, 0u, 0u);
                    b[u][4 * h] = g.x;
                    b[u][4 * h + 1] = g.y;
                    b[u][4 * h + 2] = g.z;
                    b[u][4 * h + 3] = g.w;
                }
            }
            row += drow;
            kb += dkb;
            if (kb >= KB) {
                kb -= KB;
                ++row;
            }
        }
#pragma unroll
        for (int u = 0; u < kQuantAhead; ++u) {
            float v[16];
            uint32_t top = 0;   // bit patterns of |v| order like the values, infinities and NaN on top
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[2 * j] = __uint_as_float(a[u][j] << 16);
                v[2 * j + 1] = __uint_as_float(a[u][j] & 0xFFFF0000u);
                if (SWIGLU) {
                    const float up0 = __uint_as_float(b[u][j] << 16), up1 = __uint_as_float(b[u][j] & 0xFFFF0000u);
                    v[2 * j] = silu(v[2 * j]) * up0;
                    v[2 * j + 1] = silu(v[2 * j + 1]) * up1;
                    top = max(top, __float_as_uint(v[2 * j]) & 0x7FFFFFFFu);
                    top = max(top, __float_as_uint(v[2 * j + 1]) & 0x7FFFFFFFu);
                } else {
                    top = __vmaxu2(top, a[u][j] & 0x7FFF7FFFu);
                }
            }
            if (!SWIGLU) top = max(top & 0xFFFF0000u, top << 16);
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float amax = __uint_as_float(top);
            float s;
            // amax between 2^-90 and 2^100: neither a reciprocal nor a remainder leaves fp32's range
            if (amax > 0x1p-90f && amax < 0x1p100f) {
                s = quotient(amax, 448.0f, 1.0f / 448.0f);
                const float r = __frcp_rn(s);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = quotient(v[j], s, r);
            } else {
                // 0 from amax = 0, and with SwiGLU from an amax up to 224 * 2^-149: 1 then, for 0 / 0 is NaN
                s = __fdiv_rn(amax, 448.0f);
                if (s == 0.0f) s = 1.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __fdiv_rn(v[j], s);
            }
            if (at[u] < rows) {
                const int c0 = c[u] * 128 + l8 * 16;
                if (c0 < K)
                    *reinterpret_cast<uint4 *>(codes + at[u] * ldc + c0) =
                        make_uint4(e4m3x4_code(v[0], v[1], v[2], v[3]), e4m3x4_code(v[4], v[5], v[6], v[7]),
                                   e4m3x4_code(v[8], v[9], v[10], v[11]), e4m3x4_code(v[12], v[13], v[14], v[15]));
                if (l8 == 0) scale[at[u] * KB + c[u]] = s;
            }
        }
    }
}

moe_status launch_quantize_fp8(const void *x, int64_t ldx, int rows, int K, int swiglu, void *codes, int64_t ldc,
                               float *scale, int nsm, cudaStream_t st) {
    const int KB = (K + 127) / 128;
    const int64_t blocks = ((int64_t)rows * KB + 31) / 32;
    const int grid = (int)std::min<int64_t>(blocks, (int64_t)nsm * 4);
    const int drow = grid * 32 / KB, dkb = grid * 32 % KB;
    const __nv_bfloat16 *xb = reinterpret_cast<const __nv_bfloat16 *>(x);
    uint8_t *cb = reinterpret_cast<uint8_t *>(codes);
    cudaError_t e = launch_pdl(swiglu ? quantize_fp8_kernel<true> : quantize_fp8_kernel<false>, dim3(grid), dim3(256), 0,
                               st, xb, ldx, rows, K, KB, drow, dkb, cb, ldc, scale);
    return e == cudaSuccess ? MOE_OK : set_cuda_error(e, "fp8 quantiser launch");
}

}  // namespace moe
