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
#include "mx_codec.cuh"
#include <cstdlib>

namespace moe {

constexpr int kGemmFwd = 0, kGemmDgrad = 1, kGemmWgrad = 2, kGemmFp8 = 3;

// Warps 0-3: TMA, MMA, scales, tail rows; from 4 on the epilogue: 16 warps for tiles of 256
// columns (64 sums per thread; with 8 warps and 128 sums the fp8 kernel spilled), 8 for small.
__host__ __device__ constexpr int gemm_epi_warps(int BN) { return BN >= 256 ? 16 : 8; }
__host__ __device__ constexpr int gemm_threads(int BN) { return 128 + 32 * gemm_epi_warps(BN); }
constexpr int kGemmABytes = 128 * 128;     // one CTA's A tile of a stage: 128 m x 128 bytes
constexpr int kGemmBoxRows = 32;           // rows of B in a small TMA box (K-major B); a large one has 128
constexpr int kGemmMaxStages = 10;
constexpr int kGemmXsSlots = 8;            // ring of activation scales (fp8), one slot per K block

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
    const float *xs, *ws;     // fp8 scales: [n_rows][xs_ld], [E][M][ws_ld]
    int64_t xs_ld, ws_ld, ws_estride;
};

struct GemmSmem {
    uint64_t full[kGemmMaxStages];    // operands of a stage landed (and tail rows cleared)
    uint64_t empty[kGemmMaxStages];   // the stage's MMAs have read them
    uint64_t tail[kGemmMaxStages];    // wgrad: a stage with rows to clear landed in this CTA
    uint64_t tailpeer[kGemmMaxStages];   // and the pair's other CTA has cleared its own
    uint64_t accfull[2], accempty[2];
    uint64_t scfull[kGemmXsSlots], scempty[kGemmXsSlots];
    float xs[kGemmXsSlots][256];   // fp8: a K block's scales of the tile's rows and of this CTA's 128 weight rows
    float ws[kGemmXsSlots][128];
    uint32_t tmem_base;
    int abort_flag;
    int total_items;
    int tile_start[kMaxExperts + 1];
    int2 range[kMaxExperts];          // first row and rows of each expert
};

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

// An expert's n rows are cut into ceil(n / BN) tiles of nearly equal size, a multiple of the
// MMA's N step, so 260 rows cost two tiles of about 130, not one of 256 and one of 4.
template <int CG, int BN>
__device__ __forceinline__ int gemm_tile_rows(int n) {
    const int t = (n + BN - 1) / BN;
    const int r = (n + t - 1) / t;
    constexpr int G = 16 * CG;
    return (r + G - 1) / G * G;
}

template <int MODE, int CG, int BN>
__device__ __forceinline__ GemmItem gemm_item(const GemmSmem &sm, const GemmParams &p, int item) {
    constexpr int G = 16 * CG;
    GemmItem it;
    if (MODE == kGemmWgrad) {
        const int rt = item / p.m_tiles;
        it.m0 = (item - rt * p.m_tiles) * (128 * CG);
        it.e = rt / p.j_tiles;
        it.j0 = (rt - it.e * p.j_tiles) * BN;
        it.row0 = sm.range[it.e].x;
        it.valid = sm.range[it.e].y;
        it.nt = min(BN, (p.J - it.j0 + G - 1) / G * G);
        it.kblocks = (it.valid + 63) / 64;
        return it;
    }
    const int rt = item / p.m_tiles;
    it.m0 = (item - rt * p.m_tiles) * (128 * CG);
    int lo = 0, hi = p.E - 1;   // expert with tile_start[e] <= rt < tile_start[e+1]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sm.tile_start[mid] <= rt) lo = mid; else hi = mid - 1;
    }
    it.e = lo;
    const int beg = sm.range[lo].x, n = sm.range[lo].y;
    const int tr = gemm_tile_rows<CG, BN>(n), t = rt - sm.tile_start[lo];
    it.row0 = beg + t * tr;
    it.valid = min(tr, n - t * tr);
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
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) { return pack2u(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float half2of(uint64_t p, int hi) {
    uint32_t lo, up;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(up) : "l"(p));
    return __uint_as_float(hi ? up : lo);
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

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// tcgen05.wait::ld that the loaded registers pass through, so that no use of them can be
// scheduled before it.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
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

// ------------------------------------------------------------------ kernel

template <int MODE, int CG, int BN>
__global__ void __launch_bounds__(gemm_threads(BN), 1)
gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
            const __grid_constant__ CUtensorMap bmap128, GemmParams p) {
    constexpr bool FP8 = MODE == kGemmFp8;
    constexpr bool A_MN = MODE == kGemmDgrad || MODE == kGemmWgrad, B_MN = MODE == kGemmWgrad;
    constexpr int EPI = gemm_epi_warps(BN);
    constexpr int BROWS = BN / CG;                       // j's of B that this CTA holds
    constexpr int STAGE = kGemmABytes + BROWS * 128;
    constexpr int CB = FP8 ? 128 : 64;                   // c's per stage
    constexpr uint32_t TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int ns = p.stages;
    GemmSmem &sm = *reinterpret_cast<GemmSmem *>(ring + ns * STAGE);
    volatile int *abort_flag = &sm.abort_flag;
    const int warp = warp_id(), lane = lane_id();
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int first = CG == 2 ? blockIdx.x / 2 : blockIdx.x, step = CG == 2 ? gridDim.x / 2 : gridDim.x;

    pdl_wait();
    if (threadIdx.x == 0) {
        pdl_release();
        for (int s = 0; s < ns; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
            mbar_init(&sm.tail[s], 1);
            mbar_init(&sm.tailpeer[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.accfull[b], 1);
            mbar_init(&sm.accempty[b], CG * EPI);
        }
        for (int s = 0; s < kGemmXsSlots; ++s) {
            mbar_init(&sm.scfull[s], 64);
            mbar_init(&sm.scempty[s], EPI);
        }
        sm.abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&amap);
        tma_prefetch_desc(&bmap);
        if (MODE != kGemmWgrad && BROWS >= 128) tma_prefetch_desc(&bmap128);
    }
    if (warp == 2) gemm_tmem_alloc<CG>(&sm.tmem_base, TMEM_COLS);
    if (warp == 3) {
        int run = 0;
        if (lane == 0) sm.tile_start[0] = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int nt = 0;
            if (e < p.E) {
                int beg, n;
                gemm_range(p, e, beg, n);
                sm.range[e] = make_int2(beg, n);
                nt = (n + BN - 1) / BN;
            }
            int incl = nt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
            }
            if (e < p.E) sm.tile_start[e + 1] = run + incl;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) sm.total_items = MODE == kGemmWgrad ? p.E * p.j_tiles * p.m_tiles : run * p.m_tiles;
    }
    tc_fence_before();
    __syncthreads();
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
                const GemmItem it = gemm_item<MODE, CG, BN>(sm, p, item);
                const int bj0 = it.j0 + (int)rank * (it.nt / CG);          // this CTA's share of B
                // K-major B in boxes of 128 rows, a rest of up to 96 rows in boxes of 32: few boxes
                // when the tile is full (issuing 4 KB boxes only cost a quarter of the rate), no
                // more than 31 rows too many when it is not
                const int share = it.nt / CG;
                const int big = BROWS < 128 ? 0 : (share + 31) / 128;
                const int small = big * 128 >= share ? 0 : (share - big * 128 + kGemmBoxRows - 1) / kGemmBoxRows;
                const int chunks = (share + 63) / 64;
                const uint32_t bytes = kGemmABytes + (B_MN ? chunks * 8192 : big * 16384 + small * kGemmBoxRows * 128);
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
                        } else {
                            gemm_tma_3d<CG>(a, &amap, bar, c0, m0, it.e);
                        }
                        for (int i = 0; i < big; ++i) gemm_tma_2d<CG>(b + i * 16384, &bmap128, bar, c0, bj0 + i * 128);
                        for (int i = 0; i < small; ++i)
                            gemm_tma_2d<CG>(b + big * 16384 + i * kGemmBoxRows * 128, &bmap, bar, c0,
                                            bj0 + big * 128 + i * kGemmBoxRows);
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
        // =================================================== MMA issuer (one thread of the leader)
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc0 = (1u << 4) | (FP8 ? 0u : (1u << 7) | (1u << 10)) | (A_MN ? 1u << 15 : 0u) |
                                        (B_MN ? 1u << 16 : 0u) | ((uint32_t)(128 * CG >> 4) << 24);
            int s = 0, u = 0;   // u: accumulator uses so far
            const int part = FP8 ? 1 : p.part;
            uint32_t ph = 0;
            bool ok = true;
            const uint32_t ring0 = smem_u32(ring);
            for (int item = first; item < total && ok; item += step) {
                const GemmItem it = gemm_item<MODE, CG, BN>(sm, p, item);
                const uint32_t idesc = idesc0 | ((uint32_t)(it.nt >> 3) << 17);
                int left = 0;   // blocks that this accumulator still takes
                for (int kb = 0; kb < it.kblocks; ++kb) {
                    const bool fresh = left == 0;
                    if (fresh) {
                        left = min(part, it.kblocks - kb);
                        if (!gemm_wait(&sm.accempty[u & 1], ((u >> 1) & 1) ^ 1, abort_flag)) { ok = false; break; }
                    }
                    const uint32_t d = tmem + (u & 1) * BN;
                    if (!gemm_wait(&sm.full[s], ph, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sa = ring0 + s * STAGE, sb = sa + kGemmABytes;
                    const uint64_t ad = A_MN ? smem_desc_mn_sw128(sa) : smem_desc_sw128(sa);
                    const uint64_t bd = B_MN ? smem_desc_mn_sw128(sb) : smem_desc_sw128(sb);
                    int steps = 4;
                    if (MODE == kGemmWgrad) steps = min(4, (it.valid - kb * 64 + 15) / 16);
                    for (int i = 0; i < steps; ++i)   // 16 (fp8: 32) c's each
                        gemm_mma<CG, FP8>(d, ad + (A_MN ? 128 : 2) * i, bd + (B_MN ? 128 : 2) * i, idesc,
                                          !(fresh && i == 0));
                    gemm_commit<CG>(&sm.empty[s]);
                    if (--left == 0) {
                        gemm_commit<CG>(&sm.accfull[u & 1]);
                        ++u;
                    }
                    if (++s == ns) { s = 0; ph ^= 1; }
                }
            }
        }
    } else if (FP8 && (warp == 2 || warp == 3)) {
        // =================================================== scales (fp8)
        // A K block's scales of the tile's rows and of the CTA's 128 weight rows, copied
        // asynchronously so that the whole ring of slots is in flight.
        constexpr int R = (BN + 128 + 63) / 64;   // per lane of the two warps, counting rows of x, then of w
        int x = 0;   // K blocks so far
        bool ok = true;
        for (int item = first; item < total && ok; item += step) {
            const GemmItem it = gemm_item<MODE, CG, BN>(sm, p, item);
            const int mbase = it.m0 + (int)rank * 128;
            for (int kb = 0; kb < it.kblocks; ++kb, ++x) {
                const int slot = x % kGemmXsSlots;
                if (!gemm_wait(&sm.scempty[slot], ((x / kGemmXsSlots) & 1) ^ 1, abort_flag)) { ok = false; break; }
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int r = (warp - 2) * 32 + lane + 64 * i, w = r - BN;
                    if (w >= 128) continue;
                    const bool on = w < 0 ? r < it.valid : mbase + w < p.M;
                    const float *src = w < 0 ? p.xs + (int64_t)(it.row0 + r) * p.xs_ld + kb
                                             : p.ws + (int64_t)it.e * p.ws_estride + (int64_t)(mbase + w) * p.ws_ld + kb;
                    const uint32_t dst = smem_u32(w < 0 ? &sm.xs[slot][r] : &sm.ws[slot][w]);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(on ? src : p.xs), "r"(on ? 4 : 0)
                                 : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sm.scfull[slot])) : "memory");
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < 4) {
        // =================================================== wgrad (warp 3): rows behind the expert's last
        // The last block of an expert holds rows of the next one; the up to 15 of them that
        // the last MMA step would read are cleared in both operands (0 * inf is not 0).
        if (MODE == kGemmWgrad && warp == 3) {
            int s = 0;
            uint32_t tph = 0;   // bit s: parity of tail[s]
            bool ok = true;
            for (int item = first; item < total && ok; item += step) {
                const GemmItem it = gemm_item<MODE, CG, BN>(sm, p, item);
                if (!it.kblocks) continue;
                s = (s + it.kblocks - 1) % ns;   // the stage of the last block
                if (it.valid & 15) {
                    if (!gemm_wait(&sm.tail[s], (tph >> s) & 1, abort_flag)) { ok = false; break; }
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
                        if (CG == 2 && !gemm_wait<true>(&sm.tailpeer[s], ((tph >> s) & 1) ^ 1, abort_flag)) { ok = false; break; }
                        if (lane == 0) mbar_arrive(&sm.full[s]);
                    }
                }
                s = s + 1 == ns ? 0 : s + 1;
            }
        }
    } else {
        // =================================================== epilogue
        // Warp quarter q owns TMEM lanes 32q..32q+31; the quarter's G warps take turns on units
        // of 16 columns.
        constexpr int G = EPI / 4;
        const int q = warp & 3, g = (warp - 4) >> 2;
        const uint32_t lead_empty0 = CG == 2 ? mapa_u32(smem_u32(&sm.accempty[0]), 0) : smem_u32(&sm.accempty[0]);
        constexpr int NU = BN / (16 * G);   // units per warp
        const int part = FP8 ? 1 : p.part;
        int u = 0;
        bool ok = true;
        for (int item = first; item < total && ok; item += step) {
            const GemmItem it = gemm_item<MODE, CG, BN>(sm, p, item);
            const int m = it.m0 + (int)rank * 128 + q * 32 + lane;
            const bool mok = m < p.M;
            const int jn = MODE == kGemmWgrad ? min(it.nt, p.J - it.j0) : it.valid;   // columns to store
            const int units = (it.nt / 16 + G - 1 - g) / G;
            uint64_t acc[NU][8];   // pairs of fp32
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i][j] = 0;
            for (int kb = 0; kb < it.kblocks; kb += part, ++u) {
                const int slot = u % kGemmXsSlots;   // fp8: uses and K blocks are the same
                uint64_t ws2 = 0;
                if (FP8) {
                    if (!gemm_wait(&sm.scfull[slot], (u / kGemmXsSlots) & 1, abort_flag)) { ok = false; break; }
                    const float w = sm.ws[slot][q * 32 + lane];
                    ws2 = pack2(w, w);
                }
                if (!gemm_wait(&sm.accfull[u & 1], (u >> 1) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + (u & 1) * BN + g * 16;
#pragma unroll
                for (int i = 0; i < NU; ++i) {
                    if (i < units) {
                        uint32_t c[16];
                        tmem_ld16(t + i * (16 * G), c);
                        tmem_wait_ld16(c);
                        if (FP8) {
                            const uint32_t xs4 = smem_u32(&sm.xs[slot][(i * G + g) * 16]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint64_t f0, f1;   // volatile: four scales at a time, not all sixteen, in registers
                                asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(f0), "=l"(f1) : "r"(xs4 + 16 * j));
                                acc[i][2 * j] = fma2(mul2(pack2u(c[4 * j], c[4 * j + 1]), f0), ws2, acc[i][2 * j]);
                                acc[i][2 * j + 1] = fma2(mul2(pack2u(c[4 * j + 2], c[4 * j + 3]), f1), ws2, acc[i][2 * j + 1]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) acc[i][j] = add2(acc[i][j], pack2u(c[2 * j], c[2 * j + 1]));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) mbar_arrive_remote(lead_empty0 + 8 * (u & 1));
                    else mbar_arrive(&sm.accempty[u & 1]);
                    if (FP8) mbar_arrive(&sm.scempty[slot]);
                }
            }
            if (!ok) break;
            int64_t o = (int64_t)it.j0 * p.ldo + m;
            if (MODE == kGemmWgrad) o += (int64_t)it.e * p.out_estride;
            // stores in program order (volatile), so that the compiler does not hold many of their
            // addresses and converted values at once and spill
            const int lim = mok ? jn : 0;
            if (p.out_fp32) {
                float *d = reinterpret_cast<float *>(p.out) + o + (int64_t)(g * 16) * p.ldo;
#pragma unroll
                for (int i = 0; i < NU; ++i, d += 16 * (G - 1) * p.ldo) {
#pragma unroll
                    for (int j = 0; j < 16; ++j, d += p.ldo) {
                        float v = half2of(acc[i][j >> 1], j & 1);
                        const bool on = (i * G + g) * 16 + j < lim;
                        if (MODE == kGemmWgrad) {   // read by a later kernel at most: first to leave L2
                            if (p.accumulate && on) v += *d;
                            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.cs.f32 [%0], %1;\n\t}" ::"l"(d),
                                         "f"(v), "r"((uint32_t)on)
                                         : "memory");
                        } else {
                            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.f32 [%0], %1;\n\t}" ::"l"(d),
                                         "f"(v), "r"((uint32_t)on)
                                         : "memory");
                        }
                    }
                }
            } else {
                __nv_bfloat16 *d = reinterpret_cast<__nv_bfloat16 *>(p.out) + o + (int64_t)(g * 16) * p.ldo;
#pragma unroll
                for (int i = 0; i < NU; ++i, d += 16 * (G - 1) * p.ldo) {
#pragma unroll
                    for (int j = 0; j < 16; ++j, d += p.ldo) {
                        const bool on = (i * G + g) * 16 + j < lim;
                        asm volatile(
                            "{\n\t.reg .pred p;\n\t.reg .b16 h;\n\tsetp.ne.u32 p, %2, 0;\n\tcvt.rn.bf16.f32 h, %1;\n\t"
                            "@p st.global.b16 [%0], h;\n\t}" ::"l"(d),
                            "f"(half2of(acc[i][j >> 1], j & 1)), "r"((uint32_t)on)
                            : "memory");
                    }
                }
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

// ------------------------------------------------------------------ launch

template <int MODE, int CG, int BN>
static moe_status gemm_launch(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &b128, GemmParams p, int64_t items, int nsm,
                              cudaStream_t st) {
    constexpr int STAGE = kGemmABytes + BN / CG * 128;
    constexpr int kSmemMax = 227 * 1024;
    p.stages = std::min<int>(kGemmMaxStages, (kSmemMax - 1024 - (int)sizeof(GemmSmem)) / STAGE);
    p.m_tiles = (p.M + 128 * CG - 1) / (128 * CG);
    // The tensor core truncates as it adds, an error that grows with the length of the sum: fp32
    // results add up parts of 512 in rounded fp32 (K = 4096: 4.4e-6 off in the 2-norm without).
    p.part = p.out_fp32 ? 8 : 1 << 30;
    const size_t smem = (size_t)p.stages * STAGE + sizeof(GemmSmem) + 1024;
    constexpr auto kern = gemm_kernel<MODE, CG, BN>;
    cudaError_t e = ensure_max_smem<kern>((int)smem);
    if (e != cudaSuccess) return set_cuda_error(e, "grouped product shared memory");
    const int64_t groups = std::max<int64_t>(1, std::min<int64_t>(items * p.m_tiles, nsm / CG));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups * CG));
    cfg.blockDim = dim3(gemm_threads(BN));
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
    e = cudaLaunchKernelEx(&cfg, kern, a, b, b128, p);
    return e == cudaSuccess ? MOE_OK : set_cuda_error(e, "grouped product launch");
}

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

// Most row tiles that n_rows rows of E experts can make.
static int64_t gemm_row_tiles(int n_rows, int E, int BN) {
    return (int64_t)n_rows / BN + std::min(n_rows, E);
}

template <int MODE>
static moe_status gemm_pick(const CUtensorMap &am, const CUtensorMap &bm, const CUtensorMap &bm2, const GemmParams &p, int n, int E, int nsm, cudaStream_t st) {
    const char *v = getenv("GCFG");
    const int c = v ? atoi(v) : 2;
    const bool wg = MODE == kGemmWgrad;
    if constexpr (MODE != kGemmWgrad) { if (c == 0) return gemm_launch<MODE, 1, 32>(am, bm, bm2, p, gemm_row_tiles(n, E, 32), nsm, st); }
    const int64_t it = wg ? (int64_t)E * p.j_tiles : gemm_row_tiles(n, E, 256);
    if (c == 1) return gemm_launch<MODE, 1, 256>(am, bm, bm2, p, it, nsm, st);
    return gemm_launch<MODE, 2, 256>(am, bm, bm2, p, it, nsm, st);
}

moe_status launch_grouped_gemm(const GemmArgs &a, int nsm, cudaStream_t st) {
    CUtensorMap am, bm, bm2;
    GemmParams p;
    memset(&p, 0, sizeof(p));
    p.offsets = a.offsets;
    p.E = a.E;
    p.n_rows = a.n_rows;
    p.out = a.out;
    p.ldo = a.ldo;
    p.out_fp32 = a.out_fp32;
    moe_status r;
    const int N = a.N, K = a.K;
    if (a.op == kGemmOpForward || a.op == kGemmOpFp8) {
        const int esz = a.op == kGemmOpFp8 ? 1 : 2, cb = 128 / esz;
        if ((r = gemm_map3(&am, esz, a.w, a.E, N, K, a.ldw, a.w_estride, cb, 128)) != MOE_OK) return r;
        if ((r = gemm_map2(&bm, esz, a.x, a.n_rows, K, a.ldx, cb, kGemmBoxRows)) != MOE_OK) return r;
        if ((r = gemm_map2(&bm2, esz, a.x, a.n_rows, K, a.ldx, cb, 128)) != MOE_OK) return r;
        p.M = N;
        p.C = K;
        p.xs = a.xs;
        p.ws = a.ws;
        p.xs_ld = p.ws_ld = (K + 127) / 128;
        p.ws_estride = a.ws_estride;
        if (a.op == kGemmOpFp8) return gemm_pick<kGemmFp8>(am, bm, bm2, p, a.n_rows, a.E, nsm, st);
        return gemm_pick<kGemmFwd>(am, bm, bm2, p, a.n_rows, a.E, nsm, st);
    }
    if (a.op == kGemmOpDgrad) {
        if ((r = gemm_map3(&am, 2, a.w, a.E, N, K, a.ldw, a.w_estride, 64, 64)) != MOE_OK) return r;
        if ((r = gemm_map2(&bm, 2, a.x, a.n_rows, N, a.ldx, 64, kGemmBoxRows)) != MOE_OK) return r;
        if ((r = gemm_map2(&bm2, 2, a.x, a.n_rows, N, a.ldx, 64, 128)) != MOE_OK) return r;
        p.M = K;
        p.C = N;
        return gemm_pick<kGemmDgrad>(am, bm, bm2, p, a.n_rows, a.E, nsm, st);
    }
    if ((r = gemm_map2(&am, 2, a.w, a.n_rows, K, a.ldw, 64, 64)) != MOE_OK) return r;
    if ((r = gemm_map2(&bm, 2, a.x, a.n_rows, N, a.ldx, 64, 64)) != MOE_OK) return r;
    bm2 = bm;   // not used
    p.M = K;
    p.J = N;
    p.j_tiles = (N + 255) / 256;
    p.out_estride = a.out_estride;
    p.accumulate = a.accumulate;
    return gemm_pick<kGemmWgrad>(am, bm, bm2, p, a.n_rows, a.E, nsm, st);
}

// ------------------------------------------------------------------ FP8 quantiser

// One half-warp per block of 128: 8 elements per lane. Each step is one correctly rounded
// fp32 operation, so the codes and scales are the formula's bit for bit.
template <bool SWIGLU>
__global__ void __launch_bounds__(256) quantize_fp8_kernel(const __nv_bfloat16 *x, int64_t ldx, int rows, int K,
                                                           uint8_t *codes, int64_t ldc, float *scale) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_release();
    const int KB = (K + 127) / 128;
    const int64_t total = (int64_t)rows * KB;
    const int l16 = threadIdx.x & 15;
    const int64_t stride = (int64_t)gridDim.x * 16;
    // whole half-warps leave the loop together with their partner (the shuffles name 32 lanes)
    const int64_t rounds = (total + stride - 1) / stride;
    for (int64_t i = 0; i < rounds; ++i) {
        const int64_t blk = i * stride + (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
        const bool on = blk < total;
        const int64_t row = on ? blk / KB : 0;
        const int kb = on ? (int)(blk - row * KB) : 0, c0 = kb * 128 + l16 * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        const bool in = on && c0 < K;   // K is a multiple of 16
        if (in) {
            const uint4 a = *reinterpret_cast<const uint4 *>(x + row * ldx + c0);
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(aw[j] << 16);
                v[2 * j + 1] = __uint_as_float(aw[j] & 0xFFFF0000u);
            }
            if (SWIGLU) {
                const uint4 b = *reinterpret_cast<const uint4 *>(x + row * ldx + K + c0);
                const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = __uint_as_float(j & 1 ? bw[j >> 1] & 0xFFFF0000u : bw[j >> 1] << 16);
                    v[j] = v[j] / (1.0f + expf(-v[j])) * u;
                }
            }
        }
        // bit patterns of |v| order like the values, with infinities and NaN on top
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float s = top == 0 ? 1.0f : __fdiv_rn(__uint_as_float(top), 448.0f);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j >> 2] |= e4m3_code(__fdiv_rn(v[j], s)) << (8 * (j & 3));
        if (in) *reinterpret_cast<uint2 *>(codes + row * ldc + c0) = make_uint2(w[0], w[1]);
        if (on && l16 == 0) scale[blk] = s;
    }
}

moe_status launch_quantize_fp8(const void *x, int64_t ldx, int rows, int K, int swiglu, void *codes, int64_t ldc,
                               float *scale, int nsm, cudaStream_t st) {
    const int64_t blocks = ((int64_t)rows * ((K + 127) / 128) + 15) / 16;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)nsm * 8));
    const __nv_bfloat16 *xb = reinterpret_cast<const __nv_bfloat16 *>(x);
    uint8_t *cb = reinterpret_cast<uint8_t *>(codes);
    cudaError_t e = swiglu ? launch_pdl(quantize_fp8_kernel<true>, grid, dim3(256), 0, st, xb, ldx, rows, K, cb, ldc, scale)
                           : launch_pdl(quantize_fp8_kernel<false>, grid, dim3(256), 0, st, xb, ldx, rows, K, cb, ldc, scale);
    return e == cudaSuccess ? MOE_OK : set_cuda_error(e, "fp8 quantiser launch");
}

}  // namespace moe
