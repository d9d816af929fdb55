// mxfp4_linear2.cuh -- the grouped linear's product on pairs of SMs (included
// by mxfp4_moe.cu after mxfp4_linear.cuh, whose arithmetic, epilogue and
// conventions it shares).
//
// A cluster of two CTAs multiplies 256 features by 256 tokens with one
// tcgen05.mma.cta_group::2: CTA r holds the features' half r (A), the tokens'
// half r (B), and the accumulator of its 128 features by all 256 tokens. Per
// stage a CTA loads 128 + 128 operand rows for 128 x 256 products, where the
// single-SM kernel loads 256 + 128 rows for 256 x 128, and an MMA of 256
// columns reads its A operand once for twice the columns.
//
// Roles per CTA: warp 0 loads its operand rows, its features' scale atoms and
// all 256 tokens' scales, everything by TMA that completes on CTA 0's stage
// barrier; warp 1 of CTA 0 issues the scale copies and MMAs of both CTAs, and its
// commits arrive on both CTAs' barriers; the other 16 warps are the epilogue,
// four per 64 tokens. For the tokens' scales to be TMA's, scale_tiles_kernel
// first copies them into atoms that start with each tile's first token (a
// group's rows start anywhere in an atom): 2 / k of the operands' bytes.
// Gathering them per stage instead, and relaying CTA 1's barrier to CTA 0 (a
// release at cluster scope takes half a microsecond, as long as a stage), took
// 506 us where this takes 391 (32768 x 4096 x 7168, E2M1, 32 experts; single-SM
// kernel 486). Waits are bounded as in the single-SM kernel; the CTAs meet at a
// cluster barrier before either leaves.

namespace mxfp4 {

constexpr int L2_NT = 256;      // tokens per tile
constexpr int L2_THREADS = 64 + 32 * 16;

template <int FMT>
struct __align__(1024) Ln2Smem {
    static constexpr int ATOMS = LnFmt<FMT>::ATOMS;
    static constexpr int S = 6;
    static constexpr int MAX_GROUPS = 1024;        // whose plan fits beside the stages
    static constexpr uint32_t SF_COL0 = L2_NT;     // after the accumulator
    static_assert(SF_COL0 + S * 12 * ATOMS <= LN_TMEM_COLS, "tensor memory columns");
    uint8_t w[S][128 * LN_ROW_BYTES];
    uint8_t x[S][128 * LN_ROW_BYTES];
    uint8_t sfw[S][512 * ATOMS];
    uint8_t sfx[S][ATOMS][2][512];                 // per 128 K: tokens 0-127, 128-255
    unsigned long long full[S], empty[S], acc_full, acc_empty, done;
    uint32_t tmem_base;
    int err;
};

struct Ln2Maps {
    CUtensorMap x, w;        // operand rows, 128 x 128 byte boxes
    CUtensorMap sfx, sfw;    // scale atoms of 128 words: per tile and 128 K two of the tokens; the weights' as they lie
};

// One stage's part of a tensor into this CTA, completing on CTA 0's barrier (the
// address of this CTA's with the pair's bit clear).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar & 0xFEFFFFFFu)
        : "memory");
}

// The tokens' scales by tiles: ws[unit][K column][half][atom word]; words of
// tokens behind the tile's last are whatever follows (their products are not
// stored). A CTA takes a tile and SC_COLS columns: it reads the three atoms a
// column's 256 rows can touch in whole 16-byte pieces, holds them in row order
// in shared memory, and writes the tile's two atoms; word by word in global
// memory the copy took 19 us where this takes 13 (65536 rows of 7168).
constexpr int SC_COLS = 16;

__global__ void __launch_bounds__(L2_NT) scale_tiles_kernel(const LnArgs a, uint32_t* ws)
{
    extern __shared__ __align__(16) int32_t sc_dyn[];
    __shared__ uint32_t s_word[SC_COLS][3 * 128];
    int32_t* s_tpre = sc_dyn;
    int32_t* s_rst = s_tpre + a.num_groups + 1;
    let_dependents_start();
    const int64_t units = ln_plan<L2_NT>(a, s_tpre, s_rst);
    const int64_t nblk = a.k / 32, ncb = (nblk + 3) >> 2, row_atoms = (a.m + 127) >> 7;
    const int tid = threadIdx.x;
    const int64_t c0 = (int64_t)blockIdx.y * SC_COLS;
    const int cols = (int)min((int64_t)SC_COLS, ncb - c0);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const LnTile tl = ln_tile<L2_NT>(a, s_tpre, s_rst, u, 1);
        const int64_t i0 = tl.row0 >> 7;
        const int o = (int)(tl.row0 & 127);
        for (int i = tid; i < cols * 96; i += L2_NT) {
            const int c = i / 96, l = i % 32, at = (i / 32) % 3;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (i0 + at < row_atoms)
                v = *reinterpret_cast<const uint4*>(a.sfx + ((i0 + at) * ncb + c0 + c) * 512 + 16 * l);
            uint32_t* w = s_word[c] + 128 * at + l;  // entry (row l + 32 q, K block word) is word q of piece l
            w[0] = v.x;
            w[32] = v.y;
            w[64] = v.z;
            w[96] = v.w;
        }
        __syncthreads();
        const int r = (tid & 128) + 32 * (tid & 3) + ((tid & 127) >> 2);
        for (int c = 0; c < cols; ++c)
            ws[(u * ncb + c0 + c) * 256 + tid] = s_word[c][o + r];
        __syncthreads();
    }
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on the barrier at the same offset in CTA 0 of the cluster.
__device__ __forceinline__ void arrive_leader(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// ln_wait for a barrier that the other CTA arrives on.
__device__ __forceinline__ bool ln_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint64_t t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_cluster(bar, parity))
                return true;
        const uint64_t now = global_ns();
        if (t0 == 0)
            t0 = now;
        else if (now - t0 > SG_WAIT_NS)
            return false;
    }
}

// Arrive on this barrier's offset in both CTAs once the MMAs issued so far have completed.
__device__ __forceinline__ void commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

template <int FMT>
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa_tmem,
                                         uint32_t sfb_tmem, uint32_t acc)
{
    if constexpr (FMT == MXFP4_ELEM_E2M1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sfa_tmem), "r"(sfb_tmem)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sfa_tmem), "r"(sfb_tmem)
            : "memory");
}

__device__ __forceinline__ void cp_scales_pair(uint32_t col, uint32_t lo)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(col), "l"(ln_desc(lo, LN_SCALE_HI)) : "memory");
}

// One stage, straight-line (ln_stage): scale atoms of both CTAs, then up to four MMAs.
template <int FMT>
__device__ __forceinline__ void ln2_stage(uint32_t d_tmem, uint32_t sf_col, uint32_t wlo, uint32_t xlo, uint32_t sfw, uint32_t sfx,
                                          int na, int nk, bool accumulate)
{
    using F = LnFmt<FMT>;
    constexpr int ATOMS = F::ATOMS;
#pragma unroll
    for (int i = 0; i < ATOMS; ++i) {
        if (i > 0 && i >= na)
            break;
        cp_scales_pair(sf_col + 4u * i, sfw + 32u * i);
        cp_scales_pair(sf_col + 4u * (ATOMS + 2 * i), sfx + 64u * i);           // tokens 0-127
        cp_scales_pair(sf_col + 4u * (ATOMS + 2 * i + 1), sfx + 64u * i + 32u);  // tokens 128-255
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        if (kk > 0 && kk >= nk)
            break;
        constexpr int SB = F::MMA_K / 32;
        const uint32_t ai = (uint32_t)((kk * SB) >> 2), id = (uint32_t)((kk * SB) & 3);
        // M = 256 over the pair, N = 256
        const uint32_t idesc = (id << 4) | (F::AB_FMT << 7) | (F::AB_FMT << 10) | ((uint32_t)(L2_NT >> 3) << 17) | (1u << 23) |
                               ((256u >> 4) << 24) | (id << 29);
        mma_pair<FMT>(d_tmem, ln_desc(wlo + 2u * kk, LN_OPERAND_HI), ln_desc(xlo + 2u * kk, LN_OPERAND_HI), idesc, sf_col + 4u * ai,
                      sf_col + 4u * (ATOMS + 2 * ai), kk > 0 || accumulate ? 1u : 0u);
    }
}

template <int FMT, bool F32, bool RES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(L2_THREADS, 1)
    linear2_kernel(const __grid_constant__ Ln2Maps maps, const LnArgs a)
{
    using F = LnFmt<FMT>;
    using SM = Ln2Smem<FMT>;
    constexpr int S = SM::S, ATOMS = F::ATOMS;
    extern __shared__ __align__(1024) uint8_t ln_dyn[];
    uint8_t* base = ln_dyn + ((1024u - (smem_addr(ln_dyn) & 1023u)) & 1023u);
    SM& sm = *reinterpret_cast<SM*>(base);
    int32_t* s_tpre = reinterpret_cast<int32_t*>(base + sizeof(SM));
    int32_t* s_rst = s_tpre + a.num_groups + 1;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_rank();
    if (tid == 0) {
        sm.err = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);  // CTA 0: the transactions of both CTAs
            mbar_init(smem_addr(&sm.empty[s]), 1);
        }
        mbar_init(smem_addr(&sm.acc_full), 1);
        mbar_init(smem_addr(&sm.acc_empty), 32);        // CTA 0: the epilogue warps of both
        mbar_init(smem_addr(&sm.done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem_base)),
                     "r"(LN_TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        gm_fence_before();
    }
    const int64_t units = ln_plan<L2_NT>(a, s_tpre, s_rst);  // contains __syncthreads
    wait_for_prerequisite();                                 // scale_tiles_kernel
    cluster_sync();                                          // the barriers of both CTAs are ready
    gm_fence_after();
    const uint32_t tmem = sm.tmem_base;
    if (blockIdx.x == 0 && tid == 0 && a.status)
        *a.status = units >= 0 ? MXFP4_OK : MXFP4_EINVAL;

    const int n_ft = (int)((a.n + LN_FT - 1) / LN_FT);
    const int64_t tiles = units < 0 ? 0 : units * n_ft;
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int64_t nblk = a.k / 32, ncb = (nblk + 3) >> 2;
    const int nmma = (int)(a.k / F::MMA_K);
    const int nst = (int)((a.k + F::BK - 1) / F::BK);

    if (warp == 0) {
        // ---- producer (one lane)
        int s = 0;
        uint32_t ph = 0, issued = 0;
        for (int64_t t = first; t < tiles && !sm.err; t += step) {
            const LnTile tl = ln_tile<L2_NT>(a, s_tpre, s_rst, t, n_ft);
            const bool has = rank < tl.nh;  // this half has features, hence scales
            const int wrow = (int)((int64_t)tl.g * a.n + tl.f0) + 128 * rank;
            const int watom = (int)(tl.g * (a.sfw_group_bytes >> 9) + ((int64_t)(tl.f0 >> 7) + rank) * ncb);
            const int xatom = (int)(t / n_ft * ncb * 2);
            for (int ks = 0; ks < nst; ++ks) {
                if (!__all_sync(FULL, ln_wait_cluster(smem_addr(&sm.empty[s]), ph ^ 1u))) {
                    sm.err = 1;
                    break;
                }
                if (elect_one()) {
                    const uint32_t bar = smem_addr(&sm.full[s]);
                    // boxes count whole, whatever lies outside the tensors
                    if (rank == 0)
                        mbar_expect_tx(bar, 2 * (2 * 128 * LN_ROW_BYTES + 1024 * ATOMS) + tl.nh * 512 * ATOMS);
                    tma_load_pair(smem_addr(sm.w[s]), &maps.w, ks * LN_ROW_BYTES, wrow, bar);
                    tma_load_pair(smem_addr(sm.x[s]), &maps.x, ks * LN_ROW_BYTES, (int)tl.row0 + 128 * rank, bar);
                    if (has)
                        tma_load_pair(smem_addr(sm.sfw[s]), &maps.sfw, 0, watom + ks * ATOMS, bar);
                    tma_load_pair(smem_addr(sm.sfx[s]), &maps.sfx, 0, xatom + ks * 2 * ATOMS, bar);
                }
                __syncwarp();
                issued |= 1u << s;
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // every load of both CTAs lands before they leave (the cluster barrier
        // below holds CTA 1): the last load of stage i had the parity of its turn
        if (rank == 0)
            for (int i = 0; i < S; ++i)
                if (issued & (1u << i))
                    (void)ln_wait_cluster(smem_addr(&sm.full[i]), i < s ? ph : ph ^ 1u);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // ---- MMA issuer of the pair
            int s = 0;
            uint32_t ph = 0, aph = 0;
            for (int64_t t = first; t < tiles && !sm.err; t += step) {
                if (!__all_sync(FULL, ln_wait_cluster(smem_addr(&sm.acc_empty), aph ^ 1u))) {
                    sm.err = 1;
                    break;
                }
                aph ^= 1u;
                gm_fence_after();
                for (int ks = 0; ks < nst; ++ks) {
                    if (!__all_sync(FULL, ln_wait_cluster(smem_addr(&sm.full[s]), ph))) {
                        sm.err = 1;
                        break;
                    }
                    gm_fence_after();
                    if (elect_one()) {
                        ln2_stage<FMT>(tmem, tmem + SM::SF_COL0 + (uint32_t)(12 * ATOMS * s), ln_desc_lo(smem_addr(sm.w[s])),
                                       ln_desc_lo(smem_addr(sm.x[s])), ln_desc_lo(smem_addr(sm.sfw[s])), ln_desc_lo(smem_addr(sm.sfx[s])),
                                       (int)min((int64_t)ATOMS, ncb - (int64_t)ks * ATOMS), nmma - 4 * ks, ks > 0);
                        commit_pair(smem_addr(&sm.empty[s]));
                        if (ks + 1 == nst)
                            commit_pair(smem_addr(&sm.acc_full));
                    }
                    __syncwarp();
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // every MMA issued has completed before the tensor memory is freed
            if (elect_one())
                commit_pair(smem_addr(&sm.done));
            __syncwarp();
        }
        (void)ln_wait_cluster(smem_addr(&sm.done), 0);
        __syncwarp();
    } else {
        // ---- epilogue: tensor-memory lanes 32 (warp % 4) .. + 31, tokens c0 .. c0 + 63
        const int quad = warp & 3, c0 = ((warp - 2) >> 2) * 64;
        uint32_t aph = 0;
        for (int64_t t = first; t < tiles && !sm.err; t += step) {
            const LnTile tl = ln_tile<L2_NT>(a, s_tpre, s_rst, t, n_ft);
            const int f = tl.f0 + 128 * rank + 32 * quad + lane;
            const bool fok = f < a.n;
            const float bias = a.bias && fok ? a.bias[(int64_t)tl.g * a.n + f] : 0.0f;
            if (RES && nst <= LN_SHORT && rank < tl.nh)
                ln_prefetch<F32, 64>(a, tl.row0 + c0, tl.rows - c0, f);
            __syncwarp();
            if (!__all_sync(FULL, ln_wait_cluster(smem_addr(&sm.acc_full), aph))) {
                sm.err = 1;
                break;
            }
            aph ^= 1u;
            gm_fence_after();
            float v[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t u[32];
                __syncwarp();
                gm_ld32(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(c0 + 32 * c), u);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[c][i] = __uint_as_float(u[i]) + bias;
            }
            gm_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_leader(smem_addr(&sm.acc_empty));
            if (rank < tl.nh) {
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    const int rows = tl.rows - c0 - 32 * c;
                    if (rows <= 0)
                        break;
                    if (rows >= 32 && __all_sync(FULL, fok))
                        ln_epilogue32<F32, true, RES>(a, v[0], tl.row0 + c0 + 32 * c, rows, f, fok);
                    else
                        ln_epilogue32<F32, false, RES>(a, v[0], tl.row0 + c0 + 32 * c, rows, f, fok);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[0][i] = v[1][i];
                }
            }
        }
    }

    __syncthreads();
    if (tid == 0 && sm.err && a.status)
        *a.status = MXFP4_ECUDA;
    cluster_sync();  // neither CTA leaves while the other may arrive on its barriers or read its operands
    if (warp == 1) {
        gm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(LN_TMEM_COLS) : "memory");
    }
}

}  // namespace mxfp4
