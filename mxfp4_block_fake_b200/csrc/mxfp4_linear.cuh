// mxfp4_linear.cuh -- the grouped block-scaled product with bias, activation
// and residual in its epilogue, on the fifth-generation tensor cores, and the
// epilogue's gradients (included by mxfp4_moe.cu; the definition is in
// include/mxfp4.h, mxfp4_grouped_linear).
//
//   z[t][f] = sum_k decode(A[t][k]) 2^(sA-127) decode(B_g[f][k]) 2^(sB-127) + bias_g[f]
//   y       = act(z) + residual
//
// Layout of the product: the features (rows of B_g, the expert's weight) are
// the MMA's M side and the tokens its N side, so that a tile of few tokens
// (decoding) costs few tensor-core columns instead of a padded 128-row tile,
// the weight's scale atoms are copied as they lie in memory, the bias is one
// value per thread of the epilogue, and a warp's store writes 32 consecutive
// features of one token.
//
// One CTA per SM, persistent over tiles of 256 features (two M = 128 halves
// that share the tokens' operand) x NT tokens:
//   warp 0: producer. Per stage of 128-byte rows (256 E2M1 or 128 E4M3 K
//     elements) the TMA loads of both halves and the tokens (128-byte
//     swizzle), bulk copies of the weight's scale atoms, and asynchronous
//     4-byte copies of the tokens' scales (a group's rows start anywhere in
//     an atom).
//   warp 1: copies the scale atoms into tensor memory (tcgen05.cp) and issues
//     the block-scaled MMAs.
//   the other warps: epilogue, four per half and 64 tokens. A warp reads its 32
//     features of its tokens from tensor memory into registers, hands the
//     accumulator back, and then does its arithmetic and stores while the next
//     tile is multiplied. (With 128 tokens per warp the values no longer fit
//     the registers beside the arithmetic: 347 against 172 us on 32768 x 4096 x
//     1024, swiglu.)
// Every wait on an mbarrier is bounded (SG_WAIT_NS); on expiry the CTA records
// MXFP4_ECUDA, waits (bounded) for its loads and MMAs in flight, frees the
// tensor memory and exits.

namespace mxfp4 {

constexpr int LN_FT = 256;              // features per tile
constexpr uint32_t LN_TMEM_COLS = 512;
constexpr int LN_ROW_BYTES = 128;       // bytes of an operand row per stage

template <int FMT>
struct LnFmt;
template <>
struct LnFmt<MXFP4_ELEM_E2M1> {
    static constexpr int BK = 256;       // K elements per stage
    static constexpr int ATOMS = 2;      // scale atoms (128 K) per stage
    static constexpr int MMA_K = 64;
    static constexpr uint32_t AB_FMT = 1;
};
template <>
struct LnFmt<MXFP4_ELEM_E4M3> {
    static constexpr int BK = 128;
    static constexpr int ATOMS = 1;
    static constexpr int MMA_K = 32;
    static constexpr uint32_t AB_FMT = 0;
};

template <int FMT, int NT>
struct __align__(1024) LnSmem {
    static constexpr int ATOMS = LnFmt<FMT>::ATOMS;
    static constexpr int S = 4;                    // stages (227 KB with the plan of MAX_GROUPS groups)
    static constexpr int NACC = NT > 64 ? 1 : 2;   // accumulators in tensor memory
    static constexpr int TW = NT < 64 ? NT : 64;   // tokens of an epilogue warp
    static constexpr int EPI_WARPS = 8 * (NT / TW);
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr uint32_t SF_COL0 = NACC * 2 * NT;
    // groups whose plan (two words each) fits beside the stages
    static constexpr int MAX_GROUPS = NT > 64 ? 2048 : MXFP4_MAX_GROUPS;
    static_assert(SF_COL0 + S * 12 * ATOMS <= LN_TMEM_COLS, "tensor memory columns");
    uint8_t w[S][LN_FT * LN_ROW_BYTES];
    uint8_t x[S][NT * LN_ROW_BYTES];
    uint8_t sfw[S][2][512 * ATOMS];
    uint8_t sfx[S][512 * ATOMS];
    unsigned long long full[S], empty[S], acc_full[2], acc_empty[2], done;
    uint32_t tmem_base;
    int err;
};

struct LnArgs {
    const uint8_t* sfx;     // A's scales (tokens)
    const uint8_t* sfw;     // B's scales, group g at g * sfw_group_bytes
    const float* bias;      // [groups][n] or NULL
    const void* residual;   // [m][ld_res] or NULL
    void* y;                // [m][ld_y]
    void* preact;           // [m][ld_z] or NULL
    const int64_t* group_list;
    int32_t* status;
    int64_t m, n, k, ld_res, ld_y, ld_z, sfw_group_bytes;
    int32_t num_groups, gl_type, act;
};

struct LnMaps {
    CUtensorMap x, w;
};

struct LnTile {
    int g, f0, nh;      // group, first feature, halves with features
    int64_t row0;       // first token row
    int rows;           // valid token rows (<= NT)
};

template <int NT>
__device__ __forceinline__ LnTile ln_tile(const LnArgs& a, const int32_t* s_tpre, const int32_t* s_rst, int64_t t,
                                          int n_ft)
{
    LnTile r;
    const int mt = (int)(t / n_ft);
    const int ft = (int)(t - (int64_t)mt * n_ft);
    int lo = 0, hi = a.num_groups - 1;  // largest g with s_tpre[g] <= mt (skips empty groups)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tpre[mid] <= mt)
            lo = mid;
        else
            hi = mid - 1;
    }
    r.g = lo;
    r.row0 = (int64_t)s_rst[lo] + (int64_t)(mt - s_tpre[lo]) * NT;
    r.rows = (int)min((int64_t)NT, (int64_t)s_rst[lo + 1] - r.row0);
    r.f0 = ft * LN_FT;
    r.nh = a.n - r.f0 > 128 ? 2 : 1;
    return r;
}

__device__ __forceinline__ uint32_t ln_idesc(uint32_t ab_fmt, uint32_t sf_id, uint32_t n)
{
    return (sf_id << 4) | (ab_fmt << 7) | (ab_fmt << 10) | ((n >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24) |
           (sf_id << 29);
}

// Bytes of global memory (16-byte aligned, a multiple of 16) into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// The group plan in shared memory: s_tpre[g] = sum_{j<g} ceil(n_j / BS), s_rst[g]
// = the group's first row. Without a group list all rows are one group.
// Returns the number of row tiles, -1 for an invalid list. Contains __syncthreads.
template <int BS, typename Args>
__device__ int64_t ln_plan(const Args& a, int32_t* s_tpre, int32_t* s_rst)
{
    if (!a.group_list) {
        const int64_t units = (a.m + BS - 1) / BS;
        if (threadIdx.x == 0) {
            s_tpre[0] = s_rst[0] = 0;
            s_tpre[1] = (int32_t)units;
            s_rst[1] = (int32_t)a.m;
        }
        __syncthreads();
        return units;
    }
    KArgs pa;
    memset(&pa, 0, sizeof(pa));
    pa.group_list = a.group_list;
    pa.num_groups = a.num_groups;
    pa.gl_type = a.gl_type;
    pa.rows = a.m;
    return build_plan<BS, true>(pa, s_tpre, s_rst);
}

// mbar_wait that reads the clock once in 64 tries: a read takes longer than the
// event it would delay (a stage here is half a microsecond).
__device__ __forceinline__ bool ln_wait(uint32_t bar, uint32_t parity)
{
    uint64_t t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try(bar, parity))
                return true;
        const uint64_t now = global_ns();
        if (t0 == 0)
            t0 = now;
        else if (now - t0 > SG_WAIT_NS)
            return false;
    }
}

// ---- activations -----------------------------------------------------------

// 1 / (1 + e^-z) by the approximate exponential and quotient: their errors, a few
// 2^-23 plus |z| 2^-24 relative, are of the order of z's own rounding.
__device__ __forceinline__ float act_sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// The normal distribution's mass below z, 0.5 erfc(-z / sqrt 2), and e = exp(-z^2 / 2).
// Below 0 it is e t P(t) with t = 1 / (1 + 0.42 |z|): 0.5 erfcx is smooth in t down to
// t = 0, where it goes as t, and P is the polynomial of degree 7 of least largest
// relative error on it (2.2e-7; 4.8e-7 with fp32 coefficients and Horner steps), found
// by linear programming over 1200 points of 0 <= |z| <= 14.5. Relative, so that gelu's
// small results left of 0 keep their digits: with e's argument and exponential the
// whole is off by at most (24 + 1.7 z^2) 2^-24 of itself. The other side by symmetry.
// erfcf's instructions bounded the epilogue (E4M3 2049 x 14336 x 4096, gelu, residual
// and pre-activation in fp32: 222 us against 181 with this).
__device__ __forceinline__ float normal_mass(float z, float& e)
{
    const float u = fabsf(z), t = __fdividef(1.0f, fmaf(0.42f, u, 1.0f));
    e = __expf(-0.5f * u * u);
    float q = fmaf(-0.0446484350f, t, 0.204033539f);
    q = fmaf(q, t, -0.328966498f);
    q = fmaf(q, t, 0.157051578f);
    q = fmaf(q, t, 0.0316510014f);
    q = fmaf(q, t, 0.146566480f);
    q = fmaf(q, t, 0.166723162f);
    q = fmaf(q, t, 0.167589054f) * t * e;
    return z < 0.0f ? q : 1.0f - q;
}

// act(z) of the elementwise activations. gelu_tanh: 0.5 z (1 + tanh u) is z
// times the logistic function of 2u.
__device__ __forceinline__ float act_value(float z, int act)
{
    switch (act) {
    case MXFP4_ACT_RELU:
        return z > 0.0f ? z : (z != z ? z : 0.0f);
    case MXFP4_ACT_GELU: {
        float e;
        return z * normal_mass(z, e);
    }
    case MXFP4_ACT_GELU_TANH:
        return z * act_sigmoid(1.5957691216057308f * (z + 0.044715f * z * z * z));
    case MXFP4_ACT_SILU:
        return z * act_sigmoid(z);
    default:
        return z;
    }
}

// d act / dz
__device__ __forceinline__ float act_slope(float z, int act)
{
    switch (act) {
    case MXFP4_ACT_RELU:
        return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case MXFP4_ACT_GELU: {
        float e;
        const float mass = normal_mass(z, e);
        return mass + z * 0.39894228040143268f * e;
    }
    case MXFP4_ACT_GELU_TANH: {
        if (fabsf(z) > 16.0f)  // saturated; z^2 must not overflow against a zero
            return z > 0.0f ? 1.0f : 0.0f;
        const float s = act_sigmoid(1.5957691216057308f * (z + 0.044715f * z * z * z));
        return s + z * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * z * z);
    }
    case MXFP4_ACT_SILU: {
        const float s = act_sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    default:
        return 1.0f;
    }
}

template <bool F32>
__device__ __forceinline__ float ln_load(const void* p, int64_t i)
{
    return F32 ? static_cast<const float*>(p)[i]
               : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

template <bool F32>
__device__ __forceinline__ void ln_store(void* p, int64_t i, float v)
{
    if constexpr (F32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16(v);
}

// One activation, chosen at compile time where a loop holds many of them.
template <int ACT>
__device__ __forceinline__ float act_of(float z)
{
    return act_value(z, ACT);
}

// 32 tokens of this thread's feature: v[i] = z of token i of `rows`. The
// pointers are those of token 0 and this thread's column (the activated
// width's where the activation is gated). Loads of the residual go ahead of
// the stores eight tokens at a time, since y may be the residual; without one,
// four at a time keep the temporaries in registers (what spills goes to L2: the
// stages leave the L1 cache next to nothing. 32768 x 4096 x 2048, swiglu, over 32
// experts 193 against 176 us; with a residual 8192 x 4096 x 1024 83 / 106).
template <int ACT, bool F32, bool WHOLE, bool RES>
__device__ __forceinline__ void ln_finish32(const float (&v)[32], int rows, bool fok, char* y, int64_t ld_y,
                                            const char* res, int64_t ld_res)
{
    constexpr int ESZ = F32 ? 4 : 2;
    constexpr bool GATED = ACT == MXFP4_ACT_SWIGLU;
    constexpr int STEP = GATED ? 2 : 1, BATCH = RES ? 8 : 4;
    // gated: lanes 2j and 2j + 1 hold gate j and up j; of a pair of tokens the
    // even lane finishes the first, the odd lane the second
    const bool odd = GATED && (threadIdx.x & 1);
    const int first = odd ? 1 : 0;
    y += first * ld_y * ESZ;
    if constexpr (RES)
        res += first * ld_res * ESZ;
#pragma unroll
    for (int i0 = 0; i0 < 32; i0 += BATCH * STEP) {
        float o[BATCH];
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                o[i] = WHOLE || (fok && i0 + STEP * i + first < rows) ? ln_load<F32>(res, 0) : 0.0f;
                res += ld_res * (STEP * ESZ);
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            float a;
            if constexpr (GATED) {
                const int t = i0 + 2 * i;
                const float other = __shfl_xor_sync(FULL, odd ? v[t] : v[t + 1], 1);
                const float gate = odd ? other : v[t], up = odd ? v[t + 1] : other;
                a = act_of<MXFP4_ACT_SILU>(gate) * up;
            } else {
                a = act_of<ACT>(v[i0 + i]);
            }
            o[i] = RES ? a + o[i] : a;
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (WHOLE || (fok && i0 + STEP * i + first < rows))
                ln_store<F32>(y, 0, o[i]);
            y += ld_y * (STEP * ESZ);
        }
    }
}

template <bool F32, bool WHOLE, bool RES>
__device__ __forceinline__ void ln_epilogue32(const LnArgs& a, const float (&v)[32], int64_t row0, int rows, int f, bool fok)
{
    constexpr int ESZ = F32 ? 4 : 2;
    if (a.preact) {
        char* z = static_cast<char*>(a.preact) + (row0 * a.ld_z + f) * ESZ;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (WHOLE || (fok && i < rows))
                ln_store<F32>(z, 0, v[i]);
            z += a.ld_z * ESZ;
        }
    }
    const int fo = a.act == MXFP4_ACT_SWIGLU ? f >> 1 : f;
    char* y = static_cast<char*>(a.y) + (row0 * a.ld_y + fo) * ESZ;
    const char* res = RES ? static_cast<const char*>(a.residual) + (row0 * a.ld_res + fo) * ESZ : nullptr;
    // the branch is outside the loops: one activation's code runs
    switch (a.act) {
    case MXFP4_ACT_NONE:
        return ln_finish32<MXFP4_ACT_NONE, F32, WHOLE, RES>(v, rows, fok, y, a.ld_y, res, a.ld_res);
    case MXFP4_ACT_RELU:
        return ln_finish32<MXFP4_ACT_RELU, F32, WHOLE, RES>(v, rows, fok, y, a.ld_y, res, a.ld_res);
    case MXFP4_ACT_GELU:
        return ln_finish32<MXFP4_ACT_GELU, F32, WHOLE, RES>(v, rows, fok, y, a.ld_y, res, a.ld_res);
    case MXFP4_ACT_GELU_TANH:
        return ln_finish32<MXFP4_ACT_GELU_TANH, F32, WHOLE, RES>(v, rows, fok, y, a.ld_y, res, a.ld_res);
    case MXFP4_ACT_SILU:
        return ln_finish32<MXFP4_ACT_SILU, F32, WHOLE, RES>(v, rows, fok, y, a.ld_y, res, a.ld_res);
    default:
        return ln_finish32<MXFP4_ACT_SWIGLU, F32, WHOLE, RES>(v, rows, fok, y, a.ld_y, res, a.ld_res);
    }
}

// Asks for a warp's part of the residual (32 features, TW tokens: a line each)
// ahead of the product's end, where that is at most LN_SHORT stages away (k = 1024,
// 4 stages: 69 against 83 us without; with 32 stages it came 3 % slower).
constexpr int LN_SHORT = 16;

template <bool F32, int TW>
__device__ __forceinline__ void ln_prefetch(const LnArgs& a, int64_t row0, int rows, int f)
{
    if (f >= a.n)
        return;
    const int lane = threadIdx.x & 31, fo = (a.act == MXFP4_ACT_SWIGLU ? f >> 1 : f);
    const int fw = __shfl_sync(__activemask(), fo, 0);
    for (int t = lane; t < TW && t < rows; t += 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.residual) + ((row0 + t) * a.ld_res + fw) * (F32 ? 4 : 2)));
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Low word of a shared-memory descriptor: the address in units of 16 bytes and
// a leading byte offset of 16. Advancing the address adds to this word.
__device__ __forceinline__ uint32_t ln_desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
// High words: operands (8-row groups 1024 bytes apart, version 1, 128-byte
// swizzle) and scale atoms (core matrices 128 bytes apart, no swizzle).
constexpr uint32_t LN_OPERAND_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t LN_SCALE_HI = (128u >> 4) | (1u << 14);

__device__ __forceinline__ uint64_t ln_desc(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

// One stage: its scale atoms into tensor memory, then its MMAs (up to 4 along
// K for NH halves of the features). Straight-line for a full stage: a single
// thread issues all of it, so every address must be at hand.
template <int FMT, int NT, int NH>
__device__ __forceinline__ void ln_stage(uint32_t d_tmem, uint32_t sf_col, uint32_t wlo, uint32_t xlo, uint32_t sfw,
                                         uint32_t sfx, int na, int nk, bool accumulate)
{
    using F = LnFmt<FMT>;
    constexpr int ATOMS = F::ATOMS;
#pragma unroll
    for (int i = 0; i < ATOMS; ++i) {
        if (i > 0 && i >= na)
            break;
#pragma unroll
        for (int h = 0; h < NH; ++h)
            asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(sf_col + 4u * (2 * i + h)),
                         "l"(ln_desc(sfw + (uint32_t)(512 / 16) * (ATOMS * h + i), LN_SCALE_HI))
                         : "memory");
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(sf_col + 4u * (2 * ATOMS + i)),
                     "l"(ln_desc(sfx + (uint32_t)(512 / 16) * i, LN_SCALE_HI))
                     : "memory");
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        if (kk > 0 && kk >= nk)
            break;
        // 32 bytes of K per MMA; its first scale block is byte (block % 4) of atom (block / 4)
        constexpr int SB = F::MMA_K / 32;
        const uint32_t ai = (uint32_t)((kk * SB) >> 2);
#pragma unroll
        for (int h = 0; h < NH; ++h)
            gm_mma<FMT>(d_tmem + (uint32_t)(h * NT), ln_desc(wlo + (uint32_t)(h * 128 * LN_ROW_BYTES / 16 + 2 * kk), LN_OPERAND_HI),
                        ln_desc(xlo + 2u * kk, LN_OPERAND_HI), ln_idesc(F::AB_FMT, (uint32_t)((kk * SB) & 3), NT),
                        sf_col + 4u * (2 * ai + h), sf_col + 4u * (2 * ATOMS + ai), kk > 0 || accumulate ? 1u : 0u);
    }
}

template <int FMT, int NT, bool F32, bool RES>
__global__ void __launch_bounds__(LnSmem<FMT, NT>::THREADS, 1) linear_kernel(const __grid_constant__ LnMaps maps, const LnArgs a)
{
    using F = LnFmt<FMT>;
    using SM = LnSmem<FMT, NT>;
    constexpr int S = SM::S, ATOMS = F::ATOMS, NACC = SM::NACC;
    extern __shared__ __align__(1024) uint8_t ln_dyn[];
    uint8_t* base = ln_dyn + ((1024u - (smem_addr(ln_dyn) & 1023u)) & 1023u);
    SM& sm = *reinterpret_cast<SM*>(base);
    int32_t* s_tpre = reinterpret_cast<int32_t*>(base + sizeof(SM));
    int32_t* s_rst = s_tpre + a.num_groups + 1;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sm.err = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1 + 32);  // the transactions + each producer lane's copies
            mbar_init(smem_addr(&sm.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sm.acc_full[i]), 1);
            mbar_init(smem_addr(&sm.acc_empty[i]), SM::EPI_WARPS);
        }
        mbar_init(smem_addr(&sm.done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem_base)),
                     "r"(LN_TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        gm_fence_before();
    }
    const int64_t units = ln_plan<NT>(a, s_tpre, s_rst);  // contains __syncthreads
    gm_fence_after();
    const uint32_t tmem = sm.tmem_base;
    if (blockIdx.x == 0 && tid == 0 && a.status)
        *a.status = units >= 0 ? MXFP4_OK : MXFP4_EINVAL;

    const int n_ft = (int)((a.n + LN_FT - 1) / LN_FT);
    const int64_t tiles = units < 0 ? 0 : units * n_ft;
    const int64_t nblk = a.k / 32, ncb = (nblk + 3) >> 2;
    const int nmma = (int)(a.k / F::MMA_K);           // MMAs along K
    const int nst = (int)((a.k + F::BK - 1) / F::BK);  // stages along K

    if (warp == 0) {
        // ---- producer
        int s = 0;
        uint32_t ph = 0, issued = 0;
        for (int64_t t = blockIdx.x; t < tiles && !sm.err; t += gridDim.x) {
            const LnTile tl = ln_tile<NT>(a, s_tpre, s_rst, t, n_ft);
            const int wrow = (int)((int64_t)tl.g * a.n + tl.f0);
            const uint8_t* sfw = a.sfw + tl.g * a.sfw_group_bytes + (int64_t)(tl.f0 >> 7) * ncb * 512;
            const uint8_t* px[NT / 32];
            uint32_t okx = 0;
#pragma unroll
            for (int q = 0; q < NT / 32; ++q) {
                const int r = lane + 32 * q;
                const bool ok = r < tl.rows;
                px[q] = a.sfx + (ok ? srow_off_mma(tl.row0 + r, 0, nblk) : 0);
                okx |= (ok ? 1u : 0u) << q;
            }
            for (int ks = 0; ks < nst; ++ks) {
                if (!__all_sync(FULL, ln_wait(smem_addr(&sm.empty[s]), ph ^ 1u))) {
                    sm.err = 1;
                    break;
                }
                const int na = (int)min((int64_t)ATOMS, ncb - (int64_t)ks * ATOMS);  // scale atoms of the stage
                const uint32_t bar = smem_addr(&sm.full[s]);
#pragma unroll
                for (int i = 0; i < ATOMS; ++i) {
                    const int64_t jo = ((int64_t)ks * ATOMS + i) * 512;
                    const uint32_t dst = smem_addr(sm.sfx[s]) + 512 * i + 16 * lane;
#pragma unroll
                    for (int q = 0; q < NT / 32; ++q) {
                        const bool ok = ((okx >> q) & 1u) && i < na;
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 4 * q),
                                     "l"(px[q] + (ok ? jo : 0)), "r"(ok ? 4u : 0u)
                                     : "memory");
                    }
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
                if (lane == 0) {
                    mbar_expect_tx(bar, tl.nh * (128 * LN_ROW_BYTES + 512 * na) + NT * LN_ROW_BYTES);
                    for (int h = 0; h < tl.nh; ++h) {
                        gm_tma_load(smem_addr(sm.w[s]) + h * 128 * LN_ROW_BYTES, &maps.w, ks * LN_ROW_BYTES,
                                    wrow + 128 * h, bar);
                        bulk_load(smem_addr(sm.sfw[s][h]), sfw + ((int64_t)h * ncb + (int64_t)ks * ATOMS) * 512, 512 * na,
                                  bar);
                    }
                    gm_tma_load(smem_addr(sm.x[s]), &maps.x, ks * LN_ROW_BYTES, (int)tl.row0, bar);
                }
                issued |= 1u << s;
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // every load issued lands before the CTA leaves (the last load of stage
        // i had the parity of its turn)
        if (lane == 0)
            for (int i = 0; i < S; ++i)
                if (issued & (1u << i))
                    (void)ln_wait(smem_addr(&sm.full[i]), i < s ? ph : ph ^ 1u);
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer. The whole warp walks the tiles, so that addresses and
        // descriptors stay in uniform registers; one elected lane issues.
        int s = 0, acc = 0;
        uint32_t ph = 0, aph = 0;
        for (int64_t t = blockIdx.x; t < tiles && !sm.err; t += gridDim.x) {
            const LnTile tl = ln_tile<NT>(a, s_tpre, s_rst, t, n_ft);
            if (!__all_sync(FULL, ln_wait(smem_addr(&sm.acc_empty[acc]), aph ^ 1u))) {
                sm.err = 1;
                break;
            }
            gm_fence_after();
            const uint32_t d_tmem = tmem + (uint32_t)(acc * 2 * NT);
            for (int ks = 0; ks < nst; ++ks) {
                if (!__all_sync(FULL, ln_wait(smem_addr(&sm.full[s]), ph))) {
                    sm.err = 1;
                    break;
                }
                gm_fence_after();
                // the tokens' scales were written by the producer's copies
                // (generic proxy); tcgen05.cp reads them in the async proxy
                fence_async_smem();
                if (elect_one()) {
                    const uint32_t sf_col = tmem + SM::SF_COL0 + (uint32_t)(12 * ATOMS * s);
                    const uint32_t wlo = ln_desc_lo(smem_addr(sm.w[s])), xlo = ln_desc_lo(smem_addr(sm.x[s]));
                    const int na = (int)min((int64_t)ATOMS, ncb - (int64_t)ks * ATOMS);
                    const int nk = nmma - 4 * ks;
                    if (tl.nh == 2)
                        ln_stage<FMT, NT, 2>(d_tmem, sf_col, wlo, xlo, ln_desc_lo(smem_addr(sm.sfw[s][0])),
                                             ln_desc_lo(smem_addr(sm.sfx[s])), na, nk, ks > 0);
                    else
                        ln_stage<FMT, NT, 1>(d_tmem, sf_col, wlo, xlo, ln_desc_lo(smem_addr(sm.sfw[s][0])),
                                             ln_desc_lo(smem_addr(sm.sfx[s])), na, nk, ks > 0);
                    gm_commit(smem_addr(&sm.empty[s]));
                    if (ks + 1 == nst)
                        gm_commit(smem_addr(&sm.acc_full[acc]));
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (++acc == NACC) {
                acc = 0;
                aph ^= 1u;
            }
        }
        // every MMA issued has completed before the tensor memory is freed
        if (elect_one())
            gm_commit(smem_addr(&sm.done));
        __syncwarp();
        (void)ln_wait(smem_addr(&sm.done), 0);
        __syncwarp();
    } else {
        // ---- epilogue: tensor-memory lanes 32 (warp % 4) .. + 31 of half h,
        // tokens c0 .. c0 + TW - 1 of the tile
        constexpr int TW = SM::TW;
        const int quad = warp & 3, h = ((warp - 2) >> 2) & 1, c0 = ((warp - 2) >> 3) * TW;
        int acc = 0;
        uint32_t aph = 0;
        for (int64_t t = blockIdx.x; t < tiles && !sm.err; t += gridDim.x) {
            const LnTile tl = ln_tile<NT>(a, s_tpre, s_rst, t, n_ft);
            const int f = tl.f0 + 128 * h + 32 * quad + lane;
            const bool fok = f < a.n;
            const float bias = a.bias && fok ? a.bias[(int64_t)tl.g * a.n + f] : 0.0f;
            if (RES && nst <= LN_SHORT && h < tl.nh)
                ln_prefetch<F32, TW>(a, tl.row0 + c0, tl.rows - c0, f);
            __syncwarp();
            if (!__all_sync(FULL, ln_wait(smem_addr(&sm.acc_full[acc]), aph))) {
                sm.err = 1;
                break;
            }
            gm_fence_after();
            float v[TW / 32][32];
#pragma unroll
            for (int c = 0; c < TW / 32; ++c) {
                uint32_t u[32];
                __syncwarp();
                gm_ld32(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(acc * 2 * NT + h * NT + c0 + 32 * c), u);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[c][i] = __uint_as_float(u[i]) + bias;
            }
            gm_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&sm.acc_empty[acc]));
            if (++acc == NACC) {
                acc = 0;
                aph ^= 1u;
            }
            if (h < tl.nh) {
#pragma unroll 1
                for (int c = 0; c < TW / 32; ++c) {
                    const int rows = tl.rows - c0 - 32 * c;
                    if (rows <= 0)
                        break;
                    // whole chunks (every lane a feature, 32 tokens) take no predicates
                    if (rows >= 32 && __all_sync(FULL, fok))
                        ln_epilogue32<F32, true, RES>(a, v[0], tl.row0 + c0 + 32 * c, rows, f, fok);
                    else
                        ln_epilogue32<F32, false, RES>(a, v[0], tl.row0 + c0 + 32 * c, rows, f, fok);
                    // the next 32 tokens move up, so that the code exists once
#pragma unroll
                    for (int d = 0; d + 1 < TW / 32; ++d)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[d][i] = v[d + 1][i];
                }
            }
        }
    }

    __syncthreads();
    if (tid == 0 && sm.err && a.status)
        *a.status = MXFP4_ECUDA;
    if (warp == 1) {
        gm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(LN_TMEM_COLS) : "memory");
    }
}

// ---------------------------------------------------------------------------
// Gradients of the epilogue: dz = dy act'(z) (gated: d gate = dy up silu'(gate),
// d up = dy silu(gate)), dbias_g = the sum of dz over the group's rows, in
// fp32 from the unrounded dz. Bound by memory. A CTA takes LB_ROWS rows of one
// group by a stretch of columns as wide as its threads reach (2048 bf16
// columns; narrower matrices take several rows side by side), so that it reads
// and writes long pieces of a row at a time, LB_UNROLL rows in flight. Partial
// sums (a thread's rows in order, then the rows side by side) go to
// ws[unit][n], and a second kernel adds a group's units in order.
// ---------------------------------------------------------------------------

constexpr int LB_ROWS = 32;

struct LnBwdArgs {
    const void* grad;      // [m][ld_g]
    const void* z;         // [m][ld_z]
    void* grad_z;          // [m][ld_dz]
    float* grad_bias;      // [groups][n] or NULL
    float* ws;             // [units][n]
    const int64_t* group_list;
    int32_t* status;
    int64_t m, n, ld_g, ld_z, ld_dz;
    int32_t num_groups, gl_type, act;
    int32_t across_log2;   // log2 of a row's threads
};

// PER columns of one row of z and the matching gradients, as loaded (the
// vector form keeps 16-byte words until they are used: registers bound how many
// rows are in flight) and as fp32.
template <int ESZ, bool VEC, int PER>
struct LbPiece {
    uint4 z;
    uint4 g;   // gated: the low half

    __device__ __forceinline__ void load(const LnBwdArgs& a, int64_t row, int64_t c, bool gated)
    {
        z = g = make_uint4(0u, 0u, 0u, 0u);
        if (c >= a.n)
            return;
        if constexpr (VEC) {
            z = ld_stream(static_cast<const char*>(a.z) + (row * a.ld_z + c) * ESZ);
            if (gated) {
                const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const char*>(a.grad) + (row * a.ld_g + (c >> 1)) * ESZ);
                g.x = q.x;
                g.y = q.y;
            } else {
                g = ld_stream(static_cast<const char*>(a.grad) + (row * a.ld_g + c) * ESZ);
            }
        } else {  // two columns, one element a word
            z.x = mv_load<ESZ>(a.z, row * a.ld_z + c);
            g.x = mv_load<ESZ>(a.grad, row * a.ld_g + (gated ? c >> 1 : c));
            if (c + 1 < a.n) {
                z.y = mv_load<ESZ>(a.z, row * a.ld_z + c + 1);
                if (!gated)
                    g.y = mv_load<ESZ>(a.grad, row * a.ld_g + c + 1);
            }
        }
    }

    static __device__ __forceinline__ void spread(const uint4& q, float (&v)[PER])
    {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if constexpr (VEC && ESZ == 2)
                v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
            else
                v[i] = __uint_as_float(u[i] << (ESZ == 2 ? 16 : 0));
        }
    }
};

template <int PER>
__device__ __forceinline__ void lb_slope(const LnBwdArgs& a, bool gated, const float (&z)[PER], const float (&g)[PER], float (&d)[PER])
{
    if (gated) {
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
            const float gate = z[i], s = act_sigmoid(gate);
            d[i] = g[i / 2] * z[i + 1] * (s * (1.0f + gate * (1.0f - s)));
            d[i + 1] = g[i / 2] * (gate * s);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            d[i] = g[i] * act_slope(z[i], a.act);
    }
}

constexpr int LB_UNROLL = 2;

template <int ESZ, bool VEC>
__global__ void __launch_bounds__(NTHREADS, 4) linear_bwd_kernel(const LnBwdArgs a)
{
    constexpr int PER = VEC ? 16 / ESZ : 2;   // columns of z per thread
    extern __shared__ __align__(16) int32_t lb_dyn[];
    __shared__ float s_sum[NTHREADS * PER];
    int32_t* s_tpre = lb_dyn;
    int32_t* s_rst = lb_dyn + a.num_groups + 1;
    const int64_t units = ln_plan<LB_ROWS>(a, s_tpre, s_rst);
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && tid == 0 && a.status)
        *a.status = units >= 0 ? MXFP4_OK : MXFP4_EINVAL;
    const bool gated = a.act == MXFP4_ACT_SWIGLU;
    const int across = 1 << a.across_log2;             // threads along a row
    const int down = NTHREADS >> a.across_log2;        // rows side by side
    const int64_t n_ct = (a.n + (int64_t)across * PER - 1) / (across * PER);
    const int tc = tid & (across - 1), tr = tid >> a.across_log2;
    for (int64_t w = blockIdx.x; w < (units < 0 ? 0 : units * n_ct); w += gridDim.x) {
        const uint32_t unit = (uint32_t)(w / n_ct);
        const int64_t c0 = (w - (int64_t)unit * n_ct) * across * PER, c = c0 + (int64_t)tc * PER;
        int lo = 0, hi = a.num_groups - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((uint32_t)s_tpre[mid] <= unit)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int64_t r0 = (int64_t)s_rst[lo] + (int64_t)(unit - (uint32_t)s_tpre[lo]) * LB_ROWS;
        const int nr = (int)min((int64_t)LB_ROWS, (int64_t)s_rst[lo + 1] - r0);
        float sum[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sum[i] = 0.0f;
        for (int r = tr; r < nr; r += LB_UNROLL * down) {
            LbPiece<ESZ, VEC, PER> in[LB_UNROLL];
#pragma unroll
            for (int q = 0; q < LB_UNROLL; ++q)
                if (r + q * down < nr)
                    in[q].load(a, r0 + r + q * down, c, gated);
#pragma unroll
            for (int q = 0; q < LB_UNROLL; ++q)
                if (r + q * down < nr) {
                    const int64_t row = r0 + r + q * down;
                    float z[PER], g[PER], d[PER];
                    in[q].spread(in[q].z, z);
                    in[q].spread(in[q].g, g);
                    lb_slope<PER>(a, gated, z, g, d);
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        sum[i] += d[i];
                    if constexpr (VEC) {
                        if (c < a.n)
                            piece_store<ESZ, PER>(a.grad_z, row * a.ld_dz + c, d);
                    } else {
#pragma unroll
                        for (int i = 0; i < PER; ++i)
                            if (c + i < a.n)
                                ln_store<ESZ == 4>(a.grad_z, row * a.ld_dz + c + i, d[i]);
                    }
                }
        }
        if (a.grad_bias) {
            if (down > 1) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    s_sum[(tr * across + tc) * PER + i] = sum[i];
                __syncthreads();
                if (tr == 0)
                    for (int q = 1; q < down; ++q)
#pragma unroll
                        for (int i = 0; i < PER; ++i)
                            sum[i] += s_sum[(q * across + tc) * PER + i];
                __syncthreads();
            }
            if (tr == 0)
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (c + i < a.n)
                        a.ws[(int64_t)unit * a.n + c + i] = sum[i];
        }
    }
}

// The status of a call whose matrices are empty: the list is checked all the same.
__global__ void __launch_bounds__(NTHREADS) linear_list_kernel(const LnBwdArgs a)
{
    extern __shared__ __align__(16) int32_t lb_dyn[];
    const int64_t units = ln_plan<LB_ROWS>(a, lb_dyn, lb_dyn + a.num_groups + 1);
    if (threadIdx.x == 0)
        *a.status = units >= 0 ? MXFP4_OK : MXFP4_EINVAL;
}

// grad_bias[g][c] = the sum of the group's units, in order (0 for an invalid list). Grid: column
// blocks x groups.
__global__ void __launch_bounds__(NTHREADS) linear_bias_kernel(const LnBwdArgs a)
{
    extern __shared__ __align__(16) int32_t lb_dyn[];
    int32_t* s_tpre = lb_dyn;
    int32_t* s_rst = lb_dyn + a.num_groups + 1;
    // (started early, its waiting CTAs took room from linear_bwd_kernel's: 94 against 78 us)
    const bool ok = ln_plan<LB_ROWS>(a, s_tpre, s_rst) >= 0;
    wait_for_prerequisite();
    const int64_t c = (int64_t)blockIdx.x * NTHREADS + threadIdx.x;
    if (c >= a.n)
        return;
    for (int g = blockIdx.y; g < a.num_groups; g += gridDim.y) {
        float v = 0.0f;
        const int end = ok ? s_tpre[g + 1] : s_tpre[g];  // an invalid list: no rows, and no partial sums were written
#pragma unroll 4
        for (int u = s_tpre[g]; u < end; ++u)
            v += a.ws[(int64_t)u * a.n + c];
        a.grad_bias[(int64_t)g * a.n + c] = v;
    }
}

}  // namespace mxfp4
