// mxfp4_common.cuh -- what the translation units of libmxfp4 share: kernel
// arguments, block scale parameters and element rounding, the group plan,
// mbarrier, TMA and tcgen05 wrappers, and the host helpers of the launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "mxfp4.h"

namespace mxfp4 {

constexpr unsigned FULL = 0xFFFFFFFFu;
constexpr uint32_t QNAN32 = 0x7FC00000u;
constexpr int NTHREADS = 256;

struct KArgs {
    const void* x;
    int64_t rows, cols, ld;
    float sf;
    int32_t mode;
    int32_t grad_dir;  // 0, MXFP4_ROWWISE or MXFP4_COLWISE
    void* y_row;
    void* y_col;
    int64_t ld_y;
    uint8_t* codes_row;
    uint8_t* scales_row;
    uint8_t* mask_row;
    uint8_t* codes_col;
    uint8_t* scales_col;
    uint8_t* mask_col;
    const void* g_out;
    void* g_in;
    int64_t ld_g;
    const int64_t* group_list;
    int32_t num_groups;
    int32_t gl_type;
    int32_t* status;
    uint32_t n_ct;  // column tiles of the tile kernel
    uint32_t thr;   // PAGE mode: fp32 bits of T0 (see qparams)
    uint32_t ts_flags;  // staged kernel: column-wise outputs written by TMA stores (SG_TS_*)
    int32_t srow_mma;   // scales_row in the MMA scale-factor layout (MXFP4_SCALES_MMA)
    int32_t fmt;        // MXFP4_ELEM_E2M1 or MXFP4_ELEM_E4M3
    int64_t k_alloc;    // column-wise operand layout: K slots per codes row (MXFP4_COLS_MMA)
    // 4 and 65536, set by the host: the staged kernel scales table indices and
    // moves halves with integer multiply-adds by these run-time values, which
    // the compiler cannot turn back into shifts, so that this work runs on the
    // multiply-add pipe beside the logic ops on the ALU pipe
    uint32_t mul4, mul16;
};

// Byte offset of row-wise scale (row, b) of a [rows][nblk] scale matrix:
// row-major, or the block-scaled MMA layout (atoms of 128 rows x 4 block
// columns, 512 bytes, atom rows in order; entry (r, c) of an atom at
// 16 (r mod 32) + 4 floor(r / 32) + c).
__device__ __forceinline__ int64_t srow_off_mma(int64_t row, int64_t b, int64_t nblk)
{
    const int64_t ncb = (nblk + 3) >> 2;
    return (((row >> 7) * ncb + (b >> 2)) << 9) + ((row & 31) << 4) + (((row >> 5) & 3) << 2) + (b & 3);
}

__device__ __forceinline__ int64_t srow_off(const KArgs& a, int64_t row, int64_t b, int64_t nblk)
{
    return a.srow_mma ? srow_off_mma(row, b, nblk) : row * nblk + b;
}

// ---------------------------------------------------------------------------
// Per-block parameters
// ---------------------------------------------------------------------------

struct BP {
    float inv;      // 2^-k
    float scale;    // 2^k
    uint32_t lim;   // fp32 bits of fl(6 * 2^k); +inf bits once it overflows
    uint32_t nanm;  // all ones for a non-finite block
    uint32_t e8;    // E8M0 byte
};

// fp32 bits of 2^k for k in [-127, 127] (2^-127 is the subnormal 0x00400000).
__device__ __forceinline__ uint32_t pow2_bits(int k)
{
    return k >= -126 ? (uint32_t)(k + 127) << 23 : 0x00400000u;
}

// A = fp32 bits of the block's max |x| (integer max of sign-cleared bits, so a
// NaN anywhere gives A > 0x7F800000 and an inf gives A == 0x7F800000).
__device__ __forceinline__ BP block_params(uint32_t A, int mode, float sf)
{
    int k;
    bool special = A >= 0x7F800000u;
    if (mode == MXFP4_SCALE_FLOOR) {
        // floor(log2 amax) - 2 from the biased exponent; subnormal and zero
        // amax have a biased exponent of 0 and saturate at -127.
        k = max((int)(A >> 23) - 129, -127);
    } else {
        // r = max(fl(amax / sf), 2^-30) is a normal fp32 number; round(log2 r)
        // is its exponent plus one when its significand is at or above the
        // first fp32 significand above sqrt(2) (1.0110101000001001111001100..b;
        // fraction field 0x3504F3 < frac(sqrt 2) < 0x3504F4).
        float r = fmaxf(__fdiv_rn(__uint_as_float(A), sf), 0x1p-30f);
        uint32_t rb = __float_as_uint(r);
        k = (int)(rb >> 23) - 127 + ((rb & 0x7FFFFFu) >= 0x3504F4u ? 1 : 0);
        special = special || k > 127;  // 2^128 overflows fp32: scale = inf
    }
    if (special)
        k = 0;
    BP p;
    p.inv = __uint_as_float(pow2_bits(-k));
    p.scale = __uint_as_float(pow2_bits(k));
    p.lim = k >= 126 ? 0x7F800000u : (((uint32_t)(k + 129) << 23) | 0x00400000u);
    p.nanm = special ? 0xFFFFFFFFu : 0u;
    p.e8 = special ? 0xFFu : (uint32_t)(k + 127);
    return p;
}

// One element: returns the fp32 bits of sign(y) * code * 2^k with y = x * 2^-k
// (== fl(x / 2^k)), and the E2M1 nibble and saturation flag.
__device__ __forceinline__ uint32_t qdq_elem(uint32_t xb, const BP& p, uint32_t& nib, uint32_t& sat)
{
    const float y = __fmul_rn(__uint_as_float(xb), p.inv);
    const float a = fabsf(y);
    const uint32_t i = (uint32_t)(a >= 0.25f) + (uint32_t)(a >= 0.75f) + (uint32_t)(a >= 1.25f) +
                       (uint32_t)(a >= 1.75f) + (uint32_t)(a >= 2.5f) + (uint32_t)(a >= 3.5f) +
                       (uint32_t)(a >= 5.0f);
    // code magnitude as fp32 bits: 0, 0.5, then (i << 22) + 0x3F000000 gives
    // 1, 1.5, 2, 3, 4, 6 for i = 2..7 (two significant bits per binade)
    const uint32_t cb = i >= 2u ? (i << 22) + 0x3F000000u : (i == 1u ? 0x3F000000u : 0u);
    const uint32_t neg = y < 0.0f ? 0x80000000u : 0u;  // sign(-0) and sign(+0) are 0
    const float o = __fmul_rn(__uint_as_float(cb | neg), p.scale);
    nib = (neg >> 28) | i;
    sat = (xb & 0x7FFFFFFFu) > p.lim ? 1u : 0u;
    return __float_as_uint(o);
}

// ---------------------------------------------------------------------------
// MXFP8: E4M3 elements (scale mode FLOOR, block 32)
// ---------------------------------------------------------------------------

// k = floor(log2 amax) - 8 from the biased exponent (E4M3's largest normal is
// 1.75 * 2^8 = 448), saturated at -127 (subnormal and zero amax included).
__device__ __forceinline__ int k_e4m3(uint32_t A) { return max((int)(A >> 23) - 135, -127); }

__device__ __forceinline__ BP block_params8(uint32_t A)
{
    const bool special = A >= 0x7F800000u;
    const int k = special ? 0 : k_e4m3(A);
    BP p;
    p.inv = __uint_as_float(pow2_bits(-k));
    p.scale = __uint_as_float(pow2_bits(k));
    p.lim = ((uint32_t)(k + 135) << 23) | 0x00600000u;  // fp32 bits of 448 * 2^k = 1.75 * 2^(k + 8)
    p.nanm = special ? 0xFFFFFFFFu : 0u;
    p.e8 = special ? 0xFFu : (uint32_t)(k + 127);
    return p;
}

// One element: fp32 bits of decode(code) * 2^k (exact: codes have four
// significant bits and 2^k >= 2^-127), the E4M3 code of y = x * 2^-k by the
// hardware convert (nearest even, saturating at 448, sign kept) and the
// saturation flag.
__device__ __forceinline__ uint32_t qdq8_elem(uint32_t xb, const BP& p, uint32_t& code, uint32_t& sat)
{
    const float y = __fmul_rn(__uint_as_float(xb), p.inv);
    uint16_t q;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(0.0f), "f"(y));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(q));
    float c;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(c) : "r"(h));
    code = q & 0xFFu;
    sat = (xb & 0x7FFFFFFFu) > p.lim ? 1u : 0u;
    return __float_as_uint(__fmul_rn(c, p.scale));
}

// fp32 bits -> the same bits rounded to bf16 (nearest even) in the top half;
// finite values only.
__device__ __forceinline__ uint32_t round_bf16_bits(uint32_t b)
{
    return (b + 0x7FFFu + ((b >> 16) & 1u)) & 0xFFFF0000u;
}

// Volatile: the compiler takes an asm without it for arithmetic and may execute it
// ahead of the condition that guards it, which reads outside the tensor.
__device__ __forceinline__ uint4 ld_stream(const void* p)
{
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "l"(p));
    return r;
}

__device__ __forceinline__ void st_stream(void* p, const uint4& v)
{
    __stcs(reinterpret_cast<uint4*>(p), v);
}

// ---------------------------------------------------------------------------
// group_list plan, built by every CTA in shared memory
// ---------------------------------------------------------------------------

// Writes s_rst[g] = sum_{j<g} n_j and s_bpre[g] = sum_{j<g} ceil(n_j / BS) for
// g = 0..G and returns S = s_bpre[G], or -1 when the list is not a partition
// of [0, rows): a negative count, a decreasing offset, or a wrong total.
// PART: the groups may end before `rows` (rows behind the last group are no one's).
// Every thread of the CTA must call it; the first NTHREADS hold the groups.
template <int BS, bool PART = false>
__device__ int64_t build_plan(const KArgs& a, int32_t* s_bpre, int32_t* s_rst)
{
    __shared__ long long s_wr[NTHREADS / 32], s_wb[NTHREADS / 32];
    __shared__ int s_bad;
    const int G = a.num_groups;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (G + NTHREADS - 1) / NTHREADS;
    const int g0 = min(G, tid * per), g1 = min(G, g0 + per);
    if (tid == 0)
        s_bad = 0;
    __syncthreads();

    long long lr = 0, lb = 0;
    bool bad = false;
    long long prev = (a.gl_type == 0 && g0 > 0) ? (long long)a.group_list[g0 - 1] : 0;
    for (int g = g0; g < g1; ++g) {
        long long v = a.group_list[g];
        long long n = a.gl_type == 1 ? v : v - prev;
        prev = v;
        if (n < 0 || n > a.rows) {
            bad = true;
            n = 0;
        }
        lr += n;
        lb += (n + BS - 1) / BS;
    }
    long long ir = lr, ib = lb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        long long tr = __shfl_up_sync(FULL, ir, o);
        long long tb = __shfl_up_sync(FULL, ib, o);
        if (lane >= o) {
            ir += tr;
            ib += tb;
        }
    }
    if (lane == 31 && warp < NTHREADS / 32) {  // a CTA may carry extra warps: they hold no groups
        s_wr[warp] = ir;
        s_wb[warp] = ib;
    }
    if (bad)
        atomicOr(&s_bad, 1);
    __syncthreads();
    long long er = ir - lr, eb = ib - lb, tot_r = 0, tot_b = 0;
    for (int w = 0; w < NTHREADS / 32; ++w) {
        if (w < warp) {
            er += s_wr[w];
            eb += s_wb[w];
        }
        tot_r += s_wr[w];
        tot_b += s_wb[w];
    }
    prev = (a.gl_type == 0 && g0 > 0) ? (long long)a.group_list[g0 - 1] : 0;
    for (int g = g0; g < g1; ++g) {
        long long v = a.group_list[g];
        long long n = a.gl_type == 1 ? v : v - prev;
        prev = v;
        if (n < 0 || n > a.rows)
            n = 0;
        s_rst[g] = (int32_t)er;
        s_bpre[g] = (int32_t)eb;
        er += n;
        eb += (n + BS - 1) / BS;
    }
    if (tid == 0) {
        s_rst[G] = (int32_t)tot_r;
        s_bpre[G] = (int32_t)tot_b;
    }
    __syncthreads();
    const bool ok = !s_bad && (PART ? tot_r <= a.rows : tot_r == a.rows);
    return ok ? (int64_t)tot_b : -1;
}

// ---------------------------------------------------------------------------
// Shared-memory barriers
// ---------------------------------------------------------------------------

constexpr uint64_t SG_WAIT_NS = 4000000000ull; // an mbarrier wait gives up after 4 s

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Wait for the phase of the given parity to complete; false after SG_WAIT_NS
// of global time (the caller then records an error and stops).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity)
{
    if (mbar_try(bar, parity))
        return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try(bar, parity))
        if (global_ns() - t0 > SG_WAIT_NS)
            return false;
    return true;
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Pairs of kernels on one stream, the second launched with the programmatic
// serialisation attribute: the first lets it become resident once its own CTAs
// are, and the second waits for the first's results (its writes included) before
// it touches them or writes anything itself.
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_prerequisite() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Row-wise bf16 block-32 quantisation core
// ---------------------------------------------------------------------------

// Packed unsigned 16-bit max of two words.
__device__ __forceinline__ uint32_t vmax2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Block exponent for a scale mode fixed at compile time (block_k's rule).
template <int MODE>
__device__ __forceinline__ int block_kt(uint32_t A, uint32_t thr)
{
    if constexpr (MODE == MXFP4_SCALE_FLOOR) {
        return max((int)(A >> 23) - 129, -127);
    } else {
        const int k = (int)(A >> 23) - (int)(thr >> 23) + 1 - ((A & 0x7FFFFFu) < (thr & 0x7FFFFFu) ? 1 : 0);
        return max(k, -30);
    }
}

// Fast-path exponent range of the hardware convert core: 2^k and every code * 2^k are
// normal bf16 numbers (k >= -125), and the limit bits of lim16_of_k stay
// below 0x8000 (k <= 16).
__device__ __forceinline__ bool k_fast_bf(int k) { return (uint32_t)(k + 125) <= 141u; }

// ---- E2M1 rounding by the hardware convert ---------------------------------
// The convert rounds to nearest with ties to even; the codebook's rule sends
// ties up (away from zero). Multiplying y by (1 + 2^-20) first moves exact
// midpoints above themselves and nothing else across one: y is a bf16 value
// times 2^-k (8 significant bits), so a y below a midpoint lies at least one
// bf16 ulp (2^-8 relative) below it, and the one rounding of the product
// changes it by at most 2^-24 relative. The product is formed as
// x * (2^-k (1 + 2^-20)) + 0 in one fma: adding +0 turns -0 into +0 (the
// codebook's sign rule for zero inputs) and keeps the sign of every nonzero
// product, however small. Codes above 6 saturate to 6 in the convert, as in
// the codebook. Checked against the table path for every finite bf16 value
// and every fast-path k.

// 2^-k (1 + 2^-20) for a fast-path k (mantissa bit 3 set).
__device__ __forceinline__ float inv_nudged(int k) { return __uint_as_float((0x3F800000u - ((uint32_t)k << 23)) | 8u); }

// 2^k for a fast-path k.
__device__ __forceinline__ float pow2f_k(int k) { return __uint_as_float(0x3F800000u + ((uint32_t)k << 23)); }

// Nudged scaled values of both halves of a bf16 word.
__device__ __forceinline__ void nudged_pair(uint32_t w, float invn_lo, float invn_hi, float& ylo, float& yhi)
{
    asm("fma.rn.f32 %0, %1, %2, 0f00000000;" : "=f"(ylo) : "f"(__uint_as_float(w << 16)), "f"(invn_lo));
    asm("fma.rn.f32 %0, %1, %2, 0f00000000;" : "=f"(yhi) : "f"(__uint_as_float(w & 0xFFFF0000u)), "f"(invn_hi));
}

// E2M1 bytes of four words sharing one scale, as one 32-bit nibble word.
__device__ __forceinline__ uint32_t nibs4_cvt(const uint32_t* w, float invn)
{
    float y[8];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        nudged_pair(w[u], invn, invn, y[2 * u], y[2 * u + 1]);
    uint32_t nibs;
    asm("{\n\t.reg .b8 q0, q1, q2, q3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q3, %8, %7;\n\t"
        "mov.b32 %0, {q0, q1, q2, q3};\n\t}"
        : "=r"(nibs)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return nibs;
}

__device__ __forceinline__ void ld_nc_v8(const void* p, uint32_t* v)
{
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}

__device__ __forceinline__ void st_cs_v8(void* p, const uint32_t* v)
{
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// ---------------------------------------------------------------------------
// tcgen05 wrappers of the block-scaled GEMMs
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint64_t gm_smem_desc(uint32_t saddr, uint64_t layout, uint32_t sbo)
{
    // start address, leading byte offset 16 (unused by swizzled K-major
    // layouts), stride byte offset between 8-row groups, descriptor version 1
    // (sm_100), base offset 0, layout type in the top three bits
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) |
           ((uint64_t)1 << 46) | (layout << 61);
}

// The 512-byte scale atom (32 rows of 16 bytes, no swizzle) as the source of
// a tcgen05.cp 32x128b: core matrices of 8 rows x 16 bytes, 128 bytes apart.
__device__ __forceinline__ uint64_t gm_sf_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

template <int FMT>
__device__ __forceinline__ void gm_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t acc)
{
    if constexpr (FMT == MXFP4_ELEM_E2M1) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sfa_tmem), "r"(sfb_tmem)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sfa_tmem), "r"(sfb_tmem)
            : "memory");
    }
}

__device__ __forceinline__ void gm_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void gm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void gm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive fp32 accumulator columns of this thread's tensor-memory lane.
__device__ __forceinline__ void gm_ld32(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 2-D TMA load of a byte tile (box of 128 bytes x 128 rows, 128-byte
// swizzle); the inner coordinate is a multiple of 64 bytes.
__device__ __forceinline__ void gm_tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

struct DevInfo {
    int sms = 0;
};

inline std::mutex g_mu;

inline int device_sms()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return -1;
    static DevInfo info[64];
    std::lock_guard<std::mutex> lk(g_mu);
    if (dev < 0 || dev >= 64)
        return -1;
    if (info[dev].sms == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return -1;
        info[dev].sms = n;
    }
    return info[dev].sms;
}

// Resident CTAs per SM of `fn` launched with `threads` per CTA, cached per
// (device, kernel).
inline int occupancy(const void* fn, size_t smem, int threads = NTHREADS)
{
    struct Entry {
        const void* fn;
        int dev;
        size_t smem;
        int occ;
    };
    static Entry cache[512];
    static int n = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return -1;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        for (int i = 0; i < n; ++i)
            if (cache[i].fn == fn && cache[i].dev == dev && cache[i].smem == smem)
                return cache[i].occ;
    }
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, smem) != cudaSuccess)
        return -1;
    if (occ < 1)
        occ = 1;
    std::lock_guard<std::mutex> lk(g_mu);
    if (n < 512)
        cache[n++] = Entry{fn, dev, smem, occ};
    return occ;
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline float f32_of(uint32_t u)
{
    float f;
    memcpy(&f, &u, 4);
    return f;
}

inline uint32_t u32_of(float f)
{
    uint32_t u;
    memcpy(&u, &f, 4);
    return u;
}

// PAGE-mode scale_factor range of the vector path: every threshold T0 * 2^j it
// uses stays a normal fp32 number, and |x / 2^k| < 16 keeps floor(4|y|) inside
// the 64-entry lookup table.
inline bool page_fast_ok(float sf) { return sf >= 0x1p-64f && sf <= 11.0f; }

// T0 = the smallest fp32 a with fl(a / sf) >= C, C = 0x3FB504F4 (the first fp32
// above sqrt 2), found by stepping from fl(C * sf) one ulp at a time with IEEE
// fp32 host division (a -> fl(a / sf) is monotone).
inline uint32_t page_threshold(float sf)
{
    const float C = f32_of(0x3FB504F4u);
    volatile float a = C * sf;
    for (int i = 0; i < 64; ++i) {
        volatile float prev = nextafterf(a, 0.0f);
        volatile float q = prev / sf;
        if (!(q >= C))
            break;
        a = prev;
    }
    for (int i = 0; i < 64; ++i) {
        volatile float q = a / sf;
        if (q >= C)
            break;
        a = nextafterf(a, INFINITY);
    }
    return u32_of(a);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's driver entry point (the library
// does not link libcuda directly); nullptr when unavailable.
inline EncodeTiledFn encode_tiled()
{
    static EncodeTiledFn fn = nullptr;
    static bool tried = false;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!tried) {
        tried = true;
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        else
            (void)cudaGetLastError();
    }
    return fn;
}

// One 2-D tiled map: inner dimension d0 (elements of esz bytes), outer d1,
// row pitch bytes, box b0 x b1.
inline bool encode_2d(CUtensorMap* tm, CUtensorMapDataType dt, void* base, uint64_t d0, uint64_t d1, uint64_t pitch,
                      uint32_t b0, uint32_t b1, CUtensorMapSwizzle sw)
{
    EncodeTiledFn fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d0, (cuuint64_t)d1};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)b0, (cuuint32_t)b1};
    const cuuint32_t estr[2] = {1, 1};
    return fn(tm, dt, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mxfp4
