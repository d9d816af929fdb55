// mxfp4_permute.cuh -- token rows to their experts' places and back (included
// by mxfp4_moe.cu; the definitions are in include/mxfp4.h, mxfp4_moe_dispatch,
// mxfp4_moe_combine and mxfp4_moe_combine_bwd).
//
// All of it moves memory. Each kernel walks the tokens, not the experts' rows:
// a token's row is read (and quantised) once and written to its k places, and
// the gradients of its k rows and k weights come from one read of its own
// gradient. A row index outside the buffers is skipped, so that no index list
// can make a kernel leave them.

namespace mxfp4 {

struct DispatchArgs {
    const void* x;
    const int32_t* rows;   // [tokens][k]: destination of each (token, slot); outside [0, out_rows): none
    void* y;               // [out_rows][ld_y], x's dtype
    uint8_t* codes;        // [out_rows][code bytes]
    uint8_t* scales;       // MMA layout of [out_rows][blocks]
    int64_t tokens, cols, ld, ld_y, out_rows;
    int64_t code_ld;       // bytes of a code row
    uint32_t* ws_scales;   // [tokens][block columns / 4] scale words, or NULL: scales are written directly
    int32_t* ws_pair;      // [out_rows]: the (token, slot) whose row this is, unless the rows say otherwise
    float sf;
    uint32_t thr;          // PAGE mode threshold (page_threshold)
    int32_t k, mode;
};

template <int ESZ>
__device__ __forceinline__ uint32_t mv_load(const void* p, int64_t i)
{
    if constexpr (ESZ == 2)
        return static_cast<const uint16_t*>(p)[i];
    else
        return static_cast<const uint32_t*>(p)[i];
}

// Plain rows, 16-byte vectors (VEC) or elements: one thread per (token, piece).
template <int ESZ, bool VEC>
__global__ void __launch_bounds__(NTHREADS) dispatch_values_kernel(const DispatchArgs a)
{
    constexpr int PER = VEC ? 16 / ESZ : 1;
    const uint32_t pieces = (uint32_t)(a.cols / PER);
    const int64_t total = a.tokens * pieces;
    for (int64_t u = (int64_t)blockIdx.x * NTHREADS + threadIdx.x; u < total; u += (int64_t)gridDim.x * NTHREADS) {
        const int64_t t = u / pieces;
        const int64_t c = (u - t * pieces) * PER;
        const int32_t* rp = a.rows + t * a.k;
        if constexpr (VEC) {
            const uint4 v = ld_stream(static_cast<const char*>(a.x) + (t * a.ld + c) * ESZ);
            for (int j = 0; j < a.k; ++j) {
                const uint32_t r = (uint32_t)rp[j];
                if (r < a.out_rows)
                    st_stream(static_cast<char*>(a.y) + ((int64_t)r * a.ld_y + c) * ESZ, v);
            }
        } else {
            const uint32_t v = mv_load<ESZ>(a.x, t * a.ld + c);
            for (int j = 0; j < a.k; ++j) {
                const uint32_t r = (uint32_t)rp[j];
                if (r < a.out_rows) {
                    if constexpr (ESZ == 2)
                        static_cast<uint16_t*>(a.y)[(int64_t)r * a.ld_y + c] = (uint16_t)v;
                    else
                        static_cast<uint32_t*>(a.y)[(int64_t)r * a.ld_y + c] = v;
                }
            }
        }
    }
}

// Zeros in the scale rows behind the last one (the rest of the last atom row).
__device__ __forceinline__ void pad_scale_rows(const DispatchArgs& a)
{
    const int64_t nblk = (a.cols + 31) / 32, npad = (nblk + 3) & ~(int64_t)3;
    const int64_t last = (a.out_rows + 127) & ~(int64_t)127;
    const int64_t n = (last - a.out_rows) * npad;
    for (int64_t i = (int64_t)blockIdx.x * NTHREADS + threadIdx.x; i < n; i += (int64_t)gridDim.x * NTHREADS)
        a.scales[srow_off_mma(a.out_rows + i / npad, i % npad, nblk)] = 0;
}

// Quantised rows, any width and alignment: one thread per (token, block of
// 32). The arithmetic is the row-wise quantiser's (block_params, qdq_elem and
// their E4M3 forms); the padding of a row's last scale atom is written as 0.
template <int ESZ, int FMT>
__global__ void __launch_bounds__(NTHREADS) dispatch_quant_kernel(const DispatchArgs a)
{
    const uint32_t nblk = (uint32_t)((a.cols + 31) / 32), npad = (nblk + 3) & ~3u;
    const int64_t total = a.tokens * npad;
    for (int64_t u = (int64_t)blockIdx.x * NTHREADS + threadIdx.x; u < total; u += (int64_t)gridDim.x * NTHREADS) {
        const int64_t t = u / npad;
        const uint32_t b = (uint32_t)(u - t * npad);
        const int32_t* rp = a.rows + t * a.k;
        uint32_t e8 = 0;
        uint8_t code[32];
        int bytes = 0;
        if (b < nblk) {
            const int n = (int)min((int64_t)32, a.cols - (int64_t)b * 32);
            const int64_t x0 = t * a.ld + (int64_t)b * 32;
            uint32_t A = 0;
            for (int i = 0; i < n; ++i) {
                const uint32_t v = mv_load<ESZ>(a.x, x0 + i) << (ESZ == 2 ? 16 : 0);
                A = max(A, v & 0x7FFFFFFFu);
            }
            const BP p = FMT == MXFP4_ELEM_E4M3 ? block_params8(A) : block_params(A, a.mode, a.sf);
            e8 = p.e8;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                uint32_t q = 0, sat;
                if (i < n && !p.nanm) {
                    const uint32_t v = mv_load<ESZ>(a.x, x0 + i) << (ESZ == 2 ? 16 : 0);
                    if constexpr (FMT == MXFP4_ELEM_E4M3)
                        (void)qdq8_elem(v, p, q, sat);
                    else
                        (void)qdq_elem(v, p, q, sat);
                }
                if constexpr (FMT == MXFP4_ELEM_E4M3)
                    code[i] = (uint8_t)q;
                else if (i & 1)
                    code[i >> 1] |= (uint8_t)(q << 4);
                else
                    code[i >> 1] = (uint8_t)q;
            }
            bytes = FMT == MXFP4_ELEM_E4M3 ? n : (n + 1) / 2;
        }
        for (int j = 0; j < a.k; ++j) {
            const uint32_t r = (uint32_t)rp[j];
            if (r >= a.out_rows)
                continue;
            uint8_t* cp = a.codes + (int64_t)r * a.code_ld + (int64_t)b * (FMT == MXFP4_ELEM_E4M3 ? 32 : 16);
#pragma unroll
            for (int i = 0; i < (FMT == MXFP4_ELEM_E4M3 ? 32 : 16); ++i)
                if (i < bytes)
                    cp[i] = code[i];
            a.scales[srow_off_mma(r, b, nblk)] = (uint8_t)e8;
        }
    }
    pad_scale_rows(a);
}

// A block of 32 fp32 values (bits) -> its codes: E2M1 nibbles of 8 elements
// per word (4 words), E4M3 bytes of 4 per word (8 words). E2M1: the hardware
// convert rounds to nearest with ties to even, the codebook sends ties up; a
// tie is one of the fp32 values with at most two fraction bits, so those get
// one more in their last place first, which moves codes themselves nowhere
// (zeros and what lies above 8, infinities among it, are left alone). The
// quotient y is rounded before 0 is added, so that every -0, one that
// underflowed too, becomes +0 (the codebook's sign rule).
template <int FMT, int N>
__device__ __forceinline__ void quant_block(const uint32_t (&x)[32], const BP& p, uint32_t (&code)[N])
{
    if constexpr (FMT == MXFP4_ELEM_E4M3) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = __fmul_rn(__uint_as_float(x[4 * i + j]), p.inv);
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
            code[i] = p.nanm ? 0u : (uint32_t)lo | (uint32_t)hi << 16;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(x[8 * i + j]), p.inv), 0.0f));
                const bool tie = (b & 0x1FFFFFu) == 0u && (b & 0x7FFFFFFFu) - 1u < 0x40FFFFFFu;
                y[j] = __uint_as_float(b | (tie ? 1u : 0u));
            }
            uint32_t w;
            asm("{\n\t.reg .b8 q0, q1, q2, q3;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 q0, %2, %1;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 q1, %4, %3;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 q2, %6, %5;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 q3, %8, %7;\n\t"
                "mov.b32 %0, {q0, q1, q2, q3};\n\t}"
                : "=r"(w)
                : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
            code[i] = p.nanm ? 0u : w;
        }
    }
}

// Quantised rows of whole blocks (cols % 32 == 0, 32-byte aligned rows, fewer
// than 2^31 blocks): one thread per (token, block), its 32 values by 32-byte
// loads, its codes to each of the k rows by one 16- or 32-byte store, and the
// scale bytes of four neighbouring blocks (the four lanes of a quad, a row's
// whole atom entry) as one word, the k rows shared out among the quad's lanes.
// Bound by memory: it reads x once and writes k rows of codes. bf16 blocks in
// the usual exponent range take the streaming quantiser's convert (nibs4_cvt).
template <int ESZ, int FMT>
__global__ void __launch_bounds__(NTHREADS) dispatch_stream_kernel(const DispatchArgs a)
{
    constexpr int NC = FMT == MXFP4_ELEM_E4M3 ? 8 : 4;  // code words of a block
    const uint32_t nblk = (uint32_t)(a.cols / 32), npad = (nblk + 3) & ~3u;
    constexpr int NW = 8 * ESZ;                         // words of a block
    constexpr bool AHEAD = ESZ == 2;                    // fp32: 32 more registers would halve the resident warps
    const uint32_t total = (uint32_t)a.tokens * npad, stride = gridDim.x * NTHREADS;
    auto load = [&](uint32_t v, uint32_t (&w)[NW]) {
        const uint32_t t = v / npad, b = v - t * npad;
        if (b < nblk) {
            const char* xp = static_cast<const char*>(a.x) + ((int64_t)t * a.ld + 32 * b) * ESZ;
#pragma unroll
            for (int i = 0; i < NW / 8; ++i)
                ld_nc_v8(xp + 32 * i, w + 8 * i);
        }
    };
    let_dependents_start();
    uint32_t w[NW];
    uint32_t u = blockIdx.x * NTHREADS + threadIdx.x;
    if (u < total)
        load(u, w);
    for (; u < total; u += stride) {
        const uint32_t t = u / npad, b = u - t * npad;
        const unsigned quad = 0xFu << (threadIdx.x & 28);
        const int32_t* rp = a.rows + (int64_t)t * a.k;
        uint32_t wn[AHEAD ? NW : 1];
        const bool more = u + stride < total;
        if constexpr (AHEAD) {
            if (more)
                load(u + stride, wn);  // the next block's loads are in flight while this one is worked on
        }
        uint32_t code[NC], e8 = 0;
        if (b < nblk) {
            if constexpr (ESZ == 2) {
                uint32_t m2 = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    m2 = vmax2(m2, w[i] & 0x7FFF7FFFu);
                const uint32_t A = max(m2 & 0xFFFFu, m2 >> 16) << 16;
                bool done = false;
                if constexpr (FMT == MXFP4_ELEM_E2M1) {
                    if (a.thr || a.mode == MXFP4_SCALE_FLOOR) {
                        const int k = a.mode == MXFP4_SCALE_FLOOR ? block_kt<MXFP4_SCALE_FLOOR>(A, 0u) : block_kt<MXFP4_SCALE_PAGE>(A, a.thr);
                        if (k_fast_bf(k) && A < 0x7F800000u) {
                            const float invn = inv_nudged(k);
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                code[c] = nibs4_cvt(w + 4 * c, invn);
                            e8 = (uint32_t)(k + 127);
                            done = true;
                        }
                    }
                }
                if (!done) {
                    uint32_t x[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[2 * i] = w[i] << 16;
                        x[2 * i + 1] = w[i] & 0xFFFF0000u;
                    }
                    const BP p = FMT == MXFP4_ELEM_E4M3 ? block_params8(A) : block_params(A, a.mode, a.sf);
                    e8 = p.e8;
                    quant_block<FMT>(x, p, code);
                }
            } else {
                uint32_t A = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    A = max(A, w[i] & 0x7FFFFFFFu);
                const BP p = FMT == MXFP4_ELEM_E4M3 ? block_params8(A) : block_params(A, a.mode, a.sf);
                e8 = p.e8;
                quant_block<FMT>(w, p, code);
            }
        }
        uint32_t word = e8 << (8 * (b & 3));
        word |= __shfl_xor_sync(quad, word, 1);
        word |= __shfl_xor_sync(quad, word, 2);
        for (int j0 = 0; j0 < a.k; j0 += 8) {
            uint32_t r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                r[j] = j0 + j < a.k ? (uint32_t)rp[j0 + j] : 0xFFFFFFFFu;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (r[j] < a.out_rows) {
                    if (b < nblk) {
                        uint8_t* cp = a.codes + (int64_t)r[j] * a.code_ld + (int64_t)b * (4 * NC);
                        if constexpr (NC == 8)
                            st_cs_v8(cp, code);
                        else
                            st_stream(cp, make_uint4(code[0], code[1], code[2], code[3]));
                    }
                    if (a.ws_pair) {
                        if (b == 0)
                            a.ws_pair[r[j]] = (int32_t)(t * a.k) + j0 + j;
                    } else if ((j & 3) == (int)(threadIdx.x & 3)) {
                        *reinterpret_cast<uint32_t*>(a.scales + srow_off_mma(r[j], b & ~3u, nblk)) = word;
                    }
                }
        }
        if (a.ws_scales && (b & 3) == 0)
            a.ws_scales[u >> 2] = word;
        if constexpr (AHEAD) {
            if (more)
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    w[i] = wn[i];
        } else if (more) {
            load(u + stride, w);
        }
    }
    if (!a.ws_scales)
        pad_scale_rows(a);
}

// The scale words of dispatch_stream_kernel's workspace into the atoms. Written
// directly they are 4-byte stores, eight of which (of rows far apart in the
// tokens' order) make a sector: 88 us for the whole dispatch of 8192 x 7168 to
// 8 experts each, against 59.5 without the scales' stores. Here a CTA takes the
// 128 rows of an atom row and SG_WORDS block columns of four, reads each row's
// words as they lie in its token's, and writes whole atoms. A row's pair is
// taken only if the pair's row is this one, so the list needs no initial state;
// rows that no pair names stay as they were, rows behind out_rows are zeroed.
constexpr int SG_WORDS = 32;

__global__ void __launch_bounds__(NTHREADS) dispatch_scales_kernel(const DispatchArgs a)
{
    __shared__ uint32_t s_word[128][SG_WORDS + 1];
    __shared__ int32_t s_token[128];   // a row's token; -1: no pair names the row, -2: behind the last row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t ncb = ((a.cols + 31) / 32 + 3) / 4, pairs = a.tokens * a.k;
    const int64_t row0 = (int64_t)blockIdx.x * 128, c0 = (int64_t)blockIdx.y * SG_WORDS;
    wait_for_prerequisite();
    if (threadIdx.x < 128) {
        const int64_t r = row0 + threadIdx.x;
        int32_t t = -2;
        if (r < a.out_rows) {
            const uint32_t p = (uint32_t)a.ws_pair[r];
            t = p < pairs && a.rows[p] == r ? (int32_t)(p / (uint32_t)a.k) : -1;
        }
        s_token[threadIdx.x] = t;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int32_t t = s_token[16 * warp + i];
        s_word[16 * warp + i][lane] = t >= 0 && c0 + lane < ncb ? a.ws_scales[(int64_t)t * ncb + c0 + lane] : 0u;
    }
    __syncthreads();
    // word q of an atom is row 32 (q % 4) + q / 4
    const int q = threadIdx.x & 127, i = 32 * (q & 3) + (q >> 2);
    if (s_token[i] != -1)
        for (int c = threadIdx.x >> 7; c < SG_WORDS && c0 + c < ncb; c += NTHREADS / 128)
            reinterpret_cast<uint32_t*>(a.scales)[((int64_t)blockIdx.x * ncb + c0 + c) * 128 + q] = s_word[i][c];
}

struct CombineArgs {
    const void* y;          // [y_rows][ld_y]
    const int32_t* rows;    // [tokens][k]
    const float* weights;   // [tokens][k], or NULL for ones
    const void* residual;   // [tokens][ld_res], or NULL
    void* out;              // [tokens][ld_out]
    int64_t tokens, cols, ld_y, ld_res, ld_out, y_rows;
    int32_t k;
    // backward: grad [tokens][ld_out] in, grad_y [y_rows][ld_gy] and grad_w [tokens][k] out
    const void* grad;
    void* grad_y;
    float* grad_w;
    int64_t ld_gy;
};

// Elements of a piece as fp32, and back (one rounding).
template <int ESZ, int N>
__device__ __forceinline__ void piece_load(const void* p, int64_t i, float (&v)[N])
{
    if constexpr (N * ESZ == 16) {
        const uint4 w = ld_stream(static_cast<const char*>(p) + i * ESZ);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = ESZ == 4 ? __uint_as_float(u[j]) : __uint_as_float(j & 1 ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = __uint_as_float(mv_load<ESZ>(p, i + j) << (ESZ == 2 ? 16 : 0));
    }
}

template <int ESZ, int N>
__device__ __forceinline__ void piece_store(void* p, int64_t i, const float (&v)[N])
{
    if constexpr (N * ESZ == 16) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            u[j] = ESZ == 4 ? __float_as_uint(v[j]) : bf16x2(v[(2 * j) % N], v[(2 * j + 1) % N]);
        st_stream(static_cast<char*>(p) + i * ESZ, make_uint4(u[0], u[1], u[2], u[3]));
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if constexpr (ESZ == 2)
                static_cast<uint16_t*>(p)[i + j] = (uint16_t)f32_to_bf16(v[j]);
            else
                static_cast<float*>(p)[i + j] = v[j];
    }
}

// out[t] = residual[t] + sum_j w[t][j] y[rows[t][j]], summed in fp32 in the
// slots' order and rounded once. One thread per (token, piece).
template <int ESZ, bool VEC>
__global__ void __launch_bounds__(NTHREADS) combine_kernel(const CombineArgs a)
{
    constexpr int N = VEC ? 16 / ESZ : 1;
    const uint32_t pieces = (uint32_t)(a.cols / N);
    const int64_t total = a.tokens * pieces;
    for (int64_t u = (int64_t)blockIdx.x * NTHREADS + threadIdx.x; u < total; u += (int64_t)gridDim.x * NTHREADS) {
        const int64_t t = u / pieces;
        const int64_t c = (u - t * pieces) * N;
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            acc[i] = 0.0f;
        // four rows' loads in flight at a time
        for (int j0 = 0; j0 < a.k; j0 += 4) {
            float v[4][N], w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t r = j0 + j < a.k ? (uint32_t)a.rows[t * a.k + j0 + j] : 0xFFFFFFFFu;
                const bool some = r < a.y_rows;
                w[j] = some ? (a.weights ? a.weights[t * a.k + j0 + j] : 1.0f) : 0.0f;
                if (some) {
                    piece_load<ESZ, N>(a.y, (int64_t)r * a.ld_y + c, v[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        v[j][i] = 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[i] = fmaf(w[j], v[j][i], acc[i]);
        }
        if (a.residual) {
            float v[N];
            piece_load<ESZ, N>(a.residual, t * a.ld_res + c, v);
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[i] += v[i];
        }
        piece_store<ESZ, N>(a.out, t * a.ld_out + c, acc);
    }
}

// grad_y[rows[t][j]] = w[t][j] grad[t], grad_w[t][j] = grad[t] . y[rows[t][j]].
// One CTA per token, which goes through its rows one by one (its gradient is
// read again from the caches for each). Bound by memory; what counts is many
// resident warps: holding the gradient and the next row in registers (two CTAs
// per SM instead of six) took 117 us where this takes 80, a warp per row 143
// (4099 tokens of 6 x 4096, bf16). The dot products are summed per thread, over
// the lanes and over the warps, in order.
constexpr int CB_MAX_K = 32;

template <int ESZ, bool VEC>
__global__ void __launch_bounds__(NTHREADS) combine_bwd_kernel(const CombineArgs a)
{
    constexpr int N = VEC ? 16 / ESZ : 1;
    __shared__ float s_dot[CB_MAX_K][NTHREADS / 32];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t pieces = a.cols / N;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t r = (uint32_t)a.rows[t * a.k + j];
        const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
        float dot = 0.0f;
        if (r < a.y_rows)
            for (int64_t p = tid; p < pieces; p += NTHREADS) {
                float g[N], v[N];
                piece_load<ESZ, N>(a.grad, t * a.ld_out + p * N, g);
                if (a.grad_w) {
                    piece_load<ESZ, N>(a.y, (int64_t)r * a.ld_y + p * N, v);
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        dot = fmaf(g[i], v[i], dot);
                }
                if (a.grad_y) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        g[i] *= w;
                    piece_store<ESZ, N>(a.grad_y, (int64_t)r * a.ld_gy + p * N, g);
                }
            }
        dot = warp_sum(dot);
        if (lane == 0)
            s_dot[j][warp] = dot;
    }
    __syncthreads();
    if (a.grad_w && tid < a.k) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < NTHREADS / 32; ++w)
            v += s_dot[tid][w];
        a.grad_w[t * a.k + tid] = v;
    }
}

}  // namespace mxfp4
