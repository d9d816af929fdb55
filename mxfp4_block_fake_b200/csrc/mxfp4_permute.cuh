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

__global__ void __launch_bounds__(NTHREADS) pad_scale_kernel(const DispatchArgs a) { pad_scale_rows(a); }

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
        for (int j = 0; j < a.k; ++j) {
            const uint32_t r = (uint32_t)a.rows[t * a.k + j];
            if (r >= a.y_rows)
                continue;
            const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
            float v[N];
            piece_load<ESZ, N>(a.y, (int64_t)r * a.ld_y + c, v);
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[i] = fmaf(w, v[i], acc[i]);
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

constexpr int CB_MAX_K = 32;

// grad_y[rows[t][j]] = w[t][j] grad[t], grad_w[t][j] = grad[t] . y[rows[t][j]].
// One CTA per token; the dot products are summed per thread, then over the
// warps' lanes and the warps, in a fixed order.
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
        const bool some = r < a.y_rows;
        const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
        float dot = 0.0f;
        if (some)
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
        for (int w = 0; w < NTHREADS / 32; ++w)
            v += s_dot[tid][w];
        a.grad_w[t * a.k + tid] = v;
    }
}

}  // namespace mxfp4
