// mxfp4_moe.cu -- the mixture-of-experts operators of libmxfp4.so: routing,
// dispatch and combine, and the grouped block-scaled linear (include/mxfp4.h).
#include "mxfp4_common.cuh"

namespace mxfp4 {

// fp32 -> bf16, nearest even.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t f32_to_bf16(float v) { return bf16x2(v, 0.0f) & 0xFFFFu; }

}  // namespace mxfp4

#include "mxfp4_route.cuh"
#include "mxfp4_permute.cuh"
#include "mxfp4_linear.cuh"
#include "mxfp4_linear2.cuh"

namespace mxfp4 {

static mxfp4_status launched(cudaError_t e) { return e == cudaSuccess ? MXFP4_OK : MXFP4_ECUDA; }

// Lets `fn` be launched with `smem` bytes of dynamic shared memory; asked of the
// runtime once per (kernel, device) and size above the last. Without asking, 48 KB
// are open to a kernel's static and dynamic shared memory together (the static part
// starts at 1 KB; kernels with a large dynamic part here have at most 9 KB).
static bool allow_smem(const void* fn, size_t smem)
{
    if (smem <= 32 * 1024)
        return true;
    struct Entry {
        const void* fn;
        int dev;
        size_t smem;
    };
    static Entry cache[128];
    static int n = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return false;
    std::lock_guard<std::mutex> lk(g_mu);
    int i = 0;
    while (i < n && !(cache[i].fn == fn && cache[i].dev == dev))
        ++i;
    if (i < n && cache[i].smem >= smem)
        return true;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return false;
    if (i < 128) {
        cache[i] = Entry{fn, dev, smem};
        n = i < n ? n : i + 1;
    }
    return true;
}

template <typename A>
static mxfp4_status launch1(const void* fn, int64_t grid, int threads, size_t smem, const A& arg, cudaStream_t s)
{
    if (!allow_smem(fn, smem))
        return MXFP4_ECUDA;
    A a = arg;
    void* args[] = {&a};
    return launched(cudaLaunchKernel(fn, dim3((unsigned)grid), dim3((unsigned)threads), args, smem, s));
}

// The second of a pair of kernels (wait_for_prerequisite): its launch and its start
// overlap the first's end. The first must be the launch before it on the stream.
static mxfp4_status launch_after(const void* fn, dim3 grid, int threads, size_t smem, void** args, cudaStream_t s)
{
    if (!allow_smem(fn, smem))
        return MXFP4_ECUDA;
    cudaLaunchAttribute at;
    memset(&at, 0, sizeof(at));
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelExC(&cfg, fn, args));
}

// Grid of a grid-stride kernel over `units` threads' work.
static int64_t stride_grid(const void* fn, int64_t units)
{
    const int sms = device_sms(), occ = occupancy(fn, 0);
    if (sms <= 0 || occ <= 0)
        return -1;
    const int64_t need = (units + NTHREADS - 1) / NTHREADS, most = (int64_t)sms * occ;
    return need < most ? (need < 1 ? 1 : need) : most;
}

template <typename A>
static mxfp4_status launch_stride(const void* fn, int64_t units, const A& a, cudaStream_t s)
{
    const int64_t grid = stride_grid(fn, units);
    return grid < 0 ? MXFP4_ECUDA : launch1(fn, grid, NTHREADS, 0, a, s);
}

// ---- routing ---------------------------------------------------------------

static int64_t route_chunks(int64_t tokens) { return tokens <= RT_CHUNK ? 1 : (tokens + RT_CHUNK - 1) / RT_CHUNK; }

static mxfp4_status route_args(const mxfp4_moe_route_args* A, RouteArgs* r)
{
    if (!A)
        return MXFP4_EINVAL;
    if (A->dtype != MXFP4_F32 && A->dtype != MXFP4_BF16)
        return MXFP4_EINVAL;
    if (A->tokens < 0 || A->experts < 1 || A->k < 1 || A->k > A->experts || A->ld < A->experts)
        return MXFP4_EINVAL;
    if (A->score != MXFP4_SCORE_SOFTMAX && A->score != MXFP4_SCORE_SIGMOID)
        return MXFP4_EINVAL;
    if (!(A->scale == A->scale) || isinf(A->scale))
        return MXFP4_EINVAL;
    if (A->experts > RT_MAX_EXPERTS || A->k > RT_MAX_K || A->tokens > INT32_MAX / A->k)
        return MXFP4_EUNSUPPORTED;
    memset(r, 0, sizeof(*r));
    r->logits = A->logits;
    r->tokens = A->tokens;
    r->ld = A->ld;
    r->experts = (int32_t)A->experts;
    r->k = A->k;
    r->sigmoid = A->score == MXFP4_SCORE_SIGMOID;
    r->renorm = A->renormalize != 0;
    r->bf16 = A->dtype == MXFP4_BF16;
    r->scale = A->scale;
    r->experts_out = A->chosen;
    return MXFP4_OK;
}

template <int NV, int LW>
static const void* route_fn(bool bf16, bool sigmoid)
{
    if (sigmoid)
        return bf16 ? (const void*)route_kernel<NV, true, true, LW> : (const void*)route_kernel<NV, false, true, LW>;
    return bf16 ? (const void*)route_kernel<NV, true, false, LW> : (const void*)route_kernel<NV, false, false, LW>;
}

static mxfp4_status run_route(const mxfp4_moe_route_args* A, cudaStream_t s)
{
    RouteArgs r;
    const mxfp4_status st = route_args(A, &r);
    if (st != MXFP4_OK)
        return st;
    if (A->num_groups < 1 || A->experts % A->num_groups != 0 || A->topk_groups < 1 || A->topk_groups > A->num_groups)
        return MXFP4_EINVAL;
    if (A->group_score != MXFP4_GROUP_BEST && A->group_score != MXFP4_GROUP_TOP2)
        return MXFP4_EINVAL;
    if (A->k > A->topk_groups * (A->experts / A->num_groups))
        return MXFP4_EINVAL;
    if (A->num_groups > RT_MAX_GROUPS)
        return MXFP4_EUNSUPPORTED;
    if (!A->counts || (A->tokens > 0 && (!A->logits || !A->weights || !A->chosen || !A->rows || !A->slots)))
        return MXFP4_EINVAL;
    const size_t esz = A->dtype == MXFP4_BF16 ? 2 : 4;
    if (!aligned(A->logits, esz) || !aligned(A->bias, 4) || !aligned(A->weights, 4) || !aligned(A->chosen, 4) ||
        !aligned(A->rows, 4) || !aligned(A->slots, 4) || !aligned(A->counts, 8) || !aligned(A->workspace, 16))
        return MXFP4_EINVAL;
    const int64_t need = mxfp4_moe_route_workspace(A->tokens, A->experts);
    if (need > 0 && (!A->workspace || A->workspace_bytes < need))
        return MXFP4_EINVAL;
    r.bias = A->bias;
    r.token_mask = A->token_mask;
    r.weights = A->weights;
    r.rows = A->rows;
    r.slots = A->slots;
    r.counts = A->counts;
    r.ws = static_cast<int32_t*>(A->workspace);
    r.groups = A->num_groups;
    r.topk_groups = A->topk_groups;
    r.top2 = A->group_score == MXFP4_GROUP_TOP2;
    r.chunks = (int32_t)route_chunks(A->tokens);
    const size_t smem = (size_t)RT_WARPS * r.experts * 8 + (size_t)r.experts * 8 + (size_t)RT_CHUNK * r.k * 2;
    // two tokens a warp where sixteen lanes hold eight experts each, the choices
    // and the groups (65536 tokens: 128 experts, k = 8 67 against 77 us with one
    // token, 64 experts, k = 6 53 / 64; with 256 experts, sixteen a lane, 133 / 101)
    const bool half = r.experts <= 128 && r.k < 16 && r.groups <= 16;
    int nv = half ? 4 : 1;  // experts per lane
    while ((half ? 16 : 32) * nv < r.experts)
        nv *= 2;
    r.per = r.experts / r.groups;
    r.per_magic = r.per == 1 ? 0u : (uint32_t)((0x100000000ull + r.per - 1) / r.per);
    r.lanes = r.per % nv == 0 && ((r.per / nv) & (r.per / nv - 1)) == 0 ? r.per / nv : 0;
    r.vec = r.experts % nv == 0 && aligned(A->logits, 16) && (A->ld * (int64_t)esz) % 16 == 0;
    const bool b = r.bf16, g = r.sigmoid;
    const void* fn = half ? (nv == 4 ? route_fn<4, 16>(b, g) : route_fn<8, 16>(b, g))
                     : nv == 1 ? route_fn<1, 32>(b, g) : nv == 2 ? route_fn<2, 32>(b, g) : nv == 4 ? route_fn<4, 32>(b, g)
                     : nv == 8 ? route_fn<8, 32>(b, g) : nv == 16 ? route_fn<16, 32>(b, g) : route_fn<32, 32>(b, g);
    mxfp4_status e = launch1(fn, r.chunks, RT_THREADS, smem, r, s);
    if (e != MXFP4_OK || r.chunks == 1)
        return e;
    void* args[] = {&r};
    // every CTA reading all chunks' counts costs chunks^2 * experts words: up to
    // 2^24 of them (about 3 us over the GPU) are cheaper than the scan's launch
    if ((int64_t)r.chunks * r.chunks * r.experts <= (int64_t)1 << 24)
        return launch_after((const void*)route_place_kernel<true>, dim3((unsigned)r.chunks), RT_THREADS, 0, args, s);
    e = launch_after((const void*)route_scan_kernel, dim3((unsigned)((r.experts + 31) / 32)), 1024, 0, args, s);
    if (e == MXFP4_OK)
        e = launch_after((const void*)route_place_kernel<false>, dim3((unsigned)r.chunks), RT_THREADS, 0, args, s);
    return e;
}

static mxfp4_status run_route_bwd(const mxfp4_moe_route_args* A, cudaStream_t s)
{
    RouteBwdArgs b;
    const mxfp4_status st = route_args(A, &b.r);
    if (st != MXFP4_OK)
        return st;
    if (A->ld_grad < A->experts)
        return MXFP4_EINVAL;
    if (A->tokens == 0)
        return MXFP4_OK;
    const size_t esz = A->dtype == MXFP4_BF16 ? 2 : 4;
    if (!A->logits || !A->chosen || !A->grad_weights || !A->grad_logits || !aligned(A->logits, esz) ||
        !aligned(A->chosen, 4) || !aligned(A->grad_weights, 4) || !aligned(A->grad_logits, esz))
        return MXFP4_EINVAL;
    b.grad_w = A->grad_weights;
    b.grad_logits = A->grad_logits;
    b.ld_g = A->ld_grad;
    return launch1((const void*)route_bwd_kernel, (A->tokens + RT_WARPS - 1) / RT_WARPS, RT_THREADS,
                   (size_t)RT_WARPS * A->experts * 4, b, s);
}

// ---- dispatch and combine --------------------------------------------------

static mxfp4_status check_move(const mxfp4_moe_move_args* A)
{
    if (!A)
        return MXFP4_EINVAL;
    if (A->dtype != MXFP4_F32 && A->dtype != MXFP4_BF16)
        return MXFP4_EINVAL;
    if (A->tokens < 0 || A->cols < 0 || A->row_count < 0 || A->k < 1)
        return MXFP4_EINVAL;
    if (A->k > MXFP4_MOE_MAX_K || A->tokens > INT32_MAX / A->k || A->row_count > INT32_MAX || A->cols > INT32_MAX)
        return MXFP4_EUNSUPPORTED;
    if (A->tokens > 0 && (!A->rows || !aligned(A->rows, 4)))
        return MXFP4_EINVAL;
    return MXFP4_OK;
}

static size_t esize(const mxfp4_moe_move_args* A) { return A->dtype == MXFP4_BF16 ? 2 : 4; }

// Whether rows of this pitch from this base are whole 16-byte vectors.
static bool vec_rows(const void* p, int64_t ld, size_t esz) { return aligned(p, 16) && (ld * (int64_t)esz) % 16 == 0; }

static mxfp4_status run_dispatch(const mxfp4_moe_move_args* A, cudaStream_t s)
{
    mxfp4_status st = check_move(A);
    if (st != MXFP4_OK)
        return st;
    const size_t esz = esize(A);
    const bool e4 = A->elem_format == MXFP4_ELEM_E4M3;
    if (A->ld_tokens < A->cols || (A->values && A->ld_rows < A->cols))
        return MXFP4_EINVAL;
    if (!A->values && !A->codes)  // (outputs without an element may have no address)
        return A->row_count == 0 || A->cols == 0 ? MXFP4_OK : MXFP4_EINVAL;
    if (A->codes) {
        if (!A->scales || (A->elem_format != MXFP4_ELEM_E2M1 && !e4))
            return MXFP4_EINVAL;
        if (A->scale_mode != MXFP4_SCALE_PAGE && A->scale_mode != MXFP4_SCALE_FLOOR)
            return MXFP4_EINVAL;
        if (!(A->scale_factor > 0.0f) || isinf(A->scale_factor))
            return MXFP4_EINVAL;
        if (e4 && A->scale_mode != MXFP4_SCALE_FLOOR)
            return MXFP4_EUNSUPPORTED;
    }
    if (A->cols == 0 || (A->tokens > 0 && A->row_count > 0 && (!A->x || !aligned(A->x, esz) || !aligned(A->values, esz) || !aligned(A->workspace, 4))))
        return A->cols == 0 ? MXFP4_OK : MXFP4_EINVAL;
    DispatchArgs a;
    memset(&a, 0, sizeof(a));
    a.x = A->x;
    a.rows = A->rows;
    a.y = A->values;
    a.codes = A->codes;
    a.scales = A->scales;
    a.tokens = A->tokens;
    a.cols = A->cols;
    a.ld = A->ld_tokens;
    a.ld_y = A->ld_rows;
    a.out_rows = A->row_count;
    a.code_ld = e4 ? A->cols : (A->cols + 1) / 2;
    a.sf = A->scale_factor;
    a.k = A->k;
    a.mode = A->scale_mode;
    const bool work = A->tokens > 0 && A->row_count > 0;
    if (A->values && work) {
        const bool vec = vec_rows(A->x, A->ld_tokens, esz) && vec_rows(A->values, A->ld_rows, esz) &&
                         (A->cols * esz) % 16 == 0;
        const void* fn = esz == 2 ? (vec ? (const void*)dispatch_values_kernel<2, true> : (const void*)dispatch_values_kernel<2, false>)
                                  : (vec ? (const void*)dispatch_values_kernel<4, true> : (const void*)dispatch_values_kernel<4, false>);
        st = launch_stride(fn, A->tokens * (vec ? A->cols * (int64_t)esz / 16 : A->cols), a, s);
    }
    if (A->codes && st == MXFP4_OK) {
        const int64_t npad = ((A->cols + 31) / 32 + 3) & ~(int64_t)3;
        const bool stream = A->cols % 32 == 0 && aligned(A->x, 32) && (A->ld_tokens * (int64_t)esz) % 32 == 0 &&
                            aligned(A->codes, 32) && aligned(A->scales, 4) && A->tokens * npad < INT32_MAX;
        a.thr = !e4 && A->scale_mode == MXFP4_SCALE_PAGE && page_fast_ok(A->scale_factor) ? page_threshold(A->scale_factor) : 0u;
        const void* fn = stream ? (esz == 2 ? (e4 ? (const void*)dispatch_stream_kernel<2, MXFP4_ELEM_E4M3> : (const void*)dispatch_stream_kernel<2, MXFP4_ELEM_E2M1>)
                                            : (e4 ? (const void*)dispatch_stream_kernel<4, MXFP4_ELEM_E4M3> : (const void*)dispatch_stream_kernel<4, MXFP4_ELEM_E2M1>))
                       : esz == 2 ? (e4 ? (const void*)dispatch_quant_kernel<2, MXFP4_ELEM_E4M3> : (const void*)dispatch_quant_kernel<2, MXFP4_ELEM_E2M1>)
                                  : (e4 ? (const void*)dispatch_quant_kernel<4, MXFP4_ELEM_E4M3> : (const void*)dispatch_quant_kernel<4, MXFP4_ELEM_E2M1>);
        const int64_t pad = A->row_count % 128 != 0 ? (128 - A->row_count % 128) * npad : 0;
        const int64_t units = work ? A->tokens * npad : 0;
        if (!work)
            a.tokens = 0;
        const int64_t ws = mxfp4_moe_dispatch_workspace(A->tokens, A->k, A->cols, A->row_count);
        const bool staged = stream && work && ws > 0 && A->workspace && A->workspace_bytes >= ws;
        if (staged) {
            a.ws_scales = static_cast<uint32_t*>(A->workspace);
            a.ws_pair = reinterpret_cast<int32_t*>(a.ws_scales + A->tokens * (npad / 4));
        }
        if (units > 0 || pad > 0)
            st = launch_stride(fn, units > pad ? units : pad, a, s);
        if (st == MXFP4_OK && staged) {
            DispatchArgs arg = a;
            void* args[] = {&arg};
            const dim3 grid((unsigned)((A->row_count + 127) / 128), (unsigned)((npad / 4 + SG_WORDS - 1) / SG_WORDS));
            st = launch_after((const void*)dispatch_scales_kernel, grid, NTHREADS, 0, args, s);
        }
    }
    return st;
}

static void combine_args(const mxfp4_moe_move_args* A, CombineArgs* a)
{
    memset(a, 0, sizeof(*a));
    a->y = A->y;
    a->rows = A->rows;
    a->weights = A->weights;
    a->residual = A->residual;
    a->out = A->out;
    a->tokens = A->tokens;
    a->cols = A->cols;
    a->ld_y = A->ld_rows;
    a->ld_res = A->ld_tokens;
    a->ld_out = A->ld_out;
    a->y_rows = A->row_count;
    a->k = A->k;
    a->grad = A->grad_out;
    a->grad_y = A->grad_rows;
    a->grad_w = A->grad_weights;
    a->ld_gy = A->ld_grad_rows;
}

static mxfp4_status run_combine(const mxfp4_moe_move_args* A, cudaStream_t s)
{
    const mxfp4_status st = check_move(A);
    if (st != MXFP4_OK)
        return st;
    const size_t esz = esize(A);
    if (A->ld_out < A->cols || A->ld_rows < A->cols || (A->residual && A->ld_tokens < A->cols))
        return MXFP4_EINVAL;
    if (A->tokens == 0 || A->cols == 0)
        return MXFP4_OK;
    if (!A->out || (A->row_count > 0 && !A->y) || !aligned(A->y, esz) || !aligned(A->out, esz) ||
        !aligned(A->residual, esz) || !aligned(A->weights, 4))
        return MXFP4_EINVAL;
    CombineArgs a;
    combine_args(A, &a);
    const bool vec = (A->cols * esz) % 16 == 0 && vec_rows(A->y, A->ld_rows, esz) && vec_rows(A->out, A->ld_out, esz) &&
                     (!A->residual || vec_rows(A->residual, A->ld_tokens, esz));
    const void* fn = esz == 2 ? (vec ? (const void*)combine_kernel<2, true> : (const void*)combine_kernel<2, false>)
                              : (vec ? (const void*)combine_kernel<4, true> : (const void*)combine_kernel<4, false>);
    return launch_stride(fn, A->tokens * (vec ? A->cols * (int64_t)esz / 16 : A->cols), a, s);
}

static mxfp4_status run_combine_bwd(const mxfp4_moe_move_args* A, cudaStream_t s)
{
    const mxfp4_status st = check_move(A);
    if (st != MXFP4_OK)
        return st;
    const size_t esz = esize(A);
    if (A->ld_out < A->cols || (A->grad_weights && A->ld_rows < A->cols) || (A->grad_rows && A->ld_grad_rows < A->cols))
        return MXFP4_EINVAL;
    if (A->tokens == 0)
        return MXFP4_OK;
    if (!A->grad_rows && !A->grad_weights)
        return A->row_count == 0 || A->cols == 0 ? MXFP4_OK : MXFP4_EINVAL;
    if ((A->cols > 0 && !A->grad_out) || (A->grad_weights && A->row_count > 0 && A->cols > 0 && !A->y) ||
        !aligned(A->grad_out, esz) || !aligned(A->y, esz) || !aligned(A->grad_rows, esz) || !aligned(A->weights, 4) ||
        !aligned(A->grad_weights, 4))
        return MXFP4_EINVAL;
    CombineArgs a;
    combine_args(A, &a);
    const bool vec = (A->cols * esz) % 16 == 0 && vec_rows(A->grad_out, A->ld_out, esz) &&
                     (!A->grad_weights || vec_rows(A->y, A->ld_rows, esz)) &&
                     (!A->grad_rows || vec_rows(A->grad_rows, A->ld_grad_rows, esz));
    const void* fn = esz == 2 ? (vec ? (const void*)combine_bwd_kernel<2, true> : (const void*)combine_bwd_kernel<2, false>)
                              : (vec ? (const void*)combine_bwd_kernel<4, true> : (const void*)combine_bwd_kernel<4, false>);
    return launch1(fn, A->tokens, NTHREADS, 0, a, s);
}

// ---- grouped linear --------------------------------------------------------

template <int FMT, int NT, bool F32>
static mxfp4_status launch_linear_t(const LnMaps& maps, const LnArgs& g, cudaStream_t s)
{
    using SM = LnSmem<FMT, NT>;
    const void* fn = g.residual ? (const void*)linear_kernel<FMT, NT, F32, true> : (const void*)linear_kernel<FMT, NT, F32, false>;
    const size_t smem = sizeof(SM) + 1024 + (size_t)(2 * (g.num_groups + 1)) * sizeof(int32_t);
    if (!allow_smem(fn, smem))
        return MXFP4_ECUDA;
    const int sms = device_sms();
    if (sms <= 0)
        return MXFP4_ECUDA;
    const int64_t bound = (g.m / NT + g.num_groups) * ((g.n + LN_FT - 1) / LN_FT);
    LnMaps m = maps;
    LnArgs a = g;
    void* args[] = {&m, &a};
    return launched(cudaLaunchKernel(fn, dim3((unsigned)(bound < sms ? bound : sms)), dim3(SM::THREADS), args, smem, s));
}

template <int FMT, int NT>
static mxfp4_status launch_linear_n(const mxfp4_linear_args* A, LnMaps maps, const LnArgs& g, int64_t kb, bool f32, cudaStream_t s)
{
    if (!encode_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(A->a), (uint64_t)kb, (uint64_t)A->m,
                   (uint64_t)A->lda, LN_ROW_BYTES, NT, CU_TENSOR_MAP_SWIZZLE_128B))
        return MXFP4_ECUDA;
    return f32 ? launch_linear_t<FMT, NT, true>(maps, g, s) : launch_linear_t<FMT, NT, false>(maps, g, s);
}

// Clusters of `fn` that the device holds at once, cached per (device, kernel).
static int resident_pairs(const void* fn, int threads, size_t smem)
{
    struct Entry {
        const void* fn;
        int dev;
        size_t smem;
        int pairs;
    };
    static Entry cache[64];
    static int n = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return -1;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        for (int i = 0; i < n; ++i)
            if (cache[i].fn == fn && cache[i].dev == dev && cache[i].smem == smem)
                return cache[i].pairs;
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(2 * 1024);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int pairs = 0;
    if (cudaOccupancyMaxActiveClusters(&pairs, fn, &cfg) != cudaSuccess || pairs < 1)
        return -1;
    std::lock_guard<std::mutex> lk(g_mu);
    if (n < 64)
        cache[n++] = Entry{fn, dev, smem, pairs};
    return pairs;
}

// Bytes of the tokens' scales by tiles of the pair kernel.
static int64_t scale_tiles_bytes(int64_t m, int64_t k, int64_t groups) { return (m / L2_NT + groups) * ((k + 127) / 128) * 1024; }

template <int FMT, bool F32>
static mxfp4_status launch_linear2(const mxfp4_linear_args* A, const LnMaps& maps, const LnArgs& g, int64_t kb, cudaStream_t s)
{
    using SM = Ln2Smem<FMT>;
    const uint32_t atoms = SM::ATOMS;
    const int64_t ncb = (g.k + 127) / 128;
    Ln2Maps m2;
    memset(&m2, 0, sizeof(m2));
    m2.w = maps.w;
    if (!encode_2d(&m2.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(A->a), (uint64_t)kb, (uint64_t)A->m,
                   (uint64_t)A->lda, LN_ROW_BYTES, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&m2.sfw, CU_TENSOR_MAP_DATA_TYPE_UINT32, const_cast<uint8_t*>(A->b_scales), 128,
                   (uint64_t)(g.num_groups * (g.sfw_group_bytes >> 9)), 512, 128, atoms, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_2d(&m2.sfx, CU_TENSOR_MAP_DATA_TYPE_UINT32, A->workspace, 128, (uint64_t)((g.m / L2_NT + g.num_groups) * ncb * 2), 512, 128,
                   2 * atoms, CU_TENSOR_MAP_SWIZZLE_NONE))
        return MXFP4_ECUDA;
    const void* fn = g.residual ? (const void*)linear2_kernel<FMT, F32, true> : (const void*)linear2_kernel<FMT, F32, false>;
    const size_t plan = (size_t)(2 * (g.num_groups + 1)) * sizeof(int32_t), smem = sizeof(SM) + 1024 + plan;
    if (!allow_smem(fn, smem))
        return MXFP4_ECUDA;
    const int pairs = resident_pairs(fn, L2_THREADS, smem);
    if (pairs < 1)
        return MXFP4_ECUDA;
    const int64_t units = g.m / L2_NT + g.num_groups, bound = units * ((g.n + LN_FT - 1) / LN_FT);
    LnArgs a = g;
    uint32_t* ws = static_cast<uint32_t*>(A->workspace);
    void* args1[] = {&a, &ws};
    mxfp4_status st = launched(cudaLaunchKernel((const void*)scale_tiles_kernel, dim3((unsigned)(units < 4096 ? units : 4096), (unsigned)((ncb + SC_COLS - 1) / SC_COLS)),
                                                dim3(L2_NT), args1, plan, s));
    if (st != MXFP4_OK)
        return st;
    void* args2[] = {&m2, &a};
    return launch_after(fn, dim3((unsigned)(2 * (bound < pairs ? bound : pairs))), L2_THREADS, smem, args2, s);
}

// Whether a product goes to pairs of SMs (given the workspace). Groups of 256 rows or
// more on average, which leave tiles partly empty but still came faster on ragged ones
// (65536 x 4096 x 7168, swiglu, 256 groups: equal sizes 995 against 1490 us, uniform
// draws 1446 / 1900, log-normal 1406 / 1970; k = 2048 613 / 610 and 586 / 606); tiles for most of the device (1024 x 4096 x 4096 31
// against the single-SM kernel's 24 us, 4096 x 4096 x 4096 57 / 63); and eight
// stages along K, since its one accumulator waits for both CTAs' epilogues
// (32768 x 4096 over 32 experts, E2M1, bf16 results: k = 1024 184 / 160 us, 2048 194 /
// 194, 2560 203 / 226, 7168 391 / 486; with a residual, k = 2048, 248 / 240; three fp32
// streams: E2M1 16384 rows, k = 2048 250 / 250, 4096 275 / 284, E4M3 2049 x 14336 x
// 4096 182 / 197).
static bool linear_on_pairs(const mxfp4_linear_args* A)
{
    const int64_t stage = A->elem_format == MXFP4_ELEM_E2M1 ? LnFmt<MXFP4_ELEM_E2M1>::BK : LnFmt<MXFP4_ELEM_E4M3>::BK;
    const int64_t groups = A->group_list ? A->num_groups : 1;
    return A->m / groups >= L2_NT && A->k >= 8 * stage && (A->m / L2_NT) * (A->n / LN_FT) >= 128 &&
           groups <= Ln2Smem<MXFP4_ELEM_E2M1>::MAX_GROUPS && scale_tiles_bytes(A->m, A->k, groups) / 512 <= INT32_MAX &&
           groups * (mxfp4_scales_row_bytes(A->n, A->k, 32, MXFP4_SCALES_MMA) >> 9) <= INT32_MAX &&  // 32-bit coordinates
           aligned(A->a_scales, 16);
}

template <int FMT>
static mxfp4_status launch_linear(const mxfp4_linear_args* A, const LnMaps& maps, const LnArgs& g, int64_t kb, bool f32, cudaStream_t s)
{
    // tokens per tile by the groups' mean size (their sizes are device data)
    const int64_t mean = g.m / g.num_groups;
    if (mean <= 32)
        return launch_linear_n<FMT, 32>(A, maps, g, kb, f32, s);
    if (mean <= 64 || g.num_groups > LnSmem<FMT, 128>::MAX_GROUPS)
        return launch_linear_n<FMT, 64>(A, maps, g, kb, f32, s);
    if (linear_on_pairs(A) && A->workspace && A->workspace_bytes >= scale_tiles_bytes(g.m, g.k, g.num_groups))
        return f32 ? launch_linear2<FMT, true>(A, maps, g, kb, s) : launch_linear2<FMT, false>(A, maps, g, kb, s);
    return launch_linear_n<FMT, 128>(A, maps, g, kb, f32, s);
}

static mxfp4_status check_linear(const mxfp4_linear_args* A)
{
    if (!A)
        return MXFP4_EINVAL;
    if (A->activation < MXFP4_ACT_NONE || A->activation > MXFP4_ACT_SWIGLU)
        return MXFP4_EINVAL;
    if (A->d_dtype != MXFP4_F32 && A->d_dtype != MXFP4_BF16)
        return MXFP4_EINVAL;
    if (A->m < 0 || A->n < 0 || (A->activation == MXFP4_ACT_SWIGLU && A->n % 2 != 0))
        return MXFP4_EINVAL;
    if (A->group_list && (A->num_groups < 1 || (A->group_list_type != 0 && A->group_list_type != 1) || !aligned(A->group_list, 8)))
        return MXFP4_EINVAL;
    if (A->m > INT32_MAX || A->n > INT32_MAX || (A->group_list && A->num_groups > MXFP4_MAX_GROUPS))
        return MXFP4_EUNSUPPORTED;
    return MXFP4_OK;
}

static mxfp4_status check_product(const mxfp4_linear_args* A)
{
    const mxfp4_status st = check_linear(A);
    if (st != MXFP4_OK)
        return st;
    const bool e2 = A->elem_format == MXFP4_ELEM_E2M1;
    if (!e2 && A->elem_format != MXFP4_ELEM_E4M3)
        return MXFP4_EINVAL;
    if (A->k < 1 || A->k % (e2 ? 64 : 32) != 0)
        return MXFP4_EINVAL;
    return A->k > INT32_MAX ? MXFP4_EUNSUPPORTED : MXFP4_OK;
}

// The status of a call with nothing to multiply: its list's alone.
static mxfp4_status list_status(const mxfp4_linear_args* A, cudaStream_t s)
{
    if (!aligned(A->status, 4))
        return MXFP4_EINVAL;
    if (!A->status)
        return MXFP4_OK;
    if (!A->group_list)
        return launched(cudaMemsetAsync(A->status, 0, sizeof(int32_t), s));
    LnBwdArgs b;
    memset(&b, 0, sizeof(b));
    b.group_list = A->group_list;
    b.status = A->status;
    b.m = A->m;
    b.num_groups = (int32_t)A->num_groups;
    b.gl_type = A->group_list_type;
    return launch1((const void*)linear_list_kernel, 1, NTHREADS, (size_t)(2 * (A->num_groups + 1)) * sizeof(int32_t), b, s);
}

static mxfp4_status run_linear(const mxfp4_linear_args* A, cudaStream_t s)
{
    const mxfp4_status st = check_product(A);
    if (st != MXFP4_OK)
        return st;
    const bool e2 = A->elem_format == MXFP4_ELEM_E2M1, gated = A->activation == MXFP4_ACT_SWIGLU;
    const int64_t kb = e2 ? A->k / 2 : A->k, width = gated ? A->n / 2 : A->n;
    const size_t esz = A->d_dtype == MXFP4_F32 ? 4 : 2;
    if (A->ld_y < width || (A->residual && A->ld_res < width) || (A->preact && A->ld_preact < A->n))
        return MXFP4_EINVAL;
    if (A->m == 0 || A->n == 0)
        return list_status(A, s);
    if (!A->a || !A->b || !A->a_scales || !A->b_scales || !A->y)
        return MXFP4_EINVAL;
    if (A->lda < kb || A->ldb < kb || A->lda % 16 != 0 || A->ldb % 16 != 0 || !aligned(A->a, 16) || !aligned(A->b, 16) ||
        !aligned(A->a_scales, 4) || !aligned(A->b_scales, 16))
        return MXFP4_EINVAL;
    if (!aligned(A->y, esz) || !aligned(A->residual, esz) || !aligned(A->preact, esz) || !aligned(A->bias, 4) || !aligned(A->status, 4) || !aligned(A->workspace, 16))
        return MXFP4_EINVAL;
    LnArgs g;
    memset(&g, 0, sizeof(g));
    g.num_groups = A->group_list ? (int32_t)A->num_groups : 1;
    if (A->n * g.num_groups > INT32_MAX)
        return MXFP4_EUNSUPPORTED;
    g.sfx = A->a_scales;
    g.sfw = A->b_scales;
    g.bias = A->bias;
    g.residual = A->residual;
    g.y = A->y;
    g.preact = A->preact;
    g.group_list = A->group_list;
    g.status = A->status;
    g.m = A->m;
    g.n = A->n;
    g.k = A->k;
    g.ld_res = A->ld_res;
    g.ld_y = A->ld_y;
    g.ld_z = A->ld_preact;
    g.sfw_group_bytes = mxfp4_scales_row_bytes(A->n, A->k, 32, MXFP4_SCALES_MMA);
    g.gl_type = A->group_list_type;
    g.act = A->activation;
    LnMaps maps;
    memset(&maps, 0, sizeof(maps));
    if (!encode_2d(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(A->b), (uint64_t)kb,
                   (uint64_t)(A->n * g.num_groups), (uint64_t)A->ldb, LN_ROW_BYTES, 128, CU_TENSOR_MAP_SWIZZLE_128B))
        return MXFP4_ECUDA;
    const bool f32 = A->d_dtype == MXFP4_F32;
    return e2 ? launch_linear<MXFP4_ELEM_E2M1>(A, maps, g, kb, f32, s) : launch_linear<MXFP4_ELEM_E4M3>(A, maps, g, kb, f32, s);
}

static mxfp4_status run_linear_bwd(const mxfp4_linear_args* A, cudaStream_t s)
{
    mxfp4_status st = check_linear(A);
    if (st != MXFP4_OK)
        return st;
    const bool gated = A->activation == MXFP4_ACT_SWIGLU;
    const int64_t width = gated ? A->n / 2 : A->n;
    const size_t esz = A->d_dtype == MXFP4_F32 ? 4 : 2;
    const int64_t groups = A->group_list ? A->num_groups : 1;
    if (A->ld_y < width || A->ld_preact < A->n || A->ld_grad < A->n)
        return MXFP4_EINVAL;
    if (A->n == 0)
        return list_status(A, s);
    if (A->m > 0 && (!A->grad_out || !A->preact || !A->grad_preact))
        return MXFP4_EINVAL;
    if (!aligned(A->grad_out, esz) || !aligned(A->preact, esz) || !aligned(A->grad_preact, esz) || !aligned(A->grad_bias, 4) ||
        !aligned(A->workspace, 4) || !aligned(A->status, 4))
        return MXFP4_EINVAL;
    if (A->grad_bias && (!A->workspace || A->workspace_bytes < mxfp4_grouped_linear_workspace(A->m, A->n, groups)))
        return MXFP4_EINVAL;
    LnBwdArgs b;
    memset(&b, 0, sizeof(b));
    b.grad = A->grad_out;
    b.z = A->preact;
    b.grad_z = A->grad_preact;
    b.grad_bias = A->grad_bias;
    b.ws = static_cast<float*>(A->workspace);
    b.group_list = A->group_list;
    b.status = A->status;
    b.m = A->m;
    b.n = A->n;
    b.ld_g = A->ld_y;
    b.ld_z = A->ld_preact;
    b.ld_dz = A->ld_grad;
    b.num_groups = (int32_t)groups;
    b.gl_type = A->group_list_type;
    b.act = A->activation;
    const size_t plan = (size_t)(2 * (groups + 1)) * sizeof(int32_t);
    const int per = (int)(16 / esz);
    const bool vec = A->n % per == 0 && vec_rows(A->preact, A->ld_preact, esz) && vec_rows(A->grad_preact, A->ld_grad, esz) &&
                     (gated ? aligned(A->grad_out, 8) && (A->ld_y * (int64_t)esz) % 8 == 0 : vec_rows(A->grad_out, A->ld_y, esz));
    const void* fn = esz == 2 ? (vec ? (const void*)linear_bwd_kernel<2, true> : (const void*)linear_bwd_kernel<2, false>)
                              : (vec ? (const void*)linear_bwd_kernel<4, true> : (const void*)linear_bwd_kernel<4, false>);
    const int sms = device_sms(), occ = occupancy(fn, plan);
    if (sms <= 0 || occ <= 0)
        return MXFP4_ECUDA;
    b.across_log2 = 5;
    while (b.across_log2 < 8 && ((int64_t)(vec ? per : 2) << b.across_log2) < A->n)
        ++b.across_log2;
    const int64_t ct = (int64_t)(vec ? per : 2) << b.across_log2;
    const int64_t units = (A->m / LB_ROWS + groups) * ((A->n + ct - 1) / ct), most = (int64_t)sms * occ;
    st = launch1(fn, units < most ? units : most, NTHREADS, plan, b, s);
    if (st == MXFP4_OK && A->grad_bias) {
        LnBwdArgs arg = b;
        void* args[] = {&arg};
        st = launch_after((const void*)linear_bias_kernel, dim3((unsigned)((A->n + NTHREADS - 1) / NTHREADS), (unsigned)groups), NTHREADS, plan, args, s);
    }
    return st;
}

}  // namespace mxfp4

using namespace mxfp4;

extern "C" {

int64_t mxfp4_moe_route_workspace(int64_t tokens, int64_t experts)
{
    if (tokens < 0 || experts < 0)
        return -1;
    const int64_t chunks = route_chunks(tokens);
    return chunks > 1 ? chunks * experts * (int64_t)sizeof(int32_t) : 0;
}

mxfp4_status mxfp4_moe_route(const mxfp4_moe_route_args* args, mxfp4_stream_t stream)
{
    return run_route(args, reinterpret_cast<cudaStream_t>(stream));
}

mxfp4_status mxfp4_moe_route_bwd(const mxfp4_moe_route_args* args, mxfp4_stream_t stream)
{
    return run_route_bwd(args, reinterpret_cast<cudaStream_t>(stream));
}

int64_t mxfp4_moe_dispatch_workspace(int64_t tokens, int32_t k, int64_t cols, int64_t row_count)
{
    if (tokens < 0 || k < 1 || cols < 0 || row_count < 0)
        return -1;
    // by 4-byte stores the scales cost about 8 us per million words, the second
    // kernel about 3 us and a sixth of that
    const int64_t words = (cols + 127) / 128;
    if (tokens * k * words < (int64_t)1 << 19 || (words + SG_WORDS - 1) / SG_WORDS > 65535)  // (its grid's second dimension)
        return 0;
    return (tokens * words + row_count) * 4;
}

mxfp4_status mxfp4_moe_dispatch(const mxfp4_moe_move_args* args, mxfp4_stream_t stream)
{
    return run_dispatch(args, reinterpret_cast<cudaStream_t>(stream));
}

mxfp4_status mxfp4_moe_combine(const mxfp4_moe_move_args* args, mxfp4_stream_t stream)
{
    return run_combine(args, reinterpret_cast<cudaStream_t>(stream));
}

mxfp4_status mxfp4_moe_combine_bwd(const mxfp4_moe_move_args* args, mxfp4_stream_t stream)
{
    return run_combine_bwd(args, reinterpret_cast<cudaStream_t>(stream));
}

mxfp4_status mxfp4_grouped_linear(const mxfp4_linear_args* args, mxfp4_stream_t stream)
{
    return run_linear(args, reinterpret_cast<cudaStream_t>(stream));
}

int64_t mxfp4_grouped_linear_fwd_workspace(const mxfp4_linear_args* args)
{
    if (check_product(args) != MXFP4_OK)
        return -1;
    return linear_on_pairs(args) ? scale_tiles_bytes(args->m, args->k, args->group_list ? args->num_groups : 1) : 0;
}

int64_t mxfp4_grouped_linear_workspace(int64_t m, int64_t n, int64_t num_groups)
{
    if (m < 0 || n < 0 || num_groups < 1)
        return -1;
    return (m / LB_ROWS + num_groups) * n * (int64_t)sizeof(float);
}

mxfp4_status mxfp4_grouped_linear_bwd(const mxfp4_linear_args* args, mxfp4_stream_t stream)
{
    return run_linear_bwd(args, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
