// mxfp4_route.cuh -- routing of tokens to experts: selection, weights, the
// expert-sorted order, and the gradient of the router's logits (included by
// mxfp4_moe.cu; the definition is in include/mxfp4.h, mxfp4_moe_route).
//
// Selection is decided by real numbers (the keys s_e + b_e), so it must not
// depend on how an exponential happens to round. A warp takes a token (or two, one per
// half), a lane NV consecutive experts; keys are formed in fp32 with the approximate
// exponential, and every comparison the answer rests on (between neighbours in
// the sorted choice, at its end, and between the last group kept and the first
// dropped) is checked against the keys' error bound. A token with a comparison
// inside the bound is selected again in 64 bits (rt_select64). Without a bias
// (or with a constant one) the score is monotone in the logit, and logits are
// compared as they are.
//
// The order of the (token, expert) pairs by expert is a counting sort without
// atomics on counters: a CTA takes RT_CHUNK consecutive tokens and keeps, per
// expert, one bit per token that chose it (the only atomics set bits, whose
// order cannot matter), so a pair's rank among its chunk's pairs of the same
// expert is a population count. A scan of the chunks' counts per expert and
// one of the experts' totals give every pair its row.

namespace mxfp4 {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;
constexpr int RT_CHUNK = 64;            // tokens per CTA: two words of token bits per expert
constexpr int RT_MAX_EXPERTS = 1024;
constexpr int RT_MAX_K = 32;            // a lane per chosen expert
constexpr int RT_MAX_GROUPS = 32;       // a lane per group of experts

struct RouteArgs {
    const void* logits;
    int64_t tokens, ld;
    const float* bias;
    const uint8_t* token_mask;
    float* weights;
    int32_t* experts_out;
    int32_t* rows;
    int32_t* slots;
    int64_t* counts;
    int32_t* ws;        // [chunks][experts]: counts of a chunk, then the rows before it
    float scale;
    int32_t experts, k, groups, topk_groups;
    int32_t top2, sigmoid, renorm, bf16;
    int32_t chunks;
    int32_t per;          // experts of a group
    uint32_t per_magic;   // ceil(2^32 / per): e / per is the high word of e * per_magic (e < 1024); 0: per is 1
    int32_t lanes;        // lanes of a group where groups are whole lanes, a power of two; else 0
    int32_t vec;          // rows are whole 16-byte vectors per lane
};

template <bool BF16>
__device__ __forceinline__ float rt_logit(const RouteArgs& a, int64_t t, int e)
{
    const int64_t i = t * a.ld + e;
    return BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[i] << 16)
                : static_cast<const float*>(a.logits)[i];
}

__device__ __forceinline__ float rt_logit(const RouteArgs& a, int64_t t, int e)
{
    const int64_t i = t * a.ld + e;
    return a.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[i] << 16)
                  : static_cast<const float*>(a.logits)[i];
}

// The warp's greatest value; NaN if any is NaN.
__device__ __forceinline__ float warp_max(float v)
{
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float rcp_approx(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Reductions over the LW lanes (32, or 16: two tokens a warp) of a token.
template <int LW>
__device__ __forceinline__ float part_max(float v)
{
    if constexpr (LW == 32) {
        return warp_max(v);
    } else {
#pragma unroll
        for (int o = LW / 2; o; o >>= 1)
            v = max_nan(v, __shfl_xor_sync(FULL, v, o));
        return v;
    }
}

template <int LW>
__device__ __forceinline__ uint32_t part_max(uint32_t v)
{
    if constexpr (LW == 32) {
        return __reduce_max_sync(FULL, v);
    } else {
#pragma unroll
        for (int o = LW / 2; o; o >>= 1)
            v = max(v, __shfl_xor_sync(FULL, v, o));
        return v;
    }
}

template <int LW>
__device__ __forceinline__ float part_sum(float v)
{
#pragma unroll
    for (int o = LW / 2; o; o >>= 1)
        v += __shfl_xor_sync(FULL, v, o);
    return v;
}

template <int LW>
__device__ __forceinline__ uint32_t part_ballot(bool p)
{
    const uint32_t b = __ballot_sync(FULL, p);
    return LW == 32 ? b : (b >> (threadIdx.x & 16)) & 0xFFFFu;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(FULL, v, o);
    return v;
}

__device__ __forceinline__ double rt_neg_inf() { return __longlong_as_double(0xFFF0000000000000ll); }

// The chosen experts of token t in 64 bits: lane j < k returns the j-th (-1:
// none). sk: the warp's scratch of a.experts doubles. m: the row's largest logit.
// exact: the logits' order is the keys' (scores are formed for group ranks only).
__device__ __noinline__ int rt_select64(const RouteArgs& a, int64_t t, double* sk, float m, bool exact)
{
    const int lane = threadIdx.x & 31, E = a.experts;
    const double NI = rt_neg_inf();
    double sum = 0.0;
    __syncwarp();
    for (int e = lane; e < E; e += 32) {
        const double x = (double)rt_logit(a, t, e);
        const double p = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)m);
        sk[e] = p;
        sum += p;
    }
    sum = warp_sum(sum);
    const bool ranks = a.groups > 1 && a.top2;
    for (int e = lane; e < E; e += 32) {
        const float x = rt_logit(a, t, e);
        double key = exact && !ranks ? (double)x : a.sigmoid ? sk[e] : sk[e] / sum;
        bool open = x > -INFINITY;
        if (a.bias) {
            const float b = a.bias[e];
            key += exact && !ranks ? 0.0 : (double)b;
            open = open && fabsf(b) < INFINITY;
        }
        sk[e] = open ? key : NI;
    }
    __syncwarp();
    if (a.groups > 1) {
        // lane g: the rank of group g (best key, or the best two added)
        const int per = a.per;
        double best = NI, next = NI;
        if (lane < a.groups)
            for (int i = 0; i < per; ++i) {
                const double v = sk[lane * per + i];
                if (v > best) {
                    next = best;
                    best = v;
                } else if (v > next) {
                    next = v;
                }
            }
        const double rank = a.top2 && next != NI ? best + next : best;
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double r = __shfl_sync(FULL, rank, g);
            before += r > rank || (r == rank && g < lane);
        }
        if (lane < a.groups && before >= a.topk_groups)
            for (int i = 0; i < per; ++i)
                sk[lane * per + i] = NI;
        __syncwarp();
    }
    if (exact && ranks) {
        for (int e = lane; e < E; e += 32)
            if (sk[e] != NI)
                sk[e] = (double)rt_logit(a, t, e);
        __syncwarp();
    }
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        double best = NI;
        int at = -1;
        for (int e = lane; e < E; e += 32)
            if (sk[e] > best) {
                best = sk[e];
                at = e;
            }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double v = __shfl_xor_sync(FULL, best, o);
            const int w = __shfl_xor_sync(FULL, at, o);
            if (w >= 0 && (at < 0 || v > best || (v == best && w < at))) {
                best = v;
                at = w;
            }
        }
        if (at < 0)
            break;  // no open expert is left (the same in every lane)
        if (lane == (at & 31))
            sk[at] = NI;
        if (lane == j)
            mine = at;
        __syncwarp();
    }
    return mine;
}

// Order-preserving bits of a float (not NaN): greater floats, greater words.
__device__ __forceinline__ uint32_t rt_order(float v)
{
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float rt_unorder(uint32_t u)
{
    return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// The NV logits of this lane (experts lane * NV ..): -inf behind the last expert.
template <int NV, bool BF16, int LW>
__device__ __forceinline__ void rt_load(const RouteArgs& a, int64_t t, float (&x)[NV])
{
    const int e0 = (threadIdx.x & (LW - 1)) * NV;
    const int64_t i0 = t * a.ld + e0;
    if constexpr (NV * (BF16 ? 2 : 4) >= 16) {
        if (a.vec) {
            constexpr int W = NV * (BF16 ? 2 : 4) / 16;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                if (e0 < a.experts)
                    q = ld_stream(static_cast<const char*>(a.logits) + i0 * (BF16 ? 2 : 4) + 16 * j);
                const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < NV / W; ++i)
                    x[NV / W * j + i] = BF16 ? __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16) : __uint_as_float(u[i % 4]);
            }
            if (e0 >= a.experts)
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    x[i] = -INFINITY;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        x[i] = e0 + i < a.experts ? (BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[i0 + i] << 16)
                                          : static_cast<const float*>(a.logits)[i0 + i])
                                  : -INFINITY;
}

// Descending order of a lane's NV words (Batcher's odd-even merge sort).
template <int NV>
__device__ __forceinline__ void rt_sort(uint32_t (&v)[NV])
{
#pragma unroll
    for (int p = 1; p < NV; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < NV; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < NV && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t hi = max(v[i + j], v[i + j + k]), lo = min(v[i + j], v[i + j + k]);
                        v[i + j] = hi;
                        v[i + j + k] = lo;
                    }
}

__device__ __forceinline__ float exp2_approx(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Approximate score of a logit: the logistic function, or e^(x - m) times r.
template <bool SIG>
__device__ __forceinline__ float rt_score(float x, float m, float r)
{
    if constexpr (SIG)
        return rcp_approx(1.0f + exp2_approx(-1.4426950408889634f * x));
    else
        return exp2_approx(1.4426950408889634f * (x - m)) * r;
}

// Bound on a key's error against the real s + b. The approximate exponential is
// off by 2^-22.5 + |x| 2^-23 relative (x its argument: 2^-19 up to 14; beyond,
// the value itself is below 2^-20 and the absolute term covers it), of which
// the logistic function passes on 1 - s; its sum and reciprocal, and a softmax
// sum of at most 32 terms per lane, its reciprocal and product add less than
// 2^-21.5 and 2^-18; the sum with the bias rounds by 2^-24 of the key.
template <bool SIG>
__device__ __forceinline__ float rt_key_error(float s, float key)
{
    return s * (SIG ? fmaf(1.0f - s, 0x1p-19f, 0x1p-21f) : 0x1p-17f) + fabsf(key) * 0x1p-23f + 0x1p-25f;
}

// The chosen experts of token t (lane j < k: the j-th, -1: none). x: this lane's
// logits, b: their biases (-inf: closed), bm: the largest |bias|, m: the row's
// largest logit, exact: the logits' order is the keys'. s_key: the warp's
// scratch of a.experts doubles; xe receives the choice's logit. Each lane sorts its keys once, as
// order-preserving words whose low bits hold the lane's index (the lower expert
// first); the k rounds then take the largest head and shift one lane's list.
template <int NV, bool BF16, bool SIG, int LW>
__device__ __forceinline__ int rt_select(const RouteArgs& a, int t, bool live, const float (&x)[NV], const float (&b)[NV], float bm,
                                         bool exact, float m, double* s_key, float& xe)
{
    const int lane = threadIdx.x & (LW - 1), K = a.k;
    constexpr uint32_t INDEX = NV - 1;
    float key[NV], r = 1.0f;
    bool unsure = false;
    if (exact && !(a.groups > 1 && a.top2)) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            key[i] = b[i] > -INFINITY ? x[i] + 0.0f : -INFINITY;  // (-0 becomes +0: equal logits are equal words)
    } else {
        if constexpr (!SIG) {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                total += rt_score<false>(x[i], m, 1.0f);
            r = rcp_approx(part_sum<LW>(total));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            key[i] = x[i] > -INFINITY ? rt_score<SIG>(x[i], m, r) + b[i] : -INFINITY;
        }
    }
    uint32_t kept = 0xFFFFFFFFu;  // bit g: group g stays
    if (a.groups > 1) {
        // lane g: the two best keys of group g
        float best = -INFINITY, next = -INFINITY;
        if (a.lanes > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                next = fmaxf(next, fminf(best, key[i]));
                best = fmaxf(best, key[i]);
            }
            for (int o = a.lanes >> 1; o; o >>= 1) {
                const float ob = __shfl_xor_sync(FULL, best, o), on = __shfl_xor_sync(FULL, next, o);
                next = fmaxf(fminf(best, ob), fmaxf(next, on));
                best = fmaxf(best, ob);
            }
            best = __shfl_sync(FULL, best, (lane * a.lanes) & (LW - 1), LW);
            next = __shfl_sync(FULL, next, (lane * a.lanes) & (LW - 1), LW);
        } else {
            float* s = reinterpret_cast<float*>(s_key) + ((threadIdx.x & 31) / LW) * a.experts;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (lane * NV + i < a.experts)
                    s[lane * NV + i] = key[i];
            __syncwarp();
            if (lane < a.groups)
                for (int i = 0; i < a.per; ++i) {
                    const float v = s[lane * a.per + i];
                    next = fmaxf(next, fminf(best, v));
                    best = fmaxf(best, v);
                }
            __syncwarp();
        }
        float rank = lane < a.groups ? best : -INFINITY;
        if (a.top2 && next > -INFINITY)
            rank += next;
        int before = 0;  // groups ahead of this lane's (lane g: group g)
        if (a.groups <= 8) {
            // lane (g, part): its share of the eight comparisons of group g
            constexpr int SHARE = 64 / LW;
            const int g = lane & 7, h = (lane >> 3) * SHARE;
            const float mine = __shfl_sync(FULL, rank, g, LW);
#pragma unroll
            for (int q = 0; q < SHARE; ++q) {
                const float rq = __shfl_sync(FULL, rank, h + q, LW);
                before += (int)(rq > mine || (rq == mine && h + q < g));
            }
#pragma unroll
            for (int o = 8; o < LW; o <<= 1)
                before += __shfl_xor_sync(FULL, before, o);
        } else {
#pragma unroll 4
            for (int g = 0; g < a.groups; ++g) {
                const float rg = __shfl_sync(FULL, rank, g, LW);
                before += rg > rank || (rg == rank && g < lane);
            }
        }
        const bool keep = lane < a.groups && before < a.topk_groups;
        kept = part_ballot<LW>(keep);
        if (!exact || a.top2) {
            // the least rank kept against the greatest dropped: a rank is one or
            // two keys, whose scores are at most 1 and sum to |rank| + 2 bm
            const float low = -part_max<LW>(keep ? -rank : -INFINITY), high = part_max<LW>(keep ? -INFINITY : rank);
            const float size = fmaxf(fabsf(low), fabsf(high)) + 2.0f * bm;
            const float err = fminf(size, 2.0f) * (SIG ? 0x1.4p-19f : 0x1p-17f) + size * 0x1p-22f + 0x1p-24f;
            unsure = high > -INFINITY && !(low - high > 2.0f * err);  // (ranks that overflow differ by NaN)
        }
        if (exact)  // the scores were for the groups' ranks
#pragma unroll
            for (int i = 0; i < NV; ++i)
                key[i] = b[i] > -INFINITY ? x[i] + 0.0f : -INFINITY;
    }
    // words at or below that of -inf are closed
    constexpr uint32_t CLOSED = 0x007FFFFFu;
    uint32_t v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        v[i] = (rt_order(key[i]) & ~INDEX) | (INDEX - i);
    if (a.groups > 1 && a.lanes == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t e = lane * NV + i;
            v[i] = (kept >> (a.per_magic ? __umulhi(e, a.per_magic) : e & 31u)) & 1u ? v[i] : 0u;
        }
    }
    rt_sort<NV>(v);
    if (a.groups > 1 && a.lanes > 0 && !((kept >> (lane / a.lanes)) & 1u))
        v[0] = 0u;  // a lane of one group that was dropped: its list is never entered
    uint32_t word = 0u;   // lane j: the j-th choice's word (lane K: the one behind the last)
    int src = 0;          // and its lane
    for (int j = 0; j <= K; ++j) {
        // equal keys: the lowest lane holds the lowest expert
        const uint32_t head = v[0] & ~INDEX, top = part_max<LW>(head);
        const bool some = top > CLOSED;
        if (LW == 32 ? !some : !__any_sync(FULL, some))
            break;
        const int at = __ffs(part_ballot<LW>(some && head == top)) - 1;  // -1: nothing is left to this token
        const uint32_t taken = __shfl_sync(FULL, v[0], at & (LW - 1), LW);
        if (lane == j && some) {
            word = taken;
            src = at;
        }
        if (lane == at) {
#pragma unroll
            for (int i = 0; i + 1 < NV; ++i)
                v[i] = v[i + 1];
            v[NV - 1] = 0u;
        }
    }
    const int e = word ? src * NV + (int)(INDEX - (word & INDEX)) : -1;
    // bf16 logits are whole in their words, zeros of both signs as one: nothing to check
    xe = e >= 0 ? rt_logit<BF16>(a, t, e) : -INFINITY;
    if (!(exact && BF16)) {
        const float be = e >= 0 && a.bias ? a.bias[e] : 0.0f;
        const float xn = __shfl_down_sync(FULL, xe, 1, LW), bn = __shfl_down_sync(FULL, be, 1, LW);
        const int en = __shfl_down_sync(FULL, e, 1, LW);
        const uint32_t wn = __shfl_down_sync(FULL, word, 1, LW);
        bool close;
        if (exact) {
            close = lane < K - 1 ? !(xe > xn || (xe == xn && e < en)) : ((word ^ wn) & ~INDEX) == 0u;
        } else {
            // the whole keys again; behind the last choice no key exceeds the next
            // word with its low bits full, but any expert may hold such a key: its
            // score is the key less its bias, and at most the row's largest
            const float se = rt_score<SIG>(xe, m, r), sn = rt_score<SIG>(xn, m, r), ke = se + be, kn = sn + bn;
            const bool last = lane == K - 1;
            const float bound = last ? rt_unorder(wn | INDEX) : kn;
            const float rest = fminf(bound + bm, SIG ? 1.0f : r) * (SIG ? 0x1.4p-19f : 0x1p-17f) + fabsf(bound) * 0x1p-23f + 0x1p-25f;
            close = !(ke - bound > rt_key_error<SIG>(se, ke) + (last ? rest : rt_key_error<SIG>(sn, kn)));
            if (lane < K - 1 && xe == xn && be == bn)
                close = e > en;  // equal keys: the lower expert first
        }
        // a lane whose successor exists; that of a choice in the last lane is not at hand
        // (k = 32: every token again, 65536 x 256 628 us against 193 at k = 31)
        unsure = unsure || (lane < K && e >= 0 && (K < LW || lane < LW - 1 ? en >= 0 && close : true));
    }
    int mine = lane < K ? e : -1;
    const uint32_t again = __ballot_sync(FULL, unsure && live);
    if (again) {  // the warp's tokens in doubt, one by one
#pragma unroll 1
        for (int h = 0; h < 32; h += LW)
            if ((again >> h) & (LW == 32 ? 0xFFFFFFFFu : 0xFFFFu)) {
                const int th = __shfl_sync(FULL, t, h);
                const float mh = __shfl_sync(FULL, m, h);
                const int got = __shfl_sync(FULL, rt_select64(a, th, s_key, mh, exact), lane);
                if ((int)(threadIdx.x & 31 & ~(LW - 1)) == h)
                    mine = got;
            }
        xe = mine >= 0 ? rt_logit<BF16>(a, t, mine) : -INFINITY;
    }
    if (mine < 0)
        xe = -INFINITY;
    return mine;
}

// Score of a chosen expert (fp32): softmax e^(x - m) / sum, or the logistic
// function. With renormalisation a common factor cancels, so scores that
// underflow are taken relative to the chosen ones' largest logit.
__device__ __forceinline__ float rt_sigmoid(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }

// Sum over the k slots' lanes (0 in the others).
template <int LW>
__device__ __forceinline__ float rt_sum_k(const RouteArgs& a, float v)
{
    if (a.k > 8)
#pragma unroll
        for (int o = LW / 2; o >= 8; o >>= 1)
            v += __shfl_xor_sync(FULL, v, o);
#pragma unroll
    for (int o = 4; o; o >>= 1)
        v += __shfl_xor_sync(FULL, v, o);
    return v;
}

// x: the choice's logit, -inf where there is none.
template <int LW>
__device__ __forceinline__ float rt_weight(const RouteArgs& a, int mine, float x, float m, float sum)
{
    float s;
    if (a.renorm) {
        const float top = part_max<LW>(x);
        if (a.sigmoid) {
            const float shift = top < -60.0f ? top : 0.0f;  // below that 1 + e^x is 1
            s = top < -60.0f ? expf(x - shift) : rt_sigmoid(x);
        } else {
            s = expf(x - top);
        }
        s = mine >= 0 ? s : 0.0f;
        const float total = rt_sum_k<LW>(a, s);
        return total > 0.0f ? a.scale * __fdividef(s, total) : 0.0f;
    }
    s = a.sigmoid ? rt_sigmoid(x) : expf(x - m) / sum;
    return mine >= 0 ? a.scale * s : 0.0f;
}

// Exclusive scan of n <= RT_MAX_EXPERTS counts (shared memory) into s_off by a
// CTA of RT_THREADS; returns the total.
__device__ int rt_scan(const int* s_cnt, int* s_off, int n)
{
    __shared__ int s_w[RT_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n + RT_THREADS - 1) / RT_THREADS;
    int mine = 0;
    for (int i = 0; i < per; ++i)
        if (tid * per + i < n)
            mine += s_cnt[tid * per + i];
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, inc, o);
        inc += lane >= o ? v : 0;
    }
    if (lane == 31)
        s_w[warp] = inc;
    __syncthreads();
    int off = inc - mine, total = 0;
    for (int w = 0; w < RT_WARPS; ++w) {
        off += w < warp ? s_w[w] : 0;
        total += s_w[w];
    }
    for (int i = 0; i < per; ++i)
        if (tid * per + i < n) {
            s_off[tid * per + i] = off;
            off += s_cnt[tid * per + i];
        }
    __syncthreads();
    return total;
}

// One CTA per chunk. A single chunk (chunks == 1) finishes the order itself;
// else `rows` receives ranks within the chunk and ws the chunk's counts.
template <int NV, bool BF16, bool SIG, int LW>
__global__ void __launch_bounds__(RT_THREADS, NV <= 8 ? 4 : NV == 16 ? 2 : 1) route_kernel(const __grid_constant__ RouteArgs a)
{
    extern __shared__ __align__(16) uint8_t rt_dyn[];
    const int E = a.experts, K = a.k;
    const int tid = threadIdx.x, lane = tid & (LW - 1), warp = tid >> 5;
    double* s_key = reinterpret_cast<double*>(rt_dyn) + (size_t)warp * E;
    uint32_t* s_bits = reinterpret_cast<uint32_t*>(rt_dyn + (size_t)RT_WARPS * E * 8);  // [E][2]
    int16_t* s_pick = reinterpret_cast<int16_t*>(s_bits + 2 * E);                       // [RT_CHUNK][K]
    const int64_t t0 = (int64_t)blockIdx.x * RT_CHUNK;
    const int nt = (int)min((int64_t)RT_CHUNK, a.tokens - t0);
    for (int i = tid; i < 2 * E; i += RT_THREADS)
        s_bits[i] = 0u;
    __syncthreads();
    float x[NV], b[NV];
    // biases: one that is not finite closes its expert (-inf does in the keys);
    // one value for all open experts leaves the order to the logits
    bool exact = true;
    float bm = 0.0f;
    if (a.bias) {
        float low = INFINITY, high = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            b[i] = lane * NV + i < E ? a.bias[lane * NV + i] : 0.0f;
            if (!(fabsf(b[i]) < INFINITY))
                b[i] = -INFINITY;
            else if (lane * NV + i < E) {
                low = fminf(low, b[i]);
                high = fmaxf(high, b[i]);
            }
        }
        low = -warp_max(-low);
        high = warp_max(high);
        exact = low >= high;
        bm = fmaxf(fabsf(low), fabsf(high));  // infinite where no expert is open: then no key is compared
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            b[i] = 0.0f;
    }
    constexpr int TOKENS = 32 / LW;  // of a warp at a time
    for (int i0 = warp * TOKENS; i0 < nt; i0 += RT_WARPS * TOKENS) {
        const int i = i0 + (tid & 31) / LW;
        const int64_t t = t0 + i;
        const bool here = i < nt, active = here && (!a.token_mask || a.token_mask[t]);
        float m = -INFINITY;
        if (active) {
            rt_load<NV, BF16, LW>(a, t, x);
            m = x[0];
#pragma unroll
            for (int e = 1; e < NV; ++e)
                m = max_nan(m, x[e]);
        }
        __syncwarp();
        m = part_max<LW>(m);
        const bool bad = active && !(m < INFINITY);  // a NaN or +inf
        const bool live = active && !bad && m > -INFINITY;
        int mine = bad && lane < K ? lane : -1;
        float w = bad ? __uint_as_float(QNAN32) : 0.0f;
        if (__any_sync(FULL, live)) {
            if (!live) {
                m = 0.0f;
#pragma unroll
                for (int e = 0; e < NV; ++e)
                    x[e] = -INFINITY;
            }
            __syncwarp();
            float sum = 0.0f;
            if (!SIG && !a.renorm) {
#pragma unroll
                for (int e = 0; e < NV; ++e)
                    sum += expf(x[e] - m);
                sum = part_sum<LW>(sum);
            }
            float xe;
            const int got = rt_select<NV, BF16, SIG, LW>(a, live ? (int)t : (int)t0, live, x, b, bm, exact, m, s_key, xe);
            const float gw = rt_weight<LW>(a, got, xe, m, sum);
            if (live) {
                mine = got;
                w = gw;
            }
        }
        if (here && lane < K) {
            a.weights[t * K + lane] = w;
            a.experts_out[t * K + lane] = mine;
            s_pick[i * K + lane] = (int16_t)mine;
            if (mine >= 0)
                atomicOr(&s_bits[2 * mine + (i >> 5)], 1u << (i & 31));
        }
    }
    __syncthreads();
    int* s_cnt = reinterpret_cast<int*>(rt_dyn);  // over the keys, which are done with
    int* s_off = s_cnt + E;
    if (a.chunks == 1) {
        for (int e = tid; e < E; e += RT_THREADS) {
            s_cnt[e] = __popc(s_bits[2 * e]) + __popc(s_bits[2 * e + 1]);
            a.counts[e] = s_cnt[e];
        }
        __syncthreads();
        const int total = rt_scan(s_cnt, s_off, E);
        for (int p = total + tid; p < nt * K; p += RT_THREADS)
            a.slots[p] = -1;
    } else {
        for (int e = tid; e < E; e += RT_THREADS)
            a.ws[(int64_t)blockIdx.x * E + e] = __popc(s_bits[2 * e]) + __popc(s_bits[2 * e + 1]);
    }
    for (int p = tid; p < nt * K; p += RT_THREADS) {
        const int e = s_pick[p], i = p / K;
        int r = -1;
        if (e >= 0) {
            const uint32_t low = i < 32 ? s_bits[2 * e] : s_bits[2 * e + 1];
            r = __popc(low & ((1u << (i & 31)) - 1u)) + (i < 32 ? 0 : __popc(s_bits[2 * e]));
            if (a.chunks == 1) {
                r += s_off[e];
                a.slots[r] = p;
            }
        }
        a.rows[t0 * K + p] = r;
    }
}

// Exclusive scan of the chunks' counts per expert, in place, and the totals.
// A CTA takes 32 experts; thread (lane, warp) a segment of the chunks.
__global__ void __launch_bounds__(1024) route_scan_kernel(const RouteArgs a)
{
    __shared__ int s_seg[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    const int per = (a.chunks + 31) / 32;
    const int c0 = min(a.chunks, warp * per), c1 = min(a.chunks, c0 + per);
    wait_for_prerequisite();
    int sum = 0;
    if (e < a.experts)
#pragma unroll 8
        for (int c = c0; c < c1; ++c)
            sum += a.ws[(int64_t)c * a.experts + e];
    s_seg[warp][lane] = sum;
    __syncthreads();
    int off = 0, total = 0;
    for (int w = 0; w < 32; ++w) {
        const int v = s_seg[w][lane];
        off += w < warp ? v : 0;
        total += v;
    }
    if (e >= a.experts)
        return;
    if (warp == 0)
        a.counts[e] = total;
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
        const int64_t i = (int64_t)c * a.experts + e;
        const int v = a.ws[i];
        a.ws[i] = off;
        off += v;
    }
}

// Ranks within a chunk -> rows, and the rows' slots; -1 in the slots behind
// the last row. One CTA per chunk. SCAN: the CTA adds up the chunks' counts
// itself (few chunks: one launch instead of two); else ws holds the rows of
// each expert before the chunk and `counts` the totals.
template <bool SCAN>
__global__ void __launch_bounds__(RT_THREADS) route_place_kernel(const RouteArgs a)
{
    __shared__ int s_cnt[RT_MAX_EXPERTS], s_off[RT_MAX_EXPERTS], s_base[RT_MAX_EXPERTS];
    const int tid = threadIdx.x, E = a.experts, K = a.k;
    wait_for_prerequisite();
    if constexpr (SCAN) {
        for (int e = tid; e < E; e += RT_THREADS)
            s_cnt[e] = s_base[e] = 0;
        __syncthreads();
        // threads side by side on the chunks of four experts (whole 16-byte pieces
        // where rows of counts are), integer sums, so their order does not matter
        const int per = E % 4 == 0 ? 4 : 1, cols = E / per;
        const int segs = max(1, RT_THREADS / cols);
        for (int i = tid; i < segs * cols; i += RT_THREADS) {
            const int seg = i / cols, e = (i - seg * cols) * per;
            int before[4] = {0, 0, 0, 0}, total[4] = {0, 0, 0, 0};
#pragma unroll 4
            for (int c = seg; c < a.chunks; c += segs) {
                const int* p = a.ws + (int64_t)c * E + e;
                int v[4];
                if (per == 4) {
                    const int4 q = *reinterpret_cast<const int4*>(p);
                    v[0] = q.x;
                    v[1] = q.y;
                    v[2] = q.z;
                    v[3] = q.w;
                } else {
                    v[0] = *p;
                    v[1] = v[2] = v[3] = 0;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    total[q] += v[q];
                    before[q] += c < (int)blockIdx.x ? v[q] : 0;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < per) {
                    atomicAdd(&s_cnt[e + q], total[q]);
                    atomicAdd(&s_base[e + q], before[q]);
                }
        }
        __syncthreads();
        if (blockIdx.x == 0)
            for (int e = tid; e < E; e += RT_THREADS)
                a.counts[e] = s_cnt[e];
    } else {
        for (int e = tid; e < E; e += RT_THREADS) {
            s_cnt[e] = (int)a.counts[e];
            s_base[e] = a.ws[(int64_t)blockIdx.x * E + e];
        }
        __syncthreads();
    }
    const int total = rt_scan(s_cnt, s_off, E);
    const int64_t p0 = (int64_t)blockIdx.x * RT_CHUNK * K;
    const int64_t pairs = a.tokens * K;
    const int n = (int)min((int64_t)RT_CHUNK * K, pairs - p0);
    for (int p = tid; p < n; p += RT_THREADS) {
        const int e = a.experts_out[p0 + p];
        if (e >= 0) {
            const int r = a.rows[p0 + p] + s_base[e] + s_off[e];
            a.rows[p0 + p] = r;
            a.slots[r] = (int)(p0 + p);
        }
        if (p0 + p >= total)
            a.slots[p0 + p] = -1;
    }
}

// ---------------------------------------------------------------------------
// Gradient of the logits. With w_j = c s_j / S (S = the chosen scores' sum, or
// 1), g_j the weights' gradients and h_j = c g_j / S:
//   dL/ds_j = h_j - renorm * sum_i h_i s_i / S
//   logistic: dL/dx_j = dL/ds_j s_j (1 - s_j) at the chosen experts, else 0
//   softmax:  dL/dx_e = s_e (dL/ds_e - sum_j dL/ds_j s_j); renormalised, the
//             sum is 0 and s_e / S is the softmax over the chosen logits
// A warp per token. Rows with a NaN or +inf logit get NaN.
// ---------------------------------------------------------------------------

struct RouteBwdArgs {
    RouteArgs r;              // logits, geometry, rule; experts_out is read
    const float* grad_w;
    void* grad_logits;
    int64_t ld_g;
};

__device__ __forceinline__ void rt_store(const RouteBwdArgs& b, int64_t t, int e, float v)
{
    if (b.r.bf16)
        static_cast<uint16_t*>(b.grad_logits)[t * b.ld_g + e] = (uint16_t)f32_to_bf16(v);
    else
        static_cast<float*>(b.grad_logits)[t * b.ld_g + e] = v;
}

__global__ void __launch_bounds__(RT_THREADS) route_bwd_kernel(const RouteBwdArgs b)
{
    extern __shared__ __align__(16) uint8_t rt_dyn[];
    const RouteArgs& a = b.r;
    const int E = a.experts, K = a.k;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* s_d = reinterpret_cast<float*>(rt_dyn) + (size_t)warp * E;  // dL/dx of the chosen experts
    const int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp;
    if (t >= a.tokens)
        return;
    int mine = lane < K ? a.experts_out[t * K + lane] : -1;
    mine = mine < E ? mine : -1;
    const float g = mine >= 0 ? b.grad_w[t * K + lane] : 0.0f;
    const bool some = __any_sync(FULL, mine >= 0);
    float m = -INFINITY;
    bool bad = false;
    for (int e = lane; e < E; e += 32) {  // read before it is known whether they count
        const float x = rt_logit(a, t, e);
        bad |= !(x < INFINITY);
        m = fmaxf(m, x);
    }
    bad = __any_sync(FULL, bad) && some;
    m = warp_max(m);
    for (int e = lane; e < E; e += 32)
        s_d[e] = bad ? __uint_as_float(QNAN32) : 0.0f;
    __syncwarp();
    float sub = 0.0f, sum = 1.0f;  // softmax as it is: what each s_e is multiplied by, and 1 / s_e's divisor
    const bool dense = some && !bad && !a.sigmoid && !a.renorm;
    if (some && !bad) {
        const float x = mine >= 0 ? rt_logit(a, t, mine) : -INFINITY;
        const float h = a.scale * g;
        float d;
        if (a.renorm) {
            const float top = warp_max(x);
            float s = a.sigmoid ? (top < -60.0f ? expf(x - top) : rt_sigmoid(x)) : expf(x - top);
            s = mine >= 0 ? s : 0.0f;
            const float total = warp_sum(s);
            const float share = total > 0.0f ? s / total : 0.0f;
            d = share * (h - warp_sum(h * share));
            if (a.sigmoid)
                d *= rt_sigmoid(-x);
        } else if (a.sigmoid) {
            d = h * rt_sigmoid(x) * rt_sigmoid(-x);
        } else {
            sum = 0.0f;
            for (int e = lane; e < E; e += 32)
                sum += expf(rt_logit(a, t, e) - m);
            sum = warp_sum(sum);
            d = h * expf(x - m) / sum;
            sub = warp_sum(mine >= 0 ? d : 0.0f);
        }
        // an expert chosen twice takes the sum, in the slots' order
        float total = 0.0f;
        for (int j = 0; j < K; ++j) {
            const int e = __shfl_sync(FULL, mine, j);
            const float v = __shfl_sync(FULL, d, j);
            total += e == mine ? v : 0.0f;
        }
        if (mine >= 0)
            s_d[mine] = total;
        __syncwarp();
    }
    for (int e = lane; e < E; e += 32) {
        float v = s_d[e];
        if (dense)
            v -= expf(rt_logit(a, t, e) - m) / sum * sub;
        rt_store(b, t, e, v);
    }
}

}  // namespace mxfp4
