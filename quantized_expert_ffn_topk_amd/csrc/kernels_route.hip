// kernels_route.hip -- selection of experts with groups on gfx950: softmax or
// sigmoid scores, a bias that only steers the choice, the best groups, the k
// best experts inside them, weights renormalised or as they are.
//
// One wave per token, expert e on lane e/NE (register e%NE), so that the first
// lane of a ballot holds the lowest expert.  A token's logits are read once
// and everything up to the k results stays in registers (the group scores pass
// through LDS); the time is the launch and the k dependent wave maxima.
#include "ops_common.h"

#include <cmath>

namespace moe {

struct SelectArgs {
    const void *logits;
    int64_t ld;
    const float *bias;             // NULL: none
    int T, E, k;
    int softmax, n_group, topk_group, group_best, renorm;
    float scale;
    uint32_t gs, gs_inv;           // experts per group, ceil(2^22 / gs)
    int32_t *idx;
    float *w;
    double *part2;                 // fp64 logits in two parts: the second, added and kept
};

// ---------------------------------------------------------------------------
// Ordered keys: a larger value has the larger key, equal values (zeros of both
// signs among them) equal keys; key 0 belongs to no number and marks what
// cannot be chosen.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t order_key(float c)
{
    const uint32_t u = __float_as_uint(c + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double c)
{
    const uint64_t u = (uint64_t)__double_as_longlong(c + 0.0);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ uint64_t wave_top(uint64_t v)
{
    const uint32_t hi = wave_top((uint32_t)(v >> 32));
    const uint32_t lo = wave_top((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ float lane_value(float v, int l)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ double lane_value(double v, int l)
{
    const long long u = __double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(u & 0xffffffffll), l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), l);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ float wave_sum(float v)
{
    return wave_total_f(v);
}
__device__ __forceinline__ double wave_sum(double v)
{
    return wave_total_d(v);
}
__device__ __forceinline__ float exp_of(float v)
{
    return expf(v);
}
__device__ __forceinline__ double exp_of(double v)
{
    return exp(v);
}

template <typename LT>
struct Score {
    typedef float S;               // scores of fp32 and bf16 logits
    typedef uint32_t Key;
};
template <>
struct Score<double> {
    typedef double S;
    typedef uint64_t Key;
};

__device__ __forceinline__ float widen(float v)
{
    return v;
}
__device__ __forceinline__ float widen(bf16_t v)
{
    return bf16_to_f32(v);
}
__device__ __forceinline__ double widen(double v)
{
    return v;
}

template <typename LT, int NE>
__global__ __launch_bounds__(256) void select_kernel(SelectArgs a)
{
    typedef typename Score<LT>::S S;
    typedef typename Score<LT>::Key Key;
    struct __attribute__((packed, aligned(sizeof(LT)))) Piece {
        LT v[NE];
    };
    __shared__ S lds[4][64 * NE + 64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + wave;
    if (t >= a.T)
        return;
    const int e0 = lane * NE;
    const S inf = (S)INFINITY;

    // logits and bias of this lane's experts, all loads issued before any use
    S l[NE], b[NE];
    const LT *row = static_cast<const LT *>(a.logits) + (int64_t)t * a.ld;
    if (e0 + NE <= a.E) {
        const Piece p = *reinterpret_cast<const Piece *>(row + e0);
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            l[j] = widen(p.v[j]);
            b[j] = a.bias ? (S)a.bias[e0 + j] : (S)0;
        }
    } else {
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const bool in = e0 + j < a.E;
            l[j] = in ? widen(row[e0 + j]) : -inf;
            b[j] = (in && a.bias) ? (S)a.bias[e0 + j] : (S)0;
        }
    }
    if constexpr (sizeof(LT) == 8) {
        if (a.part2) {
            double *r1 = const_cast<double *>(row), *r2 = a.part2 + (int64_t)t * a.ld;
#pragma unroll
            for (int j = 0; j < NE; ++j)
                if (e0 + j < a.E) {
                    l[j] += r2[e0 + j];
                    r1[e0 + j] = l[j];
                }
        }
    }

    // scores p (0 for a NaN) and choice values c (-inf for a NaN)
    S p[NE], c[NE];
    if (a.softmax) {
        S m = -inf;
#pragma unroll
        for (int j = 0; j < NE; ++j)
            m = (l[j] > m) ? l[j] : m;                  // a NaN is never larger
        const Key mk = wave_top(order_key(m));
        m = lane_value(m, __builtin_ctzll(__ballot(order_key(m) == mk)));
        S sum = 0;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const S e = (m == inf) ? (l[j] == inf ? (S)1 : (S)0) : exp_of(l[j] - m);
            p[j] = (l[j] > -inf) ? e : (S)0;            // 0 for -inf and NaN, whatever m is
            sum += p[j];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int j = 0; j < NE; ++j)
            p[j] = (sum > (S)0) ? p[j] / sum : (S)0;
    } else {
#pragma unroll
        for (int j = 0; j < NE; ++j)
            p[j] = (l[j] == l[j]) ? (S)1 / ((S)1 + exp_of(-l[j])) : (S)0;
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        c[j] = p[j] + b[j];
        if (l[j] != l[j] || c[j] != c[j])
            c[j] = -inf;
    }

    // the groups that stay: group g's bit at g*P, P neighbouring lanes (a power
    // of two) working on one group; a group's values lie P further from the
    // group before in LDS than their number, which spreads the banks
    uint64_t stay = 0;
    int P = 1;
    const bool limited = a.topk_group < a.n_group;
    if (limited) {
        while (2 * P * a.n_group <= 64)
            P *= 2;
        S *mine = lds[wave];
#pragma unroll
        for (int j = 0; j < NE; ++j)
            if (e0 + j < a.E)
                mine[e0 + j + (((uint32_t)(e0 + j) * a.gs_inv) >> 22) * P] = c[j];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const int g = lane / P, sub = lane & (P - 1);
        S b1 = -inf, b2 = -inf;
        if (g < a.n_group) {
            const S *mg = mine + g * ((int)a.gs + P);
            for (int i = sub; i < (int)a.gs; i += P) {
                const S v = mg[i];
                b2 = (v > b1) ? b1 : (v > b2) ? v : b2;
                b1 = (v > b1) ? v : b1;
            }
        }
        for (int o = 1; o < P; o *= 2) {
            const S o1 = __shfl_xor(b1, o, 64), o2 = __shfl_xor(b2, o, 64);
            const S lower = (b1 > o1) ? o1 : b1, second = (b2 > o2) ? b2 : o2;
            b1 = (b1 > o1) ? b1 : o1;
            b2 = (lower > second) ? lower : second;
        }
        S score = (a.group_best == 2) ? b1 + b2 : b1;
        if (score != score)
            score = -inf;
        int rank = 0;
        for (int h = 0; h < a.n_group; ++h) {
            const S other = lane_value(score, h * P);
            rank += (other > score || (other == score && h < g)) ? 1 : 0;
        }
        stay = __ballot(g < a.n_group && sub == 0 && rank < a.topk_group);
    }
    Key key[NE], top = 0;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const uint32_t g = ((uint32_t)(e0 + j) * a.gs_inv) >> 22;
        const bool in = e0 + j < a.E && (!limited || ((stay >> (g * P)) & 1ull));
        key[j] = in ? order_key(c[j]) : (Key)0;
        top = max(top, key[j]);
    }

    // k times the largest key, the lowest expert of it first
    int my_e = 0;
    S my_p = 0, den = 0;
    for (int i = 0; i < a.k; ++i) {
        const Key best = wave_top(top);
        const int owner = __builtin_ctzll(__ballot(top == best));
        int je = 0;
        S jp = 0;
#pragma unroll
        for (int j = NE - 1; j >= 0; --j)
            if (key[j] == best) {
                je = e0 + j;
                jp = p[j];
            }
        const int e = __builtin_amdgcn_readlane(je, owner);
        const S pe = lane_value(jp, owner);
        den += pe;
        if (lane == i) {
            my_e = e;
            my_p = pe;
        }
        top = 0;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            if (e0 + j == e)
                key[j] = 0;
            top = max(top, key[j]);
        }
    }
    if (lane < a.k) {
        const S v = a.renorm ? ((den > (S)0) ? my_p / den : (S)0) : my_p;
        a.idx[(int64_t)t * a.k + lane] = my_e;
        a.w[(int64_t)t * a.k + lane] = (float)(v * (S)a.scale);
    }
}

template <typename LT>
static hipError_t enqueue_select(const SelectArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)((a.T + 3) / 4);
    const int ne = (a.E + 63) / 64;
    if (ne <= 1)
        launch(select_kernel<LT, 1>, grid, 256, 0, st, a);
    else if (ne <= 2)
        launch(select_kernel<LT, 2>, grid, 256, 0, st, a);
    else if (ne <= 4)
        launch(select_kernel<LT, 4>, grid, 256, 0, st, a);
    else if (ne <= 8)
        launch(select_kernel<LT, 8>, grid, 256, 0, st, a);
    else
        launch(select_kernel<LT, 16>, grid, 256, 0, st, a);
    return hipGetLastError();
}

static moe_status check_route(const moe_route_desc *d)
{
    if (!d)
        return fail(MOE_E_INVAL, "route desc is NULL");
    if (d->n_experts < 1 || d->n_experts > 1024)
        return fail(MOE_E_INVAL, "n_experts=%d must be in [1,1024]", d->n_experts);
    if (d->score != MOE_SCORE_SIGMOID && d->score != MOE_SCORE_SOFTMAX)
        return fail(MOE_E_INVAL, "unknown score %d", d->score);
    if (d->n_group < 1 || d->n_group > 64 || d->n_experts % d->n_group)
        return fail(MOE_E_INVAL, "n_group=%d must be in [1,64] and divide n_experts=%d", d->n_group,
                    d->n_experts);
    if (d->topk_group < 1 || d->topk_group > d->n_group)
        return fail(MOE_E_INVAL, "topk_group=%d must be in [1, n_group=%d]", d->topk_group, d->n_group);
    const int gs = d->n_experts / d->n_group;
    if (d->group_best != 1 && !(d->group_best == 2 && gs >= 2))
        return fail(MOE_E_INVAL, "group_best=%d must be 1, or 2 with at least 2 experts a group",
                    d->group_best);
    if (d->top_k < 1 || d->top_k > 32 || d->top_k > d->topk_group * gs)
        return fail(MOE_E_INVAL, "top_k=%d must be in [1, min(32, topk_group*E/n_group=%d)]", d->top_k,
                    d->topk_group * gs);
    if (d->renorm != 0 && d->renorm != 1)
        return fail(MOE_E_INVAL, "renorm=%d must be 0 or 1", d->renorm);
    if (!(d->scale >= 0.0f) || !(d->scale < INFINITY))
        return fail(MOE_E_INVAL, "scale must be finite and >= 0");
    return MOE_OK;
}

static SelectArgs select_args(const moe_route_desc *d, const void *logits, int64_t ld,
                              const float *bias, int32_t T, int32_t *idx, float *w)
{
    SelectArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.bias = bias;
    a.T = T;
    a.E = d->n_experts;
    a.k = d->top_k;
    a.softmax = d->score == MOE_SCORE_SOFTMAX;
    a.n_group = d->n_group;
    a.topk_group = d->topk_group;
    a.group_best = d->group_best;
    a.renorm = d->renorm;
    a.scale = d->scale;
    a.gs = (uint32_t)(d->n_experts / d->n_group);
    a.gs_inv = ((1u << 22) + a.gs - 1) / a.gs;
    a.idx = idx;
    a.w = w;
    return a;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_route_select(const moe_route_desc *desc, const void *logits,
                                       int32_t logit_dtype, int64_t ld, const float *bias,
                                       int32_t T, int32_t *idx, float *gate_w, void *stream)
{
    moe_status st = check_route(desc);
    if (st)
        return st;
    if (!ops_dtype_ok(logit_dtype))
        return fail(MOE_E_INVAL, "unknown logit_dtype %d", logit_dtype);
    if (T < 0 || T > (1 << 20))
        return fail(MOE_E_INVAL, "T=%d out of range [0, 2^20]", T);
    if (T == 0)
        return MOE_OK;
    if (!logits || !idx || !gate_w)
        return fail(MOE_E_INVAL, "logits/idx/gate_w is NULL");
    if (ld < desc->n_experts)
        return fail(MOE_E_INVAL, "ld=%lld is below n_experts=%d", (long long)ld, desc->n_experts);
    if (!ops_aligned(logits, logit_dtype == MOE_DT_F32 ? 4 : 2) || !ops_aligned(bias, 4) ||
        !ops_aligned(idx, 4) || !ops_aligned(gate_w, 4))
        return fail(MOE_E_INVAL, "logits, bias, idx and gate_w must be aligned to their elements");
    if ((st = ops_check_device()) != MOE_OK)
        return st;
    const SelectArgs a = select_args(desc, logits, ld, bias, T, idx, gate_w);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    const hipError_t e = logit_dtype == MOE_DT_F32 ? enqueue_select<float>(a, hs)
                                                   : enqueue_select<bf16_t>(a, hs);
    return e == hipSuccess ? MOE_OK : hip_fail(e, "selection launch");
}

extern "C" moe_status moe_router_topk_grouped(moe_ctx *ctx, const moe_route_desc *desc,
                                              const void *x, int32_t T, const moe_layer_weights *w,
                                              int32_t *idx, float *gate_w, void *stream)
{
    const moe_status st = check_route(desc);
    if (st)
        return st;
    if (!ctx)
        return fail(MOE_E_INVAL, "ctx is NULL");
    if (desc->n_experts != ctx->d.n_experts)
        return fail(MOE_E_INVAL, "n_experts=%d, the layer has %d", desc->n_experts, ctx->d.n_experts);
    if (T < 0 || T > ctx->max_tokens)
        return fail(MOE_E_INVAL, "T=%d out of range [0,%d]", T, ctx->max_tokens);
    if (!w)
        return fail(MOE_E_INVAL, "weights is NULL");
    if (T == 0)
        return MOE_OK;
    if (!x || !idx || !gate_w)
        return fail(MOE_E_INVAL, "x/idx/gate_w is NULL");
    if (!w->router_w)
        return fail(MOE_E_INVAL, "router weights are NULL");
    hipStream_t hs = static_cast<hipStream_t>(stream);
    const int H = ctx->d.hidden, E = ctx->d.n_experts;
    ctx->last_T = T;
    prof_begin(ctx, MOE_PROF_ROUTER, hs);
    hipError_t e = launch_router_logits(static_cast<const uint16_t *>(x), T, H, w->router_w, E,
                                        ctx->logits, hs);
    if (e != hipSuccess)
        return hip_fail(e, "router logits launch");
    prof_end(ctx, MOE_PROF_ROUTER, hs);
    SelectArgs a = select_args(desc, ctx->logits, E, w->router_bias, T, idx, gate_w);
    if (router_ksplit(T, H, E) == 2)
        a.part2 = ctx->logits + (size_t)T * E;
    prof_begin(ctx, MOE_PROF_TOPK, hs);
    e = enqueue_select<double>(a, hs);
    if (e != hipSuccess)
        return hip_fail(e, "selection launch");
    prof_end(ctx, MOE_PROF_TOPK, hs);
    return prof_collect(ctx);
}
