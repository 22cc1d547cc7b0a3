// kernels_route.hip -- selection of experts with groups on gfx950: softmax or
// sigmoid scores, a bias that only steers the choice, the best groups, the k
// best experts inside them, weights renormalised or as they are.
//
// One wave per token, expert e on lane e/NE (register e%NE), so that the first
// lane of a ballot holds the lowest expert.  Each lane sorts its NE candidates
// once; then k times the best of the 64 first candidates is taken (a DPP
// maximum over the wave) and its lane moves on.  A token's logits are read once
// and stay in registers.  Bound by instructions, the k dependent maxima first
// among them: 16 tokens of 256 experts in 8 groups 3.9 us, 4096 5.75, 16384
// 15.7 (launches in a graph; 4.2 MB in and out at 4096 would take 1 us).  With
// the best found among all NE registers each time, the library's exp and IEEE
// quotients, 4096 took 7.4.
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
    int lanes;                     // lanes that hold a group's experts and no others, a power
                                   // of two; 0: there is no such number
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
// exp and reciprocal.  fp32: 2^(v*log2 e) with the product's remainder added, so
// that the error does not grow with |v|, and the hardware's reciprocal, each
// about a unit in the last place (the library's exp and an IEEE quotient were a
// fifth of the selection's instructions); v up to 88, 0 past -200 (for -inf too).
// fp64: the library's.
__device__ __forceinline__ float exp_of(float v, float above = 0.0f)
{
    const float L2E = 1.44269502f, L2E_LO = 1.92596303e-8f;   // log2(e) = L2E + L2E_LO
    const float a = __builtin_amdgcn_fmed3f(v, -200.0f, 88.0f);
    const float t = a * L2E;
    const float r = fmaf(a, L2E, -t) + a * L2E_LO;
    const float e = __builtin_amdgcn_exp2f(t + above);
    return fmaf(e, r * 0.693147181f, e);
}
__device__ __forceinline__ double exp_of(double v)
{
    return exp(v);
}
__device__ __forceinline__ float inverse(float v)
{
    return __builtin_amdgcn_rcpf(v);
}
__device__ __forceinline__ double inverse(double v)
{
    return 1.0 / v;
}

// The hardware's 2^t and reciprocal give 0 below 2^-126.  Scores there (v from
// -200 to -80; 0 from -104 on) keep their order as fp32's subnormals: 2^t is taken
// 2^64 higher and brought down by an exact product that rounds once.  Rarely
// needed, so a wave asks once for all its values.
__device__ __forceinline__ bool is_low(float v)
{
    return fabsf(v + 140.0f) < 60.0f;
}
__device__ __forceinline__ float exp_low(float v)
{
    return exp_of(v, 64.0f) * 0x1p-64f;
}

// p[j] = exp(v[j]), v[j] <= 0
template <int NE>
__device__ __forceinline__ void exp_each(const float (&v)[NE], float (&p)[NE])
{
    bool low = false;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        p[j] = exp_of(v[j]);
        low |= is_low(v[j]);
    }
    if (__ballot(low)) {
#pragma unroll
        for (int j = 0; j < NE; ++j)
            p[j] = is_low(v[j]) ? exp_low(v[j]) : p[j];
    }
}
template <int NE>
__device__ __forceinline__ void exp_each(const double (&v)[NE], double (&p)[NE])
{
#pragma unroll
    for (int j = 0; j < NE; ++j)
        p[j] = exp_of(v[j]);
}
// p[j] = 1/(1 + exp(-l[j])), which is exp(l[j]) in fp32 where that is low, and 0
// below (for -inf too); 0 for a NaN
template <int NE>
__device__ __forceinline__ void sigmoid_each(const float (&l)[NE], float (&p)[NE])
{
    bool low = false;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        p[j] = inverse(1.0f + exp_of(-l[j]));
        p[j] = (l[j] > -200.0f) ? p[j] : 0.0f;
        low |= is_low(l[j]);
    }
    if (__ballot(low)) {
#pragma unroll
        for (int j = 0; j < NE; ++j)
            p[j] = is_low(l[j]) ? exp_low(l[j]) : p[j];
    }
}
template <int NE>
__device__ __forceinline__ void sigmoid_each(const double (&l)[NE], double (&p)[NE])
{
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        p[j] = inverse(1.0 + exp_of(-l[j]));
        p[j] = (l[j] == l[j]) ? p[j] : 0.0;
    }
}

// A candidate: its key and its expert, in the order of choice: the larger key,
// of equal ones the lower expert.
template <typename Key>
struct Cand;
template <>
struct Cand<uint32_t> {
    uint64_t v;
    __device__ __forceinline__ void set(uint32_t key, int e)
    {
        v = (uint64_t)key << 32 | (uint32_t)~e;
    }
    __device__ __forceinline__ uint32_t key() const
    {
        return (uint32_t)(v >> 32);
    }
    __device__ __forceinline__ int expert() const
    {
        return (int)~(uint32_t)v;
    }
    __device__ __forceinline__ bool before(const Cand &o) const
    {
        return v > o.v;
    }
};
template <>
struct Cand<uint64_t> {
    uint64_t k;
    int e;
    __device__ __forceinline__ void set(uint64_t key, int expert)
    {
        k = key;
        e = expert;
    }
    __device__ __forceinline__ uint64_t key() const
    {
        return k;
    }
    __device__ __forceinline__ int expert() const
    {
        return e;
    }
    __device__ __forceinline__ bool before(const Cand &o) const
    {
        return k > o.k || (k == o.k && e < o.e);
    }
};

// Batcher's odd-even merge sort of N (a power of two) candidates, first first.
template <int N, typename C>
__device__ __forceinline__ void sort_cands(C (&c)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        C &a = c[i + j], &b = c[i + j + k];
                        const bool swap = b.before(a);
                        const C t = a;
                        a = swap ? b : a;
                        b = swap ? t : b;
                    }
}

// The two best of pairs (b1 >= b2) held by this lane and another.
template <typename S>
__device__ __forceinline__ void merge_best(S &b1, S &b2, S o1, S o2)
{
    const S lower = (b1 > o1) ? o1 : b1, second = (b2 > o2) ? b2 : o2;
    b1 = (b1 > o1) ? b1 : o1;
    b2 = (lower > second) ? lower : second;
}
template <int CTRL>
__device__ __forceinline__ float dpp_value(float v)
{
    return __int_as_float(dpp0<CTRL, 0xf>(__float_as_int(v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp_value(double v)
{
    const long long u = __double_as_longlong(v);
    const uint32_t lo = (uint32_t)dpp0<CTRL, 0xf>((int)(u & 0xffffffffll));
    const uint32_t hi = (uint32_t)dpp0<CTRL, 0xf>((int)(u >> 32));
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
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

    // logits and bias of this lane's experts, all loads issued before any use;
    // a lane past the experts reads the last one's and drops them
    struct __attribute__((packed, aligned(4))) Bias {
        float v[NE];
    };
    S l[NE], b[NE];
    const LT *row = static_cast<const LT *>(a.logits) + (int64_t)t * a.ld;
    {
        Piece lp;
        Bias bp;
        if (e0 + NE <= a.E) {
            lp = *reinterpret_cast<const Piece *>(row + e0);
            if (a.bias)
                bp = *reinterpret_cast<const Bias *>(a.bias + e0);
        } else {
#pragma unroll
            for (int j = 0; j < NE; ++j)
                lp.v[j] = row[min(e0 + j, a.E - 1)];
            if (a.bias) {
#pragma unroll
                for (int j = 0; j < NE; ++j)
                    bp.v[j] = a.bias[min(e0 + j, a.E - 1)];
            }
        }
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            l[j] = (e0 + j < a.E) ? widen(lp.v[j]) : -inf;
            b[j] = a.bias ? (S)bp.v[j] : (S)0;
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
        S sum = 0, v[NE];
#pragma unroll
        for (int j = 0; j < NE; ++j)
            v[j] = l[j] - m;
        exp_each(v, p);
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const S e = (m == inf) ? (l[j] == inf ? (S)1 : (S)0) : p[j];
            p[j] = (l[j] > -inf) ? e : (S)0;            // 0 for -inf and NaN, whatever m is
            sum += p[j];
        }
        sum = wave_sum(sum);
        const S by = (sum > (S)0) ? inverse(sum) : (S)0;
#pragma unroll
        for (int j = 0; j < NE; ++j)
            p[j] *= by;
    } else {
        sigmoid_each(l, p);
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        c[j] = p[j] + b[j];
        if (l[j] != l[j] || c[j] != c[j])
            c[j] = -inf;
    }

    // the groups that stay: group g's bit at g*P, P neighbouring lanes (a power
    // of two) working on one group.  Where a group's experts are just P lanes'
    // (256 experts in 8 groups: 8 lanes of 4) they begin with their own in
    // registers; else the values go through LDS, a group's P further from the
    // group before than their number, which spreads the banks (4096 tokens of
    // 256 experts, launches in a graph: 6.1 us through LDS, 5.75 in registers).
    uint64_t stay = 0;
    int P = 1;
    const bool limited = a.topk_group < a.n_group;
    if (limited) {
        S b1 = -inf, b2 = -inf;
        if (a.lanes) {
            P = a.lanes;
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                b2 = (c[j] > b1) ? b1 : (c[j] > b2) ? c[j] : b2;
                b1 = (c[j] > b1) ? c[j] : b1;
            }
        } else {
            while (2 * P * a.n_group <= 64)
                P *= 2;
            S *mine = lds[wave];
#pragma unroll
            for (int j = 0; j < NE; ++j) {
                // the last place is nobody's: for what lies past the experts
                const int at = e0 + j + (int)((((uint32_t)(e0 + j) * a.gs_inv) >> 22) * P);
                mine[(e0 + j < a.E) ? at : 64 * NE + 63] = c[j];
            }
            wave_lds_sync();
            const int g = lane / P;
            if (g < a.n_group) {
                const S *mg = mine + g * ((int)a.gs + P);
                int i = lane & (P - 1);
                for (; i + 3 * P < (int)a.gs; i += 4 * P) {     // four reads on their way
                    S v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        v[u] = mg[i + u * P];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        b2 = (v[u] > b1) ? b1 : (v[u] > b2) ? v[u] : b2;
                        b1 = (v[u] > b1) ? v[u] : b1;
                    }
                }
                for (; i < (int)a.gs; i += P) {
                    const S v = mg[i];
                    b2 = (v > b1) ? b1 : (v > b2) ? v : b2;
                    b1 = (v > b1) ? v : b1;
                }
            }
        }
        const int g = lane / P, sub = lane & (P - 1);
        // a group's lanes together: neighbours, pairs, then mirrored halves
        // (once four or eight lanes agree, the mirror lies in the others)
        if (P > 1)
            merge_best(b1, b2, dpp_value<0xB1>(b1), dpp_value<0xB1>(b2));      // quad_perm 1,0,3,2
        if (P > 2)
            merge_best(b1, b2, dpp_value<0x4E>(b1), dpp_value<0x4E>(b2));      // quad_perm 2,3,0,1
        if (P > 4)
            merge_best(b1, b2, dpp_value<0x141>(b1), dpp_value<0x141>(b2));    // row_half_mirror
        if (P > 8)
            merge_best(b1, b2, dpp_value<0x140>(b1), dpp_value<0x140>(b2));    // row_mirror
        if (P > 16)
            merge_best(b1, b2, (S)__shfl_xor(b1, 16, 64), (S)__shfl_xor(b2, 16, 64));
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
    // this lane's candidates in the order of choice; p for whoever is chosen
    Cand<Key> cand[NE];
    S *mine = lds[wave];
    wave_lds_sync();
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const uint32_t g = ((uint32_t)(e0 + j) * a.gs_inv) >> 22;
        const bool in = e0 + j < a.E && (!limited || ((stay >> (g * P)) & 1ull));
        cand[j].set(in ? order_key(c[j]) : (Key)0, e0 + j);
        mine[e0 + j] = p[j];
    }
    sort_cands(cand);

    // k times the largest of the lanes' first candidates, the lowest lane's
    // where they are equal; that lane moves on to its next
    int my_e = 0;
    for (int i = 0; i < a.k; ++i) {
        const Key best = wave_top(cand[0].key());
        const int owner = __builtin_ctzll(__ballot(cand[0].key() == best));
        const int e = __builtin_amdgcn_readlane(cand[0].expert(), owner);
        my_e = (lane == i) ? e : my_e;
        const bool won = lane == owner;
#pragma unroll
        for (int j = 0; j + 1 < NE; ++j)
            cand[j] = won ? cand[j + 1] : cand[j];
        if (won)
            cand[NE - 1].set((Key)0, 0);
    }
    wave_lds_sync();
    const S my_p = (lane < a.k) ? mine[my_e] : (S)0;
    const S den = wave_sum(my_p);
    if (lane < a.k) {
        const S v = a.renorm ? ((den > (S)0) ? my_p / den : (S)0) : my_p;
        a.idx[(int64_t)t * a.k + lane] = my_e;
        a.w[(int64_t)t * a.k + lane] = (float)(v * (S)a.scale);
    }
}

template <typename LT, int NE>
static void launch_select(SelectArgs a, hipStream_t st)
{
    const int lanes = (int)a.gs / NE;
    a.lanes = (a.gs % NE == 0 && (lanes & (lanes - 1)) == 0) ? lanes : 0;
    launch(select_kernel<LT, NE>, (unsigned)((a.T + 3) / 4), 256, 0, st, a);
}

template <typename LT>
static hipError_t enqueue_select(const SelectArgs &a, hipStream_t st)
{
    if (a.E <= 64)
        launch_select<LT, 1>(a, st);
    else if (a.E <= 128)
        launch_select<LT, 2>(a, st);
    else if (a.E <= 256)
        launch_select<LT, 4>(a, st);
    else if (a.E <= 512)
        launch_select<LT, 8>(a, st);
    else
        launch_select<LT, 16>(a, st);
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
