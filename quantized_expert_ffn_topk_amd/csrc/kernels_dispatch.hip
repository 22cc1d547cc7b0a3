// kernels_dispatch.hip -- the way of routed rows to their experts and back on
// gfx950: the stable grouping of (token, rank) by expert, and the weighted sum of
// a token's expert rows.
#include "ops_common.h"

namespace moe {

struct GroupArgs {
    const int32_t *idx;
    int32_t *offsets, *rows, *pos;
    int M, k, E;               // M = T*k
};

// ---------------------------------------------------------------------------
// Grouping up to 65536 ids in one launch without a workspace: a block per expert
// reads all ids, counts those below its own (its offset) and lists its own.  Wave w
// has a run of neighbouring ids, 64 at a time, so its list follows those of the
// waves before it.  Bound by the instructions of all blocks' rounds (E*M/64 in all):
// two comparisons each, no bounds in whole batches, more only where an id is found.
// In a graph 16 x 8 of 256 3.1 us, a launch; 1024 x 8 3.9; 4096 x 8 5.7; 8192 x 8 8.3.  The
// three sizes of lists are for what a block's LDS leaves to others and how many loads are worth a
// batch; the limit is that of a CU's LDS.
// ---------------------------------------------------------------------------
constexpr int GROUP_W = 16;                          // waves
constexpr int GROUP_ONE = 64 * 64 * GROUP_W;         // ids of one launch

// BATCH: rounds whose loads are in flight at once; ROUNDS: of a wave at most
template <int BATCH, int ROUNDS>
__global__ __launch_bounds__(64 * GROUP_W) void group_rows_kernel(GroupArgs a)
{
    __shared__ int below[GROUP_W], own[GROUP_W];
    __shared__ uint16_t found[GROUP_W][64 * ROUNDS]; // places in the wave's run
    const int lane = threadIdx.x & 63, e = blockIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rounds = (a.M + 64 * GROUP_W - 1) / (64 * GROUP_W), first = wave * rounds * 64;
    // an id that is no expert has no row: each block looks for them among its share
    for (int i = (int)((int64_t)a.M * e / a.E) + (int)threadIdx.x; i < (int)((int64_t)a.M * (e + 1) / a.E); i += 64 * GROUP_W)
        if ((unsigned)a.idx[i] >= (unsigned)a.E)
            a.pos[i] = -1;
    int nb = 0, no = 0;
    auto count = [&](const int (&id)[BATCH], int r0) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const unsigned long long m = __ballot(id[j] == e);
            nb += __popcll(__ballot((unsigned)id[j] < (unsigned)e));
            if (m) {
                if (id[j] == e)
                    found[wave][no + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(64 * (r0 + j) + lane);
                no += __popcll(m);
            }
        }
    };
    int r0 = 0;
    for (; r0 + BATCH <= rounds && first + 64 * (r0 + BATCH) <= a.M; r0 += BATCH) {
        int id[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            id[j] = a.idx[first + 64 * r0 + lane + 64 * j];
        count(id, r0);
    }
    for (; r0 < rounds && first + 64 * r0 < a.M; r0 += BATCH) {   // the last ids
        int id[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int i = first + 64 * (r0 + j) + lane;
            id[j] = (r0 + j < rounds && i < a.M) ? a.idx[i] : INT_MAX;
        }
        count(id, r0);
    }
    if (lane == 0) {
        below[wave] = nb;
        own[wave] = no;
    }
    __syncthreads();
    int base = 0, at = 0, total = 0;
#pragma unroll
    for (int w = 0; w < GROUP_W; ++w) {
        base += below[w];
        at += (w < wave) ? own[w] : 0;
        total += own[w];
    }
    if (threadIdx.x == 0) {
        a.offsets[e] = base;
        if (e == a.E - 1)
            a.offsets[a.E] = base + total;
    }
    for (int n = lane; n < no; n += 64) {
        const int i = first + found[wave][n], g = base + at + n;
        a.rows[g] = i / a.k;
        a.pos[i] = g;
    }
}

// ---------------------------------------------------------------------------
// More ids, in three launches: the counts of each run of GROUP_RUN ids, their
// sums over the runs, and each run's ids by these.  The counts of a run lie at the
// beginning of its own part of pos until the last step takes them out and writes
// pos itself (a run is longer than the experts are many).  27 us for 66048 ids of 256
// experts, 28 for 131072, 47 for 2^20: not the launches but few long runs (4 blocks, 8, 64) that each
// walk their ids twice in 16 rounds or more, and one block that adds up the runs.
// ---------------------------------------------------------------------------
constexpr int GROUP_RUN = 16384;
constexpr int MAX_E = 1024;

// ids [first, last) of run r: the last run has the remainder too
__device__ __forceinline__ void run_of(const GroupArgs &a, int r, int runs, int *first, int *last)
{
    *first = r * GROUP_RUN;
    *last = (r == runs - 1) ? a.M : *first + GROUP_RUN;
}

__global__ __launch_bounds__(1024) void group_count_kernel(GroupArgs a, int runs)
{
    __shared__ int count[MAX_E];
    int first, last;
    run_of(a, blockIdx.x, runs, &first, &last);
    count[threadIdx.x] = 0;
    __syncthreads();
    for (int i = first + (int)threadIdx.x; i < last; i += 1024) {
        const int id = a.idx[i];
        if ((unsigned)id < (unsigned)a.E)
            atomicAdd(&count[id], 1);                // whole numbers: any order
    }
    __syncthreads();
    if ((int)threadIdx.x < a.E)
        a.pos[first + threadIdx.x] = count[threadIdx.x];
}

__global__ __launch_bounds__(1024) void group_sum_kernel(GroupArgs a, int runs)
{
    __shared__ int waves[16];
    const int e = threadIdx.x, lane = e & 63, wave = e >> 6;
    int n = 0;
    if (e < a.E)
        for (int r = 0; r < runs; ++r)
            n += a.pos[r * GROUP_RUN + e];
    int incl = n;
#define STEP(c, r) incl += dpp0<c, r>(incl);
    MOE_DPP_STEPS(STEP)
#undef STEP
    if (lane == 63)
        waves[wave] = incl;
    __syncthreads();
    int base = incl - n;
    for (int w = 0; w < wave; ++w)
        base += waves[w];
    if (e < a.E) {
        a.offsets[e] = base;
        if (e == a.E - 1)
            a.offsets[a.E] = base + n;
        for (int r = 0; r < runs; ++r) {
            int32_t *p = a.pos + r * GROUP_RUN + e;
            const int c = *p;
            *p = base;
            base += c;
        }
    }
}

// A wave has a run of neighbouring ids of the block's; next[w][e] is where wave
// w's next id of expert e goes.  Of 64 ids a lane finds its equals by a ballot
// for each bit of an id.
__global__ __launch_bounds__(1024) void group_place_kernel(GroupArgs a, int runs)
{
    __shared__ int next[16][MAX_E];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int first, last;
    run_of(a, blockIdx.x, runs, &first, &last);
    const int rounds = (last - first + 1023) / 1024, w0 = first + wave * rounds * 64;
    const int base = ((int)threadIdx.x < a.E) ? a.pos[first + threadIdx.x] : 0;
    for (int w = 0; w < 16; ++w)
        next[w][threadIdx.x] = 0;
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
        const int i = w0 + 64 * r + lane;
        const int id = (i < last) ? a.idx[i] : -1;
        if ((unsigned)id < (unsigned)a.E)
            atomicAdd(&next[wave][id], 1);
    }
    __syncthreads();
    int at = base;
    for (int w = 0; w < 16; ++w) {
        const int c = next[w][threadIdx.x];
        next[w][threadIdx.x] = at;
        at += c;
    }
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
        const int i = w0 + 64 * r + lane;
        const int id = (i < last) ? a.idx[i] : -1;
        const bool in = (unsigned)id < (unsigned)a.E;
        unsigned long long equal = __ballot(in);
#pragma unroll
        for (int b = 0; b < 10; ++b) {
            const unsigned long long m = __ballot((id >> b) & 1);
            equal &= ((id >> b) & 1) ? m : ~m;
        }
        if (in) {
            const int before = __popcll(equal & ((1ull << lane) - 1));
            const int g = next[wave][id] + before;
            a.rows[g] = i / a.k;
            a.pos[i] = g;
            wave_lds_sync();
            if (before == 0)
                next[wave][id] += __popcll(equal);
        } else if (i < last) {
            a.pos[i] = -1;
        }
        wave_lds_sync();
    }
}

// ---------------------------------------------------------------------------
// out[t] = base[t] + sum_i w[t,i] * y[pos[t,i]], fp32 FMAs in the order of i,
// rounded once.  A thread has eight columns of a token; the loads of eight of
// its rows are in flight at once.  Bound by HBM: 4096 x 8 x 6144 with base 98 us (5.1 TB/s);
// 1 x 8 x 6144 3.1 us in a graph.  Columns behind the last eight are one thread's, row after row:
// 1 x 8 x 6143 10.5 us, 4096 x 8 x 6143 144.
// ---------------------------------------------------------------------------
struct CombineArgs {
    const void *y, *base;
    const int32_t *pos;
    const float *w;
    void *out;
    int64_t ldy, ldb, ldo;
    int R, T, k, H;
};

template <typename YT, typename OT>
__global__ __launch_bounds__(256) void combine_rows_kernel(CombineArgs a)
{
    const int t = blockIdx.y + 65535 * blockIdx.z;
    const int col = 8 * ((int)blockIdx.x * (int)blockDim.x + (int)threadIdx.x);
    if (t >= a.T || col >= a.H)
        return;
    const int32_t *pos = a.pos + (int64_t)t * a.k;
    const float *w = a.w + (int64_t)t * a.k;
    const YT *y = static_cast<const YT *>(a.y) + col;
    const OT *base = a.base ? static_cast<const OT *>(a.base) + (int64_t)t * a.ldb + col : nullptr;
    OT *out = static_cast<OT *>(a.out) + (int64_t)t * a.ldo + col;
    float v[8];
    if (col + 8 <= a.H) {
        raw8<OT> b;
        if (base)
            b.load(base);
        if (base) {
            b.widen(v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = 0.0f;
        }
        for (int i0 = 0; i0 < a.k; i0 += 8) {
            raw8<YT> r[8];
            float wi[8];
            bool in[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = (i0 + i < a.k) ? pos[i0 + i] : -1;
                in[i] = (unsigned)p < (unsigned)a.R;
                wi[i] = in[i] ? w[i0 + i] : 0.0f;
                if (in[i])
                    r[i].load(y + (int64_t)p * a.ldy);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (in[i]) {
                    float x[8];
                    r[i].widen(x);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = fmaf(wi[i], x[j], v[j]);
                }
            }
        }
        store8(out, v);
        return;
    }
    for (int j = 0; j < a.H - col; ++j) {            // the row's last columns
        float s = base ? to_f32(base[j]) : 0.0f;
        for (int i = 0; i < a.k; ++i)
            if ((unsigned)pos[i] < (unsigned)a.R)
                s = fmaf(w[i], to_f32(y[(int64_t)pos[i] * a.ldy + j]), s);
        store1(out + j, s);
    }
}

template <typename YT, typename OT>
static void enqueue_combine(const CombineArgs &a, hipStream_t st)
{
    const int cols = (a.H + 7) / 8, nt = 64;
    const dim3 grid((cols + nt - 1) / nt, a.T < 65535 ? a.T : 65535, (a.T + 65534) / 65535);
    launch(combine_rows_kernel<YT, OT>, grid, nt, 0, st, a);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_group_rows(const int32_t *idx, int32_t T, int32_t k, int32_t E,
                                     int32_t *offsets, int32_t *rows, int32_t *pos, void *stream)
{
    if (T < 0 || T > (1 << 20))
        return fail(MOE_E_INVAL, "T=%d out of range [0, 2^20]", T);
    if (k < 1 || k > 32)
        return fail(MOE_E_INVAL, "k=%d must be in [1, 32]", k);
    if (E < 1 || E > MAX_E)
        return fail(MOE_E_INVAL, "E=%d must be in [1, 1024]", E);
    if (!offsets || (T > 0 && (!idx || !rows || !pos)))
        return fail(MOE_E_INVAL, "idx/offsets/rows/pos is NULL");
    if (!ops_aligned(idx, 4) || !ops_aligned(offsets, 4) || !ops_aligned(rows, 4) || !ops_aligned(pos, 4))
        return fail(MOE_E_INVAL, "idx, offsets, rows and pos must be aligned to their elements");
    const moe_status st = ops_check_device();
    if (st)
        return st;
    const GroupArgs a{idx, offsets, rows, pos, T * k, k, E};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (a.M <= GROUP_ONE) {
        if (a.M <= 4 * 64 * GROUP_W)
            launch(group_rows_kernel<4, 4>, (unsigned)E, 64 * GROUP_W, 0, hs, a);
        else if (a.M <= 16 * 64 * GROUP_W)
            launch(group_rows_kernel<8, 16>, (unsigned)E, 64 * GROUP_W, 0, hs, a);
        else
            launch(group_rows_kernel<16, 64>, (unsigned)E, 64 * GROUP_W, 0, hs, a);
    } else {
        const int runs = a.M / GROUP_RUN;
        launch(group_count_kernel, (unsigned)runs, 1024, 0, hs, a, runs);
        launch(group_sum_kernel, 1, 1024, 0, hs, a, runs);
        launch(group_place_kernel, (unsigned)runs, 1024, 0, hs, a, runs);
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_fail(e, "grouping launch");
}

extern "C" moe_status moe_combine_rows(const void *y, int32_t y_dtype, int64_t ldy, int32_t R,
                                       const int32_t *pos, const float *gate_w, const void *base,
                                       int64_t ldb, int32_t T, int32_t k, int32_t H, void *out,
                                       int32_t out_dtype, int64_t ldo, void *stream)
{
    if (!ops_dtype_ok(y_dtype) || !ops_dtype_ok(out_dtype))
        return fail(MOE_E_INVAL, "unknown y_dtype %d or out_dtype %d", y_dtype, out_dtype);
    if (T < 0 || T > (1 << 20))
        return fail(MOE_E_INVAL, "T=%d out of range [0, 2^20]", T);
    if (k < 1 || k > 32)
        return fail(MOE_E_INVAL, "k=%d must be in [1, 32]", k);
    if (H < 1 || H > (1 << 20))
        return fail(MOE_E_INVAL, "H=%d must be in [1, 2^20]", H);
    if (R < 0)
        return fail(MOE_E_INVAL, "R=%d is negative", R);
    if (T == 0)
        return MOE_OK;
    if ((R > 0 && !y) || !pos || !gate_w || !out)
        return fail(MOE_E_INVAL, "y/pos/gate_w/out is NULL");
    if ((R > 0 && ldy < H) || (base && ldb < H) || ldo < H)
        return fail(MOE_E_INVAL, "a leading dimension is below H=%d", H);
    if (base == out && T > 1 && ldb != ldo)          // a row of out would be another one's base
        return fail(MOE_E_INVAL, "base is out, but ldb=%lld and ldo=%lld", (long long)ldb, (long long)ldo);
    const size_t os = out_dtype == MOE_DT_F32 ? 4 : 2;
    if (!ops_aligned(y, y_dtype == MOE_DT_F32 ? 4 : 2) || !ops_aligned(pos, 4) || !ops_aligned(gate_w, 4) ||
        !ops_aligned(base, os) || !ops_aligned(out, os))
        return fail(MOE_E_INVAL, "y, pos, gate_w, base and out must be aligned to their elements");
    const moe_status st = ops_check_device();
    if (st)
        return st;
    const CombineArgs a{y, base, pos, gate_w, out, ldy, ldb, ldo, R, T, k, H};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (y_dtype == MOE_DT_F32)
        out_dtype == MOE_DT_F32 ? enqueue_combine<float, float>(a, hs) : enqueue_combine<float, bf16_t>(a, hs);
    else
        out_dtype == MOE_DT_F32 ? enqueue_combine<bf16_t, float>(a, hs) : enqueue_combine<bf16_t, bf16_t>(a, hs);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_fail(e, "combine launch");
}
