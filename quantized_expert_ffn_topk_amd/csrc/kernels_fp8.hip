// kernels_fp8.hip -- rows, or the SwiGLU of rows, as E4M3 codes with an fp32 scale
// for each block of 128 neighbouring values, on gfx950.
//
// Per block: a = max |v|, s = a/448, q = e4m3(v * (448/a)), the steps in fp32, the
// code rounded to nearest even (v_cvt_pk_fp8_f32).
#include "ops_common.h"

namespace moe {

struct Fp8Args {
    const void *x;
    uint8_t *q;
    float *s;
    const int32_t *count;      // NULL: all T rows
    int64_t ldx, ldq, lds;
    int T, K;
};

// The scale of a block whose largest magnitude has the fp32 bits m, and the
// multiplier of its codes: blocks below 2^-96 are multiplied by pre = 2^64 first
// (exact), so that 448/a stays finite.  A block with a NaN or an infinity gets
// the scale NaN and codes 0.
__device__ __forceinline__ void block_scale(uint32_t m, float *s, float *pre, float *inv)
{
    const float a = __uint_as_float(m);
    *s = a / 448.0f;
    *pre = (a < 0x1p-96f) ? 0x1p64f : 1.0f;
    *inv = (m == 0u) ? 0.0f : 448.0f / (a * *pre);
    if (m >= 0x7f800000u) {
        *s = __uint_as_float(0x7fc00000u);
        *inv = 0.0f;
    }
}

// maximum over the 16 lanes of a DPP row, in each of them
__device__ __forceinline__ uint32_t row16_top(uint32_t v)
{
#define STEP(c) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, c, 0xf, 0xf, true));
    STEP(0x121)                                      // row_ror:1
    STEP(0x122)
    STEP(0x124)
    STEP(0x128)
#undef STEP
    return v;
}

// ---------------------------------------------------------------------------
// 16 lanes per block of 128, eight values a lane (16 bytes of bf16), the blocks of all
// rows in one count: one pass, no LDS, the maximum by four lane rotations.  Bound by
// HBM: SwiGLU of 32768 x 2048 63 us (5.4 TB/s read and written), 4096 x 6144 14.9 us;
// one row of 6144 2.2 us in a graph, a launch.
// ---------------------------------------------------------------------------
template <typename XT, bool SWIGLU>
__global__ __launch_bounds__(256) void quant_fp8_kernel(Fp8Args a, int blocks)
{
    const int lane = threadIdx.x & 15;
    const int rows = a.count ? min(a.T, max(*a.count, 0)) : a.T;
    const int b = (int)blockIdx.x * 16 + (int)(threadIdx.x >> 4);
    if (b >= rows * blocks)
        return;
    const int t = b / blocks, col = 128 * (b - t * blocks) + 8 * lane;
    const XT *x = static_cast<const XT *>(a.x) + (int64_t)t * a.ldx;
    const bool whole = col + 8 <= a.K;
    float v[8], w[8];
    if (whole) {
        raw8<XT> g, u;
        g.load(x + col);
        if constexpr (SWIGLU)
            u.load(x + a.K + col);
        g.widen(v);
        if constexpr (SWIGLU)
            u.widen(w);
    } else {                                         // the row's end
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = (col + j < a.K) ? to_f32(x[col + j]) : 0.0f;
            w[j] = (SWIGLU && col + j < a.K) ? to_f32(x[a.K + col + j]) : 0.0f;
        }
    }
    if constexpr (SWIGLU) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = silu_mul(v[j], w[j]);
    }
    // the maximum that keeps a NaN, then bits: NaN is largest
    float big = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        big = __builtin_elementwise_maximum(big, fabsf(v[j]));
    float s, pre, inv;
    block_scale(row16_top(__float_as_uint(big) & 0x7fffffffu), &s, &pre, &inv);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = (inv == 0.0f) ? 0.0f : (v[j] * pre) * inv;
    bytes8_a1 q;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        int d = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j], v[4 * j + 1], 0, false);
        d = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j + 2], v[4 * j + 3], d, true);
        q.d[j] = (uint32_t)d;
    }
    uint8_t *to = a.q + (int64_t)t * a.ldq + col;
    if (whole) {
        *reinterpret_cast<bytes8_a1 *>(to) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < a.K)
                to[j] = (uint8_t)(q.d[j >> 2] >> (8 * (j & 3)));
    }
    if (lane == 0)
        a.s[(int64_t)t * a.lds + (col >> 7)] = s;
}

template <typename XT, bool SWIGLU>
static void enqueue_quant(const Fp8Args &a, hipStream_t st)
{
    const int blocks = (a.K + 127) / 128;
    const int64_t all = (int64_t)a.T * blocks;
    launch(quant_fp8_kernel<XT, SWIGLU>, (unsigned)((all + 15) / 16), 256, 0, st, a, blocks);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quant_fp8(const void *x, int32_t x_dtype, int64_t ldx, int32_t act, int32_t T,
                                    int32_t K, const int32_t *count, void *q, int64_t ldq, float *s,
                                    int64_t lds, void *stream)
{
    if (!ops_dtype_ok(x_dtype))
        return fail(MOE_E_INVAL, "unknown x_dtype %d", x_dtype);
    if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU)
        return fail(MOE_E_INVAL, "unknown act %d", act);
    if (T < 0 || T > (1 << 25))
        return fail(MOE_E_INVAL, "T=%d out of range [0, 2^25]", T);
    if (K < 1 || K > (1 << 17))
        return fail(MOE_E_INVAL, "K=%d must be in [1, 2^17]", K);
    const int64_t blocks = (K + 127) / 128;
    if (T * blocks > (1 << 27))                      // the launch's limit on threads
        return fail(MOE_E_INVAL, "T*ceil(K/128)=%lld above 2^27", (long long)(T * blocks));
    if (T == 0)
        return MOE_OK;
    if (!x || !q || !s)
        return fail(MOE_E_INVAL, "x/q/s is NULL");
    if (ldx < (act == MOE_ACT_SWIGLU ? 2 : 1) * (int64_t)K || ldq < K || lds < blocks)
        return fail(MOE_E_INVAL, "a leading dimension is below its row's length");
    if (!ops_aligned(x, x_dtype == MOE_DT_F32 ? 4 : 2) || !ops_aligned(s, 4) || !ops_aligned(count, 4))
        return fail(MOE_E_INVAL, "x, s and count must be aligned to their elements");
    const moe_status st = ops_check_device();
    if (st)
        return st;
    const Fp8Args a{x, static_cast<uint8_t *>(q), s, count, ldx, ldq, lds, T, K};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (x_dtype == MOE_DT_F32)
        act == MOE_ACT_SWIGLU ? enqueue_quant<float, true>(a, hs) : enqueue_quant<float, false>(a, hs);
    else
        act == MOE_ACT_SWIGLU ? enqueue_quant<bf16_t, true>(a, hs) : enqueue_quant<bf16_t, false>(a, hs);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_fail(e, "E4M3 rows launch");
}
