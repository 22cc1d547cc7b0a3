// kernels_rows.hip -- row operators around the MoE layer on gfx950: the RMS
// norm with the residual's addition, and SwiGLU, both with int8 output (codes
// and one scale per row) beside or instead of bf16.
//
// A row needs its sum (norm) and its largest value before its first code: it is
// read once, stays in the registers of 64 to 1024 threads, and is written from
// there.  Bound by HBM from some hundred rows on, by the launch and a round trip
// to memory below (kernel times under the profiler):
//   norm   4096 x 6144, bf16, residual, codes    33.8 us, 176 MB at 5.3 TB/s (a
//          333 x 7001, fp32, residual, codes    7 to 8     large copy runs at 4.9)
//            1 x 6144, bf16, residual             2.3
//   SwiGLU 4096 x 12288, bf16, codes         46 to 48, 252 MB at 5.2 to 5.4 TB/s
//            1 x 12288                            3.4
// SwiGLU's instructions alone are three quarters of its time: hence silu_mul's
// form, the code by an addition and the maximum over two values at once.
#include "ops_common.h"

#include <cmath>

namespace moe {

// ---------------------------------------------------------------------------
// Sources of a row's fp32 values.
// ---------------------------------------------------------------------------
template <typename XT, typename RT>
struct NormArgs {
    const XT *x;
    const RT *res;             // NULL: none
    const float *gamma;        // NULL: ones
    RT *h;                     // NULL: not wanted
    int64_t ldx, ldr, ldh;
    double inv_n;              // 1/n
    float eps;
};
template <typename XT>
struct SwigluArgs {
    const XT *gu;
    int64_t ld;
};
struct RowOut {
    bf16_t *y;                 // NULL: not wanted
    int8_t *q;                 // NULL: not wanted (then s too)
    float *s;
    int64_t ldy, ldq;
    int T, n;
};

// silu(g)*u in fp32, from E = exp(-|g|) <= 1 so that nothing overflows:
// g*u/(1+E) for g >= 0, g*u*E/(1+E) for g < 0.  E is the square of 2^t with
// t = -|g|*log2(e)/2 as a rounded product and its remainder r, so that the
// exponent's rounding does not grow with |g| and E reaches the subnormals,
// which the hardware's 2^t itself does not; the reciprocal is the hardware's
// (one unit in the last place), of a number in [1,2].  Past |g| = 200 E is 0
// either way.
__device__ __forceinline__ float silu_mul(float g, float u)
{
    const float C = 0.72134751f, C_LO = 9.62981515e-9f;       // log2(e)/2 = C + C_LO
    const float a = fminf(fabsf(g), 200.0f);
    const float t = -a * C;
    const float r = fmaf(-a, C_LO, fmaf(-a, C, -t));
    const float h = __builtin_amdgcn_exp2f(t);
    float e = h * h;
    e = fmaf(e, r * 1.386294361f, e);                         // (1 + r ln 2)^2
    const float d = __builtin_amdgcn_rcpf(1.0f + e);
    return g * ((g < 0.0f) ? e * d : d) * u;
}

// ---------------------------------------------------------------------------
// One row by NT threads, NV vectors of 8 values per thread (8*NT*NV >= n >= 8),
// the row in registers between its one read and its writes.  A thread's vector
// i covers values [col, col+8), col = 8*(lane + NT*i).  One that passes the
// row's end reads the row's last 8 values instead (c < col), counts those of
// its own in the sum and writes all of them again, with the same values.
// NT = 64: a wave per row, four rows per block, no barrier.
// ---------------------------------------------------------------------------
template <int NT>
__device__ __forceinline__ double row_sum_d(double v, double *red)
{
    v = wave_total_d(v);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < NT / 64; ++w)
            v += red[w];
    }
    return v;
}

template <int NT>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v, uint32_t *red)
{
    v = wave_top(v);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < NT / 64; ++w)
            v = max(v, red[w]);
    }
    return v;
}

// fp32(1/sqrt(x)): the hardware's fp64 estimate and two Newton steps, far
// within fp32's unit (the exact fp64 root and quotient took a fifth of the
// norm's instructions); 0 for infinity, NaN for NaN
__device__ __forceinline__ float inv_sqrt(double x)
{
    const double r0 = __builtin_amdgcn_rsq(x);
    double r = r0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r = r * fma(-0.5 * x * r, r, 1.5);
    return (float)((x < (double)INFINITY) ? r : r0);
}

// The scale of a row whose largest magnitude has the fp32 bits m, and the
// multiplier of its codes: rows below 2^-96 are multiplied by pre = 2^64 first
// (exact), so that 127/max stays finite.  inv = 0 for a row of zeros and for
// one with a NaN or an infinity.
__device__ __forceinline__ void row_scale(uint32_t m, float *s, float *pre, float *inv)
{
    const float a = __uint_as_float(m);
    *s = a / 127.0f;
    *pre = (a < 0x1p-96f) ? 0x1p64f : 1.0f;
    *inv = (m == 0u) ? 0.0f : 127.0f / (a * *pre);
    if (m >= 0x7f800000u) {
        *s = __uint_as_float(0x7fc00000u);
        *inv = 0.0f;
    }
}

// rint of |p| <= 127.5 in the low byte: adding 1.5*2^23 rounds to the nearest
// whole number, ties to even
__device__ __forceinline__ uint32_t code(float p)
{
    return __float_as_uint(p + 12582912.0f);
}
// four codes in a word
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d)
{
    const uint32_t lo = __builtin_amdgcn_perm(code(b), code(a), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(code(d), code(c), 0x0c0c0400u);
    return lo | hi << 16;
}

// y_out, codes and scale of a row whose values are in v
template <int NT, int NV>
__device__ __forceinline__ void row_out(const RowOut &o, int t, int lane, bool live, uint32_t *red,
                                        float (&v)[NV][8], const int (&c)[NV])
{
    const int n = o.n;
    if (o.y && live) {
        bf16_t *yr = o.y + (int64_t)t * o.ldy;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (8 * (lane + NT * i) < n)
                store8(yr + c[i], v[i]);
    }
    if (!o.q)
        return;
    // the maximum that keeps a NaN (v_maximum3_f32), then bits: NaN is largest
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            big = __builtin_elementwise_maximum(big, fabsf(v[i][j]));
    const uint32_t m = row_max_u32<NT>(__float_as_uint(big) & 0x7fffffffu, red);
    float s, pre, inv;
    row_scale(m, &s, &pre, &inv);
    if (!live)
        return;
    if (pre != 1.0f) {                              // the whole row alike
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] *= pre;
    }
    int8_t *qr = o.q + (int64_t)t * o.ldq;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const float *p = v[i];
        bytes8_a1 b;
        b.d[0] = code4(p[0] * inv, p[1] * inv, p[2] * inv, p[3] * inv);
        b.d[1] = code4(p[4] * inv, p[5] * inv, p[6] * inv, p[7] * inv);
        if (inv == 0.0f)
            b.d[0] = b.d[1] = 0u;
        if (8 * (lane + NT * i) < n)
            *reinterpret_cast<bytes8_a1 *>(qr + c[i]) = b;
    }
    if (lane == 0)
        o.s[t] = s;
}

template <int NT>
constexpr int block_threads()
{
    return NT == 64 ? 256 : NT;
}

// Row and lane of a thread; a wave past the rows (NT = 64) repeats the last
// row and stores nothing.
template <int NT>
__device__ __forceinline__ bool row_of(int T, int *t, int *lane)
{
    const int row = (NT == 64) ? (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6) : (int)blockIdx.x;
    *lane = (NT == 64) ? threadIdx.x & 63 : threadIdx.x;
    *t = min(row, T - 1);
    return row < T;
}

// RES: there is a residual.  All loads of the row and of gamma are issued
// before any value is used (waiting for one after the other 4096 x 6144 took
// 44.5 us).  The sum is fp64: no fp32 row overflows it, and its order hardly ever
// shows.
template <int NT, int NV, typename XT, typename RT, bool RES>
__global__ __launch_bounds__(block_threads<NT>()) void rmsnorm_kernel(NormArgs<XT, RT> a, RowOut o)
{
    __shared__ double red_d[NT / 64];
    __shared__ uint32_t red_m[NT / 64];
    int t, lane;
    const bool live = row_of<NT>(o.T, &t, &lane);
    const int n = o.n;
    int c[NV];
    float v[NV][8], g[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        c[i] = min(8 * (lane + NT * i), n - 8);
    {
        raw8<XT> x[NV];
        raw8<RT> r[RES ? NV : 1];
        const XT *xr = a.x + (int64_t)t * a.ldx;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            x[i].load(xr + c[i]);
        if constexpr (RES) {
            const RT *rr = a.res + (int64_t)t * a.ldr;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                r[i].load(rr + c[i]);
        }
        if (a.gamma) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                load8(a.gamma + c[i], g[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    g[i][j] = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i].widen(v[i]);
            if constexpr (RES) {
                float w[8];
                r[i].widen(w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] += w[j];
            }
        }
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = 8 * (lane + NT * i);
        if (col + 8 <= n) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss = fma((double)v[i][j], (double)v[i][j], ss);
        } else if (col < n) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double d = (c[i] + j >= col) ? (double)v[i][j] : 0.0;
                ss = fma(d, d, ss);
            }
        }
    }
    ss = row_sum_d<NT>(ss, red_d);
    const float r = inv_sqrt(ss * a.inv_n + (double)a.eps);
    if (a.h && live) {
        RT *hr = a.h + (int64_t)t * a.ldh;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (8 * (lane + NT * i) < n)
                store8(hr + c[i], v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] = v[i][j] * r * g[i][j];
    row_out<NT, NV>(o, t, lane, live, red_m, v, c);
}

template <int NT, int NV, typename XT>
__global__ __launch_bounds__(block_threads<NT>()) void swiglu_kernel(SwigluArgs<XT> a, RowOut o)
{
    __shared__ uint32_t red_m[NT / 64];
    int t, lane;
    const bool live = row_of<NT>(o.T, &t, &lane);
    const int n = o.n;
    int c[NV];
    float v[NV][8];
    const XT *gr = a.gu + (int64_t)t * a.ld, *ur = gr + n;
    raw8<XT> g[NV], u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        c[i] = min(8 * (lane + NT * i), n - 8);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        g[i].load(gr + c[i]);
        u[i].load(ur + c[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[8];
        g[i].widen(v[i]);
        u[i].widen(w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] = silu_mul(v[i][j], w[j]);
    }
    row_out<NT, NV>(o, t, lane, live, red_m, v, c);
}

// ---------------------------------------------------------------------------
// Rows too long for the registers (n > 32768), or shorter than a vector (n < 8):
// value by value, a block reads the row again for each step; every value is read
// and written by one thread, the writes in the last step, so h_out may be an
// input here too.
// ---------------------------------------------------------------------------
template <typename XT, typename RT>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(NormArgs<XT, RT> a, RowOut o)
{
    __shared__ double red_d[16];
    __shared__ uint32_t red_m[16];
    const int t = blockIdx.x, n = o.n;
    const XT *xr = a.x + (int64_t)t * a.ldx;
    const RT *rr = a.res ? a.res + (int64_t)t * a.ldr : nullptr;
    auto value = [&](int i) {
        const float v = to_f32(xr[i]);
        return rr ? v + to_f32(rr[i]) : v;
    };
    double ss = 0.0;
    for (int i = threadIdx.x; i < n; i += 1024) {
        const double d = (double)value(i);
        ss = fma(d, d, ss);
    }
    ss = row_sum_d<1024>(ss, red_d);
    const float r = inv_sqrt(ss * a.inv_n + (double)a.eps);
    auto normed = [&](float h, int i) {
        const float y = h * r;
        return a.gamma ? y * a.gamma[i] : y;
    };
    float s = 0.0f, pre = 0.0f, inv = 0.0f;
    if (o.q) {
        uint32_t m = 0u;
        for (int i = threadIdx.x; i < n; i += 1024)
            m = max(m, __float_as_uint(normed(value(i), i)) & 0x7fffffffu);
        row_scale(row_max_u32<1024>(m, red_m), &s, &pre, &inv);
    }
    for (int i = threadIdx.x; i < n; i += 1024) {
        const float h = value(i);
        const float v = normed(h, i);
        if (a.h)
            store1(a.h + (int64_t)t * a.ldh + i, h);
        if (o.y)
            store1(o.y + (int64_t)t * o.ldy + i, v);
        if (o.q)
            o.q[(int64_t)t * o.ldq + i] = (inv == 0.0f) ? 0 : (int8_t)(code((v * pre) * inv) & 0xffu);
    }
    if (o.q && threadIdx.x == 0)
        o.s[t] = s;
}

template <typename XT>
__global__ __launch_bounds__(1024) void swiglu_long_kernel(SwigluArgs<XT> a, RowOut o)
{
    __shared__ uint32_t red_m[16];
    const int t = blockIdx.x, n = o.n;
    const XT *gr = a.gu + (int64_t)t * a.ld;
    auto value = [&](int i) { return silu_mul(to_f32(gr[i]), to_f32(gr[n + i])); };
    float s = 0.0f, pre = 0.0f, inv = 0.0f;
    if (o.q) {
        uint32_t m = 0u;
        for (int i = threadIdx.x; i < n; i += 1024)
            m = max(m, __float_as_uint(value(i)) & 0x7fffffffu);
        row_scale(row_max_u32<1024>(m, red_m), &s, &pre, &inv);
    }
    for (int i = threadIdx.x; i < n; i += 1024) {
        const float v = value(i);
        if (o.y)
            store1(o.y + (int64_t)t * o.ldy + i, v);
        if (o.q)
            o.q[(int64_t)t * o.ldq + i] = (inv == 0.0f) ? 0 : (int8_t)(code((v * pre) * inv) & 0xffu);
    }
    if (o.q && threadIdx.x == 0)
        o.s[t] = s;
}

// ---------------------------------------------------------------------------
// Shapes: threads of a row x vectors of eight per thread, one rule by the row's
// length for both operators and any number of rows.  Fewer threads with more
// vectors wait longer for each row, more threads meet later, idle vectors cost
// their instructions (us, launches in a graph, bf16 with codes, norm / SwiGLU):
//   4096 x  1024  128x1  6.4 /  6.1   64x2  6.6 /  6.1
//   4096 x  2048  256x1 10.7 /  9.0  128x2 10.4 /  9.5   64x4 10.8 / 10.2
//    100 x  2048  256x1  2.8 /  2.6  128x2  2.9 /  2.8   64x4  3.4 /  3.3
//      1 x  2560  256x2  2.7 /  2.5  128x3  2.9 /  2.8  512x1  2.6 /  2.4
//    100 x  2560  256x2  3.1 /  2.9  128x3  3.3 /  3.1  512x1  3.0 /  2.8
//   1000 x  2560  256x2  5.4 /  5.2  128x3  5.3 /  4.7  512x1  5.6 /  5.2
//   4096 x  2560  256x2 12.7 / 12.9  128x3 12.8 / 11.4  512x1 13.9 / 12.7
//   4096 x  3328  256x2 15.6 / 13.9                     512x1 16.1 / 13.7
//      1 x  4096  512x1  2.6 /  2.4  256x2  2.7 /  2.5
//   4096 x  4096  512x1 19.0 / 14.3  256x2 18.4 / 14.9
//   4096 x  6144  256x3 30.2 / 23.1  512x2 30.2 / 24.2 1024x1 34.3 / 27.2
//      1 x  6144  256x3  3.0 /  2.8  512x2  3.0 /  3.0 1024x1  3.0 /  2.9
//   4096 x  8192  512x2 38.3 / 29.4  256x4 38.7 / 30.3 1024x1 43.9 / 30.3
//      1 x  8192  512x2  3.1 /  3.0  256x4  3.4 /  3.2 1024x1  3.2 /  3.1
//   4096 x 12288  512x3 64.4 / 44.1 1024x2 79.9 / 47.1
//   4096 x 16384  512x4 85.5 / 61.4 1024x2 94.9 / 58.9
// From 2049 to 4096 no shape is best throughout: 512x1 is 0.1 us faster than
// 256x2 on up to 100 rows, and slower on thousands of the norm's, by 11 % at 2056
// and less and less from there; it is taken from where that is below 4 %.  128x3,
// with the fewest idle vectors, is 10 % faster for thousands of SwiGLU's rows, 10
// to 12 % slower for a few, and holds three quarters as many values.  At 16384 the norm
// would lose more with 1024x2 than SwiGLU gains.
// ---------------------------------------------------------------------------
constexpr int ROW_REG_MAX = 32768;

template <int V>
using num = std::integral_constant<int, V>;

template <typename F>
static void with_shape(int n, F &&f)
{
    if (n <= 512)
        return f(num<64>(), num<1>());
    if (n <= 1024)
        return f(num<128>(), num<1>());
    if (n <= 2048)
        return f(num<256>(), num<1>());
    if (n <= 3328)
        return f(num<256>(), num<2>());
    if (n <= 4096)
        return f(num<512>(), num<1>());
    if (n <= 6144)
        return f(num<256>(), num<3>());
    if (n <= 8192)
        return f(num<512>(), num<2>());
    if (n <= 12288)
        return f(num<512>(), num<3>());
    if (n <= 16384)
        return f(num<512>(), num<4>());
    if (n <= 24576)
        return f(num<1024>(), num<3>());
    f(num<1024>(), num<4>());
}

static unsigned row_grid(int T, int nt)
{
    return nt == 64 ? (unsigned)((T + 3) / 4) : (unsigned)T;
}

template <bool RES, typename XT, typename RT>
static void enqueue_norm(const NormArgs<XT, RT> &a, const RowOut &o, hipStream_t st)
{
    if (o.n > ROW_REG_MAX || o.n < 8) {
        launch(rmsnorm_long_kernel<XT, RT>, (unsigned)o.T, 1024, 0, st, a, o);
        return;
    }
    with_shape(o.n, [&](auto nt, auto nv) {
        launch(rmsnorm_kernel<nt(), nv(), XT, RT, RES>, row_grid(o.T, nt()), block_threads<nt()>(), 0, st, a, o);
    });
}

template <typename XT>
static void enqueue_swiglu(const SwigluArgs<XT> &a, const RowOut &o, hipStream_t st)
{
    if (o.n > ROW_REG_MAX || o.n < 8) {
        launch(swiglu_long_kernel<XT>, (unsigned)o.T, 1024, 0, st, a, o);
        return;
    }
    with_shape(o.n, [&](auto nt, auto nv) {
        launch(swiglu_kernel<nt(), nv(), XT>, row_grid(o.T, nt()), block_threads<nt()>(), 0, st, a, o);
    });
}

static moe_status check_rows(int32_t T, int32_t n, const char *name, const void *y, int64_t ldy,
                             const void *q, int64_t ldq, const void *s)
{
    if (T < 0 || T > (1 << 20))
        return fail(MOE_E_INVAL, "T=%d out of range [0, 2^20]", T);
    if (n < 1 || n > (1 << 20))
        return fail(MOE_E_INVAL, "%s=%d must be in [1, 2^20]", name, n);
    if ((q == nullptr) != (s == nullptr))
        return fail(MOE_E_INVAL, "q and s go together");
    if (y && ldy < n)
        return fail(MOE_E_INVAL, "ldy=%lld is below %s=%d", (long long)ldy, name, n);
    if (q && ldq < n)
        return fail(MOE_E_INVAL, "ldq=%lld is below %s=%d", (long long)ldq, name, n);
    if (!ops_aligned(y, 2) || !ops_aligned(s, 4))
        return fail(MOE_E_INVAL, "y_out and s must be aligned to their elements");
    return MOE_OK;
}

static size_t dtype_size(int32_t dt)
{
    return dt == MOE_DT_F32 ? 4 : 2;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_rmsnorm_quant(const void *x, int32_t x_dtype, int64_t ldx,
                                        const void *residual, int32_t res_dtype, int64_t ldr,
                                        const float *gamma, int32_t T, int32_t H, float eps,
                                        void *h_out, int64_t ldh, void *y_out, int64_t ldy,
                                        int8_t *q, int64_t ldq, float *s, void *stream)
{
    moe_status st = check_rows(T, H, "H", y_out, ldy, q, ldq, s);
    if (st)
        return st;
    if (!ops_dtype_ok(x_dtype))
        return fail(MOE_E_INVAL, "unknown x_dtype %d", x_dtype);
    if ((residual || h_out) && !ops_dtype_ok(res_dtype))
        return fail(MOE_E_INVAL, "unknown res_dtype %d", res_dtype);
    if (!residual && h_out && res_dtype != x_dtype)
        return fail(MOE_E_INVAL, "without a residual h_out has x's dtype");
    if (!(eps > 0.0f) || !(eps < INFINITY))
        return fail(MOE_E_INVAL, "eps must be finite and > 0");
    if (!y_out && !q && !h_out)
        return fail(MOE_E_INVAL, "no output is wanted");
    if (T == 0)
        return MOE_OK;
    if (!x)
        return fail(MOE_E_INVAL, "x is NULL");
    if (ldx < H || (residual && ldr < H) || (h_out && ldh < H))
        return fail(MOE_E_INVAL, "a leading dimension is below H=%d", H);
    const size_t rs = dtype_size(res_dtype);
    if (!ops_aligned(x, dtype_size(x_dtype)) || !ops_aligned(residual, rs) || !ops_aligned(h_out, rs) ||
        !ops_aligned(gamma, 4))
        return fail(MOE_E_INVAL, "x, residual, gamma and h_out must be aligned to their elements");
    if ((st = ops_check_device()) != MOE_OK)
        return st;
    const RowOut o{static_cast<bf16_t *>(y_out), q, s, ldy, ldq, T, H};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    auto with = [&](auto res, auto xt, auto rt) {
        typedef std::remove_const_t<decltype(xt)> XT;
        typedef std::remove_const_t<decltype(rt)> RT;
        const NormArgs<XT, RT> a{static_cast<const XT *>(x), static_cast<const RT *>(residual), gamma,
                                 static_cast<RT *>(h_out), ldx, ldr, ldh, 1.0 / (double)H, eps};
        enqueue_norm<decltype(res)::value>(a, o, hs);
    };
    const std::true_type yes;
    const std::false_type no;
    const float f = 0.0f;
    const bf16_t b = 0;
    if (!residual)                                  // h_out then has x's dtype
        x_dtype == MOE_DT_F32 ? with(no, f, f) : with(no, b, b);
    else if (x_dtype == MOE_DT_F32)
        res_dtype == MOE_DT_F32 ? with(yes, f, f) : with(yes, f, b);
    else
        res_dtype == MOE_DT_F32 ? with(yes, b, f) : with(yes, b, b);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_fail(e, "norm launch");
}

extern "C" moe_status moe_swiglu_quant(const void *gu, int32_t gu_dtype, int64_t ld, int32_t T,
                                       int32_t F, void *y_out, int64_t ldy, int8_t *q, int64_t ldq,
                                       float *s, void *stream)
{
    moe_status st = check_rows(T, F, "F", y_out, ldy, q, ldq, s);
    if (st)
        return st;
    if (!ops_dtype_ok(gu_dtype))
        return fail(MOE_E_INVAL, "unknown gu_dtype %d", gu_dtype);
    if (!y_out && !q)
        return fail(MOE_E_INVAL, "no output is wanted");
    if (T == 0)
        return MOE_OK;
    if (!gu)
        return fail(MOE_E_INVAL, "gu is NULL");
    if (ld < 2 * (int64_t)F)
        return fail(MOE_E_INVAL, "ld=%lld is below 2*F=%d", (long long)ld, 2 * F);
    if (!ops_aligned(gu, dtype_size(gu_dtype)))
        return fail(MOE_E_INVAL, "gu must be aligned to its elements");
    if ((st = ops_check_device()) != MOE_OK)
        return st;
    const RowOut o{static_cast<bf16_t *>(y_out), q, s, ldy, ldq, T, F};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (gu_dtype == MOE_DT_F32)
        enqueue_swiglu(SwigluArgs<float>{static_cast<const float *>(gu), ld}, o, hs);
    else
        enqueue_swiglu(SwigluArgs<bf16_t>{static_cast<const bf16_t *>(gu), ld}, o, hs);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_fail(e, "SwiGLU launch");
}
