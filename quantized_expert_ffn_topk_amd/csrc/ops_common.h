// ops_common.h -- pieces shared by the operators around the MoE layer
// (kernels_rows.hip, kernels_linear.hip, kernels_route.hip, kernels_fp8.hip,
// kernels_products.hip, kernels_dispatch.hip): argument checks,
// loads and stores of rows of any alignment, type conversions.
#pragma once

#include "device_common.h"
#include "host_common.h"

#include <atomic>
#include <climits>

namespace moe {

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// The current device runs this library.  The answer is kept per device (it
// does not change while the process lives).
inline moe_status ops_check_device()
{
    constexpr int MAX = 64;
    static std::atomic<bool> known[MAX];
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return fail(MOE_E_UNSUPPORTED, "no HIP device available: %s", hipGetErrorString(e));
    if (dev >= 0 && dev < MAX && known[dev].load(std::memory_order_relaxed))
        return MOE_OK;
    const moe_status st = check_device(dev);
    if (st == MOE_OK && dev >= 0 && dev < MAX)
        known[dev].store(true, std::memory_order_relaxed);
    return st;
}

inline bool ops_dtype_ok(int32_t dt)
{
    return dt == MOE_DT_F32 || dt == MOE_DT_BF16;
}

inline bool ops_aligned(const void *p, size_t a)
{
    return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// ---------------------------------------------------------------------------
// device: 8 neighbouring values of a row at their element's alignment (the
// memory unit takes 16-byte accesses at any address; an address that crosses
// a line costs a second access, an aligned one nothing)
// ---------------------------------------------------------------------------
struct __attribute__((packed, aligned(2))) bytes16_a2 {
    uint32_t d[4];
};
struct __attribute__((packed, aligned(4))) bytes16_a4 {
    uint32_t d[4];
};
struct __attribute__((packed, aligned(1))) bytes16_a1 {
    uint32_t d[4];
};
struct __attribute__((packed, aligned(1))) bytes8_a1 {
    uint32_t d[2];
};

typedef uint16_t bf16_t;     // bits

__device__ __forceinline__ float to_f32(float v)
{
    return v;
}
__device__ __forceinline__ float to_f32(bf16_t v)
{
    return bf16_to_f32(v);
}

// 8 values as they lie in memory: loaded now, widened to fp32 when used
template <typename T>
struct raw8;
template <>
struct raw8<bf16_t> {
    bytes16_a2 b;
    __device__ __forceinline__ void load(const bf16_t *p)
    {
        b = *reinterpret_cast<const bytes16_a2 *>(p);
    }
    __device__ __forceinline__ void widen(float (&v)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(b.d[j] << 16);
            v[2 * j + 1] = __uint_as_float(b.d[j] & 0xffff0000u);
        }
    }
};
template <>
struct raw8<float> {
    bytes16_a4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const bytes16_a4 *>(p);
        b = *reinterpret_cast<const bytes16_a4 *>(p + 4);
    }
    __device__ __forceinline__ void widen(float (&v)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __uint_as_float(a.d[j]);
            v[4 + j] = __uint_as_float(b.d[j]);
        }
    }
};
__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    raw8<float> r;
    r.load(p);
    r.widen(v);
}

// two fp32 -> two bf16 in one word, round to nearest even (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

__device__ __forceinline__ void store1(bf16_t *p, float v)
{
    *p = (bf16_t)(pack_bf16(v, 0.0f) & 0xffffu);
}
__device__ __forceinline__ void store1(float *p, float v)
{
    *p = v;
}
__device__ __forceinline__ void store8(bf16_t *p, const float (&v)[8])
{
    bytes16_a2 b;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        b.d[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<bytes16_a2 *>(p) = b;
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    bytes16_a4 a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a.d[j] = __float_as_uint(v[j]);
        b.d[j] = __float_as_uint(v[4 + j]);
    }
    *reinterpret_cast<bytes16_a4 *>(p) = a;
    *reinterpret_cast<bytes16_a4 *>(p + 4) = b;
}

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

// LDS written by lanes of a wave and read by others of the same wave
__device__ __forceinline__ void wave_lds_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------------------
// device: maximum and sum over a wave, in every lane.  DPP row shifts and
// broadcasts bring them to lane 63 in six dependent VALU steps (the swizzles
// of xor_lane go through the LDS unit, several times as long each).  Lanes
// that a step does not reach take 0.
// ---------------------------------------------------------------------------
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp0(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
#define MOE_DPP_STEPS(STEP)                                                              \
    STEP(0x111, 0xf)   /* row_shr:1 */                                                   \
    STEP(0x112, 0xf)                                                                     \
    STEP(0x114, 0xf)                                                                     \
    STEP(0x118, 0xf)                                                                     \
    STEP(0x142, 0xa)   /* row_bcast:15 into rows 1 and 3 */                              \
    STEP(0x143, 0xc)   /* row_bcast:31 into rows 2 and 3 */

__device__ __forceinline__ uint32_t wave_top(uint32_t v)
{
#define STEP(c, r) v = max(v, (uint32_t)dpp0<c, r>((int)v));
    MOE_DPP_STEPS(STEP)
#undef STEP
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// fixed order of additions
__device__ __forceinline__ double wave_total_d(double v)
{
#define STEP(c, r)                                                                       \
    {                                                                                    \
        const long long u = __double_as_longlong(v);                                     \
        const uint32_t lo = (uint32_t)dpp0<c, r>((int)(u & 0xffffffffll));               \
        const uint32_t hi = (uint32_t)dpp0<c, r>((int)(u >> 32));                        \
        v += __longlong_as_double((long long)((uint64_t)hi << 32 | lo));                 \
    }
    MOE_DPP_STEPS(STEP)
#undef STEP
    const long long u = __double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(u & 0xffffffffll), 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ float wave_total_f(float v)
{
#define STEP(c, r) v += __int_as_float(dpp0<c, r>(__float_as_int(v)));
    MOE_DPP_STEPS(STEP)
#undef STEP
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace moe
