// ops_common.h -- pieces shared by the operators around the MoE layer
// (kernels_rows.hip, kernels_linear.hip, kernels_route.hip): argument checks,
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

__device__ __forceinline__ void load8(const bf16_t *p, float (&v)[8])
{
    const bytes16_a2 b = *reinterpret_cast<const bytes16_a2 *>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(b.d[j] << 16);
        v[2 * j + 1] = __uint_as_float(b.d[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const bytes16_a4 a = *reinterpret_cast<const bytes16_a4 *>(p);
    const bytes16_a4 b = *reinterpret_cast<const bytes16_a4 *>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = __uint_as_float(a.d[j]);
        v[4 + j] = __uint_as_float(b.d[j]);
    }
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

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    v = max(v, (uint32_t)xor_lane<32>((int)v));
    v = max(v, (uint32_t)xor_lane<16>((int)v));
    v = max(v, (uint32_t)xor_lane<8>((int)v));
    v = max(v, (uint32_t)xor_lane<4>((int)v));
    v = max(v, (uint32_t)xor_lane<2>((int)v));
    v = max(v, (uint32_t)xor_lane<1>((int)v));
    return v;
}

}  // namespace moe
