// kernels_linear.hip -- the int8 product with scales per token and channel on
// gfx950: out[t,n] = (float(sum_k q[t,k]*w[n,k]) * s[t]) * ws[n] + bias[n].
//
// The sum is exact in int32 (v_mfma_i32_32x32x32_i8), so it does not matter
// how a kernel splits it, and the epilogue's fp32 steps are the same in every
// kernel: results are bit-identical whatever the shape of the launch.
#include "ops_common.h"

namespace moe {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

struct LinArgs {
    const int8_t *q, *w;
    const float *s, *ws, *bias;   // bias NULL: none
    void *out;
    int64_t ldq, ldw, ldo;
    int T, N, K;
};

// 16 codes of a row at k (a multiple of 16), zeros past K, at any alignment.
// The piece that passes the row's end is read as the row's last 16 bytes and
// shifted down; rows shorter than 16 byte by byte.
__device__ __forceinline__ v4i load_codes(const int8_t *row, int k, int K)
{
    v4i v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        const bytes16_a1 b = *reinterpret_cast<const bytes16_a1 *>(row + k);
        v = v4i{(int)b.d[0], (int)b.d[1], (int)b.d[2], (int)b.d[3]};
    } else if (k < K) {
        if (K >= 16) {
            const unsigned __int128 b = __builtin_bit_cast(
                unsigned __int128, *reinterpret_cast<const bytes16_a1 *>(row + K - 16));
            v = __builtin_bit_cast(v4i, b >> (8 * (k + 16 - K)));
        } else {
            unsigned __int128 b = 0;
            for (int j = 0; j < K; ++j)                      // k is 0 here
                b |= (unsigned __int128)(uint8_t)row[j] << (8 * j);
            v = __builtin_bit_cast(v4i, b);
        }
    }
    return v;
}

template <typename OT>
__device__ __forceinline__ void store_out(const LinArgs &a, int t, int n, int acc)
{
    float y = ((float)acc * a.s[t]) * a.ws[n];
    if (a.bias)
        y += a.bias[n];
    store1(static_cast<OT *>(a.out) + (int64_t)t * a.ldo + n, y);
}

// ---------------------------------------------------------------------------
// Any shape and alignment: 64 x 64 outputs per block, four waves of 32 x 32,
// K in steps of 64 codes through registers into LDS.
// ---------------------------------------------------------------------------
constexpr int LP = 64 + 16;                // LDS pitch of a 64-byte row: 16-byte reads of
                                           // 32 rows fall on different banks

template <typename OT>
__global__ __launch_bounds__(256) void linear_tile_kernel(LinArgs a)
{
    __shared__ __align__(16) uint8_t lq[64 * LP], lw[64 * LP];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int n0 = blockIdx.x * 64, t0 = blockIdx.y * 64;
    const int r = tid >> 2, c = (tid & 3) * 16;
    const int8_t *qr = a.q + (int64_t)min(t0 + r, a.T - 1) * a.ldq;
    const int8_t *wr = a.w + (int64_t)min(n0 + r, a.N - 1) * a.ldw;
    const int tq = 32 * (wave >> 1), tw = 32 * (wave & 1);
    v16i acc = {0};
    for (int k = 0; k < a.K; k += 64) {
        const v4i vq = load_codes(qr, k + c, a.K), vw = load_codes(wr, k + c, a.K);
        __syncthreads();
        *reinterpret_cast<v4i *>(lq + r * LP + c) = vq;
        *reinterpret_cast<v4i *>(lw + r * LP + c) = vw;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int o = (lane & 31) * LP + 32 * u + 16 * (lane >> 5);
            acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(*reinterpret_cast<const v4i *>(lq + tq * LP + o),
                                                        *reinterpret_cast<const v4i *>(lw + tw * LP + o),
                                                        acc, 0, 0, 0);
        }
    }
    const int n = n0 + tw + (lane & 31);
    if (n >= a.N)
        return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int t = t0 + tq + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
        if (t < a.T)
            store_out<OT>(a, t, n, acc[i]);
    }
}

template <typename OT>
static void enqueue_linear(const LinArgs &a, hipStream_t st)
{
    const dim3 grid((a.N + 63) / 64, (a.T + 63) / 64);
    launch(linear_tile_kernel<OT>, grid, 256, 0, st, a);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_linear_int8(const int8_t *q, int64_t ldq, const float *s, int32_t T,
                                      const int8_t *w, int64_t ldw, const float *ws,
                                      const float *bias, int32_t N, int32_t K, void *out,
                                      int32_t out_dtype, int64_t ldo, void *stream)
{
    if (T < 0 || T > (1 << 20))
        return fail(MOE_E_INVAL, "T=%d out of range [0, 2^20]", T);
    if (N < 1 || N > (1 << 20))
        return fail(MOE_E_INVAL, "N=%d must be in [1, 2^20]", N);
    // 2^14 per product at most: the int32 sum holds 131071 of them
    if (K < 1 || K > 131071)
        return fail(MOE_E_INVAL, "K=%d must be in [1, 131071]", K);
    if (!ops_dtype_ok(out_dtype))
        return fail(MOE_E_INVAL, "unknown out_dtype %d", out_dtype);
    if (T == 0)
        return MOE_OK;
    if (!q || !s || !w || !ws || !out)
        return fail(MOE_E_INVAL, "q/s/w/ws/out is NULL");
    if (ldq < K || ldw < K || ldo < N)
        return fail(MOE_E_INVAL, "a leading dimension is below its row's length");
    if (!ops_aligned(s, 4) || !ops_aligned(ws, 4) || !ops_aligned(bias, 4) ||
        !ops_aligned(out, out_dtype == MOE_DT_F32 ? 4 : 2))
        return fail(MOE_E_INVAL, "s, ws, bias and out must be aligned to their elements");
    const moe_status st = ops_check_device();
    if (st)
        return st;
    const LinArgs a{q, w, s, ws, bias, out, ldq, ldw, ldo, T, N, K};
    if (out_dtype == MOE_DT_F32)
        enqueue_linear<float>(a, static_cast<hipStream_t>(stream));
    else
        enqueue_linear<bf16_t>(a, static_cast<hipStream_t>(stream));
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_fail(e, "int8 product launch");
}
