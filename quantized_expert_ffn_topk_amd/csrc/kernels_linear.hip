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
// Few tokens: a stream of weights.  A block owns RT tiles of 16 weight rows and
// TB tiles of 16 tokens; its W waves split K in steps of 64 codes and add their
// exact sums through LDS.  v_mfma_i32_16x16x64_i8: lane l supplies 16 codes at
// 16*(l/16) of weight row l%16 (A) and of token l%16 (B), straight from memory;
// result register i is row 4*(l/16)+i, token l%16.
// ---------------------------------------------------------------------------
__device__ __forceinline__ v4i load16(const int8_t *p)
{
    const bytes16_a1 b = *reinterpret_cast<const bytes16_a1 *>(p);
    return v4i{(int)b.d[0], (int)b.d[1], (int)b.d[2], (int)b.d[3]};
}

template <typename OT, int RT, int TB, int W, int U>
__global__ __launch_bounds__(64 * W) void linear_stream_kernel(LinArgs a)
{
    __shared__ v4i part[W][RT * TB][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * 16 * TB;
    const int8_t *wr[RT], *qr[TB];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        wr[i] = a.w + (int64_t)min(n0 + 16 * i + (lane & 15), a.N - 1) * a.ldw + 16 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < TB; ++i)
        qr[i] = a.q + (int64_t)min(t0 + 16 * i + (lane & 15), a.T - 1) * a.ldq + 16 * (lane >> 4);
    v4i acc[RT][TB];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
            acc[i][j] = v4i{0, 0, 0, 0};
    const int steps = a.K >> 6;
    const int s_lo = (int)((int64_t)wave * steps / W), s_hi = (int)((int64_t)(wave + 1) * steps / W);
    for (int s0 = s_lo; s0 < s_hi; s0 += U) {
        v4i wv[U][RT], qv[U][TB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = 64 * (int64_t)min(s0 + u, s_hi - 1);    // clamped: unconditional loads
#pragma unroll
            for (int i = 0; i < RT; ++i)
                wv[u][i] = load16(wr[i] + k);
#pragma unroll
            for (int j = 0; j < TB; ++j)
                qv[u][j] = load16(qr[j] + k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u < s_hi) {
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < TB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u][i], qv[u][j], acc[i][j], 0, 0, 0);
            }
        }
    }
    if ((a.K & 63) && wave == W - 1) {
        const int k = (steps << 6) + 16 * (lane >> 4);
        v4i qv[TB];
#pragma unroll
        for (int j = 0; j < TB; ++j)
            qv[j] = load_codes(qr[j] - 16 * (lane >> 4), k, a.K);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const v4i wv = load_codes(wr[i] - 16 * (lane >> 4), k, a.K);
#pragma unroll
            for (int j = 0; j < TB; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, qv[j], acc[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
            part[wave][i * TB + j][lane] = acc[i][j];
    __syncthreads();
    for (int f = threadIdx.x; f < RT * TB * 64; f += 64 * W) {
        const int l = f & 63, ij = f >> 6;
        v4i sum = part[0][ij][l];
#pragma unroll
        for (int w = 1; w < W; ++w)
            sum += part[w][ij][l];
        const int n = n0 + 16 * (ij / TB) + 4 * (l >> 4), t = t0 + 16 * (ij % TB) + (l & 15);
        if (t < a.T) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N)
                    store_out<OT>(a, t, n + i, sum[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Tiles: a block computes BT = 32*WT*FT tokens x BN = 32*WN*FN channels with
// WT*WN waves of FT*FN 32x32 results, K in stages of 128 codes through two LDS
// buffers, the next stage's rows on their way while one is multiplied.
// An LDS row is 128 bytes, eight 16-byte pieces; piece c of row r sits at slot
// c ^ (r/2 & 7): two rows fill the 64 banks once, so that 16 neighbouring rows'
// reads of one piece fall on different banks.
// DMA: rows go global -> LDS by the load unit (a wave's copy is 8 rows, lane l
// writing slot l%8 of row l/8, so the lane picks the global piece that belongs
// there); needs rows of 16-byte alignment.  Otherwise they pass through
// registers.  The last, partial stage always does (load_codes gives its zeros).
// ---------------------------------------------------------------------------
template <typename OT, bool DMA, int WT, int WN, int FT, int FN>
__global__ __launch_bounds__(64 * WT * WN) void linear_tiles_kernel(LinArgs a, int tiles_t, int tiles_n)
{
    constexpr int NW = WT * WN, NT = 64 * NW, BT = 32 * WT * FT, BN = 32 * WN * FN;
    constexpr int CP = (BT + BN) / 8 / NW;               // 8-row copies per wave and stage
    constexpr int TP = BT / 8 / NW;                      // of these, token rows
    static_assert(BT % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole copies per wave");
    // two buffers as two objects: the compiler then knows that reads of one do
    // not wait for copies into the other
    __shared__ __align__(128) uint8_t buf0[(BT + BN) * 128];
    __shared__ __align__(128) uint8_t buf1[(BT + BN) * 128];

    // tiles in groups of 8 token tiles, token tile fastest, each XCD (blocks
    // with the same index mod 8) a contiguous run of them
    const int per = gridDim.x >> 3, logical = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (logical >= tiles_t * tiles_n)
        return;
    const int group = logical / (8 * tiles_n), in = logical - group * 8 * tiles_n;
    const int gt = min(8, tiles_t - 8 * group);
    const int t0 = (8 * group + in % gt) * BT, n0 = (in / gt) * BN;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));   // NW is even
    const int8_t *src[CP];                               // this lane's piece of each copy
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        const int r = 8 * (wave + NW * (i < TP ? i : i - TP)) + (lane >> 3);
        src[i] = (i < TP) ? a.q + (int64_t)min(t0 + r, a.T - 1) * a.ldq
                          : a.w + (int64_t)min(n0 + r, a.N - 1) * a.ldw;
        src[i] += 16 * piece;
    }
    auto lds_at = [&](int i) { return (i < TP ? 0 : BT * 128) + 1024 * (wave + NW * (i < TP ? i : i - TP)); };

    v16i acc[FT][FN];
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = v16i{0};
    const int wt = wave / WN, wn = wave % WN;
    // fragments of K step u (32 codes): two sets, one read while the other is multiplied
    v4i av[2][FT], bv[2][FN];
    int slot[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        slot[u] = (lane & 31) * 128 + ((2 * u + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16;
    const int a_at = 4096 * FT * wt, b_at = BT * 128 + 4096 * FN * wn;
    auto read = [&](int set, const uint8_t *buf, int u) {
#pragma unroll
        for (int i = 0; i < FT; ++i)
            av[set][i] = *reinterpret_cast<const v4i *>(buf + slot[u] + a_at + 4096 * i);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            bv[set][j] = *reinterpret_cast<const v4i *>(buf + slot[u] + b_at + 4096 * j);
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bv[set][j], av[set][i], acc[i][j], 0, 0, 0);
    };
    v4i reg[DMA ? 1 : CP];
    auto fetch = [&](uint8_t *buf, int ahead) {          // sets out a whole stage
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            if constexpr (DMA)
                __builtin_amdgcn_global_load_lds(
                    (const __attribute__((address_space(1))) void *)src[i],
                    (__attribute__((address_space(3))) void *)(buf + lds_at(i)), 16, 0, 0);
            else
                reg[i] = load16(src[i]);
            src[i] += ahead;
        }
    };
    auto land = [&](uint8_t *buf) {
        if constexpr (!DMA) {
#pragma unroll
            for (int i = 0; i < CP; ++i)
                *reinterpret_cast<v4i *>(buf + lds_at(i) + 16 * lane) = reg[i];
        }
    };
    // the copies of this wave have landed, its reads are done; then every wave's
    auto meet = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070);              // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // within a K step: a fragment's read, a product, in turn, so that every read
    // is out before the last products and back before the next step's first
    auto interleave = [&]() {
#pragma unroll
        for (int i = 0; i < FT + FN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // an LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // an MFMA
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // Stage st in four K steps.  Step 0's fragments are in set 0 on entry.
    // Before the last step is multiplied all of this stage has been read, so
    // the waves meet there: from then on the next stage can be read and the
    // one after it copied over this one.  Past the last stage the last one is
    // fetched again and not used, so that all stages are the same code.
    const int stages = a.K >> 7;
    auto stage = [&](int st, uint8_t *cur, uint8_t *other) {
        read(1, cur, 1);
        multiply(0);
        interleave();
        read(0, cur, 2);
        multiply(1);
        interleave();
        read(1, cur, 3);
        land(other);
        multiply(0);
        interleave();
        meet();
        read(0, other, 0);
        fetch(cur, st + 3 < stages ? 128 : 0);
        multiply(1);
        interleave();
    };
    if (stages > 0) {
        fetch(buf0, stages > 1 ? 128 : 0);
        land(buf0);
        meet();
        fetch(buf1, stages > 2 ? 128 : 0);
        read(0, buf0, 0);
        int st = 0;
        for (; st + 1 < stages; st += 2) {
            stage(st, buf0, buf1);
            stage(st + 1, buf1, buf0);
        }
        if (stages & 1)
            stage(st, buf0, buf1);
        meet();                                          // no copy outlives the loop
    }
    if (a.K & 127) {
        // src points at the last whole stage, or at the row's start
        const int k = (stages << 7) + 16 * piece, at = (max(stages - 1, 0) << 7) + 16 * piece;
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            *reinterpret_cast<v4i *>(buf0 + lds_at(i) + 16 * lane) = load_codes(src[i] - at, k, a.K);
            asm volatile("" ::: "memory");               // one at a time: it is a single stage
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            read(u & 1, buf0, u);
            multiply(u & 1);
        }
    }

    // Epilogue: register 4g+e of a result is channel 8g + 4*(lane/32) + e of
    // token lane%32, so a lane scales four neighbouring channels at a time.  A
    // wave passes 32 tokens x 32*FN channels at a time through LDS of its own
    // and writes them as 16 bytes per lane, whole rows of the wave's channels
    // (written straight from the registers, 2 bytes per lane, this took a
    // quarter of the time of a 4096 x 24576 x 6144 product).
    constexpr int PITCH = 32 * FN * (int)sizeof(OT) + 16;
    constexpr int LPR = 2 * FN * (int)sizeof(OT);        // lanes (16 bytes each) per row
    constexpr int VE = 16 / (int)sizeof(OT);             // values per lane
    static_assert(32 * PITCH * NW / 2 <= (BT + BN) * 128, "half of the waves' parts fit one buffer");
    const int nw0 = n0 + 32 * FN * wn, tw0 = t0 + 32 * FT * wt;
    if (a.K & 127)
        __syncthreads();                                 // buf0 has been read
    uint8_t *mine = (wave < NW / 2 ? buf0 : buf1) + (wave % (NW / 2)) * 32 * PITCH;
    float ws[FN][16], bias[FN][16];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int n = nw0 + 32 * j + 8 * g + 4 * (lane >> 5);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ws[j][4 * g + e] = a.ws[min(n + e, a.N - 1)];
                bias[j][4 * g + e] = a.bias ? a.bias[min(n + e, a.N - 1)] : 0.0f;
            }
        }
#pragma unroll
    for (int i = 0; i < FT; ++i) {
        const float st = a.s[min(tw0 + 32 * i + (lane & 31), a.T - 1)];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = ((float)acc[i][j][4 * g + e] * st) * ws[j][4 * g + e];
                    if (a.bias)
                        y[e] += bias[j][4 * g + e];
                }
                uint8_t *p = mine + (lane & 31) * PITCH + (32 * j + 8 * g + 4 * (lane >> 5)) * (int)sizeof(OT);
                if constexpr (sizeof(OT) == 2)
                    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                else
                    *reinterpret_cast<float4 *>(p) = make_float4(y[0], y[1], y[2], y[3]);
            }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int h = 0; h < LPR / 2; ++h) {              // 64/LPR rows each
            const int row = h * (64 / LPR) + lane / LPR, col = (lane % LPR) * VE;
            const int t = tw0 + 32 * i + row, n = nw0 + col;
            const uint4 v = *reinterpret_cast<const uint4 *>(mine + row * PITCH + col * (int)sizeof(OT));
            OT *o = static_cast<OT *>(a.out) + (int64_t)t * a.ldo + n;
            if (t < a.T) {
                if (n + VE <= a.N) {
                    *reinterpret_cast<bytes16_a2 *>(o) = bytes16_a2{{v.x, v.y, v.z, v.w}};
                } else {
                    const OT *e = reinterpret_cast<const OT *>(&v);
#pragma unroll
                    for (int c = 0; c < VE; ++c)
                        if (n + c < a.N)
                            o[c] = e[c];
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
}

template <typename OT, int RT, int TB, int W, int U>
static void launch_stream(const LinArgs &a, hipStream_t st)
{
    const dim3 grid((a.N + 16 * RT - 1) / (16 * RT), (a.T + 16 * TB - 1) / (16 * TB));
    launch(linear_stream_kernel<OT, RT, TB, W, U>, grid, 64 * W, 0, st, a);
}

template <typename OT, bool DMA, int WT, int WN, int FT, int FN>
static void launch_tiles(const LinArgs &a, hipStream_t st)
{
    const int tt = (a.T + 32 * WT * FT - 1) / (32 * WT * FT), tn = (a.N + 32 * WN * FN - 1) / (32 * WN * FN);
    const unsigned grid = ((unsigned)tt * tn + 7) / 8 * 8;
    launch(linear_tiles_kernel<OT, DMA, WT, WN, FT, FN>, grid, 64 * WT * WN, 0, st, a, tt, tn);
}

template <typename OT>
static void enqueue_linear(const LinArgs &a, hipStream_t st)
{
    const bool dma = ops_aligned(a.q, 16) && ops_aligned(a.w, 16) && a.ldq % 16 == 0 && a.ldw % 16 == 0;
    if (a.T <= 16)
        launch_stream<OT, 1, 1, 8, 6>(a, st);
    else if (a.T <= 64)
        launch_stream<OT, 2, 2, 8, 4>(a, st);
    else if (dma)
        launch_tiles<OT, true, 2, 4, 4, 2>(a, st);
    else
        launch_tiles<OT, false, 2, 4, 4, 2>(a, st);
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
