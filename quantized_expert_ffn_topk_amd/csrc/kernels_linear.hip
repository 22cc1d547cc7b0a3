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

__device__ __forceinline__ v4i load16(const int8_t *p)
{
    const bytes16_a1 b = *reinterpret_cast<const bytes16_a1 *>(p);
    return v4i{(int)b.d[0], (int)b.d[1], (int)b.d[2], (int)b.d[3]};
}

// 16 codes of a row at k (a multiple of 16), zeros past K, at any alignment, with
// one load: what passes the row's end is read as the row's last 16 bytes and
// shifted down.  (Rows shorter than 16 byte by byte.)
__device__ __forceinline__ v4i load_codes(const int8_t *row, int k, int K)
{
    v4i v = {0, 0, 0, 0};
    if (K >= 16) {
        if (k < K)
            v = load16(row + min(k, K - 16));
        const bool past = k < K && k + 16 > K;
        if (__ballot(past))
            v = __builtin_bit_cast(v4i, __builtin_bit_cast(unsigned __int128, v) >>
                                            (past ? 8 * (k + 16 - K) : 0));
    } else {
        unsigned __int128 b = 0;
        for (int j = k; j < K; ++j)                          // k is 0, or past the row
            b |= (unsigned __int128)(uint8_t)row[j] << (8 * j);
        v = __builtin_bit_cast(v4i, b);
    }
    return v;
}

// ---------------------------------------------------------------------------
// Few tokens: a stream of weights.  A block owns 16*RT weight rows and up to
// 8*TC tokens; its W waves take stages of 128 codes of K in turn (so that a
// block reads W*128 neighbouring bytes of each row) and add their exact sums
// through LDS at the end.  A wave works alone: it reads 8 rows x 128 bytes per
// load, neighbouring lanes on neighbouring bytes, passes them through LDS of
// its own into fragments, and has the next stage's loads in flight meanwhile.
// (Read from memory in the fragments' order, 16 rows x 64 bytes with
// neighbouring lanes on different rows, the loads took a lookup for every
// lane: 24 x 24576 x 6144 44 us, 28 like this.)
// v_mfma_i32_16x16x64_i8: lane l supplies 16 codes at 16*(l/16) of weight row
// l%16 (A) and of token l%16 (B); result register i is row 4*(l/16)+i, token
// l%16.  LDS rows are swizzled as in the tiles below.
// NT: weights read with the non-temporal hint.
// ---------------------------------------------------------------------------
__device__ __forceinline__ v4i load16_stream(const int8_t *p)
{
    typedef int v4i_a1 __attribute__((ext_vector_type(4), aligned(1)));
    return __builtin_nontemporal_load((const __attribute__((address_space(1))) v4i_a1 *)p);
}

template <typename OT, bool NT, int RT, int TC, int W>
__global__ __launch_bounds__(64 * W) void linear_stream_kernel(LinArgs a)
{
    constexpr int TB = (TC + 1) / 2;                     // 16-token tiles
    constexpr int CW = 2 * RT, CP = CW + TC;             // 8-row pieces per stage: weights, all
    constexpr int ST = 1024 * (CW + 2 * TB);             // LDS bytes per wave (whole token tiles;
                                                         // what TC = 1 leaves unwritten is not stored)
    static_assert(RT * TB * 1024 <= ST, "a wave's sums fit its LDS");
    __shared__ __align__(128) uint8_t lds[W * ST];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * RT, t0 = blockIdx.y * 8 * TC;
    const int stages = a.K >> 7;
    const int mine = (stages - wave + W - 1) / W;        // stages wave, wave + W, ...
    const int8_t *src[CP];
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        const int r = 8 * (i < CW ? i : i - CW) + (lane >> 3);
        src[i] = (i < CW) ? a.w + (int64_t)min(n0 + r, a.N - 1) * a.ldw
                          : a.q + (int64_t)min(t0 + r, a.T - 1) * a.ldq;
        src[i] += 16 * (lane & 7) + 128 * wave;
    }
    uint8_t *slot = lds + wave * ST;
    int put[2], at[2];                                   // of a piece's even and odd 8 rows; of K half u
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        put[u] = 128 * (lane >> 3) + 16 * ((lane & 7) ^ (4 * u + (lane >> 4)));
        at[u] = 128 * (lane & 15) + 16 * ((4 * u + (lane >> 4)) ^ ((lane >> 1) & 7));
    }
    // the scales of the outputs that this thread will write, on their way from the
    // beginning (read at the end, cold, they cost 1 x 6144 x 6144 7.8 us instead of
    // 7.35, 16 x 4096 x 4096 7.2 instead of 6.7)
    constexpr int IT = (RT * TB + W - 1) / W;
    float s[IT], ws[IT][4], bias[IT][4];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int f = min((int)threadIdx.x + 64 * W * it, RT * TB * 64 - 1), l = f & 63, ij = f >> 6;
        s[it] = a.s[min(t0 + 16 * (ij % TB) + (l & 15), a.T - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = min(n0 + 16 * (ij / TB) + 4 * (l >> 4) + i, a.N - 1);
            ws[it][i] = a.ws[n];
            bias[it][i] = a.bias ? a.bias[n] : 0.0f;
        }
    }
    asm volatile("" ::: "memory");
    v4i acc[RT][TB], reg[CP], wv[2][RT], qv[2][TB];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
            acc[i][j] = v4i{0, 0, 0, 0};
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            reg[i] = (NT && i < CW) ? load16_stream(src[i]) : load16(src[i]);
            src[i] += 128 * W;
        }
    };
    auto multiply = [&]() {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u][i], qv[u][j], acc[i][j], 0, 0, 0);
    };
    if (mine > 0)
        fetch();
    for (int i = 0; i < mine; ++i) {
#pragma unroll
        for (int c = 0; c < CP; ++c)
            *reinterpret_cast<v4i *>(slot + 1024 * c + put[c & 1]) = reg[c];
        if (i + 1 < mine)
            fetch();
        wave_lds_sync();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int k = 0; k < RT; ++k)
                wv[u][k] = *reinterpret_cast<const v4i *>(slot + at[u] + 2048 * k);
#pragma unroll
            for (int j = 0; j < TB; ++j)
                qv[u][j] = *reinterpret_cast<const v4i *>(slot + at[u] + 1024 * CW + 2048 * j);
        }
        wave_lds_sync();
        multiply();
    }
    if ((a.K & 127) && wave == stages % W) {             // the partial last stage
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int k = (stages << 7) + 64 * u + 16 * (lane >> 4);
#pragma unroll
            for (int i = 0; i < RT; ++i)
                wv[u][i] = load_codes(a.w + (int64_t)min(n0 + 16 * i + (lane & 15), a.N - 1) * a.ldw, k, a.K);
#pragma unroll
            for (int j = 0; j < TB; ++j)
                qv[u][j] = load_codes(a.q + (int64_t)min(t0 + 16 * j + (lane & 15), a.T - 1) * a.ldq, k, a.K);
        }
        multiply();
    }
    v4i *part = reinterpret_cast<v4i *>(slot);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
            part[(i * TB + j) * 64 + lane] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int f = (int)threadIdx.x + 64 * W * it, l = f & 63, ij = f >> 6;
        if (f >= RT * TB * 64)
            break;
        v4i sum = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < W; ++w)
            sum += reinterpret_cast<const v4i *>(lds + w * ST)[f];
        const int n = n0 + 16 * (ij / TB) + 4 * (l >> 4), c = 16 * (ij % TB) + (l & 15), t = t0 + c;
        if (c < 8 * TC && t < a.T) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y = ((float)sum[i] * s[it]) * ws[it][i];
                if (a.bias)
                    y += bias[it][i];
                if (n + i < a.N)
                    store1(static_cast<OT *>(a.out) + (int64_t)t * a.ldo + n + i, y);
            }
        }
    }
}

// 16 bytes of each lane from memory to LDS at 16 times the lane, by the load
// unit; NT_BIT 2: with the non-temporal hint
template <int NT_BIT>
__device__ __forceinline__ void copy16(const int8_t *from, uint8_t *to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 16, 0, NT_BIT);
}

// ---------------------------------------------------------------------------
// Tiles: a block computes BT = 32*WT*FT tokens x BN = 32*WN*FN channels with
// WT*WN waves of FT*FN 32x32 results, K in stages of 128 codes through NB LDS
// buffers, the next stages' rows on their way while one is multiplied.
// An LDS row is 128 bytes, eight 16-byte pieces; piece c of row r sits at slot
// c ^ (r/2 & 7): two rows fill the 64 banks once, so that 16 neighbouring rows'
// reads of one piece fall on different banks.
// DMA: rows go global -> LDS by the load unit (a wave's copy is 8 rows, lane l
// writing slot l%8 of row l/8, so the lane picks the global piece that belongs
// there); needs rows of 16-byte alignment.  Otherwise they pass through
// registers.  The last, partial stage always does (load_codes gives its zeros).
// 256 x 256 tiles of 4096 x 24576 x 6144: 531 us, 2330 TOP/s (the library's int8
// product 575), the matrix units busy 63 % of the cycles at 1.78 GHz.  Bound by
// power: copies one and a half stages ahead instead of one took 2.6 % fewer
// cycles at a 4 % lower clock, the same time; zeros for tokens are 17 % faster.
// ---------------------------------------------------------------------------
template <typename OT, bool DMA, bool NT, int AHEAD, int WT, int WN, int FT, int FN>
__global__ __launch_bounds__(64 * WT * WN) void linear_tiles_kernel(LinArgs a, int tiles_t, int tiles_n)
{
    constexpr int NW = WT * WN, BT = 32 * WT * FT, BN = 32 * WN * FN;
    constexpr int CP = (BT + BN) / 8 / NW;               // 8-row copies per wave and stage
    constexpr int BUF = (BT + BN) * 128;                 // bytes of a stage
    constexpr int TP = BT / 8 / NW;                      // of these, token rows
    static_assert(BT % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole copies per wave");
    // the buffers are objects of their own: the compiler then knows that reads
    // of one do not wait for copies into another
    constexpr int NB = DMA ? AHEAD : 2;
    static_assert(NB >= 2 && NB <= 4, "two to four buffers");
    __shared__ __align__(128) uint8_t buf0[BUF];
    __shared__ __align__(128) uint8_t buf1[BUF];
    __shared__ __align__(128) uint8_t buf2[NB > 2 ? BUF : 16];
    __shared__ __align__(128) uint8_t buf3[NB > 3 ? BUF : 16];
    __shared__ __align__(16) float scale[BT + 2 * BN];   // tokens' scales, channels', biases

    // tiles in groups of 8 token tiles, token tile fastest, each XCD (blocks
    // with the same index mod 8) a contiguous run of them
    const int per = gridDim.x >> 3, logical = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (logical >= tiles_t * tiles_n)
        return;
    const int band = logical / (8 * tiles_n), in = logical - band * 8 * tiles_n;
    const int gt = min(8, tiles_t - 8 * band);
    const int t0 = (8 * band + in % gt) * BT, n0 = (in / gt) * BN;

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

    // the epilogue's scales go to LDS ahead of all rows, 64 at a time (read at the
    // end, cold, they cost 333 x 5003 x 2048 10.1 us instead of 9.55, 1500 x 2048 x
    // 2048 12.7 instead of 11.5)
    auto bring = [&](const float *from, int first, int count, float *to, int at) {
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void *)(from + min(first + at + lane, count - 1)),
            (__attribute__((address_space(3))) void *)(to + at), 4, 0, 0);
    };
    for (int i = wave; 64 * i < BT; i += NW)
        bring(a.s, t0, a.T, scale, min(64 * i, BT - 64));
    for (int i = wave; 64 * i < BN; i += NW) {
        bring(a.ws, n0, a.N, scale + BT, 64 * i);
        if (a.bias)
            bring(a.bias, n0, a.N, scale + BT + BN, 64 * i);
    }
    v16i acc[FT][FN];
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = v16i{0};
    const int wt = wave / WN, wn = wave % WN;
    // fragments: two sets, one read while the other is multiplied; of a K step
    // (32 codes) each, or, where a step is a single product (WHOLE), of a
    // stage's four
    constexpr bool WHOLE = FT * FN == 1;
    constexpr int US = WHOLE ? 4 : 1;
    v4i av[2][US][FT], bv[2][US][FN];
    int slot[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        slot[u] = (lane & 31) * 128 + ((2 * u + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16;
    const int a_at = 4096 * FT * wt, b_at = BT * 128 + 4096 * FN * wn;
    auto read = [&](int set, const uint8_t *buf, int u) {
        const int k = WHOLE ? u : 0;
#pragma unroll
        for (int i = 0; i < FT; ++i)
            av[set][k][i] = *reinterpret_cast<const v4i *>(buf + slot[u] + a_at + 4096 * i);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            bv[set][k][j] = *reinterpret_cast<const v4i *>(buf + slot[u] + b_at + 4096 * j);
    };
    auto multiply = [&](int set, int k) {
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bv[set][k][j], av[set][k][i], acc[i][j], 0, 0, 0);
    };
    constexpr int RD = DMA ? 0 : AHEAD;                  // stages in registers on their way into LDS
    constexpr int SETS = DMA ? 1 : RD;
    v4i reg[SETS][DMA ? 1 : CP];
    auto fetch = [&](uint8_t *buf, int set) {            // sets out the next whole stage
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            if constexpr (!DMA)
                reg[set][i] = load16(src[i]);
            else if (NT && i >= TP)
                copy16<2>(src[i], buf + lds_at(i));
            else
                copy16<0>(src[i], buf + lds_at(i));
            src[i] += 128;
        }
    };
    auto land = [&](uint8_t *buf, int set) {
#pragma unroll
        for (int i = 0; i < CP; ++i)
            *reinterpret_cast<v4i *>(buf + lds_at(i) + 16 * lane) = reg[set][i];
    };
    // this wave's copies have landed but for those of the LEFT stages set out
    // last, and its reads are done; then every wave's
    auto meet = [&](auto left_) {
        constexpr int LEFT = decltype(left_)::value * CP;
        static_assert(LEFT < 64, "vmcnt counts to 63");
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | (LEFT >> 4) << 14);   // vmcnt(LEFT) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // the same where nothing is copied: loads into registers stay on their way
    auto meet_lds = [&]() {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xc07f);              // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    const std::integral_constant<int, 0> all;
    const std::integral_constant<int, NB - 2> ahead;
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
    // The waves meet once per stage, when all of stage st has been read: from
    // then on stage st + 1 can be read and stage st + LEAD be set out over this
    // one.  The stages' end (MORE = false) waits for all copies and sets out
    // none past the last.
    const int stages = a.K >> 7;
    constexpr int LEAD = DMA ? NB : 1 + RD;
    auto meet_at = [&](auto more_, int st) {
        if constexpr (!DMA) {
            meet_lds();
        } else if constexpr (decltype(more_)::value) {
            meet(ahead);
        } else {
            if (st + NB - 1 < stages)
                meet(ahead);
            else
                meet(all);
        }
    };
    // WHOLE: stage st's fragments are in set `frag`; the next stage's are read
    // while they are multiplied (read a K step ahead, a 64 x 64 tile's stage
    // waited for LDS four times: 128 x 8192 x 6144 15.4 us, 13.7 like this).
    // Else the stage is read a K step ahead, between the products, and the last
    // step multiplied after the waves have met (with the next stage's 16 reads
    // in front of its products, 128 x 128 tiles of 512 x 6144 x 6144 took 32.2
    // us for 27.1).
    auto stage = [&](auto more_, int st, uint8_t *cur, uint8_t *next, int set, int frag) {
        constexpr bool MORE = decltype(more_)::value;
        if constexpr (WHOLE) {
            if constexpr (!DMA)
                land(next, set);
            meet_at(more_, st);
            if (MORE || st + LEAD < stages)
                fetch(cur, set);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                read(1 - frag, next, u);
            __builtin_amdgcn_sched_barrier(0);           // all reads out first
#pragma unroll
            for (int u = 0; u < 4; ++u)
                multiply(frag, u);
            __builtin_amdgcn_sched_barrier(0);
        } else {
            read(1, cur, 1);
            multiply(0, 0);
            interleave();
            read(0, cur, 2);
            multiply(1, 0);
            interleave();
            read(1, cur, 3);
            if constexpr (!DMA)
                land(next, set);
            multiply(0, 0);
            interleave();
            meet_at(more_, st);
            read(0, next, 0);
            if (MORE || st + LEAD < stages)
                fetch(cur, set);
            multiply(1, 0);
            interleave();
        }
    };
    auto read_first = [&]() {
#pragma unroll
        for (int u = 0; u < (WHOLE ? 4 : 1); ++u)
            read(0, buf0, u);
    };
    if (stages > 0) {
        fetch(buf0, 0);
        if constexpr (DMA) {
            if (1 < stages)
                fetch(buf1, 0);
            if constexpr (NB > 2)
                if (2 < stages)
                    fetch(buf2, 0);
            if constexpr (NB > 3)
                if (3 < stages)
                    fetch(buf3, 0);
            // each way reads for itself: joined before the reads, the compiler
            // would wait for every copy there
            if (stages >= NB) {
                meet(std::integral_constant<int, NB - 1>());
                read_first();
            } else {
                meet(all);
                read_first();
            }
        } else {
            land(buf0, 0);
#pragma unroll
            for (int i = 1; i <= RD; ++i)
                if (i < stages)
                    fetch(buf0, i % SETS);
            meet_lds();
            read_first();
        }
        // stage i of a round: buffer i % NB, fragment set i % 2 (WHOLE), register
        // set (i + 1) % RD, all known at compile time
        constexpr int ROUND = DMA ? NB : RD % 2 ? 2 * RD : RD;
        constexpr std::true_type more{};
        constexpr std::false_type end{};
        static_assert(!WHOLE || ROUND % 2 == 0, "a round ends on the set it began with");
        auto buf = [&](int i) { return i % NB == 0 ? buf0 : i % NB == 1 ? buf1 : i % NB == 2 ? buf2 : buf3; };
        int st = 0;
        for (; st + ROUND - 1 + LEAD < stages; st += ROUND) {
#pragma unroll
            for (int i = 0; i < ROUND; ++i)
                stage(more, st + i, buf(i), buf(i + 1), (i + 1) % SETS, i % 2);
        }
        for (; st < stages; st += ROUND) {
#pragma unroll
            for (int i = 0; i < ROUND; ++i)
                if (st + i < stages)
                    stage(end, st + i, buf(i), buf(i + 1), (i + 1) % SETS, i % 2);
        }
    }
    const bool tail = (a.K & 127) != 0;
    if (tail) {
        const int k = 128 * stages + 16 * piece;         // src has come this far
#pragma unroll
        for (int i = 0; i < CP; ++i)
            *reinterpret_cast<v4i *>(buf0 + lds_at(i) + 16 * lane) = load_codes(src[i] - k, k, a.K);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            read(u & 1, buf0, u);
            multiply(u & 1, WHOLE ? u : 0);
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
    static_assert(32 * PITCH * NW / 2 <= BUF, "half of the waves' parts fit one buffer");
    const int nw0 = n0 + 32 * FN * wn, tw0 = t0 + 32 * FT * wt;
    uint8_t *mine = (wave < NW / 2 ? buf0 : buf1) + (wave % (NW / 2)) * 32 * PITCH;
    // every wave's scales are there, and its reads of buf0 done
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);                  // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    float ws[FN][16], bias[FN][16];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float *at = scale + BT + 32 * (FN * wn + j) + 8 * g + 4 * (lane >> 5);
            const float4 w = *reinterpret_cast<const float4 *>(at);
            const float4 b = *reinterpret_cast<const float4 *>(at + BN);   // not used unless there is a bias
            ws[j][4 * g] = w.x, ws[j][4 * g + 1] = w.y, ws[j][4 * g + 2] = w.z, ws[j][4 * g + 3] = w.w;
            bias[j][4 * g] = b.x, bias[j][4 * g + 1] = b.y, bias[j][4 * g + 2] = b.z, bias[j][4 * g + 3] = b.w;
        }
#pragma unroll
    for (int i = 0; i < FT; ++i) {
        const float st = scale[32 * (FT * wt + i) + (lane & 31)];
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
        wave_lds_sync();
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
        wave_lds_sync();
    }
}

template <typename OT, bool NT, int RT, int TC, int W>
static void launch_stream(const LinArgs &a, hipStream_t st)
{
    const dim3 grid((a.N + 16 * RT - 1) / (16 * RT), (a.T + 8 * TC - 1) / (8 * TC));
    launch(linear_stream_kernel<OT, NT, RT, TC, W>, grid, 64 * W, 0, st, a);
}

template <typename OT, bool DMA, int AHEAD, int WT, int WN, int FT, int FN>
static void launch_tiles(const LinArgs &a, bool nt, hipStream_t st)
{
    const int tt = (a.T + 32 * WT * FT - 1) / (32 * WT * FT), tn = (a.N + 32 * WN * FN - 1) / (32 * WN * FN);
    const unsigned grid = ((unsigned)tt * tn + 7) / 8 * 8;
    if (DMA && nt && tt == 1)                            // weights that nobody reads a second time
        launch(linear_tiles_kernel<OT, DMA, DMA, AHEAD, WT, WN, FT, FN>, grid, 64 * WT * WN, 0, st, a, tt, tn);
    else
        launch(linear_tiles_kernel<OT, DMA, false, AHEAD, WT, WN, FT, FN>, grid, 64 * WT * WN, 0, st, a, tt, tn);
}

// ---------------------------------------------------------------------------
// Choice of a kernel.  Times in us on an MI355X, launches in a row.  Those of the
// streams were taken with the outputs' scales still read at the end; now they are
// 0.3 to 1.2 less for all of them alike (24 x 24576 x 6144: 26.1).
//
// Stream: up to 32 tokens, and more where its blocks still find a CU each
// (256 x 512 x 6144: 6.4, tiles 12.0; 256 x 2048 x 7168: 11.3, 13.3; else tiles
// win: 128 x 6144 x 6144 20.3, tiles 12.7; 64 x 12288 x 6144 20.8, 15.1;
// 64 x 20000 x 512 11.4, 6.2).
//  - Blocks are as small as leaves each a CU: 8 tokens, 16, 32 or 64, at most as
//    many as there are, and 16, 32 or 48 weight rows (64 x 256 x 6144 in 16
//    tokens x 16 rows 4.4, 32 x 16 5.2; 64 x 2048 x 7168 in 32 x 16 6.9, 64 x 16
//    9.3; 171 x 896 x 5744 in 32 x 32 9.6, 64 x 32 13.7; 1748 x 192 x 8000 in
//    32 x 48 14.3, 64 x 32 18.6; 32 x 8448 x 6144, 11.0, and in 32 x 32 14.8);
//    past that 32 rows by four waves, two blocks per CU (16 x 16000 x 5760:
//    16.8, 48 x 8 waves 20.6, 16 x 8 18.7; 28 x 16080 x 4320 at odd strides
//    17.7, 22.3, 23.4).
//  - Up to 8 tokens 16 rows while 32 fit (4 x 8192 x 6144: 9.4, with 32 rows
//    9.5), in 16 waves where a CU has one block (1 x 512 x 12288: 5.5, with 8
//    waves 6.5; 8 x 2048 x 7168: 5.0, 5.4; 1 x 12288 x 2048, three blocks: 7.3,
//    6.2).
//  - The non-temporal hint from 96 MiB of weights on, of which the 256 MiB
//    last-level cache keeps hardly two (3 x 24576 x 4480: 17.7 with, 19.5
//    without; 24 x 24576 x 6144: 26.7, 29.8; tiles where a weight is read once,
//    128 x 24576 x 6144: 40.2, 44.7; at 91 MiB, 24 x 13312 x 7168 from three
//    sets of weights in turn: 20.1, 19.5).  Smaller weights may stay there from
//    one call to the next and are read plainly: 32 x 6144 x 6144 8.9 from the
//    cache, 12.1 from memory; with the hint 11.7 from either.  Where other layers
//    pass the cache between two calls they come from memory: one set of weights
//    again and again / 750 MB of them in turn, 1 x 6144 x 6144 6.9 / 9.1, 24 x 6144
//    x 6144 7.7 / 12.6, 8 x 12288 x 6144 12.9 / 15.8, 128 x 6144 x 6144 (tiles)
//    12.2 / 19.1, 1 x 2048 x 7168 3.8 / 6.1.  Rows that are not
//    whole lines share lines, which the hint would fetch twice (24 x 12288 x
//    12288 at odd strides: 45.7 with, 42.3 without).  With it, 64 rows by four
//    waves where 48 no longer fit (16 x 14336 x 8192: 64 rows 23.2, 48 25.9;
//    3 x 14336 x 8192: 22.4, 32 rows 28.7), past that 48 rows (24 x 24576 x
//    6144: 26.7, 64 rows 29, 32 rows 30), up to 8 tokens 32 (3 x 24576 x 4480:
//    17.7, 48 rows 18.0, 16 rows of eight waves 19.8).
//
// Tiles: a block's time is about its stages of 128 codes, each bound by what a
// CU takes in (some 40 bytes a clock; 64 x 64 .. 192 x 128 tiles need 16 .. 40
// KiB a stage) or by its products (256 x 256), and a fixed part, the first
// stage's way and the output.  Blocks go to 256 CUs in rounds; two of the
// smallest tiles fit a CU and share their fixed parts, and one that is alone
// takes longer per stage.  The tile whose rounds cost least is taken.  The costs
// rank the tiles and are no times: they were fitted to 139 shapes of 65 to 4096
// tokens, 64 to 12288 long, for the loss against the fastest tile, and a cost is
// 0.5 to 1.6 times the measured time (the median 0.97, of the tile taken 0.85;
// 128 x 6144 x 6144 as 64 x 64: cost 18.0, 12.2 us).  The tile taken is 0.3 %
// slower than the fastest of the eight on average, at most 8 %, on those shapes
// as on 100 others drawn afterwards; profiles/int8_product_tiles.csv has all
// times, and a test holds the costs below to them.  (With 64x64, 64x128, 128x128,
// 128x256 and 256x256 alone the fastest are 2.7 % slower.)  64x64 / 64x128 /
// 96x128 / 128x128 / 192x128 / 128x256 / 192x256 / 256x256:
//    128 x  6144 x 6144   12.2 / 17.6 / 20.7 / 23.8 / 29.0 / 35.9 / 47.8 / 60.3
//    256 x 12288 x 6144   31.8 / 30.9 / 42.8 / 27.9 / 33.6 / 36.0 / 48.9 / 62.0
//    451 x  4992 x 2688   15.5 / 15.2 / 12.4 / 13.5 / 16.0 / 19.6 / 26.0 / 33.0
//    520 x  9856 x 3008   36.5 / 33.5 / 34.2 / 36.0 / 26.1 / 28.6 / 37.5 / 39.6
//    600 x  8192 x 4096   36.4 / 33.8 / 33.0 / 36.5 / 29.3 / 28.8 / 35.0 / 44.4
//   1309 x  7360 x 1344   34.8 / 29.3 / 36.1 / 33.1 / 26.2 / 30.0 / 21.5 / 25.0
//   2048 x 24576 x 2048    218 /  173 /  186 /  171 /  143 /  135 /  132 /  110
//   3000 x  8000 x 8000    376 /  309 /  317 /  260 /  239 /  215 /  207 /  219
// Rows that are not 16-byte aligned pass through registers: each piece crosses a
// line (a quarter more time), and at odd addresses another quarter (128 x 6144 x
// 6144: 12.3 aligned, 23.5 at odd strides; 4096 x 24576 x 6144: 529, 768).
// ---------------------------------------------------------------------------
constexpr int64_t CUS = 256;

static int64_t blocks_of(const LinArgs &a, int tokens, int rows)
{
    return (int64_t)((a.T + tokens - 1) / tokens) * ((a.N + rows - 1) / rows);
}

// weights worth the non-temporal hint: too large for the last-level cache to
// keep from one call to the next, and their rows whole lines
static bool passing(const LinArgs &a)
{
    return (int64_t)a.N * a.K >= (96 << 20) && ops_aligned(a.w, 128) && a.ldw % 128 == 0;
}

template <typename OT, int TC>
static void enqueue_stream(const LinArgs &a, hipStream_t st)
{
    const bool nt = passing(a);
    auto fits = [&](int rows) { return blocks_of(a, 8 * TC, rows) <= CUS; };
    if constexpr (TC == 1) {
        if (fits(16))
            launch_stream<OT, false, 1, TC, 16>(a, st);
        else if (fits(32))
            nt ? launch_stream<OT, true, 1, TC, 8>(a, st) : launch_stream<OT, false, 1, TC, 8>(a, st);
        else if (fits(48))
            nt ? launch_stream<OT, true, 3, TC, 8>(a, st) : launch_stream<OT, false, 3, TC, 8>(a, st);
        else if (nt && fits(64))
            launch_stream<OT, true, 4, TC, 4>(a, st);
        else
            nt ? launch_stream<OT, true, 2, TC, 4>(a, st) : launch_stream<OT, false, 2, TC, 4>(a, st);
    } else if constexpr (TC == 8) {
        nt ? launch_stream<OT, true, 2, TC, 8>(a, st) : launch_stream<OT, false, 2, TC, 8>(a, st);
    } else {
        if (fits(16))
            launch_stream<OT, false, 1, TC, 8>(a, st);
        else if (fits(32))
            nt ? launch_stream<OT, true, 2, TC, 8>(a, st) : launch_stream<OT, false, 2, TC, 8>(a, st);
        else if (fits(48))
            nt ? launch_stream<OT, true, 3, TC, 8>(a, st) : launch_stream<OT, false, 3, TC, 8>(a, st);
        else if (!nt)
            launch_stream<OT, false, 2, TC, 4>(a, st);
        else if (fits(64))
            launch_stream<OT, true, 4, TC, 4>(a, st);
        else
            launch_stream<OT, true, 3, TC, 4>(a, st);
    }
}

template <typename OT, bool DMA>
static void enqueue_tiles(const LinArgs &a, hipStream_t st)
{
    struct Tile {
        int bt, bn, fit;                                 // blocks of it that fit a CU
        double stage, fixed, alone;                      // costs, see above
    };
    static constexpr Tile tile[8] = {
        {64, 64, 2, 0.211, 2.4, 0.113},  {64, 128, 2, 0.313, 3.4, 0.079}, {96, 128, 1, 0.548, 3.8, 0.0},
        {128, 128, 1, 0.514, 6.7, 0.0},  {192, 128, 1, 0.533, 6.4, 0.0},  {128, 256, 1, 0.849, 6.9, 0.0},
        {192, 256, 1, 0.992, 7.1, 0.0},  {256, 256, 1, 1.298, 9.4, 0.0}};
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < 8; ++i) {
        const Tile &t = tile[i];
        const int64_t n = (blocks_of(a, t.bt, t.bn) + CUS - 1) / CUS;
        const double k = a.K / 128.0, alone = n % t.fit ? t.alone : 0.0;
        const double cost = (n * t.stage + alone) * k + (n + t.fit - 1) / t.fit * t.fixed;
        if (i == 0 || cost < least) {
            best = i;
            least = cost;
        }
    }
    // copies: as many stages ahead as the LDS has room for, two blocks of the
    // smallest tiles to a CU; registers: as many as they hold
    const bool nt = passing(a);
    switch (best) {
    case 0: launch_tiles<OT, DMA, DMA ? 4 : 3, 2, 2, 1, 1>(a, nt, st); break;
    case 1: launch_tiles<OT, DMA, 3, 2, 2, 1, 2>(a, nt, st); break;
    case 2: launch_tiles<OT, DMA, 3, 1, 4, 3, 1>(a, nt, st); break;
    case 3: launch_tiles<OT, DMA, 3, 2, 2, 2, 2>(a, nt, st); break;
    case 4: launch_tiles<OT, DMA, 3, 2, 4, 3, 1>(a, nt, st); break;
    case 5: launch_tiles<OT, DMA, 3, 2, 4, 2, 2>(a, nt, st); break;
    case 6: launch_tiles<OT, DMA, 2, 2, 4, 3, 2>(a, nt, st); break;
    default: launch_tiles<OT, DMA, DMA ? 2 : 1, 2, 4, 4, 2>(a, nt, st); break;
    }
}

template <typename OT>
static void enqueue_linear(const LinArgs &a, hipStream_t st)
{
    if (a.T <= 8)
        enqueue_stream<OT, 1>(a, st);
    else if (a.T <= 16 || blocks_of(a, 16, 16) <= CUS)
        enqueue_stream<OT, 2>(a, st);
    else if (a.T <= 32 || blocks_of(a, 32, 48) <= CUS)
        enqueue_stream<OT, 4>(a, st);
    else if (blocks_of(a, 64, 32) <= CUS)
        enqueue_stream<OT, 8>(a, st);
    else if (ops_aligned(a.q, 16) && ops_aligned(a.w, 16) && a.ldq % 16 == 0 && a.ldw % 16 == 0)
        enqueue_tiles<OT, true>(a, st);
    else
        enqueue_tiles<OT, false>(a, st);
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
    if ((int64_t)T * N > (1ll << 38))                // the launch's limit on threads
        return fail(MOE_E_INVAL, "T*N=%lld above 2^38", (long long)T * N);
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
