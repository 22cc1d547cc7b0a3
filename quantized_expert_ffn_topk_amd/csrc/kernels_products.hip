// kernels_products.hip -- products of E4M3 or bf16 rows on gfx950, dense and
// grouped by expert.
//
// E4M3:  out[t,n] = bias[n] + sum_b (sum_{k in block b} q[t,k]*w[n,k]) * (s[t,b]*ws[n/128,b])
//        with blocks of 128 neighbouring k,
// bf16:  out[t,n] = sum_k x[t,k]*w[n,k],
// for all rows t, or for the rows of each group with the weights of its expert.
//
// Both read K in stages of 128 bytes of each row: a block of codes, or 64 bf16
// values.  Three ways to multiply a stage (MODE):
//   F8    v_mfma_f32_16x16x128_f8f6f4, the block's sum from zero, then one fp32
//         FMA per result with the block's scale.  The unit aligns the products of
//         8 neighbouring k to the largest of them and keeps 13 bits below its
//         leading one (found with single products: 2^16 + 2^3 is exact, 2^16 + 2^2
//         gives 2^16); between the eights it adds in fp32.  On normal codes a
//         block's sum is off by 1.4e-5 of its size; taken for bf16 outputs only,
//         whose own rounding is 2^-8.
//   F8X   the codes widened to bf16, exactly, and v_mfma_f32_16x16x32_bf16: sums in
//         fp32, half the rate.  Taken for fp32 outputs, and where the weights'
//         stream sets the time anyway.
//   BF16  v_mfma_f32_16x16x32_bf16 on the values as they are, one running sum.
// The unit's own rates here are 4130 TFLOP/s for F8 and 1900 for the others; widening
// takes 7 cycles of a SIMD for two codes a lane.
//
// What sets the time: few rows, the stream of weights from HBM (6.4 to 7.0 TB/s);
// many rows, the matrix unit with the scaling of its results beside it; in between,
// how many bytes are on their way per CU.  Weights are laid out as they come.
#include "copy_window.h"
#include "ops_common.h"
#include "products_choice.h"

namespace moe {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

struct ProdArgs {
    const uint8_t *x, *w;
    const float *s, *ws, *bias;         // s, ws NULL: bf16; bias NULL: none
    void *out;
    const int32_t *rows, *offsets;      // grouped: row of x of each grouped row (NULL: the same), groups
    int64_t ldx, ldw, w_stride;         // bytes
    int64_t lds, ldws, ws_stride, ldo;  // elements
    int R, M, N, E;                     // rows of x, rows of out, channels, experts
    int K;                              // bytes of a row
};

// ---------------------------------------------------------------------------
// A block's tile: rows [row0, row0 + rows) of out, channels from n0, and the
// weights and scales of their expert.
// ---------------------------------------------------------------------------
struct Tile {
    int row0, rows, n0;
    const uint8_t *w;
    const float *ws;
};

// Tile f of the groups, in the order expert, channels, rows (the rows of an expert
// share its weights while they are in the caches); each XCD (blocks with the same
// index mod 8) takes a contiguous run.  Every wave finds it for itself: a lane
// counts the row tiles of four experts, a prefix sum over the wave gives the
// lane, and the lane its expert.  Offsets are clamped to the rows of out, so that
// whatever they hold nothing outside is touched.
template <int BT>
struct GroupScan {
    int o[5], incl;
    __device__ __forceinline__ void load(const ProdArgs &a, int first, int lane)
    {
#pragma unroll
        for (int j = 0; j < 5; ++j)
            o[j] = a.offsets[min(first + 4 * lane + j, a.E)];
        int n = 0;
#pragma unroll
        for (int j = 0; j < 5; ++j)
            o[j] = min(max(o[j], j ? o[j - 1] : 0), a.M);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            n += (o[j + 1] - o[j] + BT - 1) / BT;
        incl = n;
#define STEP(c, r) incl += dpp0<c, r>(incl);
        MOE_DPP_STEPS(STEP)
#undef STEP
    }
    __device__ __forceinline__ int total() const
    {
        return __builtin_amdgcn_readlane(incl, 63);
    }
};

template <int BT, int BN>
__device__ __forceinline__ bool find_tile(const ProdArgs &a, int tiles_n, int lane, Tile &t)
{
    GroupScan<BT> g;
    int all = 0;
    for (int e = 0; e < a.E; e += 256) {
        g.load(a, e, lane);
        all += g.total();
    }
    const int64_t tiles = (int64_t)all * tiles_n;
    const int per = (int)((tiles + 7) >> 3);
    if (tiles > INT_MAX || (int)(blockIdx.x >> 3) >= per)
        return false;
    const int f = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    const int q = f / tiles_n;                       // row tile, counted over all experts' channels
    if (q >= all)
        return false;
    int before = 0, e = 0;
    for (;; e += 256) {
        if (a.E > 256)
            g.load(a, e, lane);
        const int n = g.total();
        if (q < before + n)
            break;
        before += n;
        if (e + 256 >= a.E)
            return false;
    }
    const unsigned long long above = __ballot(before + g.incl > q);
    if (!above)
        return false;
    const int src = __ffsll(above) - 1;
    int at = 0, cum = 0;
    {
        int mine = 0;                                // tiles of this lane's experts
#pragma unroll
        for (int j = 0; j < 4; ++j)
            mine += (g.o[j + 1] - g.o[j] + BT - 1) / BT;
        int c = before + g.incl - mine;
        cum = c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = (g.o[j + 1] - g.o[j] + BT - 1) / BT;
            if (c <= q && q < c + n) {
                at = j;
                cum = c;
            }
            c += n;
        }
    }
    int lo = g.o[0], hi = g.o[1];
#pragma unroll
    for (int j = 1; j < 4; ++j)
        if (at == j) {
            lo = g.o[j];
            hi = g.o[j + 1];
        }
    at = __builtin_amdgcn_readlane(at, src);
    cum = __builtin_amdgcn_readlane(cum, src);
    lo = __builtin_amdgcn_readlane(lo, src);
    hi = __builtin_amdgcn_readlane(hi, src);
    e += 4 * src + at;
    const int n = (hi - lo + BT - 1) / BT;           // this expert's row tiles
    if (e >= a.E || n < 1)
        return false;
    const int in = f - cum * tiles_n, col = in / n, row = in - col * n;
    t.row0 = lo + row * BT;
    t.rows = min(BT, hi - t.row0);
    t.n0 = col * BN;
    t.w = a.w + (int64_t)e * a.w_stride;
    t.ws = a.ws + (int64_t)e * a.ws_stride;
    return true;
}

// the row of x of row r (< M) of out
template <bool GROUPED>
__device__ __forceinline__ int64_t source_row(const ProdArgs &a, int r)
{
    if (GROUPED && a.rows)
        r = min(max(a.rows[r], 0), a.R - 1);
    return r;
}

// ---------------------------------------------------------------------------
// Loads.  A piece is 16 bytes of a row, eight pieces a stage.
// ---------------------------------------------------------------------------
__device__ __forceinline__ v4i load_piece(const uint8_t *p)
{
    const bytes16_a1 b = *reinterpret_cast<const bytes16_a1 *>(p);
    return v4i{(int)b.d[0], (int)b.d[1], (int)b.d[2], (int)b.d[3]};
}
__device__ __forceinline__ v4i load_piece_stream(const uint8_t *p)
{
    typedef int v4i_a1 __attribute__((ext_vector_type(4), aligned(1)));
    return __builtin_nontemporal_load((const __attribute__((address_space(1))) v4i_a1 *)p);
}
// the piece at byte k (a multiple of 16), zeros past K: what passes the row's end
// is read as the row's last 16 bytes and shifted down
__device__ __forceinline__ v4i load_piece_end(const uint8_t *row, int k, int K)
{
    v4i v = {0, 0, 0, 0};
    if (K >= 16) {
        if (k < K)
            v = load_piece(row + min(k, K - 16));
        if (k < K && k + 16 > K)
            v = __builtin_bit_cast(v4i, __builtin_bit_cast(unsigned __int128, v) >> (8 * (k + 16 - K)));
    } else {
        unsigned __int128 b = 0;
        for (int j = k; j < K; ++j)                  // k is 0, or past the row
            b |= (unsigned __int128)row[j] << (8 * j);
        v = __builtin_bit_cast(v4i, b);
    }
    return v;
}
// an address that is the same in every lane, in scalar registers
__device__ __forceinline__ const uint8_t *uniform(const void *p)
{
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)u);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
    return reinterpret_cast<const uint8_t *>((uint64_t)hi << 32 | lo);
}
// `bytes` of memory at p as the load unit's buffer: a word at an offset that is not all
// inside reads as 0
__device__ __forceinline__ v4i buffer_of(const uint8_t *p, uint32_t bytes)
{
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)u),
               __builtin_amdgcn_readfirstlane((int)((uint32_t)(u >> 32) & 0xffff)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// 16 bytes of each lane, at lane_at of a buffer, to LDS address `to` + 16 * lane.  The
// scalar offset is 0: what the unit checks is the lane's offset against the size.  (A vector
// addition for each copy; buffers that begin at the stage instead, in scalar instructions, make
// the 128 x 128 tiles 12 % slower.)
// In assembly: told of copies into LDS, the compiler waits for those on their way
// before it reads LDS elsewhere, unless it can tell the places apart; here the
// callers wait.  (m0 is the compiler's, and kept.)  The descriptor may have come out of
// vector registers just before: a memory instruction reads such a scalar 5 wait
// states later at the earliest, which the compiler does not see to inside assembly.
__device__ __forceinline__ void copy16(v4i from, uint32_t lane_at, int to)
{
    int m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 2\n\t"
                 "buffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(lane_at), "s"(from)
                 : "memory");
}
// the same of 4 bytes, from an address of each lane
__device__ __forceinline__ void copy4(const void *from, int to)
{
    int m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from)
                 : "memory");
}

// ---------------------------------------------------------------------------
// A row's part of a stage in a lane: two pieces (32 bytes) of row l%16, the same
// two of weights and of tokens, so it does not matter which.
// ---------------------------------------------------------------------------
template <int MODE>
struct Frag {
    v8i v;
    __device__ __forceinline__ void set(v4i a, v4i b)
    {
        v = v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
};
template <>
struct Frag<F8X> {
    v8bf v[4];
    static __device__ __forceinline__ v8bf widen(int lo, int hi)
    {
        const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, 1.0f, false);
        const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, 1.0f, true);
        const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, 1.0f, false);
        const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, 1.0f, true);
        return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    __device__ __forceinline__ void set(v4i a, v4i b)
    {
        v[0] = widen(a[0], a[1]);
        v[1] = widen(a[2], a[3]);
        v[2] = widen(b[0], b[1]);
        v[3] = widen(b[2], b[3]);
    }
};

// result register i of lane l: channel 4*(l/16) + i, token l%16
template <int MODE>
__device__ __forceinline__ v4f stage_product(const Frag<MODE> &w, const Frag<MODE> &x, v4f c)
{
    if constexpr (MODE == F8) {
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, c, 0, 0, 0, 0, 0, 0);
    } else if constexpr (MODE == F8X) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[u], x.v[u], c, 0, 0, 0);
    } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const v4i a = {w.v[4 * u], w.v[4 * u + 1], w.v[4 * u + 2], w.v[4 * u + 3]};
            const v4i b = {x.v[4 * u], x.v[4 * u + 1], x.v[4 * u + 2], x.v[4 * u + 3]};
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c,
                                                        0, 0, 0);
        }
    }
    return c;
}
// acc += a stage's product, with its scale
template <int MODE>
__device__ __forceinline__ void add_stage(v4f &acc, const Frag<MODE> &w, const Frag<MODE> &x, float scale)
{
    if constexpr (MODE == BF16) {
        acc = stage_product<MODE>(w, x, acc);
    } else {
        const v4f p = stage_product<MODE>(w, x, v4f{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[i] = fmaf(p[i], scale, acc[i]);
    }
}

// ---------------------------------------------------------------------------
// Few rows: a stream of weights, bound by HBM.  A block owns 16*RT weight rows and up to 8*TC
// rows of x; its W waves take the stages in turn (a block reads W*128 neighbouring
// bytes of each row) and their sums are added through LDS, in the waves' order.  A
// wave works alone: it reads 8 rows x 128 bytes per load, neighbouring lanes on
// neighbouring bytes, passes them through LDS of its own into fragments and has
// the next stage's loads in flight meanwhile.  LDS rows are swizzled as in the
// tiles below.
// Scales: lane l loads those of token l%16 for the wave's stage l/16 of the next
// four, and the weights' for its next 64 stages, and passes them on when their
// stage comes.
// Bytes on their way are what counts: a row of 6144 x 6144 7.0 us (5.4 TB/s) with 8 waves
// of 16 rows, 24576 x 6144 23.1 (6.5); 16 tokens to 8 each of 256 experts of
// 4096 x 6144 (some 80 have rows) 281 to 297, by card.
// ---------------------------------------------------------------------------
template <int MODE, typename OT, bool GROUPED, bool NT, int RT, int TC, int W>
__global__ __launch_bounds__(64 * W, 2) void product_stream_kernel(ProdArgs a, int tiles_n)
{
    constexpr int TB = (TC + 1) / 2;                 // 16-token tiles
    constexpr int CW = 2 * RT, CP = CW + TC;         // 8-row pieces per stage: weights, all
    constexpr int ST = 1024 * (CW + 2 * TB);         // LDS bytes per wave
    constexpr bool SCALED = MODE != BF16;
    static_assert(RT * TB * 1024 <= ST, "a wave's sums fit its LDS");
    __shared__ __align__(128) uint8_t lds[W * ST];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Tile t;
    if constexpr (GROUPED) {
        if (!find_tile<8 * TC, 16 * RT>(a, tiles_n, lane, t))
            return;
    } else {
        t = Tile{(int)blockIdx.y * 8 * TC, 0, (int)blockIdx.x * 16 * RT, a.w, a.ws};
        t.rows = min(8 * TC, a.M - t.row0);
    }
    const int stages = a.K >> 7, blocks = (a.K + 127) >> 7;
    const int mine = (stages - wave + W - 1) / W;    // stages wave, wave + W, ...
    const uint8_t *src[CP];
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        const int r = 8 * (i < CW ? i : i - CW) + (lane >> 3);
        src[i] = (i < CW) ? t.w + (int64_t)min(t.n0 + r, a.N - 1) * a.ldw
                          : a.x + source_row<GROUPED>(a, t.row0 + min(r, t.rows - 1)) * a.ldx;
        src[i] += 16 * (lane & 7) + 128 * wave;
    }
    const float *s_row[TB], *ws_row[RT];
    if constexpr (SCALED) {
#pragma unroll
        for (int j = 0; j < TB; ++j)
            s_row[j] = a.s + source_row<GROUPED>(a, t.row0 + min(16 * j + (lane & 15), t.rows - 1)) * a.lds;
#pragma unroll
        for (int i = 0; i < RT; ++i)
            ws_row[i] = t.ws + (int64_t)(min(t.n0 + 16 * i, a.N - 1) >> 7) * a.ldws;
    }
    float s4[TB], s4_next[TB], ws64[RT];
    auto load_s = [&](int i, float (&to)[TB]) {      // of the wave's stages i .. i+3
#pragma unroll
        for (int j = 0; j < TB; ++j)
            to[j] = s_row[j][min(wave + W * (i + (lane >> 4)), blocks - 1)];
    };
    auto load_ws = [&](int i) {                      // of the wave's stages i .. i+63
#pragma unroll
        for (int k = 0; k < RT; ++k)
            ws64[k] = ws_row[k][min(wave + W * (i + lane), blocks - 1)];
    };
    uint8_t *slot = lds + wave * ST;
    int put[2], at[2];                               // of a piece's even and odd 8 rows; of half u
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        put[u] = 128 * (lane >> 3) + 16 * ((lane & 7) ^ (4 * u + (lane >> 4)));
        at[u] = 128 * (lane & 15) + 16 * ((4 * u + (lane >> 4)) ^ ((lane >> 1) & 7));
    }
    v4f acc[RT][TB];
    v4i reg[CP];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
            acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            reg[i] = (NT && i < CW) ? load_piece_stream(src[i]) : load_piece(src[i]);
            src[i] += 128 * W;
        }
    };
    Frag<MODE> wf[RT], xf[TB];
    // the wave's stage i has its fragments; scales from s4, ws64
    auto multiply = [&](int i) {
        float s[TB], ws[RT];
        if constexpr (SCALED) {
#pragma unroll
            for (int j = 0; j < TB; ++j)
                s[j] = __shfl(s4[j], 16 * (i & 3) + (lane & 15), 64);
#pragma unroll
            for (int k = 0; k < RT; ++k)
                ws[k] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ws64[k]), i & 63));
        }
#pragma unroll
        for (int k = 0; k < RT; ++k)
#pragma unroll
            for (int j = 0; j < TB; ++j)
                add_stage<MODE>(acc[k][j], wf[k], xf[j], SCALED ? s[j] * ws[k] : 1.0f);
    };
    if constexpr (SCALED) {
        load_s(0, s4);
        load_ws(0);
    }
    if (mine > 0)
        fetch();
    for (int i = 0; i < mine; ++i) {
#pragma unroll
        for (int c = 0; c < CP; ++c)
            *reinterpret_cast<v4i *>(slot + 1024 * c + put[c & 1]) = reg[c];
        if (i + 1 < mine)
            fetch();
        if (SCALED && (i & 3) == 0)
            load_s(i + 4, s4_next);
        wave_lds_sync();
#pragma unroll
        for (int k = 0; k < RT; ++k)
            wf[k].set(*reinterpret_cast<const v4i *>(slot + at[0] + 2048 * k),
                      *reinterpret_cast<const v4i *>(slot + at[1] + 2048 * k));
#pragma unroll
        for (int j = 0; j < TB; ++j)
            xf[j].set(*reinterpret_cast<const v4i *>(slot + at[0] + 1024 * CW + 2048 * j),
                      *reinterpret_cast<const v4i *>(slot + at[1] + 1024 * CW + 2048 * j));
        wave_lds_sync();
        multiply(i);
        if (SCALED && (i & 3) == 3) {
#pragma unroll
            for (int j = 0; j < TB; ++j)
                s4[j] = s4_next[j];
            if ((i & 63) == 63)
                load_ws(i + 1);
        }
    }
    if ((a.K & 127) && wave == stages % W) {         // the partial last stage: this wave's stage `mine`
        const int k = stages << 7;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const uint8_t *row = t.w + (int64_t)min(t.n0 + 16 * i + (lane & 15), a.N - 1) * a.ldw;
            wf[i].set(load_piece_end(row, k + 16 * (lane >> 4), a.K), load_piece_end(row, k + 64 + 16 * (lane >> 4), a.K));
        }
#pragma unroll
        for (int j = 0; j < TB; ++j) {
            const uint8_t *row = a.x + source_row<GROUPED>(a, t.row0 + min(16 * j + (lane & 15), t.rows - 1)) * a.ldx;
            xf[j].set(load_piece_end(row, k + 16 * (lane >> 4), a.K), load_piece_end(row, k + 64 + 16 * (lane >> 4), a.K));
        }
        multiply(mine);
    }
    v4f *part = reinterpret_cast<v4f *>(slot);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
            part[(i * TB + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int f = (int)threadIdx.x; f < RT * TB * 64; f += 64 * W) {
        const int l = f & 63, ij = f >> 6;
        v4f sum = reinterpret_cast<const v4f *>(lds)[f];
#pragma unroll
        for (int w = 1; w < W; ++w)
            sum += reinterpret_cast<const v4f *>(lds + w * ST)[f];
        const int n = t.n0 + 16 * (ij / TB) + 4 * (l >> 4), c = 16 * (ij % TB) + (l & 15);
        if (c < t.rows) {
            OT *o = static_cast<OT *>(a.out) + (int64_t)(t.row0 + c) * a.ldo + n;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N)
                    store1(o + i, a.bias ? sum[i] + a.bias[n + i] : sum[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Tiles: a block computes BT = 16*WT*FT rows x BN = 16*WN*FN channels with WT*WN
// waves of FT*FN 16x16 results (the rows' tiles go to the WT in turn), K in stages
// of 128 bytes through NB LDS buffers, the next stages' rows on their way while one
// is multiplied.
// An LDS row is 128 bytes, eight pieces; piece c of row r sits at slot
// c ^ (r/2 & 7): two rows fill the 64 banks once, so that 16 neighbouring rows'
// reads of one piece fall on different banks.
// DMA: rows go global -> LDS by the load unit (a wave's copy is 8 rows, lane l
// writing slot l%8 of row l/8, so the lane picks the global piece that belongs
// there); needs rows on 4 bytes, not too far apart.  Otherwise they pass through
// registers.
// Scales: the weights' of all stages lie in LDS from the beginning, the rows'
// come four stages at a time (16 bytes of a row of scales; one by one they would
// be a line each) into one of two places while the other is read.
// A partial last stage comes by the same copies and is cleared in LDS past the rows'
// end before it is read: 333 x 5003 x 2000 11.0 us, x 2048 11.2.
//
// Measured, in us, for bf16 outputs (F8; tiles of rows x channels; 70 shapes are in
// profiles/e4m3_product_kernels.csv):
//                        64x64  64x128  128x128  128x256  256x256
//     64 x  6144 x 6144   21.8    23.1     26.6     41.3     63.3   (streams: 11.9)
//    333 x  5003 x 2048   11.5    11.2     12.5     18.4     28.2
//    128 x 24576 x 6144   44.2    36.1     30.2     42.9     65.4
//    600 x  8192 x 4096   44.0    37.9     38.7     31.3     46.6
//   4096 x 24576 x 6144   1184     919      810      620      518
// and for fp32 outputs (F8X):
//     64 x  6144 x 6144   28.4    37.6     52.7     79.2            (streams: 14.2)
//    333 x  5003 x 2048   17.6    17.9     22.9     32.3
//    512 x  6144 x 6144   58.6    59.9     54.9     81.3
//    600 x  8192 x 4096   67.7    64.7     76.5     58.9
//   4096 x 12288 x 6144    803     691      671      527
// 518 us are 2390 TFLOP/s, the unit 59 % busy at the 1.9 GHz that the card holds under
// it: without the copies 17 % less, without the scaling 11 %, without the stores 7 %.
// The small tiles wait: a stage of the 64 x 64 ones takes 0.45 us, with one wave on a SIMD
// that reads its fragments from LDS one step ahead of their products.  Of F8X's 17.6 us at
// 333 x 5003 x 2048 the widening, done by each wave for its own fragments, is some 7
// (16 stages, two waves on a SIMD, 64 conversions of 7 cycles each); widened once into LDS,
// the reads of twice the bytes would take as long.
// ---------------------------------------------------------------------------
constexpr int MAX_BLOCKS = 1024;                     // blocks of 128 codes in a row

// lambdas that hold a kernel's registers
#define INLINE __attribute__((always_inline))

// f(0), ..., f(N-1) with constants
template <int N, int I = 0, typename F>
__device__ __forceinline__ void steps_of(F &&f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        steps_of<N, I + 1>(f);
    }
}

template <int MODE, int NB, int WT, int WN, int FT, int FN>
struct TileShape {
    static constexpr bool SCALED = MODE != BF16;
    static constexpr int NW = WT * WN, BT = 16 * WT * FT, BN = 16 * WN * FN;
    static constexpr int CP = (BT + BN) / 8 / NW;    // 8-row copies per wave and stage
    static constexpr int TP = BT / 8 / NW;           // of these, rows of x
    static constexpr int BUF = (BT + BN) * 128;      // bytes of a stage
    static constexpr int WB = BN > 128 ? BN / 128 : 1;   // blocks of 128 channels
    static constexpr int SROWS = BT < 64 ? 64 : BT;  // rows of scales in LDS
    static constexpr int WSCALE = NB * BUF, TSCALE = WSCALE + (SCALED ? 4 * (WB * MAX_BLOCKS + 4) : 0);
    static constexpr int LDS = TSCALE + (SCALED ? 2 * 16 * SROWS : 0);
    static_assert(BT % (8 * NW) == 0 && BN % (8 * NW) == 0 && NW % 2 == 0, "whole copies per wave");
    static_assert(16 * FN <= 128 && SROWS <= 64 * NW, "a wave's channels share a scale");
    static_assert(NB >= 2 && LDS <= 160 * 1024, "the stages fit");
};

template <int MODE, typename OT, bool GROUPED, bool DMA, int NB, int WT, int WN, int FT, int FN>
__device__ __forceinline__ void tile_product(const ProdArgs &a, const Tile &t, uint8_t *lds)
{
    typedef TileShape<MODE, NB, WT, WN, FT, FN> S;
    constexpr bool SCALED = S::SCALED;
    constexpr int NW = S::NW, BT = S::BT, CP = S::CP, TP = S::TP, BUF = S::BUF, SROWS = S::SROWS;
    const float *wscale = reinterpret_cast<const float *>(lds + S::WSCALE);
    const float *tscale = reinterpret_cast<const float *>(lds + S::TSCALE);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lds0 = (int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    const int stages = (a.K + 127) >> 7;             // the last may be partial
    const bool gathered = GROUPED && a.rows;

    // copies
    const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));   // NW is even
    auto row_of = [&](int i) INLINE {                // the row of copy i, before this lane's piece
        const int r = 8 * (wave + NW * (i < TP ? i : i - TP)) + (lane >> 3);
        return i < TP ? a.x + source_row<GROUPED>(a, t.row0 + min(r, t.rows - 1)) * a.ldx
                      : t.w + (int64_t)min(t.n0 + r, a.N - 1) * a.ldw;
    };
    auto lds_at = [&](int i) INLINE { return (i < TP ? 0 : BT * 128) + 1024 * (wave + NW * (i < TP ? i : i - TP)); };
    const uint8_t *x0 = uniform(gathered ? a.x : a.x + (int64_t)t.row0 * a.ldx);
    const uint8_t *w0 = uniform(t.w + (int64_t)t.n0 * a.ldw);
    // the ends of the last rows, past which copies bring zeros, on whole words (a word is
    // read as 0 unless all of it is inside)
    const uint32_t x_end = ((uint32_t)(((gathered ? a.R : t.rows) - 1) * a.ldx + a.K) + 3) & ~3u;
    const uint32_t w_end = ((uint32_t)((min(S::BN, a.N - t.n0) - 1) * a.ldw + a.K) + 3) & ~3u;
    uint32_t lane_at[DMA ? CP : 1];                  // this lane's piece of each copy
    const uint8_t *src[DMA ? 1 : CP];
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        if constexpr (DMA)
            lane_at[i] = (uint32_t)(row_of(i) + 16 * piece - (i < TP ? x0 : w0));
        else
            src[i] = row_of(i) + 16 * piece;
    }
    v4i reg[DMA ? 1 : CP];
    auto fetch = [&](int i, int buf, int st) INLINE {    // sets out copy i of stage st
        if constexpr (DMA) {                         // zeros past the last stage: nothing is read
            copy16(buffer_of(i < TP ? x0 : w0, window_bytes(i < TP ? x_end : w_end, 128 * st, a.K)),
                   lane_at[i] + 128 * (uint32_t)st, lds0 + buf + lds_at(i));
        } else if ((a.K & 127) && st >= stages - 1) {
            reg[i] = load_piece_end(src[i] - 16 * piece, 128 * (stages - 1) + 16 * piece, a.K);
        } else {
            reg[i] = load_piece(src[i] + 128 * min(st, stages - 1));
        }
    };
    auto land = [&](int buf) INLINE {
        if constexpr (!DMA) {
#pragma unroll
            for (int i = 0; i < CP; ++i)
                *reinterpret_cast<v4i *>(lds + buf + lds_at(i) + 16 * lane) = reg[i];
        }
    };
    // a row's partial last stage has, past the row's end, what lies behind it: zeros take its place
    auto clean = [&](int buf) INLINE {
        const int kept = a.K & 127, np = 8 - (kept >> 4);
        for (int f = tid; f < (BT + S::BN) * np; f += 64 * NW) {
            const int row = f / np, c = (kept >> 4) + f - row * np;
            v4i *at = reinterpret_cast<v4i *>(lds + buf + 128 * row + 16 * (c ^ ((row >> 1) & 7)));
            unsigned __int128 v = 0;
            if (16 * c < kept)
                v = __builtin_bit_cast(unsigned __int128, *at) & (((unsigned __int128)1 << (8 * (kept & 15))) - 1);
            *at = __builtin_bit_cast(v4i, v);
        }
    };

    // scales: a quad is those of four stages, in LDS as [row][4]
    const uint8_t *s_first = nullptr;
    uint32_t s_end = 0, s_lane = 0;
    if constexpr (SCALED) {
        s_first = uniform(gathered ? a.s : a.s + (int64_t)t.row0 * a.lds);
        const int r = min(64 * wave + lane, t.rows - 1);
        s_lane = (uint32_t)((gathered ? source_row<GROUPED>(a, t.row0 + r) : r) * a.lds * 4);
        // the last row's end: what a quad has past it reads as 0
        s_end = (uint32_t)(((int64_t)((gathered ? a.R : t.rows) - 1) * a.lds + stages) * 4);
        for (int i = wave; i < S::WB * ((stages + 63) >> 6); i += NW) {
            const int b = i % S::WB, k = i / S::WB * 64;
            const float *row = t.ws + (int64_t)(min(t.n0 + 128 * b, a.N - 1) >> 7) * a.ldws;
            copy4(row + min(k + lane, stages - 1), lds0 + S::WSCALE + 4 * (b * MAX_BLOCKS + k));
        }
    }
    auto bring = [&](int q) INLINE {                 // sets out a quad's copy
        if (SCALED && 64 * wave < BT && 4 * q < stages)
            copy16(buffer_of(s_first, window_bytes(s_end, 16 * q, 4 * stages)), s_lane + 16 * (uint32_t)q,
                   lds0 + S::TSCALE + 16 * (SROWS * (q & 1) + 64 * wave));
    };

    v4f acc[FT][FN];
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int wt = wave / WN, wn = wave % WN;
    int at[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
        at[u] = 128 * (lane & 15) + 16 * ((4 * u + (lane >> 4)) ^ ((lane >> 1) & 7));
    const int x_at = 2048 * wt, w_at = BT * 128 + 2048 * FN * wn;
    auto read_x = [&](Frag<MODE> &f, int buf, int i) INLINE {
        f.set(*reinterpret_cast<const v4i *>(lds + buf + at[0] + x_at + 2048 * WT * i),
              *reinterpret_cast<const v4i *>(lds + buf + at[1] + x_at + 2048 * WT * i));
    };
    auto read_w = [&](Frag<MODE> &f, int buf, int j) INLINE {
        f.set(*reinterpret_cast<const v4i *>(lds + buf + at[0] + w_at + 2048 * j),
              *reinterpret_cast<const v4i *>(lds + buf + at[1] + w_at + 2048 * j));
    };

    // A stage is FT steps, a step the products of one tile of rows with the FN of
    // channels.  x and its scales are read LA steps ahead, w in the stage's last step,
    // each in the place of the fragment that was just used; products are scaled and
    // added LAG products later.  Before step TURN, whose x is the next stage's, nothing
    // of this stage is left to be read but w: the waves meet, and stage st + AHEAD sets
    // out over it, a copy at a time between the products (all at once they fill the
    // load unit's queue, and what is behind them waits).
    constexpr int XR = FT % 4 == 0 ? 4 : FT % 3 == 0 ? 3 : 2, LA = XR - 1, TURN = FT - LA, LAG = 2, SLOTS = LA * FN;
    constexpr int AHEAD = DMA ? NB : 2;              // registers hold one stage
    static_assert(FT % XR == 0 && FT % 2 == 0 && FN % LAG == 0, "places change the same way in each stage");
    Frag<MODE> wf[FN], xf[XR];
    v4f p[LAG];                                      // products not yet added
    float sv[XR], sc[2] = {0.0f, 0.0f};              // scales of rows; of this step and the one before
    float ws = 1.0f, ws_next = 1.0f;
    int s_at = 0;                                    // of the stage and this lane's rows, in tscale
#pragma unroll
    for (int j = 0; j < LAG; ++j)
        p[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto read_s = [&](int i) INLINE {
        if constexpr (SCALED)
            sv[i % XR] = tscale[s_at + 64 * WT * i];
    };
    auto scales_of = [&](int st) INLINE {
        if constexpr (SCALED) {
            ws_next = wscale[(16 * FN * wn >> 7) * MAX_BLOCKS + st];
            s_at = ((st >> 2) & 1) * 4 * SROWS + (st & 3) + 4 * (16 * wt + (lane & 15));
        }
    };
    // this wave's copies have landed but for those of the LEFT stages set out
    // last, and its reads are done; then every wave's.  (Where rows pass through
    // registers, loads stay on their way.)
    auto meet = [&](auto left_) INLINE {
        constexpr int LEFT = decltype(left_)::value * CP;
        static_assert(LEFT < 64, "vmcnt counts to 63");
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(DMA ? 0x0070 | (LEFT & 15) | (LEFT >> 4) << 14    // vmcnt(LEFT) lgkmcnt(0)
                                       : 0xc07f);                                    // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // the product LAG before product m of a stage
    auto add = [&](auto m_, float now, float before) INLINE {
        if constexpr (SCALED) {
            constexpr int m = decltype(m_)::value, of = (m - LAG + FT * FN) % (FT * FN), i = of / FN, j = of % FN;
            const float s = (i == m / FN) ? now : before;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][j][e] = fmaf(p[m % LAG][e], s, acc[i][j][e]);
            // here, and not where the compiler would sink it to: before the next stage's
            asm volatile("" : "+v"(acc[i][j]));
        }
    };
    auto meet_clean = [&](int buf) INLINE {
        clean(buf);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xc07f);          // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // stage st, whose rows are in cur
    auto run_stage = [&](int cur, int next, int st) INLINE {
        ws = ws_next;
        steps_of<FT>([&](auto i_) INLINE {
            constexpr int i = decltype(i_)::value;
            sc[i & 1] = sv[i % XR] * ws;
            if constexpr (i == TURN) {
                land(next);
                meet(std::integral_constant<int, NB - 2>());
                if (DMA && (a.K & 127) && st + 2 == stages)
                    meet_clean(next);
                if (SCALED && (st & 3) == 3)         // its quad's place is free
                    bring((st >> 2) + 2);
                scales_of(st + 1);
            }
            if constexpr (i < TURN) {
                read_x(xf[(i + LA) % XR], cur, i + LA);
                read_s(i + LA);
            } else {
                read_x(xf[(i + LA) % XR], next, i + LA - FT);
                read_s(i + LA - FT);
            }
            steps_of<FN>([&](auto j_) INLINE {
                constexpr int j = decltype(j_)::value, m = FN * i + j, slot = m - FN * TURN;
                if constexpr (SCALED) {
                    add(std::integral_constant<int, m>(), sc[i & 1], sc[1 - (i & 1)]);
                    p[m % LAG] = stage_product<MODE>(wf[j], xf[i % XR], v4f{0.0f, 0.0f, 0.0f, 0.0f});
                } else {
                    acc[i][j] = stage_product<MODE>(wf[j], xf[i % XR], acc[i][j]);
                }
                if constexpr (i >= TURN) {
#pragma unroll
                    for (int c = slot * CP / SLOTS; c < (slot + 1) * CP / SLOTS; ++c)
                        fetch(c, cur, st + AHEAD);
                    if constexpr (i == FT - 1)
                        read_w(wf[j], next, j);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        });
    };
    auto begin = [&](int buf, int st) INLINE {
        scales_of(st);
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            read_x(xf[i], buf, i);
            read_s(i);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j)
            read_w(wf[j], buf, j);
    };
    bring(0);
    bring(1);
#pragma unroll
    for (int b = 0; b < AHEAD; ++b) {
#pragma unroll
        for (int i = 0; i < CP; ++i)
            fetch(i, b * BUF, b);
        if (b == 0)
            land(0);
    }
    meet(std::integral_constant<int, NB - 1>());
    if (DMA && a.K < 128)
        meet_clean(0);
    begin(0, 0);
    int cur = 0;
    for (int st = 0; st < stages; ++st) {
        const int next = (cur == (NB - 1) * BUF) ? 0 : cur + BUF;
        run_stage(cur, next, st);
        cur = next;
    }
    steps_of<LAG>([&](auto j_) INLINE { add(j_, 0.0f, sc[(FT - 1) & 1]); });
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);                   // copies past the end are still to land
    __syncthreads();

    // Epilogue: a wave passes 16 rows x 16*FN channels at a time through LDS of its
    // own and writes them as 16 bytes per lane, whole rows of the wave's channels.
    constexpr int PITCH = 16 * FN * (int)sizeof(OT) + 16;
    constexpr int LPR = FN * (int)sizeof(OT);        // lanes (16 bytes each) per row
    constexpr int VE = 16 / (int)sizeof(OT);         // values per lane
    static_assert(16 * PITCH * NW <= NB * BUF, "the waves' parts fit the buffers");
    const int nw0 = t.n0 + 16 * FN * wn;
    uint8_t *mine = lds + wave * 16 * PITCH;
    float bias[FN][4];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            bias[j][e] = a.bias ? a.bias[min(nw0 + 16 * j + 4 * (lane >> 4) + e, a.N - 1)] : 0.0f;
#pragma unroll
    for (int i = 0; i < FT; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            v4f y = acc[i][j];
            if (a.bias) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] += bias[j][e];
            }
            uint8_t *p = mine + (lane & 15) * PITCH + (16 * j + 4 * (lane >> 4)) * (int)sizeof(OT);
            if constexpr (sizeof(OT) == 2)
                *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
            else
                *reinterpret_cast<v4f *>(p) = y;
        }
        wave_lds_sync();
#pragma unroll
        for (int h = 0; h < (16 * LPR + 63) / 64; ++h) {
            const int f = 64 * h + lane, row = f / LPR, col = (f % LPR) * VE;
            const int r = 16 * (WT * i + wt) + row, n = nw0 + col;
            if (row < 16 && r < t.rows) {
                const uint4 v = *reinterpret_cast<const uint4 *>(mine + row * PITCH + col * (int)sizeof(OT));
                OT *o = static_cast<OT *>(a.out) + (int64_t)(t.row0 + r) * a.ldo + n;
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

template <int MODE, typename OT, bool GROUPED, bool DMA, int NB, int WT, int WN, int FT, int FN>
__global__ __launch_bounds__(64 * WT * WN, 2) void product_tiles_kernel(ProdArgs a, int tiles_t, int tiles_n)
{
    typedef TileShape<MODE, NB, WT, WN, FT, FN> S;
    __shared__ __align__(128) uint8_t lds[S::LDS];
    Tile t;
    if constexpr (GROUPED) {
        if (!find_tile<S::BT, S::BN>(a, tiles_n, threadIdx.x & 63, t))
            return;
    } else {
        // tiles in groups of 8 row tiles, row tile fastest, each XCD (blocks with
        // the same index mod 8) a contiguous run of them
        const int per = gridDim.x >> 3, logical = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
        if (logical >= tiles_t * tiles_n)
            return;
        const int band = logical / (8 * tiles_n), in = logical - band * 8 * tiles_n;
        const int gt = min(8, tiles_t - 8 * band);
        t = Tile{(8 * band + in % gt) * S::BT, 0, (in / gt) * S::BN, a.w, a.ws};
        t.rows = min(S::BT, a.M - t.row0);
    }
    tile_product<MODE, OT, GROUPED, DMA, NB, WT, WN, FT, FN>(a, t, lds);
}

// The rows of a group, up to 256 at a time, as a tile of as many as there are: 64, 128,
// 192 or 256 x 256 channels, so that weights are read once for up to 256 rows and few rows
// cost few products.  Against tiles of one shape (64x128 / 128x256 / these, us):
//   1024 tokens x 8 of 256 experts of 4096 x 6144   1185 / 1160 / 1135  (HBM, 5.6 TB/s)
//   4096 x 8 of 256                                  1931 / 1605 / 1560
//   4096 x 8 of  64 of 2048 x 2048                    273 /  199 /  176
// 4096 x 8 of 256 is 1020 us of products (27 % of them for rows that only fill up tiles) and
// 1030 of weights, overlapped in part: 1165 with all weights in L2.  On their way are two stages
// (up to 96 KB) in tiles of 64 and 128 rows, one (56 and 64 KB) in those of 192 and 256, whose
// third buffer has no room in LDS.
template <int MODE, typename OT, bool DMA>
__global__ __launch_bounds__(512, 2) void product_groups_kernel(ProdArgs a, int tiles_n)
{
    __shared__ __align__(128) uint8_t lds[TileShape<MODE, 3, 2, 4, 4, 4>::LDS];
    static_assert(TileShape<MODE, 2, 2, 4, 8, 4>::LDS <= sizeof(lds) && TileShape<MODE, 2, 2, 4, 6, 4>::LDS <= sizeof(lds) &&
                  TileShape<MODE, 3, 2, 4, 2, 4>::LDS <= sizeof(lds), "every shape fits");
    Tile t;
    if (!find_tile<256, 256>(a, tiles_n, threadIdx.x & 63, t))
        return;
    if (t.rows <= 64)
        tile_product<MODE, OT, true, DMA, 3, 2, 4, 2, 4>(a, t, lds);
    else if (t.rows <= 128)
        tile_product<MODE, OT, true, DMA, 3, 2, 4, 4, 4>(a, t, lds);
    else if (t.rows <= 192)
        tile_product<MODE, OT, true, DMA, 2, 2, 4, 6, 4>(a, t, lds);
    else
        tile_product<MODE, OT, true, DMA, 2, 2, 4, 8, 4>(a, t, lds);
}

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------
// row tiles of bt rows: exact, or an upper bound for groups of unknown sizes
static int64_t row_tiles(const ProdArgs &a, bool grouped, int bt)
{
    if (!grouped)
        return ceil_div(a.M, bt);
    const int64_t e = a.E < a.M ? a.E : a.M;
    return (a.M - e) / bt + e;
}

template <int MODE, typename OT, bool GROUPED, bool NT, int RT, int TC, int W>
static void launch_stream(const ProdArgs &a, hipStream_t st)
{
    const int tn = (int)ceil_div(a.N, 16 * RT);
    const int64_t tt = row_tiles(a, GROUPED, 8 * TC);
    const dim3 grid = GROUPED ? dim3((unsigned)ceil_div(tt * tn, 8) * 8) : dim3((unsigned)tn, (unsigned)tt);
    launch(product_stream_kernel<MODE, OT, GROUPED, NT, RT, TC, W>, grid, 64 * W, 0, st, a, tn);
}

template <int MODE, typename OT, bool GROUPED, bool DMA, int NB, int WT, int WN, int FT, int FN>
static void launch_tiles(const ProdArgs &a, hipStream_t st)
{
    const int tn = (int)ceil_div(a.N, 16 * WN * FN);
    const int64_t tt = row_tiles(a, GROUPED, 16 * WT * FT);
    launch(product_tiles_kernel<MODE, OT, GROUPED, DMA, NB, WT, WN, FT, FN>, (unsigned)ceil_div(tt * tn, 8) * 8,
           64 * WT * WN, 0, st, a, (int)tt, tn);
}

template <int MODE, typename OT, bool DMA>
static void launch_groups(const ProdArgs &a, hipStream_t st)
{
    const int tn = (int)ceil_div(a.N, 256);
    const int64_t tt = row_tiles(a, true, 256);
    launch(product_groups_kernel<MODE, OT, DMA>, (unsigned)ceil_div(tt * tn, 8) * 8, 512, 0, st, a, tn);
}

// products_choice.h's rule with these launches
template <typename OT, bool GROUPED>
struct Launches {
    const ProdArgs &a;
    hipStream_t st;
    template <int MODE, bool NT, int RT, int TC, int W>
    void stream()
    {
        launch_stream<MODE, OT, GROUPED, NT, RT, TC, W>(a, st);
    }
    template <int MODE, bool DMA, int NB, int WT, int WN, int FT, int FN>
    void tiles()
    {
        launch_tiles<MODE, OT, GROUPED, DMA, NB, WT, WN, FT, FN>(a, st);
    }
    template <int MODE, bool DMA>
    void groups()
    {
        launch_groups<MODE, OT, DMA>(a, st);
    }
};

template <int MODE, int TILE_MODE, typename OT, bool GROUPED>
static void enqueue(const ProdArgs &a, hipStream_t st)
{
    const ProductSizes sizes{a.M, a.N, a.K, a.E, copies_rows(a.x, a.w, a.ldx, a.ldw, a.w_stride, a.rows ? a.R : 0)};
    Launches<OT, GROUPED> launch{a, st};
    if constexpr (GROUPED)
        choose_grouped<MODE, TILE_MODE>(sizes, launch);
    else
        choose_dense<MODE, TILE_MODE>(sizes, launch);
}

static moe_status check_product(int32_t N, int32_t n_max, int32_t K, int32_t out_dtype)
{
    if (N < 1 || N > n_max)
        return fail(MOE_E_INVAL, "N=%d must be in [1, %d]", N, n_max);
    if (K < 1 || K > 128 * MAX_BLOCKS)
        return fail(MOE_E_INVAL, "K=%d must be in [1, 2^17]", K);
    if (!ops_dtype_ok(out_dtype))
        return fail(MOE_E_INVAL, "unknown out_dtype %d", out_dtype);
    return MOE_OK;
}

static moe_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? MOE_OK : hip_fail(e, what);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_linear_fp8(const void *q, int64_t ldq, const float *s, int64_t lds, int32_t T,
                                     const void *w, int64_t ldw, const float *ws, int64_t ldws,
                                     const float *bias, int32_t N, int32_t K, void *out,
                                     int32_t out_dtype, int64_t ldo, void *stream)
{
    if (T < 0 || T > (1 << 20))
        return fail(MOE_E_INVAL, "T=%d out of range [0, 2^20]", T);
    moe_status st = check_product(N, 1 << 20, K, out_dtype);
    if (st)
        return st;
    if ((int64_t)T * N > (1ll << 35))                // the launch's limit on threads
        return fail(MOE_E_INVAL, "T*N=%lld above 2^35", (long long)T * N);
    if (T == 0)
        return MOE_OK;
    if (!q || !s || !w || !ws || !out)
        return fail(MOE_E_INVAL, "q/s/w/ws/out is NULL");
    const int64_t blocks = (K + 127) / 128;
    if (ldq < K || ldw < K || ldo < N || lds < blocks || ldws < blocks)
        return fail(MOE_E_INVAL, "a leading dimension is below its row's length");
    if (lds > (1 << 21))                             // a tile's scales are within 2^31 bytes
        return fail(MOE_E_INVAL, "lds=%lld above 2^21", (long long)lds);
    if (!ops_aligned(s, 4) || !ops_aligned(ws, 4) || !ops_aligned(bias, 4) ||
        !ops_aligned(out, out_dtype == MOE_DT_F32 ? 4 : 2))
        return fail(MOE_E_INVAL, "s, ws, bias and out must be aligned to their elements");
    if ((st = ops_check_device()) != MOE_OK)
        return st;
    const ProdArgs a{static_cast<const uint8_t *>(q), static_cast<const uint8_t *>(w), s, ws, bias, out,
                     nullptr, nullptr, ldq, ldw, 0, lds, ldws, 0, ldo, T, T, N, 1, K};
    if (out_dtype == MOE_DT_F32)
        enqueue<F8X, F8X, float, false>(a, static_cast<hipStream_t>(stream));
    else
        enqueue<F8X, F8, bf16_t, false>(a, static_cast<hipStream_t>(stream));
    return launched("E4M3 product launch");
}

extern "C" moe_status moe_grouped_linear(const void *x, int32_t x_dtype, int64_t ldx, const float *s,
                                         int64_t lds, int32_t R, const int32_t *rows,
                                         const int32_t *offsets, int32_t E, int32_t M, const void *w,
                                         int64_t ldw, int64_t w_stride, const float *ws, int64_t ldws,
                                         int64_t ws_stride, int32_t N, int32_t K, void *out,
                                         int32_t out_dtype, int64_t ldo, void *stream)
{
    if (x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_FP8)
        return fail(MOE_E_INVAL, "x_dtype=%d must be MOE_DT_BF16 or MOE_DT_FP8", x_dtype);
    if (E < 1 || E > 1024)
        return fail(MOE_E_INVAL, "E=%d must be in [1, 1024]", E);
    if (M < 0 || M > (1 << 25))
        return fail(MOE_E_INVAL, "M=%d out of range [0, 2^25]", M);
    moe_status st = check_product(N, 1 << 17, K, out_dtype);
    if (st)
        return st;
    if ((int64_t)M * N > (1ll << 33))                // the launch's limit on threads
        return fail(MOE_E_INVAL, "M*N=%lld above 2^33", (long long)M * N);
    if (M == 0)
        return MOE_OK;
    const bool f8 = x_dtype == MOE_DT_FP8;
    if (R < 1 || (!rows && R < M))
        return fail(MOE_E_INVAL, "x has R=%d rows, M=%d are wanted", R, M);
    if (!x || !offsets || !w || !out || (f8 && (!s || !ws)))
        return fail(MOE_E_INVAL, "x/s/offsets/w/ws/out is NULL");
    const int64_t blocks = (K + 127) / 128, nblocks = (N + 127) / 128;
    if (ldx < K || ldw < K || ldo < N || (f8 && (lds < blocks || ldws < blocks)))
        return fail(MOE_E_INVAL, "a leading dimension is below its row's length");
    if (f8 && (lds > (rows ? (1 << 29) / R : 1 << 21)))   // a tile's scales are within 2^31 bytes
        return fail(MOE_E_INVAL, "lds=%lld too large", (long long)lds);
    if (E > 1 && (w_stride < (int64_t)(N - 1) * ldw + K || (f8 && ws_stride < (nblocks - 1) * ldws + blocks)))
        return fail(MOE_E_INVAL, "w_stride or ws_stride is below an expert's size");
    if (!ops_aligned(rows, 4) || !ops_aligned(offsets, 4) || (f8 && (!ops_aligned(s, 4) || !ops_aligned(ws, 4))) ||
        (!f8 && (!ops_aligned(x, 2) || !ops_aligned(w, 2))) || !ops_aligned(out, out_dtype == MOE_DT_F32 ? 4 : 2))
        return fail(MOE_E_INVAL, "pointers must be aligned to their elements");
    if ((st = ops_check_device()) != MOE_OK)
        return st;
    const int64_t b = f8 ? 1 : 2;
    const ProdArgs a{static_cast<const uint8_t *>(x), static_cast<const uint8_t *>(w), s, ws, nullptr, out,
                     rows, offsets, ldx * b, ldw * b, w_stride * b, lds, ldws, ws_stride, ldo, R, M, N, E,
                     (int)(K * b)};
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (f8 && out_dtype == MOE_DT_F32)
        enqueue<F8X, F8X, float, true>(a, hs);
    else if (f8)
        enqueue<F8X, F8, bf16_t, true>(a, hs);
    else if (out_dtype == MOE_DT_F32)
        enqueue<BF16, BF16, float, true>(a, hs);
    else
        enqueue<BF16, BF16, bf16_t, true>(a, hs);
    return launched("grouped product launch");
}
