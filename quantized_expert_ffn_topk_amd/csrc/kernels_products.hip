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
#include "ops_common.h"

namespace moe {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

enum { F8 = 0, F8X = 1, BF16 = 2 };

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
// 16 (4) bytes of each active lane from memory to LDS at 16 (4) times the lane
__device__ __forceinline__ void copy16(const void *from, void *to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}
__device__ __forceinline__ void copy4(const void *from, void *to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 4, 0, 0);
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
// Few rows: a stream of weights.  A block owns 16*RT weight rows and up to 8*TC
// rows of x; its W waves take the stages in turn (a block reads W*128 neighbouring
// bytes of each row) and their sums are added through LDS, in the waves' order.  A
// wave works alone: it reads 8 rows x 128 bytes per load, neighbouring lanes on
// neighbouring bytes, passes them through LDS of its own into fragments and has
// the next stage's loads in flight meanwhile.  LDS rows are swizzled as in the
// tiles below.
// Scales: lane l loads those of token l%16 for the wave's stage l/16 of the next
// four, and the weights' for its next 64 stages, and passes them on when their
// stage comes.
// ---------------------------------------------------------------------------
template <int MODE, typename OT, bool GROUPED, bool NT, int RT, int TC, int W>
__global__ __launch_bounds__(64 * W) void product_stream_kernel(ProdArgs a, int tiles_n)
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
// waves of FT*FN 16x16 results, K in stages of 128 bytes through NB LDS buffers,
// the next stages' rows on their way while one is multiplied.
// An LDS row is 128 bytes, eight pieces; piece c of row r sits at slot
// c ^ (r/2 & 7): two rows fill the 64 banks once, so that 16 neighbouring rows'
// reads of one piece fall on different banks.
// DMA: rows go global -> LDS by the load unit (a wave's copy is 8 rows, lane l
// writing slot l%8 of row l/8, so the lane picks the global piece that belongs
// there); needs rows of 16-byte alignment.  Otherwise they pass through
// registers.  The last, partial stage always does (load_piece_end's zeros).
// Scales: the weights' of all stages lie in LDS from the beginning, the rows'
// come four stages at a time (16 bytes of a row of scales; one by one they would
// be a line each), into one of two buffers while the other is read.
// ---------------------------------------------------------------------------
constexpr int MAX_BLOCKS = 1024;                     // blocks of 128 codes in a row

template <int MODE, typename OT, bool GROUPED, bool DMA, int NB, int WT, int WN, int FT, int FN>
__global__ __launch_bounds__(64 * WT * WN) void product_tiles_kernel(ProdArgs a, int tiles_t, int tiles_n)
{
    constexpr int NW = WT * WN, BT = 16 * WT * FT, BN = 16 * WN * FN;
    constexpr int CP = (BT + BN) / 8 / NW;           // 8-row copies per wave and stage
    constexpr int TP = BT / 8 / NW;                  // of these, rows of x
    constexpr int BUF = (BT + BN) * 128;             // bytes of a stage
    constexpr bool SCALED = MODE != BF16;
    constexpr int WB = BN > 128 ? BN / 128 : 1;      // blocks of 128 channels
    constexpr int TPW = BT / NW;                     // rows whose scales a wave brings
    static_assert(BT % (8 * NW) == 0 && BN % (8 * NW) == 0 && NW % 2 == 0, "whole copies per wave");
    static_assert(16 * FN <= 128 && TPW <= 64, "a wave's channels share a scale");
    static_assert(NB >= 2 && NB <= 4, "two to four buffers");
    // the buffers are objects of their own: the compiler then knows that reads
    // of one do not wait for copies into another
    __shared__ __align__(128) uint8_t buf0[BUF];
    __shared__ __align__(128) uint8_t buf1[BUF];
    __shared__ __align__(128) uint8_t buf2[NB > 2 ? BUF : 16];
    __shared__ __align__(128) uint8_t buf3[NB > 3 ? BUF : 16];
    __shared__ __align__(16) float wscale[SCALED ? WB * MAX_BLOCKS : 4];
    __shared__ __align__(16) float tscale0[SCALED ? 4 * BT : 4];
    __shared__ __align__(16) float tscale1[SCALED ? 4 * BT : 4];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Tile t;
    if constexpr (GROUPED) {
        if (!find_tile<BT, BN>(a, tiles_n, lane, t))
            return;
    } else {
        // tiles in groups of 8 row tiles, row tile fastest, each XCD (blocks with
        // the same index mod 8) a contiguous run of them
        const int per = gridDim.x >> 3, logical = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
        if (logical >= tiles_t * tiles_n)
            return;
        const int band = logical / (8 * tiles_n), in = logical - band * 8 * tiles_n;
        const int gt = min(8, tiles_t - 8 * band);
        t = Tile{(8 * band + in % gt) * BT, 0, (in / gt) * BN, a.w, a.ws};
        t.rows = min(BT, a.M - t.row0);
    }

    const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));   // NW is even
    const uint8_t *src[CP];                          // this lane's piece of each copy
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        const int r = 8 * (wave + NW * (i < TP ? i : i - TP)) + (lane >> 3);
        src[i] = (i < TP) ? a.x + source_row<GROUPED>(a, t.row0 + min(r, t.rows - 1)) * a.ldx
                          : t.w + (int64_t)min(t.n0 + r, a.N - 1) * a.ldw;
        src[i] += 16 * piece;
    }
    auto lds_at = [&](int i) { return (i < TP ? 0 : BT * 128) + 1024 * (wave + NW * (i < TP ? i : i - TP)); };
    const int stages = a.K >> 7, blocks = (a.K + 127) >> 7;

    // scales
    const float *s_row = nullptr;
    bool wide = false;                               // four scales of a row in one load
    if constexpr (SCALED) {
        s_row = a.s + source_row<GROUPED>(a, t.row0 + min(TPW * wave + min(lane, TPW - 1), t.rows - 1)) * a.lds;
        wide = (reinterpret_cast<uintptr_t>(a.s) & 15) == 0 && (a.lds & 3) == 0;
        for (int i = wave; i < WB * ((blocks + 63) >> 6); i += NW) {
            const int b = i % WB, k = i / WB * 64;
            const float *row = t.ws + (int64_t)(min(t.n0 + 128 * b, a.N - 1) >> 7) * a.ldws;
            copy4(row + min(k + lane, blocks - 1), wscale + b * MAX_BLOCKS + k);
        }
    }
    // the scales of stages 4*quad .. 4*quad+3: [row][4] where `wide` and all exist, else [4][row]
    auto quad_wide = [&](int quad) { return wide && 4 * quad + 4 <= blocks; };
    auto bring = [&](int quad) {
        if (4 * quad >= blocks || lane >= TPW)
            return;
        float *to = (quad & 1) ? tscale1 : tscale0;
        if (quad_wide(quad)) {
            copy16(s_row + 4 * quad, to + 4 * TPW * wave);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                copy4(s_row + min(4 * quad + c, blocks - 1), to + c * BT + TPW * wave);
        }
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
    const int x_at = 2048 * FT * wt, w_at = BT * 128 + 2048 * FN * wn;
    auto read_x = [&](Frag<MODE> &f, const uint8_t *buf, int i) {
        f.set(*reinterpret_cast<const v4i *>(buf + at[0] + x_at + 2048 * i),
              *reinterpret_cast<const v4i *>(buf + at[1] + x_at + 2048 * i));
    };
    auto read_w = [&](Frag<MODE> &f, const uint8_t *buf, int j) {
        f.set(*reinterpret_cast<const v4i *>(buf + at[0] + w_at + 2048 * j),
              *reinterpret_cast<const v4i *>(buf + at[1] + w_at + 2048 * j));
    };
    float sc[FT];
    auto read_scales = [&](int st) {                 // of stage st, for this lane's rows
        if constexpr (SCALED) {
            const float *q = ((st >> 2) & 1) ? tscale1 : tscale0;
            const bool w4 = quad_wide(st >> 2);
            const int step = w4 ? 4 : 1, first = w4 ? (st & 3) : (st & 3) * BT;
            const float ws = wscale[(16 * FN * wn >> 7) * MAX_BLOCKS + st];
#pragma unroll
            for (int i = 0; i < FT; ++i)
                sc[i] = q[first + step * (16 * (FT * wt + i) + (lane & 15))] * ws;
        }
    };

    v4i reg[DMA ? 1 : CP];
    auto fetch = [&](uint8_t *buf) {                 // sets out the next whole stage
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            if constexpr (DMA)
                copy16(src[i], buf + lds_at(i));
            else
                reg[i] = load_piece(src[i]);
            src[i] += 128;
        }
    };
    auto land = [&](uint8_t *buf) {
        if constexpr (!DMA) {
#pragma unroll
            for (int i = 0; i < CP; ++i)
                *reinterpret_cast<v4i *>(buf + lds_at(i) + 16 * lane) = reg[i];
        }
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
    const std::integral_constant<int, 0> all;
    Frag<MODE> wf[FN], xf[2];
    // a stage whose rows are in buf
    auto multiply_stage = [&](const uint8_t *buf, int st) {
        read_scales(st);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            read_w(wf[j], buf, j);
        read_x(xf[0], buf, 0);
#pragma unroll
        for (int i = 0; i < FT; ++i) {
            if (i + 1 < FT)
                read_x(xf[(i + 1) & 1], buf, i + 1);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                add_stage<MODE>(acc[i][j], wf[j], xf[i & 1], sc[i]);
        }
    };
    if constexpr (SCALED) {
        bring(0);
        bring(1);
    }
    auto buf = [&](int i) { return i == 0 ? buf0 : i == 1 ? buf1 : i == 2 ? buf2 : buf3; };
    if constexpr (DMA) {
#pragma unroll
        for (int i = 0; i < NB - 1; ++i)
            if (i < stages)
                fetch(buf(i));
        for (int st = 0; st < stages; st += NB) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                if (st + i >= stages)
                    break;
                // stage st+i has landed, and everyone is done with the stage before
                if (st + i + NB - 2 < stages)
                    meet(std::integral_constant<int, NB - 2>());
                else
                    meet(all);
                if (st + i + NB - 1 < stages)
                    fetch(buf((i + NB - 1) % NB));
                if (SCALED && ((st + i) & 3) == 0 && st + i > 0)
                    bring(((st + i) >> 2) + 1);
                multiply_stage(buf(i), st + i);
            }
        }
    } else {
        if (stages > 0)
            fetch(buf0);
        for (int st = 0; st < stages; ++st) {
            uint8_t *cur = (st & 1) ? buf1 : buf0;
            land(cur);
            if (st + 1 < stages)
                fetch(nullptr);
            __syncthreads();
            if (SCALED && (st & 3) == 0 && st > 0)
                bring((st >> 2) + 1);
            multiply_stage(cur, st);
        }
    }
    __syncthreads();
    if (a.K & 127) {
        const int k = 128 * stages + 16 * piece;     // src has come this far
#pragma unroll
        for (int i = 0; i < CP; ++i)
            *reinterpret_cast<v4i *>(buf0 + lds_at(i) + 16 * lane) = load_piece_end(src[i] - k, k, a.K);
        meet(all);
        multiply_stage(buf0, stages);
        __syncthreads();
    }

    // Epilogue: a wave passes 16 rows x 16*FN channels at a time through LDS of its
    // own and writes them as 16 bytes per lane, whole rows of the wave's channels.
    constexpr int PITCH = 16 * FN * (int)sizeof(OT) + 16;
    constexpr int LPR = FN * (int)sizeof(OT);        // lanes (16 bytes each) per row
    constexpr int VE = 16 / (int)sizeof(OT);         // values per lane
    static_assert(16 * PITCH * NW <= BUF, "the waves' parts fit a buffer");
    const int nw0 = t.n0 + 16 * FN * wn, tw0 = 16 * FT * wt;
    uint8_t *mine = buf0 + wave * 16 * PITCH;
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
            const int r = tw0 + 16 * i + row, n = nw0 + col;
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

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------


static int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

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

template <int MODE, typename OT, bool GROUPED, bool DMA>
static void enqueue_tiles(const ProdArgs &a, int64_t rows, hipStream_t st)
{
    launch_tiles<MODE, OT, GROUPED, DMA, DMA ? 4 : 2, 2, 2, 2, 2>(a, st);
}

// rows: of a group on average
template <int MODE, int TILE_MODE, typename OT, bool GROUPED>
static void enqueue_product(const ProdArgs &a, hipStream_t st)
{
    const int64_t rows = GROUPED ? ceil_div(a.M, a.E) : a.M;
    if (rows <= 8)
        launch_stream<MODE, OT, GROUPED, false, 2, 1, 4>(a, st);
    else if (rows <= 16)
        launch_stream<MODE, OT, GROUPED, false, 2, 2, 4>(a, st);
    else if (rows <= 32)
        launch_stream<MODE, OT, GROUPED, false, 2, 4, 4>(a, st);
    else if (ops_aligned(a.x, 16) && ops_aligned(a.w, 16) && a.ldx % 16 == 0 && a.ldw % 16 == 0 && a.w_stride % 16 == 0)
        enqueue_tiles<TILE_MODE, OT, GROUPED, true>(a, rows, st);
    else
        enqueue_tiles<TILE_MODE, OT, GROUPED, false>(a, rows, st);
}

// E4M3: fp32 outputs take exact products everywhere
template <bool GROUPED>
static void enqueue_f8(const ProdArgs &a, int32_t out_dtype, hipStream_t st)
{
    if (out_dtype == MOE_DT_F32)
        enqueue_product<F8X, F8X, float, GROUPED>(a, st);
    else
        enqueue_product<F8X, F8, bf16_t, GROUPED>(a, st);
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
    if (!ops_aligned(s, 4) || !ops_aligned(ws, 4) || !ops_aligned(bias, 4) ||
        !ops_aligned(out, out_dtype == MOE_DT_F32 ? 4 : 2))
        return fail(MOE_E_INVAL, "s, ws, bias and out must be aligned to their elements");
    if ((st = ops_check_device()) != MOE_OK)
        return st;
    const ProdArgs a{static_cast<const uint8_t *>(q), static_cast<const uint8_t *>(w), s, ws, bias, out,
                     nullptr, nullptr, ldq, ldw, 0, lds, ldws, 0, ldo, T, T, N, 1, K};
    enqueue_f8<false>(a, out_dtype, static_cast<hipStream_t>(stream));
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
    if (f8)
        enqueue_f8<true>(a, out_dtype, hs);
    else if (out_dtype == MOE_DT_F32)
        enqueue_product<BF16, BF16, float, true>(a, hs);
    else
        enqueue_product<BF16, BF16, bf16_t, true>(a, hs);
    return launched("grouped product launch");
}
