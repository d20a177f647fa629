// The kernel of the tiled products of 8-bit tensors for more than a few rows (fp8.hip holds the layout, the rounding and
// the products for few rows; fp8_gemm.hip and fp8_gated.hip choose the tiles): y = act(A W^T + bias + residual), the gated
// pair act(A G^T) (A U^T) to the type or to 8-bit codes, and the pair's gradient dG = dy (A U^T) act'(A G^T), dU = dy
// act(A G^T).
//
// A workgroup computes a BM x BN tile in steps of one 128-column panel; in the gated forms the BN weight rows are BN / 2
// of each weight, so a lane holds both projections of its outputs and they meet in registers.  A step's operands, BM +
// BN rows of 128 code bytes and a word with the scales of four panels, are contiguous runs that DMA brings into a ring
// of ST stages.  LDS rows of 128 bytes hold 16-byte chunk q at slot q ^ (row / 2 % 8): a ds_read_b128 serves lanes
// {0-7, 24-31}, {8-15, 16-23} (and the same in the upper half) one group a cycle, and the lanes of a fragment read the
// same chunk of 32 rows, so every group reaches 16 distinct 16-byte slots of two rows.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes row l % 32 and half of the instruction's 64 columns from lane l; which half's
// bytes they are is the same on both sides and a block's 128 columns have one scale, so a lane reads two neighbouring
// chunks.  It multiplies by the blocks' powers of two itself: no scaling, and no second accumulator, in the loop.
//
// What that instruction keeps (measured): of every eight products that it adds at a time, each is cut off below 2^-13 of
// the largest; the sums of these are held in 32 bits.  On normally distributed values that is 1.5e-5 of a result (2-norm),
// whatever k, a hundredth of a rounding to bfloat16 and a fourteenth of one to float16, and at most 7 2^-13 of the sum of
// the terms' magnitudes.  Results of 16 and 8 bits are computed so.  Float32 results are not (WIDE; nor are codes of up to
// 16 rows, fp8.hip): their operands are widened to bfloat16, exactly (fp8_widen says where), between LDS and the matrix
// units, which then add products of full precision at half the rate (1.7 POP/s against 3.4 in a loop of the instruction
// alone).
//
// A step's second half is read while its first half multiplies, the next step's first half while the second multiplies,
// across the one barrier of the step; stage s + ST is requested once stage s is read.
//
// What bounds it: 8192 x 8192 x 8192 in 256 x 256 tiles takes 405 to 415 us, 2.7 POP/s, at a clock that power holds near
// 1.6 GHz.  A workgroup takes 4.5 k cycles until its first panel, 142 k for 64 steps (92 % of them the matrix units' own)
// and 10 k to store the tile; at k = 2048 the first and the last are a third of its time (2.3 POP/s).
#pragma once

#include <type_traits>

#include "device_common.h"
#include "ifx_internal.h"
#include "lowp.h"

namespace ifx {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v8i join(v4i lo, v4i hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_;
    static constexpr int W = WM * WN, T = 64 * W;
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
    static constexpr int CODES = (BM + BN) * 128;
    static constexpr int STAGE = CODES + (BM + BN) * 4;
    static constexpr int CA = BM / 8 / W, CB = BN / 8 / W;  // 1 KB DMAs of A's and of W's codes per wave and stage
    static constexpr int SC = (BM + BN) / 64;               // 256-byte scale DMAs per stage
    static constexpr int SPW = (SC + W - 1) / W;            // of them per wave (the last ones may repeat others')
    static constexpr int LPS = CA + CB + SPW;               // DMAs per wave and stage
    static constexpr int ROW = TN * 4 + 32;       // bytes of a wave's staged output row: 4 rows apart, half the banks on
    static constexpr int ROW8 = BN * 2 + 32;      // the same of a workgroup's row of BN / 2 values
    static constexpr int OUT = 32 * (ROW * W > ROW8 * WM ? ROW * W : ROW8 * WM);
    static constexpr int LDS = ST * STAGE > OUT ? ST * STAGE : OUT;
    static constexpr int PER_CU = kLdsBytes / LDS < 2048 / T ? kLdsBytes / LDS : 2048 / T;
    static_assert(CA * 8 * W == BM && CB * 8 * W == BN && CA % 2 == 0 && CB % 2 == 0, "whole DMAs, their swizzles in turn");
    static_assert(STAGE % 256 == 0, "the swizzle counts from a stage's start");
    static_assert((ST - 1) * LPS < 64, "requests that a wait can count");
};

// Waits until at most `later` stages of N requests each are in flight.
template <int MOST, int N>
__device__ __forceinline__ void wait_later(int later)
{
    if constexpr (MOST > 0) {
        if (later >= MOST)
            wait_vmcnt<MOST * N>();
        else
            wait_later<MOST - 1, N>(later);
    } else {
        wait_vmcnt<0>();
    }
}

// How results leave the tile.
enum Form { kFormProduct, kFormGated, kFormGated8, kFormGrad };

template <typename C, int FORM, int TYPE, int AF>
__global__ __launch_bounds__(C::T, waves_per_simd(C::T, C::PER_CU > 2 ? 2 : C::PER_CU)) void fp8_tile_kernel(
    Fp8Args a, int tiles_m, int tiles_n, int per_xcd)
{
    typedef typename Elem<TYPE>::type E;
    constexpr bool TWO = FORM != kFormProduct, WIDE = TYPE == 0 && FORM != kFormGated8;
    constexpr int NB = TWO ? C::BN / 2 : C::BN;  // output columns of the tile
    __shared__ __attribute__((aligned(1024))) int8_t smem[C::LDS];
    // XCD x (blockIdx & 7) owns a run of tiles, in bands of four tile rows, columns outermost, so the
    // workgroups of an XCD share their operands in its L2
    const int id = (int)(blockIdx.x & 7u) * per_xcd + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per_xcd || id >= tiles_m * tiles_n) return;
    const int band = id / (4 * tiles_n), in_band = id - band * 4 * tiles_n;
    const int bh = min(4, tiles_m - 4 * band);
    const int tn = in_band / bh, tm = 4 * band + in_band - tn * bh;
    const int m0 = tm * C::BM, n0 = tn * NB;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), l = threadIdx.x & 63;
    const int wm = w / C::WN, wn = w - wm * C::WN;
    const int c = l & 31, g = l >> 5;

    // This wave's DMAs of a step: CA and CB kilobytes of codes, eight rows each, SPW times 64 rows' scale words.
    // Rows past a tensor's end lie past a resource's range and read as zeros; their scales are the last row's.
    const int a_rows = min(C::BM, a.m - m0), w_rows = min(NB, a.n - n0);
    const int a_at = w * C::CA * 1024, w_at = w * C::CB * 1024;
    const bool of_up = TWO && w_at >= NB * 128;
    const int w_first = of_up ? w_at - NB * 128 : w_at;  // from its weight's first row
    const uint8_t *a_src = a.a_codes + (long long)m0 * 128 + a_at;
    const uint8_t *w_src = (of_up ? a.u_codes : a.w_codes) + (long long)n0 * 128 + w_first;
    const long long a_step = (long long)a.m * 128, w_step = (long long)a.n * 128;
    const unsigned even_off = (unsigned)((l >> 3) * 128 + (((l & 7) ^ (l >> 4)) * 16)), odd_off = even_off ^ 64u;
    const uint8_t *s_src[C::SPW];
    unsigned s_pitch[C::SPW];
#pragma unroll
    for (int i = 0; i < C::SPW; ++i) {
        const int t = (w * C::SPW + i) % C::SC * 64 + l, tb = t - C::BM;
        const bool of_a = t < C::BM, up = TWO && tb >= NB;
        const int row = of_a ? m0 + min(t, a_rows - 1) : n0 + min(up ? tb - NB : tb, w_rows - 1);
        s_src[i] = (of_a ? a.a_scales : up ? a.u_scales : a.w_scales) + (long long)row * 4;
        s_pitch[i] = (unsigned)(of_a ? a.m : a.n);
    }
    typedef __attribute__((address_space(3))) void *Lds;
    typedef const __attribute__((address_space(1))) void *Global;

    // DMA j of this wave's LPS for step s
    auto issue1 = [&](int s, auto jj) __attribute__((always_inline)) {
        constexpr int j = decltype(jj)::value;
        int8_t *st = smem + (s % C::ST) * C::STAGE;
        // the instruction's offset counts in memory and in LDS alike, up to 4095
        if constexpr (j < C::CA) {
            constexpr int far = j / 4 * 4096;
            ifx_raw_buffer_load_lds(make_rsrc(a_src + s * a_step + far, (long long)a_rows * 128 - a_at - far),
                                    (Lds)(st + a_at + far), 16, j % 2 ? odd_off : even_off, 0, j % 4 * 1024, 0);
        } else if constexpr (j < C::CA + C::CB) {
            constexpr int i = j - C::CA, far = i / 4 * 4096;
            ifx_raw_buffer_load_lds(make_rsrc(w_src + s * w_step + far, (long long)w_rows * 128 - w_first - far),
                                    (Lds)(st + C::BM * 128 + w_at + far), 16, i % 2 ? odd_off : even_off, 0, i % 4 * 1024, 0);
        } else {
            constexpr int i = j - C::CA - C::CB;
            __builtin_amdgcn_global_load_lds((Global)(s_src[i] + (long long)(s >> 2) * s_pitch[i] * 4),
                                             (Lds)(st + C::CODES + (w * C::SPW + i) % C::SC * 256), 4, 0, 0);
        }
    };
    auto issue_some = [&](int s, auto after, auto upto) __attribute__((always_inline)) {
        auto one = [&](auto j) __attribute__((always_inline)) { issue1(s, j); };
        each_from<decltype(after)::value, decltype(upto)::value>(one);
    };
    auto issue = [&](int s) __attribute__((always_inline)) { issue_some(s, Int<0>(), Int<C::LPS>()); };

    const int k1 = a.k1;
#pragma unroll
    for (int s = 0; s < C::ST; ++s)
        if (s < k1) issue(s);

    v16f acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = (v16f){};

    // rows of the wave's fragments: of the gated forms' FN / 2 columns of fragments are each weight's
    const int q00 = ((2 * g) ^ (c >> 1 & 7)) * 16;
    const int a_row = (wm * C::TM + c) * 128, b_row = (C::BM + wn * (TWO ? C::TN / 2 : C::TN) + c) * 128;
    const int a_sc = C::CODES + (wm * C::TM + c) * 4, b_sc = C::CODES + (C::BM + wn * (TWO ? C::TN / 2 : C::TN) + c) * 4;
    constexpr int MF = C::FM * C::FN;
    auto b_frag = [](int j) __attribute__((always_inline)) {
        return TWO && j >= C::FN / 2 ? NB + (j - C::FN / 2) * 32 : j * 32;
    };
    // A half step's fragments: A's and the last of W's twice, for this half and the next one; W's others once, each
    // read anew behind its last matrix instruction (a second copy would not fit beside 128 accumulators).
    v4i af[2][C::FM][2], bf[C::FN - 1 > 0 ? C::FN - 1 : 1][2], bl[2][2];
    int as[C::FM], bs[C::FN];
    auto read_a = [&](auto half, const int8_t *st, int t) __attribute__((always_inline)) {
        constexpr int HALF = decltype(half)::value;
        const int i = t / 2, h = t % 2;
        af[HALF][i][h] = *(const v4i *)(st + a_row + i * 4096 + (q00 ^ (HALF * 64) ^ (h * 16)));
        if (!HALF && h == 0) as[i] = *(const int *)(st + a_sc + i * 128);
    };
    auto read_b = [&](auto half, const int8_t *st, int j) __attribute__((always_inline)) {
        constexpr int HALF = decltype(half)::value;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            (j == C::FN - 1 ? bl[HALF] : bf[j])[h] = *(const v4i *)(st + b_row + b_frag(j) * 128 + (q00 ^ (HALF * 64) ^ (h * 16)));
        if (!HALF) bs[j] = *(const int *)(st + b_sc + b_frag(j) * 4);
    };

    wait_later<C::ST - 1, C::LPS>(min(C::ST - 1, k1 - 1));
    ring_barrier();
#pragma unroll
    for (int t = 0; t < 2 * C::FM; ++t) read_a(Slot0(), smem, t);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) read_b(Slot0(), smem, j);
    int slot = 0;
    int sa[C::FM], sb[C::FN];
    // The matrix instructions of one half, and between them the reads of the next half (of stage nst, where there
    // is one) and a share of the requests for stage `ahead`.  Reads and requests go out one by one: issued together
    // they would hold up both waves of a SIMD at once.
    auto half_step = [&](auto half, auto further, const int8_t *nst, int ahead) __attribute__((always_inline)) {
        constexpr int H = decltype(half)::value;
        constexpr bool MORE = decltype(further)::value > 0, STEADY = decltype(further)::value > 1;
        typedef Int<1 - H> Next;
        constexpr int RA = (2 * C::FM + C::FN - 1) / C::FN;  // of A's reads, beside each column of fragments
        lowp_v8b aw[WIDE ? C::FM : 1][4], bw[4];
        each(Int<MF>(), [&](auto tt) __attribute__((always_inline)) {
            constexpr int t = decltype(tt)::value, j = t / C::FM, i = t % C::FM;
            const v4i *b = j == C::FN - 1 ? bl[H] : bf[j];
            if constexpr (WIDE) {
                if (j == 0) fp8_widen<AF>(af[H][i][0], af[H][i][1], sa[i], aw[i]);
                if (i == 0) fp8_widen<0>(b[0], b[1], sb[j], bw);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(aw[i][q], bw[q], acc[i][j], 0, 0, 0);
            } else {
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(af[H][i][0], af[H][i][1]), join(b[0], b[1]),
                                                                            acc[i][j], AF, 0, 0, sa[i], 0, sb[j]);
            }
            if constexpr (MORE) {
                if (i == 0) {
                    if (j == 0) read_b(Next(), nst, C::FN - 1);
#pragma unroll
                    for (int u = j * RA; u < (j + 1) * RA && u < 2 * C::FM; ++u) read_a(Next(), nst, u);
                }
                if (i == C::FM - 1 && j < C::FN - 1) read_b(Next(), nst, j);
            }
            if constexpr (STEADY) issue_some(ahead, Int<t * C::LPS / MF>(), Int<(t + 1) * C::LPS / MF>());
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // one step; further: 2 with a stage to request, 1 with one more to multiply, 0 the last
    auto step = [&](auto further, int s) __attribute__((always_inline)) {
        constexpr int FURTHER = decltype(further)::value;
        const int8_t *st = smem + slot * C::STAGE;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) sa[i] = (int)((unsigned)as[i] >> (8 * (s & 3)));
#pragma unroll
        for (int j = 0; j < C::FN; ++j) sb[j] = (int)((unsigned)bs[j] >> (8 * (s & 3)));
        __builtin_amdgcn_s_setprio(1);
        half_step(Slot0(), Slot1(), st, 0);
        __builtin_amdgcn_s_setprio(0);
        slot = slot + 1 == C::ST ? 0 : slot + 1;
        if constexpr (FURTHER > 0) {
            if constexpr (FURTHER > 1)
                wait_vmcnt<(C::ST - 2) * C::LPS>();
            else
                wait_later<C::ST - 2, C::LPS>(min(C::ST - 2, k1 - 2 - s));
            lds_barrier();  // the reads of stage s are complete, stage s + 1 has landed
        }
        half_step(Slot1(), further, smem + slot * C::STAGE, s + C::ST);
    };
    int s = 0;
    for (; s + C::ST < k1; ++s) step(Slot2(), s);
    for (; s + 1 < k1; ++s) step(Slot1(), s);
    step(Slot0(), s);

    // Epilogue, 32 rows of the wave's tile at a time: the accumulators (lane l: column l % 32, rows
    // 8 (i / 4) + 4 (l / 32) + i % 4) go through LDS into rows, so operands and results move several columns a lane in
    // whole rows.
    lds_barrier();
    // the lane anew: values kept from before the loop would cost registers in it
    int el = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(el));
    const auto value_row = [&](int e) __attribute__((always_inline)) { return 8 * (e / 4) + 4 * (el >> 5) + e % 4; };
    // act(gate) times the other projection, fragment jj of FN / 2
    const auto combine = [&](auto act, int i, int jj, int e) __attribute__((always_inline)) {
        return act_of<decltype(act)::value>(acc[i][jj][e]) * acc[i][jj + C::FN / 2][e];
    };

    if constexpr (FORM == kFormGated8) {
        // the waves of a tile row stage 32 rows of NB = 128 values together; sixteen lanes round a row
        static_assert(C::WN <= 2 || C::TM == 32 * C::FM, "");
        int8_t *out = smem + wm * 32 * C::ROW8;
        constexpr int ROWS = 32 / C::WN;  // that a wave rounds
        const int n1 = (a.n + 127) / 128, panel = n0 / 128;
        with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                if (i > 0) lds_barrier();
#pragma unroll
                for (int jj = 0; jj < C::FN / 2; ++jj)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        *(float *)(out + value_row(e) * C::ROW8 + (wn * C::TN / 2 + jj * 32 + (el & 31)) * 4) = combine(act, i, jj, e);
                lds_barrier();
#pragma unroll
                for (int p = 0; p < ROWS / 4; ++p) {
                    const int r = wn * ROWS + p * 4 + (el >> 4), v = el & 15;
                    const int8_t *src = out + r * C::ROW8 + v * 32;
                    const v4f lo = *(const v4f *)src, hi = *(const v4f *)(src + 16);
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = lo[e], f[4 + e] = hi[e];
                    // (columns past n are zero weights: their values are zero, or a NaN of the row's own)
                    const int left = a.n - n0 - v * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e >= left) f[e] = 0.0f;
                    const unsigned sc = fp8_scale<0>(row_max(top_bits(f)));
                    const uint2 q = fp8_codes<0>(f, sc);
                    const int row = m0 + wm * C::TM + i * 32 + r;
                    if (row < a.m) {
                        ((uint2 *)a.codes)[((long long)panel * a.m + row) * 16 + v] = q;
                        if (v == 0) {
                            uint8_t *at = a.scales + ((long long)(panel >> 2) * a.m + row) * 4;
                            at[panel & 3] = (uint8_t)sc;
                            if (panel == n1 - 1)  // the word's other bytes
                                for (int b = (panel & 3) + 1; b < 4; ++b) at[b] = 0;
                        }
                    }
                }
            }
        });
    } else {
        constexpr int TO = TWO ? C::TN / 2 : C::TN;  // columns of the wave's results
        int8_t *out = smem + w * 32 * C::ROW;
        constexpr int LPR = TO / 4, RPP = 64 / LPR, P = 32 / RPP;  // lanes per row, rows per pass, passes
        // the wave's first row and column, the lane's place in a pass
        const int r0 = m0 + wm * C::TM, c0 = n0 + wn * TO, lr = el / LPR, lc = el % LPR * 4;
        const int8_t *const src = out + lr * C::ROW + lc * 4;
        const int col = c0 + lc, left = a.n - col;
        float bias[4] = {};
        if constexpr (!TWO) {
#pragma unroll
            for (int e = 0; e < 4; ++e) bias[e] = a.bias && left >= 4 ? a.bias[col + e] : 0.0f;
        }
        // 32 rows of accumulators staged
        auto stage = [&](auto act, int i) __attribute__((always_inline)) {
            if constexpr (FORM == kFormGated) {
#pragma unroll
                for (int jj = 0; jj < C::FN / 2; ++jj)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        *(float *)(out + value_row(e) * C::ROW + (jj * 32 + (el & 31)) * 4) = combine(act, i, jj, e);
            } else {
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) *(float *)(out + value_row(e) * C::ROW + (j * 32 + (el & 31)) * 4) = acc[i][j][e];
            }
            wave_lds_sync();
        };
        // One result (of the gradient the first of two, `second` the other) from the staged value, the other
        // projection's and the operand that is read beside them.
        const auto first = [](auto act, float v, float u, float r) __attribute__((always_inline)) {
            constexpr int ACT = decltype(act)::value;
            return FORM == kFormProduct ? act_of<ACT>(v + r) : FORM == kFormGated ? v : r * u * act_slope<ACT>(v);
        };
        const auto second = [](auto act, float v, float r) __attribute__((always_inline)) {
            return r * act_of<decltype(act)::value>(v);
        };
        typedef unsigned QuadWords __attribute__((ext_vector_type(sizeof(E)), aligned(sizeof(E))));
        // A tile that lies whole in the result: addresses are a uniform base and the lane's offset, nothing is
        // predicated.  RES: an operand is read.  (Eight columns a lane, 16-byte accesses, and all operands requested at
        // once measured the same.)
        auto whole = [&](auto act, auto res_tag, auto past) __attribute__((always_inline)) {
            constexpr bool RES = decltype(res_tag)::value;
            const unsigned off = (unsigned)((lr * (int)a.ld_y + lc) * (int)sizeof(E));
            const unsigned off2 = FORM == kFormGrad ? (unsigned)((lr * (int)a.ld_y2 + lc) * (int)sizeof(E)) : 0u;
            const unsigned off_r = RES ? (unsigned)((lr * (int)a.ld_res + lc) * (int)sizeof(E)) : 0u;
            // the passes' uniform bases, on by RPP rows each time
            const auto base_of = [&](const void *p, long long ld) __attribute__((always_inline)) {
                return (char *)p + (r0 * ld + c0) * (long long)sizeof(E);
            };
            const long long step_y = RPP * a.ld_y * (long long)sizeof(E), step_y2 = RPP * a.ld_y2 * (long long)sizeof(E);
            const long long step_r = RPP * a.ld_res * (long long)sizeof(E);
            char *y = base_of(a.y, a.ld_y), *y2 = FORM == kFormGrad ? base_of(a.y2, a.ld_y2) : nullptr;
            const char *r_at = RES ? base_of(a.res, a.ld_res) : nullptr;
            const auto put = [&](char *&base, long long step, unsigned o, const float (&f)[4]) __attribute__((always_inline)) {
                QuadWords v;
                if constexpr (sizeof(E) == 4) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(f[e]);
                } else {
                    v[0] = pack2<E>(f[0], f[1]);
                    v[1] = pack2<E>(f[2], f[3]);
                }
                if constexpr (decltype(past)::value) {
                    __builtin_nontemporal_store(v, (QuadWords *)(base + o));
                    keep_apart();
                } else {
                    *(QuadWords *)(base + o) = v;
                }
                base += step;
            };
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                Quad<E> res[P];
                if constexpr (RES) {  // requested before the rows are staged
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        res[p] = *(const Quad<E> *)(r_at + off_r);
                        r_at += step_r;
                    }
                }
                stage(act, i);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const v4f f = *(const v4f *)(src + p * RPP * C::ROW);
                    v4f u = {};
                    if constexpr (FORM == kFormGrad) u = *(const v4f *)(src + p * RPP * C::ROW + TO * 4);
                    float q[4], q2[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float r = RES ? (float)res[p].v[e] : 0.0f, v = FORM == kFormProduct ? f[e] + bias[e] : f[e];
                        q[e] = RES || FORM != kFormProduct ? first(act, v, u[e], r) : act_of<decltype(act)::value>(v);
                        if constexpr (FORM == kFormGrad) q2[e] = second(act, v, r);
                    }
                    put(y, step_y, off, q);
                    if constexpr (FORM == kFormGrad) put(y2, step_y2, off2, q2);
                }
                wave_lds_sync();
            }
        };
        // A tile that ends inside: rows predicated by lane, the last one to three columns value by value.
        auto ragged = [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                if (r0 + i * 32 >= a.m) break;
                const long long row0 = r0 + i * 32 + lr;
                Quad<E> res[P];
                if (a.res) {
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        if (left >= 4 && row0 + p * RPP < a.m) res[p] = *(const Quad<E> *)((const E *)a.res + (row0 + p * RPP) * a.ld_res + col);
                }
                stage(act, i);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    if (left < 4 || row0 + p * RPP >= a.m) continue;
                    const v4f f = *(const v4f *)(src + p * RPP * C::ROW);
                    v4f u = {};
                    if constexpr (FORM == kFormGrad) u = *(const v4f *)(src + p * RPP * C::ROW + TO * 4);
                    Quad<E> q, q2;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float r = a.res ? (float)res[p].v[e] : 0.0f, v = FORM == kFormProduct ? f[e] + bias[e] : f[e];
                        q.v[e] = (E)first(act, v, u[e], r);
                        if constexpr (FORM == kFormGrad) q2.v[e] = (E)second(act, v, r);
                    }
                    *(Quad<E> *)((E *)a.y + (row0 + p * RPP) * a.ld_y + col) = q;
                    if constexpr (FORM == kFormGrad) *(Quad<E> *)((E *)a.y2 + (row0 + p * RPP) * a.ld_y2 + col) = q2;
                }
                if (left > 0 && left < 4) {
#pragma unroll 1
                    for (int k = 0; k < P * left; ++k) {
                        const int p = k / left, e = k - p * left;
                        const long long row = row0 + p * RPP;
                        if (row >= a.m) break;
                        float v = *(const float *)(src + p * RPP * C::ROW + e * 4), u = 0.0f, r = 0.0f;
                        if constexpr (FORM == kFormGrad) u = *(const float *)(src + p * RPP * C::ROW + TO * 4 + e * 4);
                        if constexpr (!TWO)
                            if (a.bias) v += a.bias[col + e];
                        if (a.res) r = (float)((const E *)a.res)[row * a.ld_res + col + e];
                        ((E *)a.y)[row * a.ld_y + col + e] = (E)first(act, v, u, r);
                        if constexpr (FORM == kFormGrad) ((E *)a.y2)[row * a.ld_y2 + col + e] = (E)second(act, v, r);
                    }
                }
                wave_lds_sync();
            }
        };
        const long long most = 1LL << 24;  // pitches whose offsets within a pass fit 32 bits
        const bool inside = m0 + C::BM <= a.m && n0 + NB <= a.n && a.ld_y <= most && a.ld_y2 <= most && a.ld_res <= most;
        with_act(a.act, [&](auto act) __attribute__((always_inline)) {
            auto with_past = [&](auto res_tag) __attribute__((always_inline)) {
                if (a.past)
                    whole(act, res_tag, std::true_type());
                else
                    whole(act, res_tag, std::false_type());
            };
            if (!inside)
                ragged(act);
            else if (FORM == kFormGrad || (FORM == kFormProduct && a.res))
                with_past(std::integral_constant<bool, FORM != kFormGated>());
            else if constexpr (FORM != kFormGrad)
                with_past(std::false_type());
        });
    }
}

// Widened operands (float32 results) have no registers beside more than four accumulators of 32 x 32 a wave.
template <typename C, int FORM, int AF>
hipError_t launch_tile(const Fp8Args &a, hipStream_t s)
{
    constexpr int NB = FORM == kFormProduct ? C::BN : C::BN / 2;
    static_assert(FORM != kFormGated8 || NB == 128, "a block of the result a tile");
    const int tiles_m = (a.m - 1) / C::BM + 1, tiles_n = (a.n - 1) / NB + 1;
    const int per_xcd = (int)(((long long)tiles_m * tiles_n + 7) / 8);
    void (*f)(Fp8Args, int, int, int) = nullptr;
    if constexpr (FORM == kFormGated8) {
        f = fp8_tile_kernel<C, FORM, 0, AF>;
    } else {
        f = a.type == 1 ? fp8_tile_kernel<C, FORM, 1, AF> : fp8_tile_kernel<C, FORM, 2, AF>;
        if constexpr (C::FM * C::FN <= 4)
            if (a.type == 0) f = fp8_tile_kernel<C, FORM, 0, AF>;
    }
    hipLaunchKernelGGL(f, dim3((unsigned)per_xcd * 8u), dim3(C::T), 0, s, a, tiles_m, tiles_n, per_xcd);
    return hipGetLastError();
}

// Tiles of BM rows and `columns` columns of the result.
template <typename C>
long long tiles(const Fp8Args &a, int columns)
{
    return ((a.m - 1LL) / C::BM + 1) * ((a.n - 1LL) / columns + 1);
}

// TileX moves the fewest bytes to LDS a product and has a CU to itself; two workgroups of TileM fit one, or one of TileN,
// the same with a deeper ring.
typedef Tile<256, 256, 4, 2, 2> TileX;
typedef Tile<128, 128, 2, 2, 2> TileM;
typedef Tile<128, 128, 2, 2, 4> TileN;
typedef Tile<64, 128, 2, 2, 3> TileG;

// Of the two, the deeper ring while every workgroup has a CU to itself, as long as that fills most of the CUs (us, TileN /
// TileM): 2048 x 2048 x 8192 (256 tiles) 35.3 / 44.9, 2048^3 13.0 / 14.7; (TileN / TileG) 1500 x 2048 x 4096 (192) 19.6 /
// 21.4, 1024 x 2048 x 8192 (128) 29.0 / 23.6
template <int FORM, int AF>
bool launch_middle(const Fp8Args &a, int cus, hipStream_t s, hipError_t *e)
{
    const long long t = tiles<TileM>(a, FORM == kFormProduct ? 128 : 64);
    if (4 * t < 3LL * cus) return false;
    *e = t <= cus ? launch_tile<TileN, FORM, AF>(a, s) : launch_tile<TileM, FORM, AF>(a, s);
    return true;
}

}  // namespace
}  // namespace ifx
