// The tiled product of two microscaled 4-bit tensors: y = act(A W^T + bias + residual) for more than
// a few rows (mx4.hip holds the layout, the rounding and the product for few rows).
//
// What bounds it: at large sizes the matrix units (v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 cycles
// a wave for 131072 operations; measured alone on operands that change: 6.5 POP/s at 2 waves per
// SIMD, the 16x16x128 form 5.7), at short sums (k of a few hundred) the output's bytes.  The matrix units'
// rate follows the chip's power: on zeros they reach 9.9 POP/s at 2.37 GHz, on changing codes 6.5 at 1.67 GHz,
// with this kernel's LDS reads beside them 5.9.  8192^3 to bf16 takes 250-261 us, 4.2-4.4 POP/s, at 1.6 GHz
// with the units busy about 60 % of the time; 4096 x 16384 x 16384 483 us, 4.6; 100352 x 128 x 512 15 us;
// 2048 x 1000 x 2048, launch and latency, 8.3.
//
// A workgroup computes a BM x BN tile in steps of one 128-column panel.  A step's operands, BM + BN
// rows of 64 code bytes and 4 scale bytes, are contiguous runs that buffer->LDS DMA brings into a ring of ST
// stages.  LDS rows of 64 bytes hold chunk (block) q at slot q ^ (row / 4 % 4): a ds_read_b128
// serves lanes {0-7, 24-31}, {8-15, 16-23} (and the same in the upper half) one group a cycle, and
// the fragment lane (c = l % 32, g = l / 32) reads block 2 ks + g of row c, so every group reaches 16
// distinct 16-byte slots.  One 32-bit word holds a row's four scales; a lane shifts its block's scale
// to the lowest byte, and the instruction's byte selector takes byte 0 (blocks 0, 1) or 2 (blocks 2, 3).
//
// A step's second half is read while its first half multiplies, the next step's first half while
// the second multiplies, across the one barrier of the step.
#include "device_common.h"
#include "ifx_internal.h"
#include "lowp.h"

namespace ifx {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kFp4 = 4;  // the matrix instruction's operand format: 4-bit e2m1

__device__ __forceinline__ v8i wide(v4i x) { return (v8i){x[0], x[1], x[2], x[3], 0, 0, 0, 0}; }

template <int N>
struct Int {
    static constexpr int value = N;
};

// f(Int<0>()) .. f(Int<N - 1>())
template <int I, int N, typename F>
__device__ __forceinline__ void each_from(F &f)
{
    if constexpr (I < N) {
        f(Int<I>());
        each_from<I + 1, N>(f);
    }
}
template <int N, typename F>
__device__ __forceinline__ void each(Int<N>, F f)
{
    each_from<0, N>(f);
}

// Four consecutive output values at any element boundary.
template <typename E>
struct Quad {
    E v[4];
};

template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_;
    static constexpr int W = WM * WN, T = 64 * W;
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
    static constexpr int CODES = (BM + BN) * 64;
    static constexpr int STAGE = CODES + (BM + BN) * 4;
    static constexpr int CA = BM / 16 / W, CB = BN / 16 / W;  // 1 KB DMAs of A's and of W's codes per wave and stage
    static constexpr int SC = (BM + BN) / 64;                 // 256-byte scale DMAs per stage
    static constexpr int SPW = (SC + W - 1) / W;              // of them per wave (the last waves may repeat others')
    static constexpr int LPS = CA + CB + SPW;                 // DMAs per wave and stage
    static constexpr int ROW = TN * 4 + 32;         // bytes of a staged output row: 4 rows apart, half the banks on
    static constexpr int OUT = 32 * ROW * W;
    // whether large results go past the caches: TileS gets small ones, and with a second copy of its epilogue
    // 2048 x 1000 x 2048 took 9.0 us instead of 8.8
    static constexpr bool PAST = BM * BN > 64 * 64 || ST == 2;
    static constexpr int LDS = ST * STAGE > OUT ? ST * STAGE : OUT;
    static constexpr int PER_CU = kLdsBytes / LDS < 2048 / T ? kLdsBytes / LDS : 2048 / T;
    static_assert(BM % (16 * W) == 0 && BN % (16 * W) == 0, "every wave brings as much of A and of W");
    static_assert(SC % SPW == 0 && BM / 64 % SPW == 0, "a wave's scale DMAs are all of A or all of W");
};

template <int N>
__device__ __forceinline__ void wait_later(int later)
{
    if (later >= 2)
        wait_vmcnt<2 * N>();
    else if (later == 1)
        wait_vmcnt<N>();
    else
        wait_vmcnt<0>();
}

template <typename C, int TYPE>
__global__ __launch_bounds__(C::T, waves_per_simd(C::T, C::PER_CU > 2 ? 2 : C::PER_CU)) void mx4_tile_kernel(
    Mx4Args a, int tiles_m, int tiles_n, int per_xcd)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ __attribute__((aligned(1024))) int8_t smem[C::LDS];
    // XCD x (blockIdx & 7) owns a run of tiles, in bands of four tile rows, columns outermost, so the
    // workgroups of an XCD share their operands in its L2
    const int id = (int)(blockIdx.x & 7u) * per_xcd + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per_xcd || id >= tiles_m * tiles_n) return;
    const int band = id / (4 * tiles_n), in_band = id - band * 4 * tiles_n;
    const int bh = min(4, tiles_m - 4 * band);
    const int tn = in_band / bh, tm = 4 * band + in_band - tn * bh;
    const int m0 = tm * C::BM, n0 = tn * C::BN;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), l = threadIdx.x & 63;
    const int wm = w / C::WN, wn = w - wm * C::WN;
    const int c = l & 31, g = l >> 5;

    // this wave's DMAs of a step: CA and CB kilobytes of codes, SPW times 64 rows of scales.  Rows past a
    // tensor's end lie past a resource's range and read as zeros.
    const long long a_rows = min(C::BM, a.m - m0), w_rows = min(C::BN, a.n - n0);
    const uint8_t *a_src = a.a_codes + (long long)m0 * 64, *w_src = a.w_codes + (long long)n0 * 64;
    const long long a_step = (long long)a.m * 64, w_step = (long long)a.n * 64;
    const int run = w * C::SPW % C::SC;
    const bool s_of_a = run < C::BM / 64;
    const uint8_t *s_src = s_of_a ? a.a_scales + (long long)m0 * 4 : a.w_scales + (long long)n0 * 4;
    const long long s_step = (s_of_a ? a_step : w_step) / 16, s_rows = s_of_a ? a_rows : w_rows;
    // One lane offset serves every code DMA: the wave's place goes into the resource's base, the DMA's into
    // the instruction's offset, which counts in memory and in LDS alike.
    const unsigned lane_off = (unsigned)((l >> 2) * 64 + (((l & 3) ^ (l >> 4)) * 16));
    const unsigned scale_off = (unsigned)((s_of_a ? run : run - C::BM / 64) * 256 + l * 4);
    static_assert(C::CA <= 4 && C::CB <= 4, "instruction offsets below 4096");

    // DMA j of this wave's LPS for step s
    auto issue1 = [&](int s, auto jj) __attribute__((always_inline)) {
        constexpr int j = decltype(jj)::value;
        int8_t *st = smem + (s % C::ST) * C::STAGE;
        typedef __attribute__((address_space(3))) void *Lds;
        if constexpr (j < C::CA) {
            const int at = w * C::CA * 1024;
            ifx_raw_buffer_load_lds(make_rsrc(a_src + s * a_step + at, a_rows * 64 - at), (Lds)(st + at), 16, lane_off, 0,
                                    j * 1024, 0);
        } else if constexpr (j < C::CA + C::CB) {
            const int at = w * C::CB * 1024;
            ifx_raw_buffer_load_lds(make_rsrc(w_src + s * w_step + at, w_rows * 64 - at), (Lds)(st + C::BM * 64 + at), 16,
                                    lane_off, 0, (j - C::CA) * 1024, 0);
        } else {
            constexpr int i = (j - C::CA - C::CB) * 256;
            ifx_raw_buffer_load_lds(make_rsrc(s_src + s * s_step, s_rows * 4), (Lds)(st + C::CODES + run * 256), 4, scale_off,
                                    0, i, 0);
        }
    };
    auto issue_some = [&](int s, auto after, auto upto) __attribute__((always_inline)) {
        auto one = [&](auto j) __attribute__((always_inline)) { issue1(s, j); };
        each_from<decltype(after)::value, decltype(upto)::value>(one);
    };
    auto issue = [&](int s) __attribute__((always_inline)) { issue_some(s, Int<0>(), Int<C::LPS>()); };

    const int k1 = a.k1;
#pragma unroll
    for (int s = 0; s < C::ST - 1; ++s)
        if (s < k1) issue(s);

    v16f acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = (v16f){};

    const int q0 = (g ^ ((c >> 2) & 3)) * 16, q1 = q0 ^ 32;  // slots of blocks g and 2 + g
    const int a_row = (wm * C::TM + c) * 64, b_row = C::BM * 64 + (wn * C::TN + c) * 64;
    const int a_sc = C::CODES + (wm * C::TM + c) * 4, b_sc = C::CODES + (C::BM + wn * C::TN + c) * 4;
    v4i a0[C::FM], b0[C::FN], a1[C::FM], b1[C::FN];
    int as[C::FM], bs[C::FN];
    // fragment t of a step's first (HALF 0, with its rows' scales) or second half
    constexpr int FR = C::FM + C::FN, MF = C::FM * C::FN;
    constexpr int RD = (2 * FR + MF - 1) / MF;  // reads after a matrix instruction: all in the half's first half
    auto read = [&](auto half, const int8_t *st, int t) __attribute__((always_inline)) {
        constexpr int HALF = decltype(half)::value;
        const int q = HALF ? q1 : q0;
        const bool of = t < C::FM;
        const int i = of ? t : t - C::FM;
        const v4i v = *(const v4i *)(st + (of ? a_row : b_row) + q + i * 2048);
        if (of)
            (HALF ? a1 : a0)[i] = v;
        else
            (HALF ? b1 : b0)[i] = v;
        if (!HALF) {
            const int sc = *(const int *)(st + (of ? a_sc : b_sc) + i * 128);
            if (of)
                as[i] = sc;
            else
                bs[i] = sc;
        }
    };

    wait_later<C::LPS>(min(C::ST - 2, k1 - 1));
    ring_barrier();
#pragma unroll
    for (int t = 0; t < FR; ++t) read(Slot0(), smem, t);
    int slot = 0;
    // one step; `steady`: a further stage is requested and ST - 2 later ones stay in flight.  Reads and
    // requests go out one by one between the matrix instructions: issued together they would hold up
    // both waves of a SIMD at once.
    auto step = [&](auto steady, int s) __attribute__((always_inline)) {
        constexpr bool STEADY = decltype(steady)::value != 0;
        const int8_t *st = smem + slot * C::STAGE;
        int sa[C::FM], sb[C::FN];
        __builtin_amdgcn_s_setprio(1);
        each(Int<MF>(), [&](auto tt) __attribute__((always_inline)) {
            constexpr int t = decltype(tt)::value, i = t / C::FN, j = t % C::FN;
            if (j == 0) sa[i] = (int)((unsigned)as[i] >> (8 * g));
            if (i == 0) sb[j] = (int)((unsigned)bs[j] >> (8 * g));
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(a0[i]), wide(b0[j]), acc[i][j], kFp4, kFp4, 0,
                                                                        sa[i], 0, sb[j]);
#pragma unroll
            for (int u = t * RD; u < (t + 1) * RD && u < FR; ++u) read(Slot1(), st, u);
            if (STEADY) issue_some(s + C::ST - 1, Int<t * C::LPS / MF>(), Int<(t + 1) * C::LPS / MF>());
            __builtin_amdgcn_sched_barrier(0);
        });
        __builtin_amdgcn_s_setprio(0);
        slot = slot + 1 == C::ST ? 0 : slot + 1;
        const bool more = STEADY || s + 1 < k1;
        if (more) {
            if (STEADY)
                wait_vmcnt<(C::ST - 2) * C::LPS>();
            else
                wait_later<C::LPS>(min(C::ST - 2, k1 - 2 - s));
            lds_barrier();  // the reads of stage s are complete, stage s + 1 has landed
        }
        const int8_t *next = smem + slot * C::STAGE;
#pragma unroll
        for (int t = 0; t < MF; ++t) {
            const int i = t / C::FN, j = t % C::FN;
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(a1[i]), wide(b1[j]), acc[i][j], kFp4, kFp4, 2,
                                                                        sa[i], 2, sb[j]);
            if (more)
#pragma unroll
                for (int u = t * RD; u < (t + 1) * RD && u < FR; ++u) read(Slot0(), next, u);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int s = 0;
    for (; s + C::ST - 1 < k1; ++s) step(Slot1(), s);
    for (; s < k1; ++s) step(Slot0(), s);

    // Epilogue, 32 rows of the wave's tile at a time: the accumulators (lane l: column l % 32, rows
    // 8 (i / 4) + 4 (l / 32) + i % 4) go through LDS into rows, so bias, residual and output move four
    // columns a lane in whole rows.  The rows' residual is requested before they are staged.
    lds_barrier();
    // the lane anew: values kept from before the loop would cost registers in it
    int el = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(el));
    int8_t *out = smem + w * 32 * C::ROW;
    constexpr int LPR = C::TN / 4, RPP = 64 / LPR, P = 32 / RPP;  // lanes per row, rows per pass, passes
    const int col = n0 + wn * C::TN + (el % LPR) * 4, left = a.n - col;
    const bool whole = left >= 4;  // all of the lane's columns exist
    float bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) bias[e] = a.bias && whole ? a.bias[col + e] : 0.0f;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
        const int r0 = m0 + wm * C::TM + i * 32;
        if (r0 >= a.m) break;
        const long long row0 = r0 + el / LPR;
        Quad<E> res[P];
        if (a.res) {
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (whole && row0 + p * RPP < a.m) res[p] = *(const Quad<E> *)((const E *)a.res + (row0 + p * RPP) * a.ld_res + col);
        }
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                *(float *)(out + (8 * (e / 4) + 4 * (el >> 5) + e % 4) * C::ROW + (j * 32 + (el & 31)) * 4) = acc[i][j][e];
        wave_lds_sync();
        with_act(a.act, [&](auto act) __attribute__((always_inline)) {
            constexpr int ACT = decltype(act)::value;
            auto rows = [&](auto past) __attribute__((always_inline)) {
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const v4f f = *(const v4f *)(out + (p * RPP + el / LPR) * C::ROW + (el % LPR) * 16);
                    Quad<E> q;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = f[e] + bias[e];
                        if (a.res) v += (float)res[p].v[e];
                        q.v[e] = (E)act_of<ACT>(v);
                    }
                    if (!whole || row0 + p * RPP >= a.m) continue;
                    E *const dst = (E *)a.y + (row0 + p * RPP) * a.ld_y + col;
                    if constexpr (decltype(past)::value) {
                        typedef unsigned Words __attribute__((ext_vector_type(sizeof(E)), aligned(sizeof(E))));
                        __builtin_nontemporal_store(__builtin_bit_cast(Words, q), (Words *)dst);
                        keep_apart();
                    } else {
                        *(Quad<E> *)dst = q;
                    }
                }
            };
            if (C::PAST && a.past)
                rows(std::true_type());
            else
                rows(std::false_type());
            if (left > 0 && !whole) {  // the last one to three columns of y, value by value
#pragma unroll 1
                for (int k = 0; k < P * left; ++k) {
                    const int p = k / left, e = k - p * left;
                    const long long row = row0 + p * RPP;
                    if (row >= a.m) break;
                    float v = *(const float *)(out + (p * RPP + el / LPR) * C::ROW + (el % LPR) * 16 + e * 4);
                    if (a.bias) v += a.bias[col + e];
                    if (a.res) v += (float)((const E *)a.res)[row * a.ld_res + col + e];
                    ((E *)a.y)[row * a.ld_y + col + e] = (E)act_of<ACT>(v);
                }
            }
        });
        wave_lds_sync();
    }
}

// TileX moves the fewest bytes to LDS a product, but has a CU to itself and pays its epilogue in full: for long
// sums.  Two of TileL's or TileM's workgroups fit a CU (one's epilogue behind the other's steps), eight of TileR's,
// which is for sums of one or two steps whose residual has to arrive as well.
typedef Tile<256, 256, 4, 2, 3> TileX;
typedef Tile<256, 128, 4, 2, 3> TileL;
typedef Tile<128, 128, 4, 2, 3> TileM;
typedef Tile<64, 64, 2, 2, 4> TileS;
typedef Tile<64, 64, 2, 2, 2> TileR;

template <typename C>
hipError_t launch(const Mx4Args &a, hipStream_t s)
{
    const int tiles_m = (a.m - 1) / C::BM + 1, tiles_n = (a.n - 1) / C::BN + 1;
    const int per_xcd = (int)(((long long)tiles_m * tiles_n + 7) / 8);
    auto *f = a.type == 0 ? mx4_tile_kernel<C, 0> : a.type == 1 ? mx4_tile_kernel<C, 1> : mx4_tile_kernel<C, 2>;
    hipLaunchKernelGGL(f, dim3((unsigned)per_xcd * 8u), dim3(C::T), 0, s, a, tiles_m, tiles_n, per_xcd);
    return hipGetLastError();
}

template <typename C>
long long tiles(const Mx4Args &a)
{
    return ((a.m - 1LL) / C::BM + 1) * ((a.n - 1LL) / C::BN + 1);
}

}  // namespace

hipError_t launch_mx4_tiles(Mx4Args a, hipStream_t s)
{
    a.past = stored_past(a.y, a.m, a.ld_y, a.type == 0 ? 4 : 2);
    const int cus = cus_or_default();
    // The largest tile that gives every CU one (256 CUs; us, large / middle / small tile):
    //   8192 x 2048 x 256 (512 large tiles)    12.4 / 14.4 / 16.8
    //   4096 x 2048 x 2048 (256 large)         17.4 / 18.1 / 21.6
    //   2048 x 2048 x 2048 (256 middle)        13.7 / 11.1 / 12.8
    //   1024 x 2048 x 2048 (128 middle)        12.5 /  9.9 /  8.5
    // and with a residual (bf16, operands from HBM; us, large tile / TileR):
    //   50176 x 512 x 128   34.9 / 29.0      200704 x 256 x 64   64.0 / 51.4      65536 x 512 x 256   45.5 / 43.7
    //   32768 x 2048 x 256  81.5 / 85.6 (the one loss seen)     32768 x 2048 x 512    92 / 103 (so not for longer)
    if (a.res && a.k1 <= 2) return launch<TileR>(a, s);
    // and for long sums (us, TileX / large tile):
    //   8192 x 8192 x 8192   261 / 280       4096 x 4096 x 4096   39.7 / 41.7     8192 x 8192 x 2048   102 / 89
    if (a.k1 >= 32 && tiles<TileX>(a) >= cus) return launch<TileX>(a, s);
    if (tiles<TileL>(a) >= cus) return launch<TileL>(a, s);
    if (tiles<TileM>(a) >= cus) return launch<TileM>(a, s);
    return launch<TileS>(a, s);
}

}  // namespace ifx
