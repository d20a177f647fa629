// The tiled product of two microscaled 4-bit tensors: y = act(A W^T + bias + residual) for more than
// a few rows (mx4.hip holds the layout, the rounding and the product for few rows).
//
// What bounds it: at large sizes the matrix units (v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 cycles
// a wave for 131072 operations; measured alone on operands that change: 6.5 POP/s at 2 waves per
// SIMD, the 16x16x128 form 5.7), at short sums (k of a few hundred) the output's bytes.
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
    static constexpr int CPW = (BM + BN) / 16 / W;  // 1 KB code DMAs per wave and stage
    static constexpr int SC = (BM + BN) / 64;       // 256-byte scale DMAs per stage
    static constexpr int SPW = SC > W ? SC / W : 1; // of them per wave (waves past SC / SPW repeat others')
    static constexpr int LPS = CPW + SPW;           // DMAs per wave and stage
    static constexpr int ROW = TN * 4 + 32;         // bytes of a staged output row: 4 rows apart, half the banks on
    static constexpr int OUT = 32 * ROW * W;
    static constexpr int LDS = ST * STAGE > OUT ? ST * STAGE : OUT;
    static constexpr int PER_CU = kLdsBytes / LDS < 2048 / T ? kLdsBytes / LDS : 2048 / T;
    static_assert(BM / 16 % CPW == 0, "a wave's code DMAs are all of A or all of W");
    static_assert(SC <= W || SC % W == 0, "waves share the runs of scales evenly");
    static_assert(BM / 64 % SPW == 0, "a wave's scale DMAs are all of A or all of W");
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

    // this wave's DMAs of a step: CPW kilobytes of A's or W's codes and 64 rows of scales
    const bool of_a = w * C::CPW < C::BM / 16;
    const int chunk0 = of_a ? w * C::CPW : w * C::CPW - C::BM / 16;
    const long long rows = of_a ? a.m : a.n;
    const int row0 = of_a ? m0 : n0;
    const uint8_t *code_src = (of_a ? a.a_codes : a.w_codes) + (long long)row0 * 64;
    const long long code_range = min((long long)(of_a ? C::BM : C::BN), rows - row0) * 64;
    const int sc = w * C::SPW % C::SC;
    const bool s_of_a = sc < C::BM / 64;
    const long long s_rows = s_of_a ? a.m : a.n;
    const int s_row0 = s_of_a ? m0 : n0, s_chunk = s_of_a ? sc : sc - C::BM / 64;
    const uint8_t *scale_src = (s_of_a ? a.a_scales : a.w_scales) + (long long)s_row0 * 4;
    const long long scale_range = min((long long)(s_of_a ? C::BM : C::BN), s_rows - s_row0) * 4;
    const unsigned code_off = (unsigned)(chunk0 * 1024 + (l >> 2) * 64 + (((l & 3) ^ (l >> 4)) * 16));
    const unsigned scale_off = (unsigned)(s_chunk * 256 + l * 4);
    const int code_dst = w * C::CPW * 1024, scale_dst = C::CODES + sc * 256;

    // DMA j of this wave's LPS for step s
    auto issue1 = [&](int s, int j) __attribute__((always_inline)) {
        int8_t *st = smem + (s % C::ST) * C::STAGE;
        if (j < C::CPW) {
            load16_lds(make_rsrc(code_src + (long long)s * rows * 64, code_range), st + code_dst + j * 1024, code_off + j * 1024);
        } else {
            const int i = (j - C::CPW) * 256;
            ifx_raw_buffer_load_lds(make_rsrc(scale_src + (long long)s * s_rows * 4, scale_range),
                                    (__attribute__((address_space(3))) void *)(st + scale_dst + i), 4, scale_off + i, 0, 0, 0);
        }
    };
    auto issue = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < C::LPS; ++j) issue1(s, j);
    };

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
#pragma unroll
        for (int t = 0; t < MF; ++t) {
            const int i = t / C::FN, j = t % C::FN;
            if (j == 0) sa[i] = (int)((unsigned)as[i] >> (8 * g));
            if (i == 0) sb[j] = (int)((unsigned)bs[j] >> (8 * g));
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(a0[i]), wide(b0[j]), acc[i][j], kFp4, kFp4, 0,
                                                                        sa[i], 0, sb[j]);
#pragma unroll
            for (int u = t * RD; u < (t + 1) * RD && u < FR; ++u) read(Slot1(), st, u);
            if (STEADY)
#pragma unroll
                for (int u = t * C::LPS / MF; u < (t + 1) * C::LPS / MF; ++u) issue1(s + C::ST - 1, u);
            __builtin_amdgcn_sched_barrier(0);
        }
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
    // columns a lane in whole rows.
    lds_barrier();
    int8_t *out = smem + w * 32 * C::ROW;
    constexpr int LPR = C::TN / 4, RPP = 64 / LPR;  // lanes per row, rows per pass
    const int col = n0 + wn * C::TN + (l % LPR) * 4, left = a.n - col;
    float bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) bias[e] = a.bias && e < left ? a.bias[col + e] : 0.0f;
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int r0 = m0 + wm * C::TM + i * 32;
            if (r0 >= a.m) break;
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    *(float *)(out + (8 * (e / 4) + 4 * g + e % 4) * C::ROW + (j * 32 + c) * 4) = acc[i][j][e];
            wave_lds_sync();
#pragma unroll
            for (int p = 0; p < 32 / RPP; ++p) {
                const int r = p * RPP + l / LPR;
                const long long row = r0 + r;
                if (row >= a.m || left <= 0) continue;
                const v4f f = *(const v4f *)(out + r * C::ROW + (l % LPR) * 16);
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = f[e] + bias[e];
                if (left >= 4) {
                    if (a.res) {
                        const Quad<E> q = *(const Quad<E> *)((const E *)a.res + row * a.ld_res + col);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] += (float)q.v[e];
                    }
                    Quad<E> q;
#pragma unroll
                    for (int e = 0; e < 4; ++e) q.v[e] = (E)act_of<decltype(act)::value>(v[e]);
                    *(Quad<E> *)((E *)a.y + row * a.ld_y + col) = q;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left) {
                            if (a.res) v[e] += (float)((const E *)a.res)[row * a.ld_res + col + e];
                            ((E *)a.y)[row * a.ld_y + col + e] = (E)act_of<decltype(act)::value>(v[e]);
                        }
                }
            }
            wave_lds_sync();
        }
    });
}

typedef Tile<256, 256, 4, 2, 4> Tile256;
typedef Tile<128, 128, 2, 2, 4> Tile128;
typedef Tile<64, 64, 2, 2, 4> Tile64;

template <typename C>
hipError_t launch(const Mx4Args &a, hipStream_t s)
{
    const int tiles_m = (a.m - 1) / C::BM + 1, tiles_n = (a.n - 1) / C::BN + 1;
    const int per_xcd = (int)(((long long)tiles_m * tiles_n + 7) / 8);
    auto *f = a.type == 0 ? mx4_tile_kernel<C, 0> : a.type == 1 ? mx4_tile_kernel<C, 1> : mx4_tile_kernel<C, 2>;
    hipLaunchKernelGGL(f, dim3((unsigned)per_xcd * 8u), dim3(C::T), 0, s, a, tiles_m, tiles_n, per_xcd);
    return hipGetLastError();
}

long long tiles(const Mx4Args &a, int size) { return ((a.m - 1LL) / size + 1) * ((a.n - 1LL) / size + 1); }

}  // namespace

hipError_t launch_mx4_tiles(const Mx4Args &a, hipStream_t s)
{
    int cus = 0;
    if (current_cus(&cus) != hipSuccess) cus = 256;
    if (tiles(a, 256) >= cus) return launch<Tile256>(a, s);
    if (tiles(a, 128) >= cus) return launch<Tile128>(a, s);
    return launch<Tile64>(a, s);
}

}  // namespace ifx
