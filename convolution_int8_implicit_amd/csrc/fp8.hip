// 8-bit floating point with one power of two per block of 128: rounding, also of the transpose, the values back,
// and the products for few rows (fp8_tile.h holds the tiled ones).
//
// A tensor of `rows` rows and k columns holds blocks of 128 consecutive columns of a row: one byte a column (e4m3
// or e5m2) and one power of two per block, 2^(s - 127) with the byte s (255: NaN).  The layout is blocked by 128
// columns as the 4-bit tensors are: codes [K1][rows][128] bytes, K1 = ceil(k / 128), columns past k zero, so a step
// of a product over any run of rows is one contiguous run of codes.  One block a row and panel leaves one byte a
// row, too few for a load of its own: the scales of four panels share a word, [ceil(K1 / 4)][rows][4] bytes.
#include "device_common.h"
#include "ifx_internal.h"
#include "lowp.h"

namespace ifx {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v8i join(v4i lo, v4i hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

// ------------------------------------------------------------------------------------------
// Rounding by rows.  Streaming, HBM-bound: a thread rounds eight consecutive columns, sixteen threads a row's
// block, so the block's maximum is one of sixteen lanes and a row's codes of a panel are one 128-byte line.  A
// workgroup covers 16 rows of four panels: four loads in flight per thread, and the four panels' scales are one
// word.  8192 x 8192 bf16 32.6 us, 6.2 TB/s (33.6 with x read past the caches, as the 4-bit rounding's is).
// ------------------------------------------------------------------------------------------
constexpr int kQRows = 16, kQPanels = 4;

template <int TYPE, int FMT>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(const void *x, long long ld, int rows, int k, int k1, int groups,
                                                           uint8_t *codes, uint8_t *scales)
{
    typedef typename Elem<TYPE>::type E;
    const int rt = (int)(blockIdx.x / (unsigned)groups), pg = (int)(blockIdx.x - (unsigned)rt * (unsigned)groups);
    const int t = threadIdx.x, v = t & 15;
    const int row = rt * kQRows + (t >> 4);
    const bool live = row < rows;
    const E *src = (const E *)x + (long long)(live ? row : rows - 1) * ld;
    Oct<E> raw[kQPanels];
#pragma unroll
    for (int i = 0; i < kQPanels; ++i) {
        // (a panel past the last one may begin past 31 bits)
        const int p = pg * kQPanels + i, col = p * 128 + v * 8;
        raw[i] = p < k1 && col < k ? load8(src + col, k - col) : Oct<E>{};
    }
    unsigned word = 0;
#pragma unroll
    for (int i = 0; i < kQPanels; ++i) {
        const int p = pg * kQPanels + i;
        const int valid = p < k1 ? k - (p * 128 + v * 8) : 0;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = raw[i].get(e);
        if (valid < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= valid) f[e] = 0.0f;
        }
        const unsigned s = fp8_scale<FMT>(row_max(top_bits(f)));
        const uint2 r = fp8_codes<FMT>(f, s);
        word |= s << (8 * i);
        if (live && p < k1) ((uint2 *)codes)[((long long)p * rows + row) * 16 + v] = r;
    }
    if (live && v == 0) ((unsigned *)scales)[(long long)pg * rows + row] = word;
}

// ------------------------------------------------------------------------------------------
// Rounding of the transpose: rows of the result are x's columns, its blocks 128 consecutive rows of x.  A
// workgroup brings 128 rows of 128 bytes of x (64 columns of a 16-bit type, 32 of float32) through LDS: rows of 32
// words and 8 words more behind every 16 rows, so that eight lanes reading the same words of rows 16 apart, eight
// words each, reach all 64 banks.  Eight neighbouring lanes hold a block, 16 values each (of two columns at once
// in 16 bits): 16 bytes of codes a lane, 128 a block.  x is read in lines, the codes of neighbouring columns are
// neighbouring lines.  8192 x 8192 bf16 37 us, 5.4 TB/s; 6241 x 2048 float32 11.1, 5.7.
// ------------------------------------------------------------------------------------------
constexpr int kTPad = 8, kTWords = 128 * 32 + 8 * kTPad;
__device__ __forceinline__ int t_word(int row, int word) { return row * 32 + (row >> 4) * kTPad + word; }

// Maximum over the eight lanes 8i .. 8i + 7.
__device__ __forceinline__ unsigned eight_max(unsigned u)
{
    u = quad_max(u);
    return max(u, (unsigned)__builtin_amdgcn_mov_dpp((int)u, 0x141, 0xf, 0xf, true));
}

// 16 values of a column: its scale byte, and the codes to p's panel and chunk.
template <int FMT>
__device__ __forceinline__ void put_column(const float (&f)[16], int chunk, long long row, int rows, int panel, int k1,
                                           uint8_t *codes, uint8_t *scales, bool live)
{
    float a[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = f[e], b[e] = f[8 + e];
    const unsigned s = fp8_scale<FMT>(eight_max(max(top_bits(a), top_bits(b))));
    const uint2 lo = fp8_codes<FMT>(a, s), hi = fp8_codes<FMT>(b, s);
    if (!live) return;
    ((uint4 *)codes)[((long long)panel * rows + row) * 8 + chunk] = make_uint4(lo.x, lo.y, hi.x, hi.y);
    if (chunk == 0) {
        uint8_t *at = scales + ((long long)(panel >> 2) * rows + row) * 4;
        at[panel & 3] = (uint8_t)s;
        if (panel == k1 - 1)  // the word's other bytes
            for (int i = (panel & 3) + 1; i < 4; ++i) at[i] = 0;
    }
}

template <int TYPE, int FMT>
__global__ __launch_bounds__(256) void fp8_quantize_t_kernel(const void *x, long long ld, int rows, int k, int k1, int groups,
                                                             uint8_t *codes, uint8_t *scales)
{
    typedef typename Elem<TYPE>::type E;
    constexpr int PER = 4 / sizeof(E), COLS = 32 * PER;  // columns of a word and of the workgroup
    __shared__ unsigned tile[kTWords];
    const int panel = (int)(blockIdx.x / (unsigned)groups), cg = (int)(blockIdx.x - (unsigned)panel * (unsigned)groups);
    const int t = threadIdx.x, c0 = cg * COLS, r0 = panel * 128;
    // 32 rows at a time, eight threads a row, 16 bytes each
    typedef typename Words<sizeof(E)>::type V;
    V raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = r0 + i * 32 + (t >> 3), col = c0 + (t & 7) * 4 * PER;
        const E *src = (const E *)x + (long long)min(row, k - 1) * ld + col;
        const int valid = row < k ? rows - col : 0;
        raw[i] = (V){0, 0, 0, 0};
        if (valid >= 4 * PER) {
            raw[i] = *(const V *)src;
        } else if (valid > 0) {
            if constexpr (PER == 1) {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (e < valid) raw[i][e] = ((const unsigned *)src)[e];
            } else {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (e < valid) raw[i][e / 2] |= (unsigned)((const unsigned short *)src)[e] << (16 * (e & 1));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) *(v4i *)&tile[t_word(i * 32 + (t >> 3), (t & 7) * 4)] = __builtin_bit_cast(v4i, raw[i]);
    __syncthreads();
    const int chunk = t & 7, word = t >> 3;
    unsigned w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = tile[t_word(chunk * 16 + e, word)];
    const int row = c0 + word * PER;
    float f[16];
    if constexpr (PER == 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(w[e]);
        put_column<FMT>(f, chunk, row, rows, panel, k1, codes, scales, row < rows);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                Oct<E> o;
                o.w[0] = w[e];
                f[e] = o.get(h);
            }
            put_column<FMT>(f, chunk, row + h, rows, panel, k1, codes, scales, row + h < rows);
        }
    }
}

// The values back: eight columns per thread, 8 bytes of codes in, one 16-byte store of a 16-bit type out.  HBM-bound:
// 8192 x 8192 to bf16 36.2 us, 5.6 TB/s, to float32 78, 4.3.
template <int TYPE, int FMT>
__global__ __launch_bounds__(256) void fp8_dequantize_kernel(const uint8_t *codes, const uint8_t *scales, int rows, int k,
                                                             int k1, int groups, void *y, long long ld, int past)
{
    typedef typename Elem<TYPE>::type E;
    const int rt = (int)(blockIdx.x / (unsigned)groups), pg = (int)(blockIdx.x - (unsigned)rt * (unsigned)groups);
    const int t = threadIdx.x, v = t & 15;
    const int row = rt * kQRows + (t >> 4);
    if (row >= rows) return;
    const unsigned word = ((const unsigned *)scales)[(long long)pg * rows + row];
    uint2 c[kQPanels];
#pragma unroll
    for (int i = 0; i < kQPanels; ++i) {
        const int p = pg * kQPanels + i;
        c[i] = ((const uint2 *)codes)[((long long)(p < k1 ? p : k1 - 1) * rows + row) * 16 + v];
    }
#pragma unroll
    for (int i = 0; i < kQPanels; ++i) {
        const int p = pg * kQPanels + i;
        if (p >= k1) break;  // (its columns may pass 31 bits)
        const int col = p * 128 + v * 8;
        if (col >= k) break;
        const float sf = __uint_as_float((word >> (8 * i) & 255u) << 23);
        float f[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const unsigned q = e ? c[i].y : c[i].x;
            typedef float v2f __attribute__((ext_vector_type(2)));
            v2f a, b;
            if constexpr (FMT) {
                a = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(q, sf, false);
                b = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(q, sf, true);
            } else {
                a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, sf, false);
                b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, sf, true);
            }
            f[4 * e] = a[0], f[4 * e + 1] = a[1], f[4 * e + 2] = b[0], f[4 * e + 3] = b[1];
        }
        E *const dst = (E *)y + (long long)row * ld + col;
        if (past && k - col >= 8)
            store8<true>(dst, f);
        else
            store8(dst, k - col, f);
    }
}

// ------------------------------------------------------------------------------------------
// Few rows: y = act(A W^T + bias + residual), act(A G^T) (A U^T), or the latter's gradient at both projections.
//
// For up to 16 rows of A.  A workgroup of kRowWaves waves takes 16 weight rows (of both weights in the gated forms); its
// waves take panels in turn straight from memory, several requested at once, and the partial sums meet in LDS, added in
// wave order.  What bounds it: the weights, read once (one row of 8192 x 8192, launch included, 12.8 us, 5.2 TB/s, with
// three weights in turn, which the memory-side cache holds in part, 16.6 with eight; 16 rows 19.5 and 20.5).  From 17 rows
// on the tiles are as fast or faster: 32 rows of 8192 x 8192 20.0 us against 29.6 with two groups of 16 rows here, 64 rows
// 22.1 against 45.8 (20 rows of 2048 x 8192 16.1 against 12.8 is the one loss seen).
// The 16x16x128 instruction takes row l % 16 and 32 of the panel's columns from lane l; which 32 is the same on
// both sides, so a lane takes the chunks that make its two loads whole 64-byte runs.  Lane l's results are column
// l % 16 (a row of A here) and rows 4 (l / 16) .. + 3 (weight rows).
// KS > 1, for at most 16 / KS rows of A over few weight rows: the instruction's 16 rows are KS panels of 16 / KS
// weight rows and of as many rows of A, of whose products the KS blocks on the diagonal count, so a workgroup takes
// 16 / KS weight rows and KS times as many workgroups share the bytes.
// WIDE: products in bfloat16 (fp8_tile.h says when and why).
// ------------------------------------------------------------------------------------------
constexpr int kRowWaves = 8;

template <int KS, int MODE, int AF, bool WIDE>
__global__ __launch_bounds__(64 * kRowWaves) void fp8_rows_kernel(Fp8Args a)
{
    constexpr int R = 16 / KS, NW = MODE == kProduct ? 1 : 2, AHEAD = 4 / NW;
    __shared__ float part[kRowWaves][NW][256];
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, c = l & 15, g = l >> 4;
    const int slice = c / R, r = c % R, n0 = (int)blockIdx.x * R;
    const int wr = min(n0 + r, a.n - 1), ar = min(r, a.m - 1);
    const uint8_t *wc[2] = {a.w_codes, a.u_codes}, *wsc[2] = {a.w_scales, a.u_scales};
    v4f acc[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j) acc[j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = w * KS; p0 < a.k1; p0 += AHEAD * kRowWaves * KS) {
        v4i wv[AHEAD][NW][2], av[AHEAD][2];
        int ws[AHEAD][NW], as[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int p = p0 + u * kRowWaves * KS + slice;
            const bool in = p < a.k1;
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                wv[u][j][0] = wv[u][j][1] = (v4i){0, 0, 0, 0};
                ws[u][j] = 0;
                if (in) {
                    const v4i *src = (const v4i *)wc[j] + ((long long)p * a.n + wr) * 8 + g;
                    wv[u][j][0] = src[0];
                    wv[u][j][1] = src[4];
                    ws[u][j] = wsc[j][((long long)(p >> 2) * a.n + wr) * 4 + (p & 3)];
                }
            }
            av[u][0] = av[u][1] = (v4i){0, 0, 0, 0};
            as[u] = 0;
            if (in) {
                const v4i *src = (const v4i *)a.a_codes + ((long long)p * a.m + ar) * 8 + g;
                av[u][0] = src[0];
                av[u][1] = src[4];
                as[u] = a.a_scales[((long long)(p >> 2) * a.m + ar) * 4 + (p & 3)];
            }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if constexpr (WIDE) {
                lowp_v8b x[4];
                fp8_widen<AF>(av[u][0], av[u][1], as[u], x);
#pragma unroll
                for (int j = 0; j < NW; ++j) {
                    lowp_v8b y[4];
                    fp8_widen<0>(wv[u][j][0], wv[u][j][1], ws[u][j], y);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[q], x[q], acc[j], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int j = 0; j < NW; ++j)
                    acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(wv[u][j][0], wv[u][j][1]), join(av[u][0], av[u][1]),
                                                                              acc[j], 0, AF, 0, ws[u][j], 0, as[u]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NW; ++j) *(v4f *)&part[w][j][c * 16 + 4 * g] = acc[j];
    __syncthreads();
    const int t = threadIdx.x;
    if (t < R * R) {
        const int m = t / R, ni = t % R, n = n0 + ni;
        if (m >= a.m || n >= a.n) return;
        float f[NW];
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            f[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < kRowWaves; ++i)
#pragma unroll
                for (int k = 0; k < KS; ++k) f[j] += part[i][j][(m + k * R) * 16 + ni + k * R];
        }
        with_act(a.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            if constexpr (MODE == kProduct) {
                float v = f[0];
                if (a.bias) v += a.bias[n];
                if (a.res) v += load_any(a.res, a.type, (long long)m * a.ld_res + n);
                store_any(a.y, a.type, (long long)m * a.ld_y + n, act_of<ACT>(v));
            } else if constexpr (MODE == kGated) {
                store_any(a.y, a.type, (long long)m * a.ld_y + n, act_of<ACT>(f[0]) * f[1]);
            } else {
                const float dy = load_any(a.res, a.type, (long long)m * a.ld_res + n);
                store_any(a.y, a.type, (long long)m * a.ld_y + n, dy * f[1] * act_slope<ACT>(f[0]));
                store_any(a.y2, a.type, (long long)m * a.ld_y2 + n, dy * act_of<ACT>(f[0]));
            }
        });
    }
}

template <int KS, int MODE, int AF, bool WIDE>
hipError_t launch_rows(const Fp8Args &a, hipStream_t s)
{
    hipLaunchKernelGGL((fp8_rows_kernel<KS, MODE, AF, WIDE>), dim3((unsigned)((a.n - 1) / (16 / KS) + 1)), dim3(64 * kRowWaves), 0,
                       s, a);
    return hipGetLastError();
}

template <int MODE, int AF, bool WIDE>
hipError_t rows_form(const Fp8Args &a, hipStream_t s)
{
    // few weight rows and enough panels for every wave (us of a graph's node, KS 4 or 2 / KS 1): 1 x 2048 x 8192 5.8 / 7.7,
    // 8 x 2048 x 8192 6.7 / 9.2, 1 x 1000 x 2048 2.9 / 3.2, 1 x 500 x 16384 5.1 / 12.7; but 1 x 4096 x 8192 10.9 / 8.6
    const int cus = cus_or_default();
    if (a.m <= 4 && a.n <= 8 * cus && a.k1 >= 4 * kRowWaves) return launch_rows<4, MODE, AF, WIDE>(a, s);
    if (a.m <= 8 && a.n <= 8 * cus && a.k1 >= 2 * kRowWaves) return launch_rows<2, MODE, AF, WIDE>(a, s);
    return launch_rows<1, MODE, AF, WIDE>(a, s);
}

template <int MODE, int AF>
hipError_t rows_of_type(const Fp8Args &a, hipStream_t s)
{
    return a.type == 0 ? rows_form<MODE, AF, true>(a, s) : rows_form<MODE, AF, false>(a, s);
}

}  // namespace

hipError_t launch_fp8_quantize(const void *x, int type, long long ld, int rows, int k, int format, uint8_t *codes,
                               uint8_t *scales, hipStream_t s)
{
    const int k1 = (k - 1) / 128 + 1, groups = (k1 - 1) / kQPanels + 1;
    const dim3 grid((unsigned)((rows + kQRows - 1LL) / kQRows * groups));
    auto pick = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        return type == 0 ? fp8_quantize_kernel<0, F> : type == 1 ? fp8_quantize_kernel<1, F> : fp8_quantize_kernel<2, F>;
    };
    auto *f = format ? pick(Slot1()) : pick(Slot0());
    hipLaunchKernelGGL(f, grid, dim3(256), 0, s, x, ld, rows, k, k1, groups, codes, scales);
    return hipGetLastError();
}

hipError_t launch_fp8_quantize_t(const void *x, int type, long long ld, int rows, int k, int format, uint8_t *codes,
                                 uint8_t *scales, hipStream_t s)
{
    const int k1 = (k - 1) / 128 + 1, cols = type == 0 ? 32 : 64, groups = (rows - 1) / cols + 1;
    const dim3 grid((unsigned)((long long)k1 * groups));
    auto pick = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        return type == 0 ? fp8_quantize_t_kernel<0, F> : type == 1 ? fp8_quantize_t_kernel<1, F> : fp8_quantize_t_kernel<2, F>;
    };
    auto *f = format ? pick(Slot1()) : pick(Slot0());
    hipLaunchKernelGGL(f, grid, dim3(256), 0, s, x, ld, rows, k, k1, groups, codes, scales);
    return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t *codes, const uint8_t *scales, int format, int rows, int k, void *y,
                                 int type, long long ld, hipStream_t s)
{
    const int k1 = (k - 1) / 128 + 1, groups = (k1 - 1) / kQPanels + 1;
    const dim3 grid((unsigned)((rows + kQRows - 1LL) / kQRows * groups));
    auto pick = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        return type == 0 ? fp8_dequantize_kernel<0, F> : type == 1 ? fp8_dequantize_kernel<1, F> : fp8_dequantize_kernel<2, F>;
    };
    auto *f = format ? pick(Slot1()) : pick(Slot0());
    const int past = stored_past(y, rows, ld, type == 0 ? 4 : 2);
    hipLaunchKernelGGL(f, grid, dim3(256), 0, s, codes, scales, rows, k, k1, groups, y, ld, past);
    return hipGetLastError();
}

bool fp8_few_rows(int m, int n) { return m <= 16 && n <= 1 << 24; }

hipError_t launch_fp8(Fp8Args a, Fp8Mode mode, hipStream_t s)
{
    if (!fp8_few_rows(a.m, a.n)) return mode == kProduct ? launch_fp8_product(a, s) : launch_fp8_gated(a, mode, s);
    if (mode == kProduct) return a.a_format ? rows_of_type<kProduct, 1>(a, s) : rows_of_type<kProduct, 0>(a, s);
    if (mode == kGatedGrad) return rows_of_type<kGatedGrad, 0>(a, s);
    if (!a.codes) return rows_of_type<kGated, 0>(a, s);
    // A block's 128 columns are eight workgroups': their values in 32 bits first, by the kernel of float32 results, then the
    // rounding in a launch of its own (4 us).  One launch whose workgroups take 128 columns of both weights reads no faster
    // than 35 GB/s a CU: 1 x 8192 x 2048 18.2 us against 12.1, 1 x 2048 x 8192 59.6 against 12.1 (1 x 1000 x 500 9.4 against
    // 11.7).
    a.y = a.ws;
    a.type = 0;
    a.ld_y = a.n;
    const hipError_t e = rows_form<kGated, 0, true>(a, s);
    if (e != hipSuccess) return e;
    return launch_fp8_quantize(a.ws, 0, a.n, a.m, a.n, 0, a.codes, a.scales, s);
}

}  // namespace ifx
