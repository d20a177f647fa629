// Microscaled 4-bit floating point: rounding, the values back, and the product of two such tensors.
//
// A tensor of `rows` rows and k columns holds blocks of 32 consecutive columns of a row: 4-bit
// codes (sign, two exponent bits, one mantissa bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one
// power of two per block, 2^(s - 127) with the byte s (255: NaN).  The layout is blocked by
// 128 columns as the int8 activations are by 32 channels: codes [K1][rows][64] bytes and scales
// [K1][rows][4] bytes, K1 = ceil(k / 128), columns past k zero.  128 columns are what one wave's
// matrix instruction reads (16 rows) or what two read (32 rows), so a step of a product over
// any run of rows is one contiguous run of codes and one of scales.
#include "device_common.h"
#include "ifx_internal.h"
#include "lowp.h"

namespace ifx {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kFp4 = 4;  // the matrix instruction's operand format: 4-bit e2m1

__device__ __forceinline__ v8i wide(v4i x) { return (v8i){x[0], x[1], x[2], x[3], 0, 0, 0, 0}; }

// ------------------------------------------------------------------------------------------
// Rounding.  Streaming, HBM-bound: a thread rounds eight consecutive columns (one 16-byte load of
// a 16-bit type), four threads a block, sixteen a row's 128-column panel, so a workgroup covers
// 16 rows of a panel: 64-byte codes of 16 consecutive rows are a contiguous kilobyte of the
// output.  Four panels per workgroup keep four loads in flight per thread.  200704 x 512 bf16: 43 us
// and back 38 us for 260 MB either way, 6.0 and 6.8 TB/s.
// ONCE: x is read past the caches.  For 16-bit rows that begin on 128-byte lines, where a wave's accesses cover
// whole lines: the above takes 43 us instead of 47, and with the values back 81 instead of 104, as the codes
// stay cached.  Elsewhere neighbouring accesses share lines: 100000 x 999 bf16 takes 49 us cached and 52 past the
// caches, float32 of 1000 columns, two accesses a line, 91 and 108.
// ------------------------------------------------------------------------------------------
constexpr int kQRows = 16, kQPanels = 4;

template <int TYPE, bool ONCE>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const void *x, long long ld, int rows, int k, int k1,
                                                           int groups, uint8_t *codes, uint8_t *scales)
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
        const int col = (pg * kQPanels + i) * 128 + v * 8;
        raw[i] = col < k ? load8<ONCE>(src + col, k - col) : Oct<E>{};
    }
#pragma unroll
    for (int i = 0; i < kQPanels; ++i) {
        const int p = pg * kQPanels + i, col = p * 128 + v * 8;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = raw[i].get(e);
        if (k - col < 8) {  // (col + 8 may pass 32 bits)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= k - col) f[e] = 0.0f;
        }
        unsigned s;
        const unsigned r = mx4_codes(f, s);
        if (live && p < k1) {
            const long long at = (long long)p * rows + row;
            ((unsigned *)codes)[at * 16 + v] = r;
            if ((v & 3) == 0) scales[at * 4 + (v >> 2)] = (uint8_t)s;
        }
    }
}

// The values back: eight columns per thread, 4 bytes of codes in, one 16-byte store of a 16-bit
// type out.  Every value of a finite block is exact in bfloat16.
template <int TYPE>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t *codes, const uint8_t *scales, int rows,
                                                             int k, int k1, int groups, void *y, long long ld, int past)
{
    typedef typename Elem<TYPE>::type E;
    const int rt = (int)(blockIdx.x / (unsigned)groups), pg = (int)(blockIdx.x - (unsigned)rt * (unsigned)groups);
    const int t = threadIdx.x, v = t & 15;
    const int row = rt * kQRows + (t >> 4);
    if (row >= rows) return;
    unsigned c[kQPanels], s[kQPanels];
#pragma unroll
    for (int i = 0; i < kQPanels; ++i) {
        const int p = pg * kQPanels + i;
        const long long at = (long long)(p < k1 ? p : k1 - 1) * rows + row;
        c[i] = ((const unsigned *)codes)[at * 16 + v];
        s[i] = scales[at * 4 + (v >> 2)];
    }
#pragma unroll
    for (int i = 0; i < kQPanels; ++i) {
        const int col = (pg * kQPanels + i) * 128 + v * 8;
        if (col >= k) break;
        const float sf = __uint_as_float(s[i] << 23);
        float f[8];
        auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sf, 0);
        auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sf, 1);
        auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sf, 2);
        auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sf, 3);
        f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1], f[4] = d[0], f[5] = d[1], f[6] = e[0], f[7] = e[1];
        E *const dst = (E *)y + (long long)row * ld + col;
        if (past && k - col >= 8)
            store8<true>(dst, f);
        else
            store8(dst, k - col, f);
    }
}

// ------------------------------------------------------------------------------------------
// Product y[m, n] = act(sum_k A[m, k] W[n, k] + bias[n] + residual[m, n]).
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ float load_any(const void *p, int type, long long i)
{
    return type == 0 ? ((const float *)p)[i] : type == 1 ? (float)((const __bf16 *)p)[i] : (float)((const _Float16 *)p)[i];
}
__device__ __forceinline__ void store_any(void *p, int type, long long i, float f)
{
    if (type == 0)
        ((float *)p)[i] = f;
    else if (type == 1)
        ((__bf16 *)p)[i] = (__bf16)f;
    else
        ((_Float16 *)p)[i] = (_Float16)f;
}

// Few rows: a workgroup of kRowWaves waves takes 16 weight rows and 16 MT rows of A; wave w multiplies
// panels w, w + kRowWaves, ... straight from memory (16 rows of a panel are one contiguous kilobyte,
// one 16-byte load per lane), kAhead of them requested at once, and the partial sums meet in LDS,
// added in wave order.  What bounds it: the weights, read once for MT = 1.
// The 16x16x128 instruction takes row l % 16 and columns 32 (l / 16) .. + 31 from lane l, one
// block with its scale in the lowest byte; lane l's results are column l % 16 (a row of A here)
// and rows 4 (l / 16) .. + 3 (weight rows).
// 8 waves and 4 panels ahead measured best (one row of 8192 x 8192 from HBM 9.8 us, launch included, 3.6 TB/s;
// 16 waves 11.5, 8 panels ahead 11.8, 2 panels 10.0, 4 waves 9.9).
constexpr int kRowWaves = 8, kAhead = 4;

template <int MT>
__global__ __launch_bounds__(64 * kRowWaves) void mx4_rows_kernel(Mx4Args a, int tiles_n)
{
    __shared__ float part[kRowWaves][MT * 256];
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, c = l & 15, g = l >> 4;
    const unsigned tm = blockIdx.x / (unsigned)tiles_n, tn = blockIdx.x - tm * (unsigned)tiles_n;
    const int m0 = (int)tm * 16 * MT, n0 = (int)tn * 16;
    const int wr = min(n0 + c, a.n - 1);
    v4f acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = w; p0 < a.k1; p0 += kAhead * kRowWaves) {
        v4i wv[kAhead], av[kAhead][MT];
        int ws[kAhead], as[kAhead][MT];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const long long p = p0 + u * kRowWaves;
            if (p < a.k1) {
                const long long wi = (p * a.n + wr) * 4 + g;
                wv[u] = ((const v4i *)a.w_codes)[wi];
                ws[u] = a.w_scales[wi];
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const long long ai = (p * a.m + min(m0 + 16 * t + c, a.m - 1)) * 4 + g;
                    av[u][t] = ((const v4i *)a.a_codes)[ai];
                    as[u][t] = a.a_scales[ai];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (p0 + u * kRowWaves < a.k1)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(wv[u]), wide(av[u][t]), acc[t], kFp4, kFp4,
                                                                             0, ws[u], 0, as[u][t]);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[w][t * 256 + c * 16 + 4 * g + i] = acc[t][i];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * 256; t += 64 * kRowWaves) {
        float f = 0.0f;
#pragma unroll
        for (int i = 0; i < kRowWaves; ++i) f += part[i][t];
        const int m = m0 + (t >> 4), n = n0 + (t & 15);
        if (m < a.m && n < a.n) {
            if (a.bias) f += a.bias[n];
            if (a.res) f += load_any(a.res, a.type, (long long)m * a.ld_res + n);
            with_act(a.act, [&](auto act) { store_any(a.y, a.type, (long long)m * a.ld_y + n, act_of<decltype(act)::value>(f)); });
        }
    }
}

template <int MT>
void launch_rows(const Mx4Args &a, hipStream_t s)
{
    const int tiles_n = (a.n - 1) / 16 + 1;
    const dim3 grid((unsigned)(((a.m - 1) / (16 * MT) + 1) * tiles_n));
    hipLaunchKernelGGL(mx4_rows_kernel<MT>, grid, dim3(64 * kRowWaves), 0, s, a, tiles_n);
}

}  // namespace

hipError_t launch_mx4_quantize(const void *x, int type, long long ld, int rows, int k, uint8_t *codes, uint8_t *scales,
                               hipStream_t s)
{
    const int k1 = (k - 1) / 128 + 1, groups = (k1 - 1) / kQPanels + 1;
    const dim3 grid((unsigned)((rows + kQRows - 1LL) / kQRows * groups));
    const bool once = ld % 64 == 0 && ((uintptr_t)x & 127) == 0;
    auto *f = type == 0   ? mx4_quantize_kernel<0, false>
              : type == 1 ? (once ? mx4_quantize_kernel<1, true> : mx4_quantize_kernel<1, false>)
                          : (once ? mx4_quantize_kernel<2, true> : mx4_quantize_kernel<2, false>);
    hipLaunchKernelGGL(f, grid, dim3(256), 0, s, x, ld, rows, k, k1, groups, codes, scales);
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int rows, int k, void *y, int type,
                                 long long ld, hipStream_t s)
{
    const int k1 = (k - 1) / 128 + 1, groups = (k1 - 1) / kQPanels + 1;
    const dim3 grid((unsigned)((rows + kQRows - 1LL) / kQRows * groups));
    auto *f = type == 0 ? mx4_dequantize_kernel<0> : type == 1 ? mx4_dequantize_kernel<1> : mx4_dequantize_kernel<2>;
    const int past = stored_past(y, rows, ld, type == 0 ? 4 : 2);
    hipLaunchKernelGGL(f, grid, dim3(256), 0, s, codes, scales, rows, k, k1, groups, y, ld, past);
    return hipGetLastError();
}

hipError_t launch_mx4_matmul(const Mx4Args &a, hipStream_t s)
{
    // The few-rows form reads the weights once a group of 64 rows, a tile of 64 rows costs the same from
    // 1 row to 64 (us, few rows / tiles, weights from HBM): 1 x 8192 x 8192 9.8 / 17.9, 32 rows 13.9 / 18.0,
    // 64 rows 21.9 / 18.2; 64 x 4096 x 4096, one workgroup a CU, 7.2 / 8.8; 64 x 1000 x 2048 5.0 / 5.8.
    const int cus = cus_or_default();
    if (a.m > 64 || (a.m > 32 && a.n > 16 * cus) || a.n > (1 << 24)) return launch_mx4_tiles(a, s);  // (the grid)
    if (a.m <= 16)
        launch_rows<1>(a, s);
    else if (a.m <= 32)
        launch_rows<2>(a, s);
    else
        launch_rows<4>(a, s);
    return hipGetLastError();
}

}  // namespace ifx
