// Root mean square norm over rows of c values, with the residual's addition and an output of the type or in 8-bit
// codes, and its gradient:
//   h = x + residual (rounded to the type, as it is kept), rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd weight
//   d = dy weight, xhat = h rstd: dx = dh + rstd (d - xhat mean(d xhat)), dweight = sum over rows of dy xhat
// Sums are held in 32 bits and taken in one order, so results repeat bit for bit.
//
// What bounds both: memory (8192 x 8192 bf16 with the residual 99 us, 5.4 TB/s; the gradient of 16384 x 4096 with dh 99,
// 5.4).  A row stays in the registers of the TPR threads that share it (NV vectors of eight
// columns each), so every tensor crosses memory once.  Sixteen neighbouring lanes hold a block of 128 columns: the
// 8-bit form rounds out of registers, one maximum over sixteen lanes a block.
#include <type_traits>

#include "device_common.h"
#include "ifx_internal.h"
#include "lowp.h"

namespace ifx {
namespace {

constexpr int threads_of(int tpr) { return tpr > 256 ? tpr : 256; }

// Sum over the TPR threads of a row, in every one of them.  Rows wider than a wave go through `red`, one word a wave.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red)
{
    v = lanes_sum(v, TPR < 64 ? TPR : 64);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += red[i];
    }
    return v;
}

// weight's eight values from column col on, `valid` of them (1 where there is none).
__device__ __forceinline__ void load_weight(const float *weight, int col, int valid, float (&w)[8])
{
    if (weight && valid > 0) {
        const Oct<float> o = load8(weight + col, valid);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = o.get(e);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    }
}

template <int TYPE, int TPR, int NV, bool CODES>
__global__ __launch_bounds__(threads_of(TPR)) void rms_kernel(RmsArgs a)
{
    typedef typename Elem<TYPE>::type E;
    constexpr int RPB = threads_of(TPR) / TPR;
    __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
    const int row = (int)(blockIdx.x * (unsigned)RPB) + (int)(threadIdx.x / TPR), t = threadIdx.x % TPR;
    const bool live = row < a.rows;
    const long long r = live ? row : a.rows - 1;
    Oct<E> h[NV];
    {
        Oct<E> res[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (t + j * TPR) * 8;
            h[j] = col < a.c ? load8((const E *)a.x + r * a.ld_x + col, a.c - col) : Oct<E>{};
        }
        if (a.res) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (t + j * TPR) * 8;
                res[j] = col < a.c ? load8((const E *)a.res + r * a.ld_res + col, a.c - col) : Oct<E>{};
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = h[j].get(e) + res[j].get(e);
                if constexpr (sizeof(E) == 4) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[j].w[e] = __float_as_uint(f[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[j].w[e] = pack2<E>(f[2 * e], f[2 * e + 1]);
                }
            }
        }
    }
    // the sum of the squares of h * scale
    auto squares = [&](float scale) __attribute__((always_inline)) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int valid = a.c - (t + j * TPR) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = h[j].get(e) * scale;
                ss = e < valid ? fmaf(f, f, ss) : ss;
            }
        }
        return ss;
    };
    const float ss = row_sum<TPR>(squares(1.0f), red[0]);
    float rstd = 1.0f / sqrtf(ss / (float)a.c + a.eps);
    // Squares of values past 2^63 overflow: the same in units of 2^80 (where an eps of ordinary size is nothing).
    const bool over = ss > 3.4e38f;
    if (TPR > 64 ? over : __any(over)) {
        const float big = row_sum<TPR>(squares(0x1p-80f), red[1]);
        if (over) rstd = 0x1p-80f / sqrtf(big / (float)a.c + a.eps * 0x1p-80f * 0x1p-80f);
    }
    if (live && t == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (t + j * TPR) * 8, valid = a.c - col;
        float w[8], f[8];
        load_weight(a.weight, col, valid, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = h[j].get(e);
        if (a.h && live && valid > 0) {
            E *dst = (E *)a.h + r * a.ld_h + col;
            store8(dst, valid, f);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * w[e];
        if constexpr (CODES) {
            if (valid < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= valid) f[e] = 0.0f;
            }
            const unsigned s = fp8_scale<0>(row_max(top_bits(f)));
            const uint2 q = fp8_codes<0>(f, s);
            const int panel = col >> 7, v = col >> 3 & 15, k1 = (a.c + 127) >> 7;
            if (live && panel < k1) {
                ((uint2 *)a.codes)[((long long)panel * a.rows + row) * 16 + v] = q;
                if (v == 0) {
                    uint8_t *at = a.scales + ((long long)(panel >> 2) * a.rows + row) * 4;
                    at[panel & 3] = (uint8_t)s;
                    if (panel == k1 - 1)  // the word's other bytes
                        for (int b = (panel & 3) + 1; b < 4; ++b) at[b] = 0;
                }
            }
        } else if (live && valid > 0) {
            E *dst = (E *)a.y + r * a.ld_y + col;
            if (valid >= 8 && a.past) {
                keep_apart();
                store8<true>(dst, f);
                keep_apart();
            } else {
                store8(dst, valid, f);
            }
        }
    }
}

// ------------------------------------------------------------------------------------------
// Gradient.  A workgroup takes rows blockIdx, blockIdx + gridDim, ... (RPB at a time), its threads the same columns
// of each, so dweight's parts stay in registers until the end, where the workgroup's are added in LDS and written as
// one row of partial sums.  AHEAD: the next rows are requested before this one's sum is taken.
// ------------------------------------------------------------------------------------------
// A thread's vector is always eight whole columns: the last one of a ragged row begins at c - 8, and its first
// `skip` values, which are its neighbour's, are left out of the sums and not stored (c >= 8; shorter rows take
// WHOLE = false, element by element).  Partial vectors would cost as many registers again.
template <int TYPE, int TPR, int NV, bool AHEAD, bool WHOLE>
__global__ __launch_bounds__(threads_of(TPR)) void rms_grad_kernel(RmsArgs a)
{
    typedef typename Elem<TYPE>::type E;
    constexpr int T = threads_of(TPR), RPB = T / TPR;
    __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
    __shared__ float add[RPB > 1 ? (RPB - 1) * TPR * 8 : 1];
    const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;
    struct Row {
        Oct<E> dy[NV], h[NV], dh[AHEAD ? NV : 1];
        float rstd;
    };
    // first column of vector j, and how many of its values are another's (8: all)
    auto column = [&](int j) __attribute__((always_inline)) {
        const int col = (t + j * TPR) * 8;
        return WHOLE ? min(col, a.c - 8) : min(col, a.c - 1);
    };
    auto skipped = [&](int j) __attribute__((always_inline)) {
        const int col = (t + j * TPR) * 8;
        return WHOLE ? min(col - min(col, a.c - 8), 8) : col < a.c ? 0 : 8;
    };
    auto get = [&](const void *p, long long r, long long ld, int j) __attribute__((always_inline)) {
        const int col = column(j);
        const E *at = (const E *)p + r * ld + col;
        return WHOLE ? load8(at) : load8(at, a.c - col);
    };
    // whether value e of vector j is this thread's
    auto mine = [&](int j, int e) __attribute__((always_inline)) {
        return WHOLE ? e >= skipped(j) : (t + j * TPR) * 8 + e < a.c;
    };
    auto load = [&](int row, Row &o) __attribute__((always_inline)) {
        const long long r = min(row, a.rows - 1);
        o.rstd = a.rstd[r];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            o.dy[j] = get(a.dy, r, a.ld_dy, j);
            o.h[j] = get(a.x, r, a.ld_x, j);
            if constexpr (AHEAD)
                if (a.dh) o.dh[j] = get(a.dh, r, a.ld_dh, j);
        }
    };
    // the weight stays in registers too where there are some to spare
    constexpr bool KEEP = TPR <= 256 && NV <= 2;
    float dw[NV][8], kept[KEEP ? NV : 1][8];
    auto weights = [&](int j, float (&w)[8]) __attribute__((always_inline)) {
        const int col = column(j);
        load_weight(a.weight, col, WHOLE ? 8 : a.c - col, w);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if constexpr (KEEP) weights(j, kept[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    }
    const int step = (int)gridDim.x * RPB;
    const float inv_c = 1.0f / (float)a.c;
    int parity = 0;
    auto one = [&](long long row, Row &o) __attribute__((always_inline)) {
        const bool live = row < a.rows;
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float w[8];
            if constexpr (!KEEP) weights(j, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = o.dy[j].get(e), xhat = o.h[j].get(e) * o.rstd;
                if (live && mine(j, e)) {
                    dw[j][e] = fmaf(d, xhat, dw[j][e]);
                    m = fmaf(d * (KEEP ? kept[j][e] : w[e]), xhat, m);
                }
            }
            o.dy[j].forget();
            o.h[j].forget();
        }
        m = row_sum<TPR>(m, red[parity]) * inv_c;
        parity ^= 1;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int skip = skipped(j);
            if (!live || skip >= 8) continue;
            float f[8], w[8];
            if constexpr (!KEEP) weights(j, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xhat = o.h[j].get(e) * o.rstd;
                f[e] = o.rstd * fmaf(-xhat, m, o.dy[j].get(e) * (KEEP ? kept[j][e] : w[e]));
            }
            if (a.dh) {
                Oct<E> dh;
                if constexpr (AHEAD)
                    dh = o.dh[j];
                else
                    dh = get(a.dh, row, a.ld_dh, j);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] += dh.get(e);
            }
            E *dst = (E *)a.y + row * a.ld_y + column(j);
            if constexpr (WHOLE) {
                if (skip > 0) {
#pragma unroll
                    for (int e = 1; e < 8; ++e)
                        if (e >= skip) dst[e] = (E)f[e];
                } else if (a.past) {
                    keep_apart();
                    store8<true>(dst, f);
                    keep_apart();
                } else {
                    store8(dst, f);
                }
            } else {
                store8(dst, a.c - column(j), f);
            }
        }
    };
    // (every thread of the workgroup goes round as often: the first row of the workgroup decides)
    const int first = (int)blockIdx.x * RPB;
    if constexpr (AHEAD) {
        Row now, next;
        load(first + sub, now);
        for (long long r = first; r < a.rows; r += step) {
            if (r + step < a.rows) load((int)min(r + step + sub, (long long)a.rows - 1), next);
            one(r + sub, now);
            now = next;
        }
    } else {
        for (long long r = first; r < a.rows; r += step) {
            Row now;
            load((int)min(r + sub, (long long)a.rows - 1), now);
            one(r + sub, now);
        }
    }
    if (!a.part) return;
    float *const part = a.part + (long long)blockIdx.x * a.c;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if constexpr (RPB > 1) {
            __syncthreads();
            if (sub > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) add[((sub - 1) * 8 + e) * TPR + t] = dw[j][e];
            }
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int i = 0; i < RPB - 1; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[j][e] += add[(i * 8 + e) * TPR + t];
            }
        }
        if (sub == 0) {
            const int skip = skipped(j);
            if (WHOLE && skip == 0) {
                store8(part + column(j), dw[j]);
            } else if (skip < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (mine(j, e)) part[column(j) + e] = dw[j][e];
            }
        }
    }
}

// dweight out of the workgroups' rows of partial sums: 32 columns a workgroup, 32 lanes of rows, added in a fixed
// order.  Without rows (no samples) zeros.
__global__ __launch_bounds__(1024) void rms_grad_join_kernel(const float *part, int chunks, int c, float *dweight)
{
    __shared__ float add[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = (int)blockIdx.x * 32 + x;
    float f = 0.0f;
    if (col < c) {
#pragma unroll 4
        for (int i = y; i < chunks; i += 32) f += part[(long long)i * c + col];
    }
    add[y][x] = f;
    __syncthreads();
    if (y == 0 && col < c) {
        f = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) f += add[i][x];
        dweight[col] = f;
    }
}

template <int TPR, int NV>
hipError_t launch_rows(const RmsArgs &a, hipStream_t s)
{
    constexpr int RPB = threads_of(TPR) / TPR;
    auto *f = a.codes ? (a.type == 0   ? rms_kernel<0, TPR, NV, true>
                         : a.type == 1 ? rms_kernel<1, TPR, NV, true>
                                       : rms_kernel<2, TPR, NV, true>)
                      : (a.type == 0   ? rms_kernel<0, TPR, NV, false>
                         : a.type == 1 ? rms_kernel<1, TPR, NV, false>
                                       : rms_kernel<2, TPR, NV, false>);
    hipLaunchKernelGGL(f, dim3((unsigned)((a.rows - 1) / RPB + 1)), dim3(threads_of(TPR)), 0, s, a);
    return hipGetLastError();
}

// TYPES: the float32 (1) and the 16-bit (2) instances that the plan below may take.
template <int TPR, int NV, bool WHOLE = true, int TYPES = 3>
hipError_t launch_grad(const RmsArgs &a, hipStream_t s)
{
    // float32 rows past 8192 columns and any past 16384 leave no registers for a second row
    void (*f)(RmsArgs) = nullptr;
    if constexpr (TYPES & 1)
        if (a.type == 0) f = rms_grad_kernel<0, TPR, NV, (TPR * NV < 2048), WHOLE>;
    if constexpr (TYPES & 2) {
        if (a.type == 1) f = rms_grad_kernel<1, TPR, NV, (TPR * NV <= 2048), WHOLE>;
        if (a.type == 2) f = rms_grad_kernel<2, TPR, NV, (TPR * NV <= 2048), WHOLE>;
    }
    hipLaunchKernelGGL(f, dim3((unsigned)a.chunks), dim3(threads_of(TPR)), 0, s, a);
    return hipGetLastError();
}

// Threads that share a row in the gradient.  From 4097 to 8192 columns (us, 256 threads / 512 / 1024): 8192 x 8192 bf16
// 106 / 88 / 97, 3000 x 8000 float32 79 / 69 / 62.
int grad_tpr(int c, int type)
{
    return c <= 128 ? 16 : c <= 1024 ? 64 : c <= 4096 ? 256 : c <= 8192 && type != 0 ? 512 : 1024;
}

// Workgroups of the gradient: two a CU of the 256 that an MI355X has (no device is asked: this sizes the caller's
// workspace too), one where it fills the CU (4000 x 15000 bf16 98 / 91 us, two / one a CU) or half of it with few rows to
// take (700 x 8192 18.1 / 16.5; but 1517 x 510 float16 12.9 / 13.9), at most one a row (or few rows).
int grad_chunks(int rows, int c, int type)
{
    const int tpr = grad_tpr(c, type), rpb = threads_of(tpr) / tpr;
    const int groups = (rows - 1) / rpb + 1, most = tpr == 1024 || (tpr == 512 && groups < 2048) ? 256 : 512;
    return groups < most ? groups : most;
}

}  // namespace

size_t rms_workspace_bytes(int rows, int c, int type)
{
    return rows > 0 ? (size_t)grad_chunks(rows, c, type) * (size_t)c * 4 : 0;
}

hipError_t launch_rms_norm(RmsArgs a, hipStream_t s)
{
    const int cus = cus_or_default();
    // us, past the caches / cached: 8192 x 8192 bf16 49.7 / 51.3, with the residual 99.3 / 101.1; 60000 x 1024 43.6 / 45.1
    // (the gradient 68.4 / 69.2, 16384 x 4096 74.0 / 76.0)
    a.past = !a.codes && stored_past(a.y, a.rows, a.ld_y, a.type == 0 ? 4 : 2);
    // Few rows: more threads a row (us of a graph's node, to 8 bits): 1 x 8192 bf16 2.7 / 3.9, 512 x 8192 4.5 / 4.9, 512 x
    // 1000 2.7 / 3.0, 1 x 4096 2.4 / 2.7; but 512 x 4096 float32 3.9 / 3.5
    const bool few = a.rows <= (a.c <= 1024 || a.c > 4096 ? 2 * cus : cus);
    if (a.c <= 128) return launch_rows<16, 1>(a, s);
    if (a.c <= 512) return launch_rows<64, 1>(a, s);
    if (a.c <= 1024 && !few) return launch_rows<64, 2>(a, s);
    if (a.c <= 2048) return launch_rows<256, 1>(a, s);
    if (a.c <= 8192 && few) return launch_rows<1024, 1>(a, s);
    if (a.c <= 4096) return launch_rows<256, 2>(a, s);
    if (a.c <= 8192) return launch_rows<256, 4>(a, s);
    if (a.c <= 16384) return launch_rows<1024, 2>(a, s);
    return launch_rows<1024, 3>(a, s);
}

hipError_t launch_rms_norm_grad(RmsArgs a, float *dweight, hipStream_t s)
{
    if (a.rows > 0) {
        a.chunks = grad_chunks(a.rows, a.c, a.type);
        a.past = stored_past(a.y, a.rows, a.ld_y, a.type == 0 ? 4 : 2);
        if (!dweight)
            a.part = nullptr;
        else if (a.chunks == 1)
            a.part = dweight;  // the only row of partial sums
        const hipError_t e = a.c < 8        ? launch_grad<16, 1, false>(a, s)
                             : a.c <= 128   ? launch_grad<16, 1>(a, s)
                             : a.c <= 512   ? launch_grad<64, 1>(a, s)
                             : a.c <= 1024  ? launch_grad<64, 2>(a, s)
                             : a.c <= 2048  ? launch_grad<256, 1>(a, s)
                             : a.c <= 4096  ? launch_grad<256, 2>(a, s)
                             : a.c <= 8192  ? (a.type == 0 ? launch_grad<1024, 1, true, 1>(a, s) : launch_grad<512, 2, true, 2>(a, s))
                             : a.c <= 16384 ? launch_grad<1024, 2>(a, s)
                                            : launch_grad<1024, 3>(a, s);
        if (e != hipSuccess || !dweight || a.chunks == 1) return e;
    }
    if (!dweight) return hipSuccess;
    hipLaunchKernelGGL(rms_grad_join_kernel, dim3((unsigned)((a.c - 1) / 32 + 1)), dim3(1024), 0, s, a.part, a.chunks, a.c,
                       dweight);
    return hipGetLastError();
}

}  // namespace ifx
