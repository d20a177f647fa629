// Group norm with an activation over channels-last tensors, its gradient, and the form that rounds
// its result to microscaled 4-bit codes.
//
// A sample is hw pixels of c channels, channels innermost (a pixel every ld elements); group g is
// the c / groups channels from g * c / groups on.  With the mean and variance of a sample's group
// over pixels and channels:
//   xhat = (x - mean) * rstd, rstd = 1 / sqrt(var + eps), z = xhat * weight + bias, y = act(z)
//   dz = dy act'(z), dweight = sum dz xhat, dbias = sum dz, d = dz weight,
//   dx = rstd (d - mean(d) - xhat mean(d xhat))          (means over the sample's group)
// Every statistic is held in 32 bits.  Variances never come from a difference of squares: a
// thread sums squares about the mean of eight pixels that it holds in registers and joins such
// parts by their means and counts, as do threads and workgroups, always in one order.
//
// Threads take eight consecutive channels (one 16-byte access of a 16-bit type), neighbouring
// threads neighbouring channels, so a wave reads whole pixels whatever the group size; values
// of a group meet through per-channel sums in LDS, so a group may be part of a thread's eight
// channels or many threads'.
#include "device_common.h"
#include "ifx_internal.h"
#include "lowp.h"

namespace ifx {
namespace {

constexpr int kMaxC = 8192;  // channels: eight per thread, 1024 threads
constexpr int kBatch = 8;    // pixels a thread holds at once

// The thread's place: channel vector `vec` of `tcv`, pixel lane `pl` of `tp`.
struct Place {
    int tcv, tp, pl, vec;
    bool active;
};

template <int T>
__device__ __forceinline__ Place place(int tcv)
{
    Place p;
    p.tcv = tcv;
    p.tp = T / tcv;
    p.pl = (int)threadIdx.x / tcv;
    p.vec = (int)threadIdx.x - p.pl * tcv;
    p.active = p.pl < p.tp;
    return p;
}

template <int N>
__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
#pragma unroll
    for (int d = 1; d < N; d *= 2)
        if (d < lanes) v += __shfl_xor(v, d);
    return v;
}

// Sums of v over each group: out[g] for every group g, from the eight per-channel values of every
// active thread.  red: T * 8 floats.  lpg lanes (a power of two, at most 64) sum one group.
template <int T>
__device__ __forceinline__ void group_sums(const float (&v)[8], const Place &p, const GnArgs &a, float *red, float *out)
{
    if (p.active) {
#pragma unroll
        for (int e = 0; e < 8; ++e) red[((int)threadIdx.x) * 8 + e] = v[e];
    }
    __syncthreads();
    const int sub = (int)threadIdx.x & (a.lpg - 1);
    for (int g = (int)threadIdx.x / a.lpg; g < a.groups; g += T / a.lpg) {
        float s = 0.0f;
        for (int j = sub; j < p.tp * a.cg; j += a.lpg) {
            const int q = fdiv(j, a.cg_mul, a.cg_shr);
            s += red[q * p.tcv * 8 + g * a.cg + (j - q * a.cg)];
        }
        s = lanes_sum<64>(s, a.lpg);
        if (sub == 0) out[g] = s;
    }
    __syncthreads();
}

// The group of each of the thread's channels (channels past c: the last group).
__device__ __forceinline__ void groups_of(const Place &p, const GnArgs &a, int (&g)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = fdiv(min(p.vec * 8 + e, a.c - 1), a.cg_mul, a.cg_shr);
}

// Per-channel weight and bias of the thread (1 and 0 where there is none; 0 past c).
__device__ __forceinline__ void params_of(const Place &p, const GnArgs &a, float (&w)[8], float (&b)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int ch = p.vec * 8 + e;
        const bool in = ch < a.c;
        w[e] = !in ? 0.0f : a.weight ? a.weight[ch] : 1.0f;
        b[e] = !in || !a.bias ? 0.0f : a.bias[ch];
    }
}

// First half of the forward pass: mean and sum of squares about it of every group over pixels
// [chunk * px, + px) of sample blockIdx.x / chunks, to ws[sample][chunk][group][2].
template <int T, int TYPE>
__global__ __launch_bounds__(T) void gn_stats_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float red[T * 8], gs[T * 8];
    const int n = (int)(blockIdx.x / (unsigned)a.chunks), k = (int)(blockIdx.x - (unsigned)n * (unsigned)a.chunks);
    const int p0 = k * a.px, p1 = min(a.hw, p0 + a.px);
    const Place p = place<T>((a.c + 7) / 8);
    const E *src = (const E *)a.x + (long long)n * a.hw * a.ld_x + p.vec * 8;
    const int valid = a.c - p.vec * 8;
    int cnt = 0;
    float mean[8] = {}, m2[8] = {};
    if (p.active) {
        for (int q = p0 + p.pl; q < p1; q += kBatch * p.tp) {
            float f[kBatch][8];
            int have = 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const bool in = q + i * p.tp < p1;
                E raw[8];
                load8(src + (long long)(in ? q + i * p.tp : q) * a.ld_x, valid, raw);
                have += in;
#pragma unroll
                for (int e = 0; e < 8; ++e) f[i][e] = (float)raw[e];
            }
            const float inv = 1.0f / (float)have, part = (float)have / (float)(cnt + have), both = (float)cnt * part;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float s = 0.0f, s2 = 0.0f;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) s += i < have ? f[i][e] : 0.0f;
                const float m = s * inv;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float d = i < have ? f[i][e] - m : 0.0f;
                    s2 += d * d;
                }
                const float d = m - mean[e];
                mean[e] += d * part;
                m2[e] += s2 + d * d * both;
            }
            cnt += have;
        }
    }
    int g[8];
    groups_of(p, a, g);
    const float total = (float)(p1 - p0) * (float)a.cg;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)cnt * mean[e];
    group_sums<T>(v, p, a, red, gs);
    float *out = a.ws + (long long)blockIdx.x * a.groups * 2;
    for (int i = threadIdx.x; i < a.groups; i += T) out[2 * i] = gs[i] / total;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float d = mean[e] - gs[g[e]] / total;
        v[e] = m2[e] + (float)cnt * d * d;
    }
    __syncthreads();
    group_sums<T>(v, p, a, red, gs);
    for (int i = threadIdx.x; i < a.groups; i += T) out[2 * i + 1] = gs[i];
}

// Joins the chunks' statistics of sample n: smean[g], srstd[g].
template <int T>
__device__ __forceinline__ void join_stats(const GnArgs &a, int n, float *smean, float *srstd)
{
    const float *ws = a.ws + (long long)n * a.chunks * a.groups * 2;
    const float total = (float)a.hw * (float)a.cg;
    const int sub = (int)threadIdx.x & (a.lpg - 1);
    for (int g = (int)threadIdx.x / a.lpg; g < a.groups; g += T / a.lpg) {
        float s = 0.0f;
        for (int k = sub; k < a.chunks; k += a.lpg)
            s += ws[((long long)k * a.groups + g) * 2] * ((float)(min(a.hw, (k + 1) * a.px) - k * a.px) * (float)a.cg);
        const float mean = lanes_sum<64>(s, a.lpg) / total;
        s = 0.0f;
        for (int k = sub; k < a.chunks; k += a.lpg) {
            const float d = ws[((long long)k * a.groups + g) * 2] - mean;
            s += ws[((long long)k * a.groups + g) * 2 + 1] +
                 d * d * ((float)(min(a.hw, (k + 1) * a.px) - k * a.px) * (float)a.cg);
        }
        const float var = lanes_sum<64>(s, a.lpg) / total;
        if (sub == 0) {
            smean[g] = mean;
            srstd[g] = 1.0f / sqrtf(var + a.eps);
        }
    }
    __syncthreads();
}

// Second half of the forward pass: the chunks joined, then each pixel normalised.  MX4: rounded to
// codes instead; threads then also cover the columns up to the next multiple of 128.
template <int T, int TYPE, bool MX4>
__global__ __launch_bounds__(T) void gn_apply_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float smean[T * 8], srstd[T * 8];
    const int n = (int)(blockIdx.x / (unsigned)a.chunks), k = (int)(blockIdx.x - (unsigned)n * (unsigned)a.chunks);
    const int p0 = k * a.px, p1 = min(a.hw, p0 + a.px);
    join_stats<T>(a, n, smean, srstd);
    if (k == 0)
        for (int i = threadIdx.x; i < a.groups; i += T) {
            if (a.mean) a.mean[(long long)n * a.groups + i] = smean[i];
            if (a.rstd) a.rstd[(long long)n * a.groups + i] = srstd[i];
        }
    const Place p = place<T>(MX4 ? (a.c + 127) / 128 * 16 : (a.c + 7) / 8);
    if (!p.active) return;
    float w[8], b[8], m[8];
    params_of(p, a, w, b);
    int g[8];
    groups_of(p, a, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m[e] = smean[g[e]];
        w[e] *= srstd[g[e]];
    }
    const int valid = a.c - p.vec * 8;
    const E *src = (const E *)a.x + (long long)n * a.hw * a.ld_x + (valid > 0 ? p.vec * 8 : 0);
    for (int q = p0 + p.pl; q < p1; q += p.tp) {
        E raw[8];
        load8(src + (long long)q * a.ld_x, valid, raw);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = act_any(a.act, ((float)raw[e] - m[e]) * w[e] + b[e]);
        const long long row = (long long)n * a.hw + q;
        if (MX4) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= valid) f[e] = 0.0f;
            unsigned s;
            const unsigned r = mx4_codes(f, s);
            const long long at = (long long)(p.vec >> 4) * a.n * a.hw + row;
            ((unsigned *)a.codes)[at * 16 + (p.vec & 15)] = r;
            if ((p.vec & 3) == 0) a.scales[at * 4 + ((p.vec & 15) >> 2)] = (uint8_t)s;
        } else {
            store8((E *)a.y + row * a.ld_y + p.vec * 8, valid, f);
        }
    }
}

// dz and xhat of one value.  z takes the operations of its formula one at a time, unfused, so that the
// side of a ReLU's corner on which a value lies is the formula's own.
__device__ __forceinline__ float grad_of(int act, float xv, float dy, float mean, float rstd, float w, float b,
                                         float &xhat)
{
#pragma clang fp contract(off)
    xhat = (xv - mean) * rstd;
    const float z = xhat * w + b;
    if (act == 1) return z > 0.0f ? dy : 0.0f;
    if (act == 2) {
        const float s = sigmoid(z);
        return dy * (s * (1.0f + z * (1.0f - s)));
    }
    return dy;
}

// First half of the gradient: per-channel sums of dz xhat and dz over a chunk's pixels, to
// ws[sample][chunk][2][c], and each group's sums of d xhat and d, to gsum[sample][chunk][group][2].
template <int T, int TYPE>
__global__ __launch_bounds__(T) void gn_grad_sums_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float red[T * 8], gs[T * 8];
    const int n = (int)(blockIdx.x / (unsigned)a.chunks), k = (int)(blockIdx.x - (unsigned)n * (unsigned)a.chunks);
    const int p0 = k * a.px, p1 = min(a.hw, p0 + a.px);
    const Place p = place<T>((a.c + 7) / 8);
    const int valid = a.c - p.vec * 8;
    float s1[8] = {}, s2[8] = {}, w[8] = {};
    if (p.active) {
        const long long first = (long long)n * a.hw;
        const E *src = (const E *)a.x + first * a.ld_x + p.vec * 8, *dsrc = (const E *)a.dy + first * a.ld_dy + p.vec * 8;
        float b[8], m[8], r[8];
        params_of(p, a, w, b);
        int g[8];
        groups_of(p, a, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m[e] = a.mean[(long long)n * a.groups + g[e]];
            r[e] = a.rstd[(long long)n * a.groups + g[e]];
        }
        for (int q = p0 + p.pl; q < p1; q += p.tp) {
            E raw[8], draw[8];
            load8(src + (long long)q * a.ld_x, valid, raw);
            load8(dsrc + (long long)q * a.ld_dy, valid, draw);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float xhat;
                const float dz = grad_of(a.act, (float)raw[e], (float)draw[e], m[e], r[e], w[e], b[e], xhat);
                s1[e] += dz * xhat;
                s2[e] += dz;
            }
        }
    }
    float *out = a.ws + (long long)blockIdx.x * a.c * 2, *gout = a.gsum + (long long)blockIdx.x * a.groups * 2;
    float v[8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (half ? s2[e] : s1[e]);
        // channel sums over the pixel lanes
        if (p.active) {
#pragma unroll
            for (int e = 0; e < 8; ++e) red[(int)threadIdx.x * 8 + e] = v[e];
        }
        __syncthreads();
        for (int ch = threadIdx.x; ch < a.c; ch += T) {
            float s = 0.0f;
            for (int q = 0; q < p.tp; ++q) s += red[q * p.tcv * 8 + ch];
            out[half * a.c + ch] = s;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= w[e];
        group_sums<T>(v, p, a, red, gs);
        for (int i = threadIdx.x; i < a.groups; i += T) gout[2 * i + half] = gs[i];
        __syncthreads();
    }
}

// Second half: dx from the group's joined sums.
template <int T, int TYPE>
__global__ __launch_bounds__(T) void gn_grad_apply_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float g1[T * 8], g2[T * 8];
    const int n = (int)(blockIdx.x / (unsigned)a.chunks), k = (int)(blockIdx.x - (unsigned)n * (unsigned)a.chunks);
    const int p0 = k * a.px, p1 = min(a.hw, p0 + a.px);
    {
        const float *gsum = a.gsum + (long long)n * a.chunks * a.groups * 2;
        const float inv = 1.0f / ((float)a.hw * (float)a.cg);
        const int sub = (int)threadIdx.x & (a.lpg - 1);
        for (int g = (int)threadIdx.x / a.lpg; g < a.groups; g += T / a.lpg) {
            float x1 = 0.0f, x2 = 0.0f;
            for (int i = sub; i < a.chunks; i += a.lpg) {
                x1 += gsum[((long long)i * a.groups + g) * 2];
                x2 += gsum[((long long)i * a.groups + g) * 2 + 1];
            }
            x1 = lanes_sum<64>(x1, a.lpg);
            x2 = lanes_sum<64>(x2, a.lpg);
            if (sub == 0) {
                g1[g] = x1 * inv;
                g2[g] = x2 * inv;
            }
        }
        __syncthreads();
    }
    const Place p = place<T>((a.c + 7) / 8);
    if (!p.active) return;
    const int valid = a.c - p.vec * 8;
    const long long first = (long long)n * a.hw;
    const E *src = (const E *)a.x + first * a.ld_x + p.vec * 8, *dsrc = (const E *)a.dy + first * a.ld_dy + p.vec * 8;
    E *dst = (E *)a.y + first * a.ld_y + p.vec * 8;
    float w[8], b[8], m[8], r[8], c1[8], c2[8];
    params_of(p, a, w, b);
    int g[8];
    groups_of(p, a, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        m[e] = a.mean[(long long)n * a.groups + g[e]];
        r[e] = a.rstd[(long long)n * a.groups + g[e]];
        c1[e] = g1[g[e]];
        c2[e] = g2[g[e]];
    }
    for (int q = p0 + p.pl; q < p1; q += p.tp) {
        E raw[8], draw[8];
        load8(src + (long long)q * a.ld_x, valid, raw);
        load8(dsrc + (long long)q * a.ld_dy, valid, draw);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float xhat;
            const float dz = grad_of(a.act, (float)raw[e], (float)draw[e], m[e], r[e], w[e], b[e], xhat);
            f[e] = r[e] * (dz * w[e] - c2[e] - xhat * c1[e]);
        }
        store8(dst + (long long)q * a.ld_y, valid, f);
    }
}

// dweight and dbias: columns of the per-chunk sums [rows][2 c] added up, 32 columns and 32 row
// lanes per workgroup, in one order.
__global__ __launch_bounds__(1024) void gn_grad_join_kernel(const float *ws, int rows, int c, float *dweight,
                                                            float *dbias)
{
    __shared__ float part[32][33];
    const int col = (int)blockIdx.x * 32 + ((int)threadIdx.x & 31), r0 = (int)threadIdx.x >> 5;
    float s = 0.0f;
    if (col < 2 * c)
        for (int r = r0; r < rows; r += 32) s += ws[(long long)r * 2 * c + col];
    part[r0][threadIdx.x & 31] = s;
    __syncthreads();
    if (threadIdx.x < 32 && col < 2 * c) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
        float *out = col < c ? dweight : dbias;
        if (out) out[col < c ? col : col - c] = s;
    }
}

// Threads of a workgroup and pixels of a chunk: a chunk gives every thread at least one batch,
// and there are about 2048 workgroups where the work allows it.
struct Plan {
    int threads, chunks, px;
};

Plan plan_split(int n, int hw, int c)
{
    Plan p;
    p.threads = c <= 2048 ? 256 : 1024;
    const int tp = p.threads / ((c + 7) / 8);
    const int most = (hw + kBatch * tp - 1) / (kBatch * tp);
    const int want = n > 0 ? (2048 + n - 1) / n : 1;
    int chunks = want < most ? want : most;
    if (chunks > 256) chunks = 256;
    if (chunks < 1) chunks = 1;
    p.px = (hw + chunks - 1) / chunks;
    p.chunks = (hw + p.px - 1) / p.px;
    return p;
}

void fill(GnArgs &a, const Plan &p)
{
    a.chunks = p.chunks;
    a.px = p.px;
    a.cg = a.c / a.groups;
    fastdiv_magic((unsigned)a.cg, &a.cg_mul, &a.cg_shr);
    a.lpg = 1;
    while (a.lpg < 64 && a.lpg * 2 * a.groups <= p.threads) a.lpg *= 2;
}

#define IFX_GN_TYPES(kernel, T, ...)                                                            \
    (a.type == 0 ? kernel<T, 0, ##__VA_ARGS__> : a.type == 1 ? kernel<T, 1, ##__VA_ARGS__> : kernel<T, 2, ##__VA_ARGS__>)

}  // namespace

size_t gn_workspace_bytes(int n, int hw, int c, int groups, bool grad)
{
    const Plan p = plan_split(n, hw, c);
    const size_t rows = (size_t)n * p.chunks;
    return rows * 4 * 2 * ((size_t)groups + (grad ? (size_t)c : 0));
}

bool gn_supported(int n, int hw, int c)
{
    if (c > kMaxC) return false;
    const Plan p = plan_split(n, hw, c);
    return (long long)n * p.chunks * p.threads <= 0xffffffffLL;
}

hipError_t launch_group_norm(GnArgs a, hipStream_t s)
{
    const Plan p = plan_split(a.n, a.hw, a.c);
    fill(a, p);
    const dim3 grid((unsigned)(a.n * p.chunks)), block((unsigned)p.threads);
    const bool mx4 = a.codes != nullptr;
    if (p.threads == 256) {
        hipLaunchKernelGGL(IFX_GN_TYPES(gn_stats_kernel, 256), grid, block, 0, s, a);
        if (mx4)
            hipLaunchKernelGGL(IFX_GN_TYPES(gn_apply_kernel, 256, true), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL(IFX_GN_TYPES(gn_apply_kernel, 256, false), grid, block, 0, s, a);
    } else {
        hipLaunchKernelGGL(IFX_GN_TYPES(gn_stats_kernel, 1024), grid, block, 0, s, a);
        if (mx4)
            hipLaunchKernelGGL(IFX_GN_TYPES(gn_apply_kernel, 1024, true), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL(IFX_GN_TYPES(gn_apply_kernel, 1024, false), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_group_norm_grad(GnArgs a, float *dweight, float *dbias, hipStream_t s)
{
    const Plan p = plan_split(a.n, a.hw, a.c);
    fill(a, p);
    const int rows = a.n * p.chunks;
    const dim3 grid((unsigned)rows), block((unsigned)p.threads);
    a.gsum = a.ws + (size_t)rows * a.c * 2;
    if (rows > 0) {
        if (p.threads == 256) {
            hipLaunchKernelGGL(IFX_GN_TYPES(gn_grad_sums_kernel, 256), grid, block, 0, s, a);
            hipLaunchKernelGGL(IFX_GN_TYPES(gn_grad_apply_kernel, 256), grid, block, 0, s, a);
        } else {
            hipLaunchKernelGGL(IFX_GN_TYPES(gn_grad_sums_kernel, 1024), grid, block, 0, s, a);
            hipLaunchKernelGGL(IFX_GN_TYPES(gn_grad_apply_kernel, 1024), grid, block, 0, s, a);
        }
    }
    if (dweight || dbias)
        hipLaunchKernelGGL(gn_grad_join_kernel, dim3((unsigned)((2 * a.c + 31) / 32)), dim3(1024), 0, s, a.ws, rows, a.c,
                           dweight, dbias);
    return hipGetLastError();
}

}  // namespace ifx
