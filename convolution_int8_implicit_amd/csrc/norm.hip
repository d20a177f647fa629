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
                const Oct<E> raw = load8(src + (long long)(in ? q + i * p.tp : q) * a.ld_x, valid);
                have += in;
#pragma unroll
                for (int e = 0; e < 8; ++e) f[i][e] = raw.get(e);
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
        const Oct<E> raw = load8(src + (long long)q * a.ld_x, valid);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = act_any(a.act, (raw.get(e) - m[e]) * w[e] + b[e]);
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
            const Oct<E> raw = load8(src + (long long)q * a.ld_x, valid);
            const Oct<E> draw = load8(dsrc + (long long)q * a.ld_dy, valid);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float xhat;
                const float dz = grad_of(a.act, raw.get(e), draw.get(e), m[e], r[e], w[e], b[e], xhat);
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
        const Oct<E> raw = load8(src + (long long)q * a.ld_x, valid);
        const Oct<E> draw = load8(dsrc + (long long)q * a.ld_dy, valid);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float xhat;
            const float dz = grad_of(a.act, raw.get(e), draw.get(e), m[e], r[e], w[e], b[e], xhat);
            f[e] = r[e] * (dz * w[e] - c2[e] - xhat * c1[e]);
        }
        store8(dst + (long long)q * a.ld_y, valid, f);
    }
}

// ------------------------------------------------------------------------------------------
// A whole slab at once: a workgroup keeps all pixels of a span of groups in registers, so x is read once
// and each of the two passes of a variance is exact.
// ------------------------------------------------------------------------------------------

// The span's groups and channels of a workgroup, and its sample.  XCD x (blockIdx & 7) owns a run
// of (sample, span) pairs, spans innermost: spans that share 128-byte lines meet in one L2.
struct Slab {
    int n, g0, ng, c0, cs;  // sample, first group, groups, first channel, channels
    bool live;
};

__device__ __forceinline__ Slab slab_of(const GnArgs &a)
{
    Slab s;
    const int i = (int)(blockIdx.x >> 3), id = (int)(blockIdx.x & 7u) * a.per_xcd + i;
    s.live = i < a.per_xcd && id < a.n * a.spans;
    s.n = id / a.spans;
    const int span = id - s.n * a.spans;
    s.g0 = span * a.gs;
    s.ng = min(a.gs, a.groups - s.g0);
    s.c0 = s.g0 * a.cg;
    s.cs = s.ng * a.cg;
    return s;
}

// Per-group values of the thread's eight channels.  VEC: cg is a multiple of 8, so they are one group's
// and one register serves all eight.
template <bool VEC>
struct PerGroup {
    float v[VEC ? 1 : 8];
    __device__ __forceinline__ float get(int e) const { return v[VEC ? 0 : e]; }
    // f(slab's group of channel ch of the slab) for the thread's channels (past the span: the last group)
    template <typename F>
    __device__ __forceinline__ void set(const Place &p, const Slab &s, const GnArgs &a, F f)
    {
#pragma unroll
        for (int e = 0; e < (VEC ? 1 : 8); ++e) v[e] = f(fdiv(min(p.vec * 8 + e, s.cs - 1), a.cg_mul, a.cg_shr));
    }
};

// Sums over each group of the slab of the thread's per-channel values v (VEC: their sum in v[0]); values of
// channels past the span are not looked at.  out[g] for the slab's groups.
template <int T, bool VEC>
__device__ __forceinline__ void slab_sums(const float *v, const Place &p, const Slab &s, const GnArgs &a, float *red,
                                          float *out)
{
    const int sub = (int)threadIdx.x & (a.lpg - 1);
    // a group's values of a pixel lane: cg / 8 threads' or cg channels
    const int per = VEC ? a.cg / 8 : a.cg, width = VEC ? p.tcv : p.tcv * 8;
    const unsigned mul = VEC ? a.cgv_mul : a.cg_mul;
    const int shr = VEC ? a.cgv_shr : a.cg_shr;
#pragma unroll
    for (int e = 0; e < (VEC ? 1 : 8); ++e) red[threadIdx.x * (VEC ? 1 : 8) + e] = v[e];
    __syncthreads();
    for (int g = (int)threadIdx.x / a.lpg; g < s.ng; g += T / a.lpg) {
        float f = 0.0f;
        for (int j = sub; j < p.tp * per; j += a.lpg) {
            const int q = fdiv(j, mul, shr);
            f += red[q * width + g * per + (j - q * per)];
        }
        f = lanes_sum<64>(f, a.lpg);
        if (sub == 0) out[g] = f;
    }
    __syncthreads();
}

__device__ __forceinline__ void slab_params(const Place &p, const Slab &s, const GnArgs &a, float (&w)[8], float (&b)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int ch = p.vec * 8 + e;
        const bool in = ch < s.cs;
        w[e] = !in ? 0.0f : a.weight ? a.weight[s.c0 + ch] : 1.0f;
        b[e] = !in || !a.bias ? 0.0f : a.bias[s.c0 + ch];
    }
}

template <int T, int NV, int TYPE, bool MX4, bool VEC>
__global__ __launch_bounds__(T, T / 256) void gn_slab_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    constexpr int LDS = T * (VEC ? 1 : 8);
    __shared__ float red[LDS], gs[LDS];
    const Slab s = slab_of(a);
    if (!s.live) return;
    // the last span of a 4-bit result also covers the columns up to the next multiple of 128
    const bool last = MX4 && s.c0 + s.cs == a.c;
    const Place p = place<T>(last ? (a.c + 127) / 128 * 16 - s.c0 / 8 : (s.cs + 7) / 8);
    const int valid = s.cs - p.vec * 8;
    const long long first = (long long)s.n * a.hw;
    const E *src = (const E *)a.x + first * a.ld_x + s.c0 + (valid > 0 ? p.vec * 8 : 0);
    Oct<E> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int q = p.pl + i * p.tp;
        const bool in = p.active && q < a.hw;
        raw[i] = load8(src + (long long)(in ? q : 0) * a.ld_x, in ? valid : 0);
    }
    float v[VEC ? 1 : 8] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float t = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (VEC)
                t += raw[i].get(e);
            else
                v[e % (VEC ? 1 : 8)] += raw[i].get(e);
        }
        if (VEC) v[0] += t;
        raw[i].forget();
    }
    const float total = (float)a.hw * (float)a.cg;
    slab_sums<T, VEC>(v, p, s, a, red, gs);
    PerGroup<VEC> m;
    m.set(p, s, a, [&](int g) { return gs[g] / total; });
    if (a.mean)
        for (int i = threadIdx.x; i < s.ng; i += T) a.mean[(long long)s.n * a.groups + s.g0 + i] = gs[i] / total;
#pragma unroll
    for (int e = 0; e < (VEC ? 1 : 8); ++e) v[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (p.pl + i * p.tp < a.hw) {
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = raw[i].get(e) - m.get(e);
                if (VEC)
                    t += d * d;
                else
                    v[e % (VEC ? 1 : 8)] += d * d;
            }
            if (VEC) v[0] += t;
        }
        raw[i].forget();
    }
    __syncthreads();
    slab_sums<T, VEC>(v, p, s, a, red, gs);
    if (a.rstd)
        for (int i = threadIdx.x; i < s.ng; i += T)
            a.rstd[(long long)s.n * a.groups + s.g0 + i] = 1.0f / sqrtf(gs[i] / total + a.eps);
    if (!p.active) return;
    float w[8], b[8];
    slab_params(p, s, a, w, b);
    PerGroup<VEC> r;
    r.set(p, s, a, [&](int g) { return 1.0f / sqrtf(gs[g] / total + a.eps); });
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= r.get(e);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int q = p.pl + i * p.tp;
        if (q >= a.hw) break;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = act_any(a.act, (raw[i].get(e) - m.get(e)) * w[e] + b[e]);
        if (MX4) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= valid) f[e] = 0.0f;
            unsigned sc;
            const unsigned code = mx4_codes(f, sc);
            const int vec = s.c0 / 8 + p.vec;
            const long long at = (long long)(vec >> 4) * a.n * a.hw + first + q;
            ((unsigned *)a.codes)[at * 16 + (vec & 15)] = code;
            if ((vec & 3) == 0) a.scales[at * 4 + ((vec & 15) >> 2)] = (uint8_t)sc;
        } else {
            store8((E *)a.y + (first + q) * a.ld_y + s.c0 + p.vec * 8, valid, f);
        }
    }
}

// The gradient of a slab: x and dy in registers, per-channel sums of dz xhat and dz over the pixels
// to ws[sample][2][c], the groups' sums from those, then dx.
template <int T, int NV, int TYPE, bool VEC>
__global__ __launch_bounds__(T, T / 256) void gn_grad_slab_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float red[T * 16], part[T], gs[2][T * (VEC ? 1 : 8)];
    const Slab s = slab_of(a);
    if (!s.live) return;
    const Place p = place<T>((s.cs + 7) / 8);
    const int valid = s.cs - p.vec * 8;
    const long long first = (long long)s.n * a.hw;
    const E *src = (const E *)a.x + first * a.ld_x + s.c0 + p.vec * 8;
    const E *dsrc = (const E *)a.dy + first * a.ld_dy + s.c0 + p.vec * 8;
    Oct<E> raw[NV], draw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int q = p.pl + i * p.tp;
        const bool in = p.active && q < a.hw;
        raw[i] = load8(src + (long long)(in ? q : 0) * a.ld_x, in ? valid : 0);
        draw[i] = load8(dsrc + (long long)(in ? q : 0) * a.ld_dy, in ? valid : 0);
    }
    const long long stat = (long long)s.n * a.groups + s.g0;
    const int width = p.tcv * 8, items = 2 * width;
    {
        float w[8], b[8], s1[8] = {}, s2[8] = {};
        slab_params(p, s, a, w, b);
        PerGroup<VEC> m, r;
        m.set(p, s, a, [&](int g) { return a.mean[stat + g]; });
        r.set(p, s, a, [&](int g) { return a.rstd[stat + g]; });
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p.pl + i * p.tp < a.hw) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float xhat;
                    const float dz = grad_of(a.act, raw[i].get(e), draw[i].get(e), m.get(e), r.get(e), w[e], b[e], xhat);
                    s1[e] += dz * xhat;
                    s2[e] += dz;
                }
            }
            raw[i].forget();
            draw[i].forget();
        }
        // channel sums over the pixel lanes: item (half, channel), `parts` threads each
        if (p.active) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                red[p.pl * items + p.vec * 8 + e] = s1[e];
                red[p.pl * items + width + p.vec * 8 + e] = s2[e];
            }
        }
    }
    __syncthreads();
    float *sums = red;  // [2][width]
    if (items <= T) {
        const int parts = T / items, at = (int)threadIdx.x / items, item = (int)threadIdx.x - at * items;
        float f = 0.0f;
        if (at < parts)
            for (int q = at; q < p.tp; q += parts) f += red[q * items + item];
        part[threadIdx.x] = f;
        __syncthreads();
        if ((int)threadIdx.x < items) {
            f = 0.0f;
            for (int q = 0; q < parts; ++q) f += part[q * items + threadIdx.x];
            sums[threadIdx.x] = f;
        }
    } else {
        for (int item = threadIdx.x; item < items; item += T) {
            float f = 0.0f;
            for (int q = 0; q < p.tp; ++q) f += red[q * items + item];
            sums[item] = f;  // row 0 of this very item: no other thread reads it
        }
    }
    __syncthreads();
    float *out = a.ws + (long long)s.n * a.c * 2 + s.c0;
    for (int i = threadIdx.x; i < 2 * s.cs; i += T) {
        const int half = i >= s.cs, ch = i - half * s.cs;
        out[(long long)half * a.c + ch] = sums[half * width + ch];
    }
    // group sums of d xhat and d
    const int sub = (int)threadIdx.x & (a.lpg - 1);
    const float inv = 1.0f / ((float)a.hw * (float)a.cg);
    for (int j = (int)threadIdx.x / a.lpg; j < 2 * s.ng; j += T / a.lpg) {
        const int half = j >= s.ng, gg = j - half * s.ng;
        float f = 0.0f;
        for (int ch = gg * a.cg + sub; ch < (gg + 1) * a.cg; ch += a.lpg)
            f += sums[half * width + ch] * (a.weight ? a.weight[s.c0 + ch] : 1.0f);
        f = lanes_sum<64>(f, a.lpg);
        if (sub == 0) gs[half][gg] = f * inv;
    }
    __syncthreads();
    if (!p.active) return;
    float w[8], b[8];  // read again: kept across the sums they would cost registers that the slab needs
    slab_params(p, s, a, w, b);
    PerGroup<VEC> m, r, c1, c2;
    m.set(p, s, a, [&](int g) { return a.mean[stat + g]; });
    r.set(p, s, a, [&](int g) { return a.rstd[stat + g]; });
    c1.set(p, s, a, [&](int g) { return gs[0][g]; });
    c2.set(p, s, a, [&](int g) { return gs[1][g]; });
    E *dst = (E *)a.y + first * a.ld_y + s.c0 + p.vec * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int q = p.pl + i * p.tp;
        if (q >= a.hw) break;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float xhat;
            const float dz = grad_of(a.act, raw[i].get(e), draw[i].get(e), m.get(e), r.get(e), w[e], b[e], xhat);
            f[e] = r.get(e) * (dz * w[e] - c2.get(e) - xhat * c1.get(e));
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

// How a call runs.  threads = 0: not supported.
struct Plan {
    int threads;
    int nv, gs, spans;  // resident: vectors per thread, groups of a span, spans; nv = 0: split
    int chunks, px;     // split: chunks of a sample and their pixels
};

// Split: a chunk gives every thread at least one batch, and there are about 2048 workgroups where the
// work allows it.
Plan plan_split(int n, int hw, int c)
{
    Plan p = {};
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

// The threads and vectors per thread of the slab kernels, by rising capacity.
struct Variant {
    int threads, nv;
};
constexpr Variant kSlab[] = {{256, 2}, {256, 8}, {1024, 4}, {1024, 8}, {1024, 16}};
constexpr Variant kGradSlab[] = {{256, 2}, {256, 4}, {1024, 2}, {1024, 4}, {1024, 8}};

// Resident where a span of whole groups that reads at least 128 (else 64, else 32) bytes of a pixel fits the
// registers of a workgroup.  A 4-bit result needs spans of whole blocks of 32 columns.
Plan plan(int n, int hw, int c, int groups, int type, bool grad, bool mx4)
{
    const int cg = c / groups, bytes = type == 0 ? 4 : 2;
    // registers for raw values: 64 of a thread's 128, half where a channel's group takes registers of its own
    int most = (type == 0 ? 8 : 16) / (grad ? 2 : 1);
    if (cg % 8 && (type != 0 || grad)) most /= 2;
    for (int least = 128; least >= 32; least /= 2)
        for (int gs = 1; gs <= groups; ++gs) {
            if (groups % gs) continue;
            const int cs = gs * cg;
            if (cs * bytes < least && gs < groups) continue;
            if (mx4 && cs % 32 && gs < groups) continue;
            // a last span of 4-bit codes is padded to whole panels
            const int tcv = mx4 ? (cs + 7) / 8 + 15 : (cs + 7) / 8;
            for (const Variant &v : grad ? kGradSlab : kSlab) {
                if (v.nv > most || tcv > v.threads || (long long)v.threads / tcv * v.nv < hw) continue;
                if (n > 0 && (long long)n * (groups / gs) * v.threads > 0x7fffffffLL) continue;
                Plan p = {};
                p.threads = v.threads;
                p.nv = v.nv;
                p.gs = gs;
                p.spans = groups / gs;
                return p;
            }
            break;  // a wider span fits no better
        }
    return plan_split(n, hw, c);
}

void fill(GnArgs &a, const Plan &p)
{
    a.cg = a.c / a.groups;
    fastdiv_magic((unsigned)a.cg, &a.cg_mul, &a.cg_shr);
    fastdiv_magic((unsigned)(a.cg / 8 > 0 ? a.cg / 8 : 1), &a.cgv_mul, &a.cgv_shr);
    a.chunks = p.chunks;
    a.px = p.px;
    a.gs = p.gs;
    a.spans = p.spans;
    a.per_xcd = (a.n * p.spans + 7) / 8;
    const int sums = p.nv ? p.gs : a.groups;
    a.lpg = 1;
    while (a.lpg < 64 && a.lpg * 2 * sums <= p.threads) a.lpg *= 2;
}

#define IFX_GN_TYPES(kernel, T, ...)                                                            \
    (a.type == 0 ? kernel<T, 0, ##__VA_ARGS__> : a.type == 1 ? kernel<T, 1, ##__VA_ARGS__> : kernel<T, 2, ##__VA_ARGS__>)

typedef void (*GnKernel)(GnArgs);

template <int T, int NV, bool MX4, bool VEC>
GnKernel slab_kernel(int type)
{
    if constexpr (NV <= 8)
        if (type == 0) return gn_slab_kernel<T, NV, 0, MX4, VEC>;
    return type == 1 ? gn_slab_kernel<T, NV, 1, MX4, VEC> : gn_slab_kernel<T, NV, 2, MX4, VEC>;
}

template <bool MX4, bool VEC>
GnKernel slab_kernel_of(const Plan &p, int type)
{
    if (p.threads == 256)
        return p.nv == 2 ? slab_kernel<256, 2, MX4, VEC>(type) : slab_kernel<256, 8, MX4, VEC>(type);
    if constexpr (VEC)
        if (p.nv == 16) return slab_kernel<1024, 16, MX4, VEC>(type);
    return p.nv == 4 ? slab_kernel<1024, 4, MX4, VEC>(type) : slab_kernel<1024, 8, MX4, VEC>(type);
}

template <int T, int NV, bool VEC>
GnKernel grad_slab_kernel(int type)
{
    if constexpr (NV <= (VEC ? 4 : 2))
        if (type == 0) return gn_grad_slab_kernel<T, NV, 0, VEC>;
    return type == 1 ? gn_grad_slab_kernel<T, NV, 1, VEC> : gn_grad_slab_kernel<T, NV, 2, VEC>;
}

template <bool VEC>
GnKernel grad_slab_kernel_of(const Plan &p, int type)
{
    if (p.threads == 256) return p.nv == 2 ? grad_slab_kernel<256, 2, VEC>(type) : grad_slab_kernel<256, 4, VEC>(type);
    if constexpr (VEC)
        if (p.nv == 8) return grad_slab_kernel<1024, 8, VEC>(type);
    return p.nv == 2 ? grad_slab_kernel<1024, 2, VEC>(type) : grad_slab_kernel<1024, 4, VEC>(type);
}

}  // namespace

size_t gn_workspace_bytes(int n, int hw, int c, int groups, int type, bool grad, bool mx4)
{
    const Plan p = plan(n, hw, c, groups, type, grad, mx4);
    if (p.nv) return grad ? (size_t)n * 2 * c * 4 : 0;
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
    const bool mx4 = a.codes != nullptr;
    const Plan p = plan(a.n, a.hw, a.c, a.groups, a.type, false, mx4);
    fill(a, p);
    const dim3 block((unsigned)p.threads);
    if (p.nv) {
        const bool vec = a.cg % 8 == 0;
        GnKernel f = mx4 ? (vec ? slab_kernel_of<true, true>(p, a.type) : slab_kernel_of<true, false>(p, a.type))
                         : (vec ? slab_kernel_of<false, true>(p, a.type) : slab_kernel_of<false, false>(p, a.type));
        hipLaunchKernelGGL(f, dim3((unsigned)a.per_xcd * 8u), block, 0, s, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(a.n * p.chunks));
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
    const Plan p = plan(a.n, a.hw, a.c, a.groups, a.type, true, false);
    fill(a, p);
    const dim3 block((unsigned)p.threads);
    const int rows = p.nv ? a.n : a.n * p.chunks;
    if (rows > 0 && p.nv) {
        GnKernel f = a.cg % 8 == 0 ? grad_slab_kernel_of<true>(p, a.type) : grad_slab_kernel_of<false>(p, a.type);
        hipLaunchKernelGGL(f, dim3((unsigned)a.per_xcd * 8u), block, 0, s, a);
    } else if (rows > 0) {
        const dim3 grid((unsigned)rows);
        a.gsum = a.ws + (size_t)rows * a.c * 2;
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
