// Gradient of the group norm with an activation (norm_common.h has the formulas and the two forms).
//
// One sum over the pixels serves everything: with S1[ch] = sum dz xhat and S2[ch] = sum dz, dweight and
// dbias are their sums over the samples, and a group's sums of d xhat and d are those of weight S1 and
// weight S2 over its channels.  What bounds it: three passes of memory (x, dy, dx) in the slab form,
// and the vector units (about 45 operations a value with SiLU).
#include "norm_common.h"

namespace ifx {
namespace {

// dz and xhat of one value.  z takes the operations of its formula one at a time, unfused, so that the
// side of a ReLU's corner on which a value lies is the formula's own.
template <int ACT>
__device__ __forceinline__ float grad_of(float xv, float dy, float mean, float rstd, float w, float b, float &xhat)
{
#pragma clang fp contract(off)
    xhat = (xv - mean) * rstd;
    const float z = xhat * w + b;
    if (ACT == 1) return z > 0.0f ? dy : 0.0f;
    if (ACT == 2) {
        const float s = sigmoid(z);
        return dy * (s * fmaf(z, 1.0f - s, 1.0f));
    }
    return dy;
}

// Channel sums over the pixel lanes: of the active threads' s1 and s2 the sums [2][tcv * 8], left at the start
// of red (T * 16 values); part: T values.  Several threads add up one channel where there are
// more threads than channels, always in one order.
template <int T>
__device__ __forceinline__ void channel_sums(const float (&s1)[8], const float (&s2)[8], const Place &p, float *red, float *part)
{
    const int width = p.tcv * 8, items = 2 * width;
    if (p.active) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            red[p.pl * items + p.vec * 8 + e] = s1[e];
            red[p.pl * items + width + p.vec * 8 + e] = s2[e];
        }
    }
    __syncthreads();
    if (items <= T) {
        const int parts = T / items, at = (int)threadIdx.x / items, item = (int)threadIdx.x - at * items;
        float f = 0.0f;
        if (at < parts)
#pragma unroll 4
            for (int q = at; q < p.tp; q += parts) f += red[q * items + item];
        part[threadIdx.x] = f;
        __syncthreads();
        if ((int)threadIdx.x < items) {
            f = 0.0f;
            for (int q = 0; q < parts; ++q) f += part[q * items + threadIdx.x];
            red[threadIdx.x] = f;
        }
    } else {
        for (int item = threadIdx.x; item < items; item += T) {
            float f = 0.0f;
#pragma unroll 4
            for (int q = 0; q < p.tp; ++q) f += red[q * items + item];
            red[item] = f;  // row 0 of this very item: no other thread reads it
        }
    }
    __syncthreads();
}

// A group's sums of d xhat (half 0) and d (half 1) from the channel sums; out(half, group, sum) by one lane.
template <int T, typename F>
__device__ __forceinline__ void weighted_sums(const float *sums, int width, const float *w, const Slab &s, const GnArgs &a, F out)
{
    const int sub = (int)threadIdx.x & (a.lpg - 1);
    for (int j = (int)threadIdx.x / a.lpg; j < 2 * s.ng; j += T / a.lpg) {
        const int half = j >= s.ng, g = j - half * s.ng;
        float f = 0.0f;
        for (int ch = g * a.cg + sub; ch < (g + 1) * a.cg; ch += a.lpg) f = fmaf(sums[half * width + ch], w[ch], f);
        f = lanes_sum(f, a.lpg);
        if (sub == 0) out(half, g, f);
    }
}

// ------------------------------------------------------------------------------------------
// Slab form: x and dy in registers; channel sums to ws[sample][2][c].
// ------------------------------------------------------------------------------------------
template <int T, int NV, int TYPE, bool VEC>
__global__ __launch_bounds__(T, T / 256 > 1 ? T / 256 : 1) void gn_grad_slab_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float red[T * 16], part[T], gs[2][2 * T];
    __shared__ __attribute__((aligned(16))) float pw[2 * T], pb[2 * T];
    const Slab s = slab_of(a);
    if (!s.live) return;
    const Place p = place<T>((s.cs + 7) / 8);
    const int valid = s.cs - p.vec * 8;
    const long long first = (long long)s.n * a.hw;
    const Pixels<E> x(a.x, a, a.ld_x), dy(a.dy, a, a.ld_dy);
    Oct<E> raw[NV], draw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int q = p.pl + i * p.tp;
        if (p.active && q < a.hw) {
            raw[i] = x.get(first + q, s.c0 + p.vec * 8, valid);
            draw[i] = dy.get(first + q, s.c0 + p.vec * 8, valid);
        } else {
            raw[i] = {};
            draw[i] = {};
        }
    }
    stage_params<T>(s, a, pw, pb);
    const long long stat = (long long)s.n * a.groups + s.g0;
    PerGroup<VEC> m, r;
    m.set(p, s, a, [&](int g) { return a.mean[stat + g]; });
    r.set(p, s, a, [&](int g) { return a.rstd[stat + g]; });
    __syncthreads();
    {
        float w[8], b[8], s1[8] = {}, s2[8] = {};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = pw[p.vec * 8 + e];
            b[e] = pb[p.vec * 8 + e];
        }
        with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (p.pl + i * p.tp >= a.hw) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float xhat;
                    const float dz = grad_of<decltype(act)::value>(raw[i].get(e), draw[i].get(e), m.get(e), r.get(e), w[e],
                                                                   b[e], xhat);
                    s1[e] = fmaf(dz, xhat, s1[e]);
                    s2[e] += dz;
                }
            }
        });
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            raw[i].forget();
            draw[i].forget();
        }
        channel_sums<T>(s1, s2, p, red, part);
    }
    const int width = p.tcv * 8;
    float *out = a.ws + (long long)s.n * a.c * 2 + s.c0;
    for (int i = threadIdx.x; i < 2 * s.cs; i += T) {
        const int half = i >= s.cs, ch = i - half * s.cs;
        out[(long long)half * a.c + ch] = red[half * width + ch];
    }
    const float inv = 1.0f / ((float)a.hw * (float)a.cg);
    weighted_sums<T>(red, width, pw, s, a, [&](int half, int g, float f) { gs[half][g] = f * inv; });
    __syncthreads();
    if (!p.active) return;
    float w[8], b[8];  // read again: kept across the sums they would cost registers that the slab needs
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        w[e] = pw[p.vec * 8 + e];
        b[e] = pb[p.vec * 8 + e];
    }
    PerGroup<VEC> c1, c2;
    c1.set(p, s, a, [&](int g) { return gs[0][g]; });
    c2.set(p, s, a, [&](int g) { return gs[1][g]; });
    E *dst = (E *)a.y + first * a.ld_y + s.c0 + p.vec * 8;
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int q = p.pl + i * p.tp;
            if (q >= a.hw) break;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float xhat;
                const float dz = grad_of<decltype(act)::value>(raw[i].get(e), draw[i].get(e), m.get(e), r.get(e), w[e], b[e],
                                                               xhat);
                f[e] = r.get(e) * (fmaf(dz, w[e], -c2.get(e)) - xhat * c1.get(e));
            }
            store8(dst + (long long)q * a.ld_y, valid, f);
        }
    });
}

// ------------------------------------------------------------------------------------------
// Split form: channel sums of a chunk to ws[sample][chunk][2][c], the groups' sums of d xhat and d to
// gsum[sample][chunk][group][2]; then dx from the groups' joined sums.
// ------------------------------------------------------------------------------------------
template <int T, int TYPE>
__global__ __launch_bounds__(T) void gn_grad_sums_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float red[T * 16], part[T];
    const Chunk s = chunk_of(a);
    const Place p = place<T>((a.c + 7) / 8);
    const int valid = a.c - p.vec * 8;
    float s1[8] = {}, s2[8] = {};
    if (p.active) {
        const long long first = (long long)s.n * a.hw, stat = (long long)s.n * a.groups;
        const Pixels<E> x(a.x, a, a.ld_x), dy(a.dy, a, a.ld_dy);
        float w[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int ch = min(p.vec * 8 + e, a.c - 1);
            w[e] = a.weight ? a.weight[ch] : 1.0f;
            b[e] = a.bias ? a.bias[ch] : 0.0f;
        }
        PerGroup<false> m, r;
        m.set(p, s, a, [&](int g) { return a.mean[stat + g]; });
        r.set(p, s, a, [&](int g) { return a.rstd[stat + g]; });
        with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll 2
            for (int q = s.p0 + p.pl; q < s.p1; q += p.tp) {
                const Oct<E> raw = x.get(first + q, p.vec * 8, valid), draw = dy.get(first + q, p.vec * 8, valid);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float xhat;
                    const float dz = grad_of<decltype(act)::value>(raw.get(e), draw.get(e), m.get(e), r.get(e), w[e], b[e],
                                                                   xhat);
                    s1[e] = fmaf(dz, xhat, s1[e]);
                    s2[e] += dz;
                }
            }
        });
    }
    channel_sums<T>(s1, s2, p, red, part);
    const int width = p.tcv * 8;
    float *out = a.ws + (long long)blockIdx.x * a.c * 2, *gout = a.gsum + (long long)blockIdx.x * a.groups * 2;
    for (int i = threadIdx.x; i < 2 * a.c; i += T) {
        const int half = i >= a.c, ch = i - half * a.c;
        const float f = red[half * width + ch];
        out[i] = f;
        red[half * width + ch] = f * (a.weight ? a.weight[ch] : 1.0f);
    }
    __syncthreads();
    const int sub = (int)threadIdx.x & (a.lpg - 1);
    for (int j = (int)threadIdx.x / a.lpg; j < 2 * a.groups; j += T / a.lpg) {
        const int half = j >= a.groups, g = j - half * a.groups;
        float f = 0.0f;
        for (int ch = g * a.cg + sub; ch < (g + 1) * a.cg; ch += a.lpg) f += red[half * width + ch];
        f = lanes_sum(f, a.lpg);
        if (sub == 0) gout[2 * g + half] = f;
    }
}

template <int T, int TYPE>
__global__ __launch_bounds__(T) void gn_grad_apply_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    typedef float v2f __attribute__((ext_vector_type(2)));
    __shared__ float g1[T * 8], g2[T * 8];
    const Chunk s = chunk_of(a);
    {
        const v2f *gsum = (const v2f *)a.gsum + (long long)s.n * a.chunks * a.groups;
        const float inv = 1.0f / ((float)a.hw * (float)a.cg);
        const int sub = (int)threadIdx.x & (a.lpg - 1);
        for (int g = (int)threadIdx.x / a.lpg; g < a.groups; g += T / a.lpg) {
            float x1 = 0.0f, x2 = 0.0f;
#pragma unroll 8
            for (int i = sub; i < a.chunks; i += a.lpg) {
                const v2f t = gsum[i * a.groups + g];
                x1 += t.x;
                x2 += t.y;
            }
            x1 = lanes_sum(x1, a.lpg);
            x2 = lanes_sum(x2, a.lpg);
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
    const long long first = (long long)s.n * a.hw, stat = (long long)s.n * a.groups;
    const Pixels<E> x(a.x, a, a.ld_x), dy(a.dy, a, a.ld_dy);
    E *dst = (E *)a.y + first * a.ld_y + p.vec * 8;
    float w[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int ch = min(p.vec * 8 + e, a.c - 1);
        w[e] = a.weight ? a.weight[ch] : 1.0f;
        b[e] = a.bias ? a.bias[ch] : 0.0f;
    }
    PerGroup<false> m, r, c1, c2;
    m.set(p, s, a, [&](int g) { return a.mean[stat + g]; });
    r.set(p, s, a, [&](int g) { return a.rstd[stat + g]; });
    c1.set(p, s, a, [&](int g) { return g1[g]; });
    c2.set(p, s, a, [&](int g) { return g2[g]; });
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
        for (int q = s.p0 + p.pl; q < s.p1; q += p.tp) {
            const Oct<E> raw = x.get(first + q, p.vec * 8, valid), draw = dy.get(first + q, p.vec * 8, valid);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float xhat;
                const float dz = grad_of<decltype(act)::value>(raw.get(e), draw.get(e), m.get(e), r.get(e), w[e], b[e], xhat);
                f[e] = r.get(e) * (fmaf(dz, w[e], -c2.get(e)) - xhat * c1.get(e));
            }
            store8(dst + (long long)q * a.ld_y, valid, f);
        }
    });
}

// dweight and dbias: columns of the sums [rows][2 c] added up, 32 columns and 32 row lanes per
// workgroup, in one order.
__global__ __launch_bounds__(1024) void gn_grad_join_kernel(const float *ws, int rows, int c, float *dweight,
                                                            float *dbias)
{
    __shared__ float part[32][33];
    const int col = (int)blockIdx.x * 32 + ((int)threadIdx.x & 31), r0 = (int)threadIdx.x >> 5;
    float s = 0.0f;
    if (col < 2 * c)
#pragma unroll 8
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
    if constexpr (VEC) {
        if (p.threads == 1024) return grad_slab_kernel<1024, 8, VEC>(type);
        if (p.nv == 8) return grad_slab_kernel<512, 8, VEC>(type);
    }
    return grad_slab_kernel<512, 4, VEC>(type);
}

}  // namespace

hipError_t launch_group_norm_grad(GnArgs a, float *dweight, float *dbias, hipStream_t s)
{
    const Plan p = gn_plan(a.n, a.hw, a.c, a.groups, a.type, true, false);
    gn_fill(a, p);
    const dim3 block((unsigned)p.threads);
    const int rows = p.nv ? a.n : a.n * p.chunks;
    if (rows > 0 && p.nv) {
        GnKernel f = a.cg % 8 == 0 ? grad_slab_kernel_of<true>(p, a.type) : grad_slab_kernel_of<false>(p, a.type);
        hipLaunchKernelGGL(f, dim3((unsigned)a.per_xcd * 8u), block, 0, s, a);
    } else if (rows > 0) {
        const dim3 grid((unsigned)rows);
        a.gsum = a.ws + (size_t)rows * a.c * 2;
        const bool small = p.threads == 256;
        GnKernel sums = small ? IFX_GN_TYPES(gn_grad_sums_kernel, 256) : IFX_GN_TYPES(gn_grad_sums_kernel, 1024);
        GnKernel apply = small ? IFX_GN_TYPES(gn_grad_apply_kernel, 256) : IFX_GN_TYPES(gn_grad_apply_kernel, 1024);
        hipLaunchKernelGGL(sums, grid, block, 0, s, a);
        hipLaunchKernelGGL(apply, grid, block, 0, s, a);
    }
    if (dweight || dbias)
        hipLaunchKernelGGL(gn_grad_join_kernel, dim3((unsigned)((2 * a.c + 31) / 32)), dim3(1024), 0, s, a.ws, rows, a.c,
                           dweight, dbias);
    return hipGetLastError();
}

}  // namespace ifx
