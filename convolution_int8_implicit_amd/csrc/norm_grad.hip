// Gradient of the group norm with an activation (norm_common.h has the formulas and the two forms).
//
// One sum over the pixels serves everything: with S1[ch] = sum dz xhat and S2[ch] = sum dz, dweight and
// dbias are their sums over the samples, and a group's sums of d xhat and d are those of weight S1 and
// weight S2 over its channels.  What bounds it: three passes of memory (x, dy, dx) in the slab form,
// and the vector units (about 40 operations a value with SiLU: dz is computed twice, since keeping it would take
// the registers that hold the slab), each of which takes turns with the other: 64 x 784 x 512 bf16 with SiLU 43 us for
// 154 MB, 3.6 TB/s, the vector units active 78 % of the time, and 3 us for dweight and dbias.  With them, on one tensor / on
// three in turn: SiLU 42 / 50 us, no activation 32 / 43, float32 with SiLU 76 / 79; split form 1 x 16384 x 512 31 / 32.
#include <iterator>

#include "norm_common.h"

namespace ifx {
namespace {

// Gradient of one channel's values.  With xc = x - mean: xhat = xc rstd, S1 = rstd sum dz xc, and
// dx = rstd weight dz - xc rstd^2 mean(d xhat) - rstd mean(d), two fused operations.  z is one too, but for a
// ReLU it takes its formula's operations one at a time, unfused, so that the side of the corner on which a
// value lies is the formula's own.
template <bool VEC>
struct Channels {
    float w[8], b[8];  // weight and bias
    PerGroup<VEC> m, r;
    float rw[8];

    __device__ __forceinline__ void set(const PerGroup<VEC> &mean, const PerGroup<VEC> &rstd)
    {
        m = mean;
        r = rstd;
#pragma unroll
        for (int e = 0; e < 8; ++e) rw[e] = rstd.get(e) * w[e];
    }
    // dz and xc of a value of channel e
    template <int ACT>
    __device__ __forceinline__ float dz(float x, float dy, int e, float &xc) const
    {
        xc = x - m.get(e);
        if (ACT == 1) {
#pragma clang fp contract(off)
            const float h = xc * r.get(e);
            const float wh = h * w[e];
            return wh + b[e] > 0.0f ? dy : 0.0f;
        }
        if (ACT == 2) {
            const float z = fmaf(xc, rw[e], b[e]);
            const float s = sigmoid(z);
            return dy * (s * fmaf(z, 1.0f - s, 1.0f));
        }
        return dy;
    }
};

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
template <int T, int NV, int TYPE, Mode MODE>
__global__ __launch_bounds__(T, T / 256 > 1 ? T / 256 : 1) void gn_grad_slab_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    constexpr bool VEC = MODE == kVec, WHOLE = MODE != kRagged;
    __shared__ float red[T * 16], part[T], gs[2][2 * T];
    __shared__ __attribute__((aligned(16))) float pw[2 * T], pb[2 * T];
    const Slab s = slab_of(a);
    if (!s.live) return;
    const Place p = place<T>((s.cs + 7) / 8);
    const int valid = s.cs - p.vec * 8;
    const long long first = (long long)s.n * a.hw;
    Oct<E> raw[NV], draw[NV];
    {
        const Pixels<E, WHOLE> x(a.x, a, a.ld_x, first + p.pl, p.tp, s.c0 + p.vec * 8, valid);
        const Pixels<E, WHOLE> dy(a.dy, a, a.ld_dy, first + p.pl, p.tp, s.c0 + p.vec * 8, valid);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (p.active && p.pl + i * p.tp < a.hw) {
                raw[i] = x.get(i);
                draw[i] = dy.get(i);
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
    auto channels = [&]() __attribute__((always_inline)) {
        Channels<VEC> ch;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ch.w[e] = pw[p.vec * 8 + e];
            ch.b[e] = pb[p.vec * 8 + e];
        }
        ch.set(m, r);
        return ch;
    };
    {
        const Channels<VEC> ch = channels();
        float s1[8] = {}, s2[8] = {};
        with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (p.pl + i * p.tp >= a.hw) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float xc;
                    const float dz = ch.template dz<decltype(act)::value>(raw[i].get(e), draw[i].get(e), e, xc);
                    s1[e] = fmaf(dz, xc, s1[e]);
                    s2[e] += dz;
                }
            }
        });
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            raw[i].forget();
            draw[i].forget();
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s1[e] *= r.get(e);
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
    // the parameters read again: kept across the sums they would cost registers that the slab needs
    const Channels<VEC> ch = channels();
    PerGroup<VEC> c1, c2;  // rstd^2 mean(d xhat), rstd mean(d)
    c1.set(p, s, a, [&](int g) { return gs[0][g]; });
    c2.set(p, s, a, [&](int g) { return gs[1][g]; });
#pragma unroll
    for (int e = 0; e < (VEC ? 1 : 8); ++e) {
        c1.v[e] *= r.v[e] * r.v[e];
        c2.v[e] *= r.v[e];
    }
    const Pixels<E, WHOLE> dx(a.y, a, a.ld_y, first + p.pl, p.tp, s.c0 + p.vec * 8, valid);
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p.pl + i * p.tp >= a.hw) break;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float xc;
                const float dz = ch.template dz<decltype(act)::value>(raw[i].get(e), draw[i].get(e), e, xc);
                f[e] = fmaf(dz, ch.rw[e], fmaf(-xc, c1.get(e), -c2.get(e)));
            }
            dx.put(i, f);
        }
    });
}

// ------------------------------------------------------------------------------------------
// Split form: channel sums of a chunk to ws[sample][chunk][2][c], the groups' sums of d xhat and d to
// gsum[sample][chunk][group][2]; then dx from the groups' joined sums.
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ Channels<false> all_channels(const Place &p, const Slab &s, const GnArgs &a, long long stat)
{
    Channels<false> ch;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = min(p.vec * 8 + e, a.c - 1);
        ch.w[e] = a.weight ? a.weight[i] : 1.0f;
        ch.b[e] = a.bias ? a.bias[i] : 0.0f;
    }
    PerGroup<false> m, r;
    m.set(p, s, a, [&](int g) { return a.mean[stat + g]; });
    r.set(p, s, a, [&](int g) { return a.rstd[stat + g]; });
    ch.set(m, r);
    return ch;
}

template <int T, int TYPE, bool WHOLE>
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
        Pixels<E, WHOLE> x(a.x, a, a.ld_x, first + s.p0 + p.pl, p.tp, p.vec * 8, valid);
        Pixels<E, WHOLE> dy(a.dy, a, a.ld_dy, first + s.p0 + p.pl, p.tp, p.vec * 8, valid);
        const Channels<false> ch = all_channels(p, s, a, stat);
        with_act(a.act, [&](auto act) __attribute__((always_inline)) {
            constexpr int AHEAD = T == 1024 ? 2 : 4;  // pixels in flight
            for (int q = s.p0 + p.pl; q < s.p1; q += AHEAD * p.tp) {
                Oct<E> raw[AHEAD], draw[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (q + i * p.tp < s.p1) {
                        raw[i] = x.get(i);
                        draw[i] = dy.get(i);
                    }
                x.advance(AHEAD);
                dy.advance(AHEAD);
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (q + i * p.tp >= s.p1) break;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float xc;
                        const float dz = ch.template dz<decltype(act)::value>(raw[i].get(e), draw[i].get(e), e, xc);
                        s1[e] = fmaf(dz, xc, s1[e]);
                        s2[e] += dz;
                    }
                }
            }
        });
#pragma unroll
        for (int e = 0; e < 8; ++e) s1[e] *= ch.r.get(e);
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

// The chunks' sums of sample n added up: the groups' means of d xhat and d.  A lane has all of its chunks'
// parts in flight at once.
template <int T>
__device__ __forceinline__ void join_sums(const GnArgs &a, int n, float *g1, float *g2)
{
    typedef float v2f __attribute__((ext_vector_type(2)));
    const v2f *gsum = (const v2f *)a.gsum + (long long)n * a.chunks * a.groups;
    const float inv = 1.0f / ((float)a.hw * (float)a.cg);
    const int sub = (int)threadIdx.x & (a.lpg - 1);
    for (int g = (int)threadIdx.x / a.lpg; g < a.groups; g += T / a.lpg) {
        v2f t[kJoin];
        float x1 = 0.0f, x2 = 0.0f;
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            const int k = sub + i * a.lpg;
            t[i] = k < a.chunks ? gsum[k * a.groups + g] : (v2f){0.0f, 0.0f};
        }
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            x1 += t[i].x;
            x2 += t[i].y;
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

template <int T, int TYPE, bool WHOLE>
__global__ __launch_bounds__(T) void gn_grad_apply_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float g1[T * 8], g2[T * 8];
    constexpr int AHEAD = T == 1024 ? 1 : 2;  // pixels in flight
    const Chunk s = chunk_of(a);
    const Place p = place<T>((a.c + 7) / 8);
    const int valid = a.c - p.vec * 8;
    const long long first = (long long)s.n * a.hw, stat = (long long)s.n * a.groups;
    Pixels<E, WHOLE> x(a.x, a, a.ld_x, first + s.p0 + p.pl, p.tp, p.vec * 8, valid);
    Pixels<E, WHOLE> dy(a.dy, a, a.ld_dy, first + s.p0 + p.pl, p.tp, p.vec * 8, valid);
    Pixels<E, WHOLE> dx(a.y, a, a.ld_y, first + s.p0 + p.pl, p.tp, p.vec * 8, valid, a.past);
    Oct<E> raw[AHEAD], draw[AHEAD];
    auto request = [&](int q) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (p.active && q + i * p.tp < s.p1) {
                raw[i] = x.get(i);
                draw[i] = dy.get(i);
            }
        x.advance(AHEAD);
        dy.advance(AHEAD);
    };
    if (T == 1024) join_sums<T>(a, s.n, g1, g2);  // first here: 128 registers do not hold both
    request(s.p0 + p.pl);
    const Channels<false> ch = all_channels(p, s, a, stat);
    if (T != 1024) join_sums<T>(a, s.n, g1, g2);
    if (!p.active) return;
    PerGroup<false> c1, c2;  // rstd^2 mean(d xhat), rstd mean(d)
    c1.set(p, s, a, [&](int g) { return g1[g]; });
    c2.set(p, s, a, [&](int g) { return g2[g]; });
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        c1.v[e] *= ch.r.v[e] * ch.r.v[e];
        c2.v[e] *= ch.r.v[e];
    }
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
        for (int q = s.p0 + p.pl; q < s.p1; q += AHEAD * p.tp) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (q + i * p.tp >= s.p1) break;
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float xc;
                    const float dz = ch.template dz<decltype(act)::value>(raw[i].get(e), draw[i].get(e), e, xc);
                    f[e] = fmaf(dz, ch.rw[e], fmaf(-xc, c1.get(e), -c2.get(e)));
                }
                dx.put(i, f);
            }
            dx.advance(AHEAD);
            request(q + AHEAD * p.tp);
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

// Entry `at` of kGradSlab.
template <int TYPE, Mode MODE, int I = 0>
Instance grad_slab_entry(int at)
{
    if constexpr (I < (int)std::size(kGradSlab)) {
        if (at != I) return grad_slab_entry<TYPE, MODE, I + 1>(at);
        constexpr Variant v = kGradSlab[I];
        if constexpr (slab_holds(v, TYPE, MODE == kVec, true))
            return {gn_grad_slab_kernel<v.threads, v.nv, TYPE, MODE>, v.threads, v.nv};
    }
    return {};
}

template <int T, bool WHOLE>
GnKernel grad_sums_of(const GnArgs &a)
{
    return IFX_GN_TYPES(gn_grad_sums_kernel, T, WHOLE);
}
template <int T, bool WHOLE>
GnKernel grad_apply_of(const GnArgs &a)
{
    return IFX_GN_TYPES(gn_grad_apply_kernel, T, WHOLE);
}

}  // namespace

hipError_t launch_group_norm_grad(GnArgs a, float *dweight, float *dbias, hipStream_t s)
{
    const Plan p = gn_plan(a.n, a.hw, a.c, a.groups, a.type, true, false);
    gn_fill(a, p);
    const bool slab = p.slab >= 0;
    const int rows = slab ? a.n : a.n * p.chunks;
    if (rows > 0 && slab) {
        const Mode mode = mode_of(p.gs * a.cg, a.cg);
        const Instance k = with_type_mode(a.type, mode, [&](auto type, auto m) { return grad_slab_entry<type.value, m.value>(p.slab); });
        if (!k.kernel) return hipErrorInvalidDeviceFunction;
        if (answer_query("gn_grad_slab_kernel<%d, %d, %d, (ifx::Mode)%d>", k.threads, k.nv, a.type, mode)) return hipSuccess;
        hipLaunchKernelGGL(k.kernel, dim3((unsigned)a.per_xcd * 8u), dim3((unsigned)k.threads), 0, s, a);
    } else if (rows > 0) {
        const dim3 grid((unsigned)rows), block((unsigned)p.threads);
        a.gsum = a.ws + (size_t)rows * a.c * 2;
        const bool wide = p.threads == 1024, whole = a.c % 8 == 0;
        if (answer_query("gn_grad_sums_kernel<%d, %d, %s>", p.threads, a.type, tf(whole))) return hipSuccess;
        a.past = stored_past(a.y, (long long)a.n * a.hw, a.ld_y, a.type == 0 ? 4 : 2);
        GnKernel sums = wide ? (whole ? grad_sums_of<1024, true>(a) : grad_sums_of<1024, false>(a))
                             : (whole ? grad_sums_of<512, true>(a) : grad_sums_of<512, false>(a));
        GnKernel apply = wide ? (whole ? grad_apply_of<1024, true>(a) : grad_apply_of<1024, false>(a))
                              : (whole ? grad_apply_of<512, true>(a) : grad_apply_of<512, false>(a));
        hipLaunchKernelGGL(sums, grid, block, 0, s, a);
        hipLaunchKernelGGL(apply, grid, block, 0, s, a);
    }
    if (dweight || dbias)
        hipLaunchKernelGGL(gn_grad_join_kernel, dim3((unsigned)((2 * a.c + 31) / 32)), dim3(1024), 0, s, a.ws, rows, a.c,
                           dweight, dbias);
    return hipGetLastError();
}

}  // namespace ifx
