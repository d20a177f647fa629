// Group norm with an activation over channels-last tensors, and the form that rounds its result to
// microscaled 4-bit codes (norm_common.h has the formulas and the two forms).
//
// Variances never come from a difference of squares: the slab form sums squares about the mean that
// it has from a first pass over its registers; a thread of the split form does so over the pixels it
// holds at once and joins such parts by their means and counts, as do threads and chunks.
//
// What bounds it: memory (each value read and written once in the slab form), closely followed by the
// vector units: about 19 operations a value with SiLU, whose exponential and reciprocal cost four
// each.  Hence the activation chosen outside the loops, z as one subtraction and one fused multiply-add, and addresses by
// uniform strides.  With SiLU, on one tensor / on three in turn (the memory-side cache holds part of the one):
// 128 x 784 x 512 bf16 43 / 51 us, 4.8 / 4.1 TB/s of the 5.2 that a copy reaches, float32 87 / 87, 4.7; 128 x 3136 x 256 bf16,
// one slab of 1024 threads a CU so that loads, sums and stores take turns, 108 / 109 us, 3.8 TB/s; the 4-bit form of the first
// 41 / 45 us, its vector units active 91 % of the time, in float32 43 / 57.  Split form: 1 x 16384 x 512 bf16 20 / 22 us.
#include <algorithm>
#include <iterator>

#include "norm_common.h"

namespace ifx {
namespace {

// A value's z from the group's mean and rstd and the channel's weight and bias.  The mean is subtracted first, also
// from 16-bit values: as x w' + (b - mean w') it would be one operation less, but off by the rounding of mean w', which
// in a nearly constant group (w' up to weight / sqrt(eps)) is far more than the bias.
template <bool VEC>
struct Affine {
    float w[8], b[8];
    PerGroup<VEC> m;
    __device__ __forceinline__ void set(const PerGroup<VEC> &mean, const PerGroup<VEC> &rstd)
    {
        m = mean;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= rstd.get(e);
    }
    template <int ACT>
    __device__ __forceinline__ void scale()
    {
        if (ACT == 2)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] *= pre_scale<ACT>();
                b[e] *= pre_scale<ACT>();
            }
    }
    // pre_scale times it, after scale()
    __device__ __forceinline__ float z(float x, int e) const { return fmaf(x - m.get(e), w[e], b[e]); }
};

// Where a thread's results go: eight channels from channel ch on of pixels row + i * step.
template <int TYPE, bool MX4, bool WHOLE>
struct Results {
    typedef typename Elem<TYPE>::type E;
    Pixels<E, WHOLE> y;
    unsigned *codes;  // of pixel `row`
    uint8_t *scale;   // of the block, or null in three threads of four
    int step, valid;

    __device__ __forceinline__ Results(const GnArgs &a, long long row, int step_, int ch, int valid_, bool past = false)
        : y(a.y, a, a.ld_y, row, step_, ch, valid_, past), step(step_), valid(valid_)
    {
        if (MX4) {
            const int vec = ch >> 3;
            const long long at = (long long)(vec >> 4) * a.n * a.hw + row;
            codes = (unsigned *)a.codes + at * 16 + (vec & 15);
            scale = (vec & 3) == 0 ? a.scales + at * 4 + ((vec & 15) >> 2) : nullptr;
        }
    }

    template <int ACT, bool VEC>
    __device__ __forceinline__ void put(int i, const Oct<E> &raw, const Affine<VEC> &f) const
    {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = act_scaled<ACT>(f.z(raw.get(e), e));
        if constexpr (MX4) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (WHOLE ? valid <= 0 : e >= valid) v[e] = 0.0f;
            unsigned sc;
            const unsigned code = mx4_codes(v, sc);
            codes[(long long)i * step * 16] = code;
            if (scale) scale[(long long)i * step * 4] = (uint8_t)sc;
        } else {
            y.put(i, v);
        }
    }
    __device__ __forceinline__ void advance(int i)
    {
        if constexpr (MX4) {
            codes += (long long)i * step * 16;
            if (scale) scale += (long long)i * step * 4;
        } else {
            y.advance(i);
        }
    }
};

// ------------------------------------------------------------------------------------------
// Slab form
// ------------------------------------------------------------------------------------------
template <int T, int NV, int TYPE, bool MX4, Mode MODE>
__global__ __launch_bounds__(T, T / 256 > 1 ? T / 256 : 1) void gn_slab_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    constexpr bool VEC = MODE == kVec, WHOLE = MODE != kRagged;
    constexpr int LDS = T * (VEC ? 1 : 8);
    __shared__ float red[LDS], gs[2 * T];
    __shared__ __attribute__((aligned(16))) float pw[2 * T], pb[2 * T];
    const Slab s = slab_of(a);
    if (!s.live) return;
    // the last span of a 4-bit result also covers the columns up to the next multiple of 128
    const bool last = MX4 && s.c0 + s.cs == a.c;
    const Place p = place<T>(last ? (a.c + 127) / 128 * 16 - s.c0 / 8 : (s.cs + 7) / 8);
    const int valid = s.cs - p.vec * 8;
    const long long first = (long long)s.n * a.hw;
    const Pixels<E, WHOLE> x(a.x, a, a.ld_x, first + p.pl, p.tp, s.c0 + p.vec * 8, valid);
    Oct<E> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (p.active && p.pl + i * p.tp < a.hw && valid > 0)
            raw[i] = x.get(i);
        else
            raw[i] = {};
    stage_params<T>(s, a, pw, pb);
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
    const float total = (float)a.hw * (float)a.cg;  // divided by, so a constant group's mean is exact
    group_sums<T, VEC>(v, p, s, a, red, gs);
    PerGroup<VEC> m, r;
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
                    t = fmaf(d, d, t);
                else
                    v[e % (VEC ? 1 : 8)] = fmaf(d, d, v[e % (VEC ? 1 : 8)]);
            }
            if (VEC) v[0] += t;
        }
        raw[i].forget();
    }
    __syncthreads();
    group_sums<T, VEC>(v, p, s, a, red, gs);
    r.set(p, s, a, [&](int g) { return 1.0f / sqrtf(gs[g] / total + a.eps); });
    if (a.rstd)
        for (int i = threadIdx.x; i < s.ng; i += T)
            a.rstd[(long long)s.n * a.groups + s.g0 + i] = 1.0f / sqrtf(gs[i] / total + a.eps);
    if (!p.active) return;
    Affine<VEC> f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f.w[e] = pw[p.vec * 8 + e];
        f.b[e] = pb[p.vec * 8 + e];
    }
    f.set(m, r);
    const Results<TYPE, MX4, WHOLE> y(a, first + p.pl, p.tp, s.c0 + p.vec * 8, valid);
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
        f.template scale<ACT>();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p.pl + i * p.tp >= a.hw) break;
            y.template put<ACT>(i, raw[i], f);
        }
    });
}

// ------------------------------------------------------------------------------------------
// Split form
// ------------------------------------------------------------------------------------------

// Mean and sum of squares about it of every group over a chunk's pixels, to ws[sample][chunk][group][2].
template <int T, int TYPE, Mode MODE>
__global__ __launch_bounds__(T) void gn_stats_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    constexpr bool VEC = MODE == kVec, WHOLE = MODE != kRagged;
    constexpr int LDS = T * (VEC ? 1 : 8);
    constexpr int P = VEC ? 1 : 8;  // parts a thread keeps: of its vector or of each channel
    __shared__ float red[LDS], gs[LDS];
    const Chunk s = chunk_of(a);
    const Place p = place<T>((a.c + 7) / 8);
    const int valid = a.c - p.vec * 8;
    const long long first = (long long)s.n * a.hw;
    Pixels<E, WHOLE> x(a.x, a, a.ld_x, first + s.p0 + p.pl, p.tp, p.vec * 8, valid);
    int cnt = 0;  // pixels joined
    float mean[P] = {}, m2[P] = {};
    if (p.active) {
        for (int q = s.p0 + p.pl; q < s.p1; q += kBatch * p.tp) {
            Oct<E> raw[kBatch];
            int have = 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const bool in = q + i * p.tp < s.p1;
                raw[i] = x.get(in ? i : 0);
                have += in;
            }
            x.advance(kBatch);
            const float each = (float)(VEC ? 8 * have : have), part = (float)have / (float)(cnt + have);
            const float both = (float)(VEC ? 8 * cnt : cnt) * part;
            float sum[P] = {}, sq[P] = {};
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i < have)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[e % P] += raw[i].get(e);
#pragma unroll
            for (int e = 0; e < P; ++e) sum[e] = have == kBatch ? sum[e] * (1.0f / (8 / P * kBatch)) : sum[e] / each;
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i < have)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float d = raw[i].get(e) - sum[e % P];
                        sq[e % P] = fmaf(d, d, sq[e % P]);
                    }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float d = sum[e] - mean[e];
                mean[e] = fmaf(d, part, mean[e]);
                m2[e] += fmaf(d, d * both, sq[e]);  // d is the mean itself while nothing is joined: both first, 0 then
            }
            cnt += have;
        }
    }
    const float total = (float)(s.p1 - s.p0) * (float)a.cg, each = (float)(VEC ? 8 * cnt : cnt);
    float v[P];
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = each * mean[e];
    group_sums<T, VEC>(v, p, s, a, red, gs);
    float *out = a.ws + (long long)blockIdx.x * a.groups * 2;
    for (int i = threadIdx.x; i < a.groups; i += T) out[2 * i] = gs[i] / total;
    PerGroup<VEC> m;
    m.set(p, s, a, [&](int g) { return gs[g] / total; });
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const float d = mean[e] - m.get(e);
        v[e] = fmaf(d, d * each, m2[e]);
    }
    __syncthreads();
    group_sums<T, VEC>(v, p, s, a, red, gs);
    for (int i = threadIdx.x; i < a.groups; i += T) out[2 * i + 1] = gs[i];
}

// Joins the chunks' statistics of sample n: smean[g], srstd[g].  A lane has all of its chunks' parts in
// flight at once.
template <int T>
__device__ __forceinline__ void join_stats(const GnArgs &a, int n, float *smean, float *srstd)
{
    typedef float v2f __attribute__((ext_vector_type(2)));
    const v2f *ws = (const v2f *)a.ws + (long long)n * a.chunks * a.groups;
    const float total = (float)a.hw * (float)a.cg;
    // values of a chunk's group; the last chunk may be shorter
    const float full = (float)a.px * (float)a.cg, rest = (float)(a.hw - (a.chunks - 1) * a.px) * (float)a.cg;
    const int sub = (int)threadIdx.x & (a.lpg - 1);
    for (int g = (int)threadIdx.x / a.lpg; g < a.groups; g += T / a.lpg) {
        v2f t[kJoin];
        float f = 0.0f;
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            const int k = sub + i * a.lpg;
            t[i] = k < a.chunks ? ws[k * a.groups + g] : (v2f){0.0f, 0.0f};
        }
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            const int k = sub + i * a.lpg;
            f = fmaf(t[i].x, k < a.chunks - 1 ? full : k == a.chunks - 1 ? rest : 0.0f, f);
        }
        const float mean = lanes_sum(f, a.lpg) / total;
        f = 0.0f;
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            const int k = sub + i * a.lpg;
            const float d = t[i].x - mean;
            f += fmaf(d, d * (k < a.chunks - 1 ? full : k == a.chunks - 1 ? rest : 0.0f), t[i].y);
        }
        const float var = lanes_sum(f, a.lpg) / total;
        if (sub == 0) {
            smean[g] = mean;
            srstd[g] = 1.0f / sqrtf(var + a.eps);
        }
    }
    __syncthreads();
}

// The chunks joined, then each pixel normalised.  MX4: threads also cover the columns up to the next
// multiple of 128.  The first pixels and the parameters are requested before the join.
template <int T, int TYPE, bool MX4, bool WHOLE>
__global__ __launch_bounds__(T) void gn_apply_kernel(GnArgs a)
{
    typedef typename Elem<TYPE>::type E;
    __shared__ float smean[T * 8], srstd[T * 8];
    constexpr int AHEAD = T == 1024 ? 2 : 4;  // loads in flight
    const Chunk s = chunk_of(a);
    const Place p = place<T>(MX4 ? (a.c + 127) / 128 * 16 : (a.c + 7) / 8);
    const int valid = a.c - p.vec * 8;
    const long long first = (long long)s.n * a.hw;
    Pixels<E, WHOLE> x(a.x, a, a.ld_x, first + s.p0 + p.pl, p.tp, p.vec * 8, valid);
    Oct<E> raw[AHEAD];
    auto request = [&](int q) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (q + i * p.tp < s.p1 && p.active && valid > 0)
                raw[i] = x.get(i);
            else
                raw[i] = {};
        x.advance(AHEAD);
    };
    if (T == 1024) join_stats<T>(a, s.n, smean, srstd);  // first here: 128 registers do not hold both
    request(s.p0 + p.pl);
    Affine<false> f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int ch = p.vec * 8 + e;
        f.w[e] = e >= valid ? 0.0f : a.weight ? a.weight[ch] : 1.0f;
        f.b[e] = e >= valid || !a.bias ? 0.0f : a.bias[ch];
    }
    if (T != 1024) join_stats<T>(a, s.n, smean, srstd);
    if (s.k == 0)
        for (int i = threadIdx.x; i < a.groups; i += T) {
            if (a.mean) a.mean[(long long)s.n * a.groups + i] = smean[i];
            if (a.rstd) a.rstd[(long long)s.n * a.groups + i] = srstd[i];
        }
    if (!p.active) return;
    PerGroup<false> m, r;
    m.set(p, s, a, [&](int g) { return smean[g]; });
    r.set(p, s, a, [&](int g) { return srstd[g]; });
    f.set(m, r);
    Results<TYPE, MX4, WHOLE> y(a, first + s.p0 + p.pl, p.tp, p.vec * 8, valid, a.past);
    with_act(a.act, [&](auto act) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
        f.template scale<ACT>();
        for (int q = s.p0 + p.pl; q < s.p1; q += AHEAD * p.tp) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (q + i * p.tp < s.p1) y.template put<ACT>(i, raw[i], f);
            y.advance(AHEAD);
            request(q + AHEAD * p.tp);
        }
    });
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------

// Lanes that sum one group where `groups` groups are summed at once.
int sum_lanes(int groups, int threads)
{
    int lanes = 1;
    while (lanes < 64 && lanes * 2 * groups <= threads) lanes *= 2;
    return lanes;
}

// A chunk gives every thread at least one batch (one pixel where that leaves fewer than 256 workgroups), a lane
// of the join has at most kJoin chunks, and there are at most 512 workgroups, two on each of 256 CUs, so that
// they run at once (16 x 2500 x 640: 848 took 48 us, 512 38).
Plan plan_split(int n, int hw, int c, int groups)
{
    Plan p = {};
    p.slab = -1;
    p.threads = c <= 2048 ? 512 : 1024;
    const int tp = p.threads / ((c + 7) / 8);
    int most = (hw + kBatch * tp - 1) / (kBatch * tp);
    const int want = n > 0 && n < 512 ? 512 / n : 1;
    // few chunks: one pixel a thread before idle CUs
    if ((long long)n * most < 256) most = std::min((hw + tp - 1) / tp, 256 / (n > 0 ? n : 1));
    if (most < 1) most = 1;
    int chunks = want < most ? want : most;
    const int limit = kJoin * sum_lanes(groups, p.threads);
    if (chunks > limit) chunks = limit;
    if (chunks < 1) chunks = 1;
    p.px = (hw + chunks - 1) / chunks;
    p.chunks = (hw + p.px - 1) / p.px;
    return p;
}

// Entry `at` of kSlab.
template <int TYPE, bool MX4, Mode MODE, int I = 0>
Instance slab_entry(int at)
{
    if constexpr (I < (int)std::size(kSlab)) {
        if (at != I) return slab_entry<TYPE, MX4, MODE, I + 1>(at);
        constexpr Variant v = kSlab[I];
        if constexpr (slab_holds(v, TYPE, MODE == kVec, false))
            return {gn_slab_kernel<v.threads, v.nv, TYPE, MX4, MODE>, v.threads, v.nv};
    }
    return {};
}

template <int T>
GnKernel stats_kernel_of(const GnArgs &a, Mode mode)
{
    return mode == kVec     ? IFX_GN_TYPES(gn_stats_kernel, T, kVec)
           : mode == kWhole ? IFX_GN_TYPES(gn_stats_kernel, T, kWhole)
                            : IFX_GN_TYPES(gn_stats_kernel, T, kRagged);
}

template <int T>
GnKernel apply_kernel_of(const GnArgs &a, bool mx4, Mode mode)
{
    if (mx4)
        return mode != kRagged ? IFX_GN_TYPES(gn_apply_kernel, T, true, true) : IFX_GN_TYPES(gn_apply_kernel, T, true, false);
    return mode != kRagged ? IFX_GN_TYPES(gn_apply_kernel, T, false, true) : IFX_GN_TYPES(gn_apply_kernel, T, false, false);
}

}  // namespace

// Slab where a span of whole groups fits the registers of a workgroup.  The span reads at least 128 bytes of
// a pixel; at least 64 where that makes a slab of more than 32768 values (us, bf16, 128 / 64 bytes: 64 x 784
// x 512 24.8 / 23.7, its gradient 53 / 45, but 256 x 196 x 1024 41 / 48) or does not fit; and down to 16 where
// the spans are too few to give every CU one (1 x 3136 x 256: 16.7 at 64 bytes, 8.6 at 16; the
// neighbouring spans of so small a tensor meet in the caches) or 64 does not fit.  A 4-bit result
// needs spans of whole blocks of 32 columns.
// The plan also sizes the caller's workspace, before any device is chosen: it counts on the MI355X's compute
// units and asks no device for its own.
constexpr int kCus = 256;
Plan gn_plan(int n, int hw, int c, int groups, int type, bool grad, bool mx4)
{
    const int cg = c / groups, bytes = type == 0 ? 4 : 2;
    Plan best = {};
    best.slab = -1;
    for (int least = 128; least >= 16; least /= 2) {
        int gs = 1;
        while (gs < groups && (groups % gs || gs * cg * bytes < least || (mx4 && gs * cg % 32))) ++gs;
        const int cs = gs * cg;
        // a last span of 4-bit codes is padded to whole panels
        const int tcv = (cs + 7) / 8 + (mx4 ? (c + 127) / 128 * 16 - (c + 7) / 8 : 0);
        if ((long long)n * (groups / gs) > (1 << 20)) break;  // the grid
        // spans of 16 bytes only while their workgroups run at once: the gradient of 32 x 3136 x 256, four a CU,
        // takes 78 us in them and 69 in the split form, of 128 samples 244 and 228, of 2 samples 16 and 22
        if (least < 32 && gs * cg * bytes < 32 && (long long)n * (groups / gs) > 2 * kCus) break;
        const bool enough = n == 0 || (long long)n * (groups / gs) >= kCus;
        if (best.slab >= 0 && ((least < 64 && best.spans * (long long)n >= kCus) || best.gs == gs)) break;
        const Variant *v = grad ? std::begin(kGradSlab) : std::begin(kSlab);
        const Variant *const end = grad ? std::end(kGradSlab) : std::end(kSlab);
        for (; v != end; ++v)
            if (slab_holds(*v, type, cg % 8 == 0, grad) && tcv <= v->threads / 4 &&
                (long long)v->threads / tcv * v->nv >= hw) {
                best.threads = v->threads;
                best.slab = (int)(v - (grad ? std::begin(kGradSlab) : std::begin(kSlab)));
                best.gs = gs;
                best.spans = groups / gs;
                break;
            }
        if (best.slab >= 0 && enough && (long long)hw * cs <= 32768) break;
    }
    return best.slab >= 0 ? best : plan_split(n, hw, c, groups);
}

void gn_fill(GnArgs &a, const Plan &p)
{
    a.cg = a.c / a.groups;
    fastdiv_magic((unsigned)a.cg, &a.cg_mul, &a.cg_shr);
    fastdiv_magic((unsigned)(a.cg / 8 > 0 ? a.cg / 8 : 1), &a.cgv_mul, &a.cgv_shr);
    a.chunks = p.chunks;
    a.px = p.px;
    a.gs = p.gs;
    a.spans = p.spans;
    a.per_xcd = (int)(((long long)a.n * p.spans + 7) / 8);
    a.lpg = sum_lanes(p.slab >= 0 ? p.gs : a.groups, p.threads);
}

size_t gn_workspace_bytes(int n, int hw, int c, int groups, int type, bool grad, bool mx4)
{
    const Plan p = gn_plan(n, hw, c, groups, type, grad, mx4);
    if (p.slab >= 0) return grad ? (size_t)n * 2 * c * 4 : 0;
    const size_t rows = (size_t)n * p.chunks;
    return rows * 4 * 2 * ((size_t)groups + (grad ? (size_t)c : 0));
}

bool gn_supported(int n, int hw, int c, int groups)
{
    if (c > kMaxC) return false;
    const Plan p = plan_split(n, hw, c, groups);
    return (long long)n * p.chunks * p.threads <= 0xffffffffLL;
}

hipError_t launch_group_norm(GnArgs a, hipStream_t s)
{
    const bool mx4 = a.codes != nullptr;
    const Plan p = gn_plan(a.n, a.hw, a.c, a.groups, a.type, false, mx4);
    gn_fill(a, p);
    const Mode mode = mode_of(p.slab >= 0 ? p.gs * a.cg : a.c, a.cg);
    if (p.slab >= 0) {
        const Instance k = with_type_mode(a.type, mode, [&](auto type, auto m) {
            return mx4 ? slab_entry<type.value, true, m.value>(p.slab) : slab_entry<type.value, false, m.value>(p.slab);
        });
        if (!k.kernel) return hipErrorInvalidDeviceFunction;
        if (answer_query("gn_slab_kernel<%d, %d, %d, %s, (ifx::Mode)%d>", k.threads, k.nv, a.type, tf(mx4), mode)) return hipSuccess;
        hipLaunchKernelGGL(k.kernel, dim3((unsigned)a.per_xcd * 8u), dim3((unsigned)k.threads), 0, s, a);
        return hipGetLastError();
    }
    if (answer_query("gn_stats_kernel<%d, %d, (ifx::Mode)%d>", p.threads, a.type, mode)) return hipSuccess;
    const dim3 grid((unsigned)(a.n * p.chunks)), block((unsigned)p.threads);
    const bool wide = p.threads == 1024;
    a.past = !mx4 && stored_past(a.y, (long long)a.n * a.hw, a.ld_y, a.type == 0 ? 4 : 2);
    GnKernel stats = wide ? stats_kernel_of<1024>(a, mode) : stats_kernel_of<512>(a, mode);
    GnKernel apply = wide ? apply_kernel_of<1024>(a, mx4, mode) : apply_kernel_of<512>(a, mx4, mode);
    hipLaunchKernelGGL(stats, grid, block, 0, s, a);
    hipLaunchKernelGGL(apply, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace ifx
