// What the group norm kernels (norm.hip, norm_grad.hip) share.
//
// A sample is hw pixels of c channels, channels innermost (a pixel every ld elements); group g is
// the c / groups channels from g * c / groups on.  With the mean and variance of a sample's group
// over pixels and channels:
//   xhat = (x - mean) * rstd, rstd = 1 / sqrt(var + eps), z = xhat * weight + bias, y = act(z)
//   dz = dy act'(z), dweight = sum dz xhat, dbias = sum dz, d = dz weight,
//   dx = rstd (d - mean(d) - xhat mean(d xhat))          (means over the sample's group)
// Every statistic is held in 32 bits and summed in one order, so results repeat bit for bit.
//
// Threads take eight consecutive channels (one 16-byte access of a 16-bit type), neighbouring
// threads neighbouring channels, so a wave reads whole runs of a pixel.  There are two forms:
//   slab   a workgroup keeps all pixels of a span of groups in registers: x (and dy) cross memory
//          once.  Taken where such a slab fits.
//   split  a first kernel reduces chunks of pixels over all channels, a second joins the chunks'
//          parts and reads x again.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "ifx_internal.h"
#include "lowp.h"

namespace ifx {

constexpr int kMaxC = 8192;  // channels: eight per thread, 1024 threads
constexpr int kBatch = 8;    // pixels a thread of the split form holds at once
constexpr int kJoin = 16;    // chunks' parts that a lane joins at most

// ------------------------------------------------------------------------------------------
// Device side
// ------------------------------------------------------------------------------------------

// What a kernel may take for granted of its threads' vectors of eight channels.
enum Mode {
    kRagged,  // the last one may hold fewer of the workgroup's channels
    kWhole,   // all eight are the workgroup's (cs is a multiple of 8)
    kVec      // and all eight of one group (cg is a multiple of 8)
};
inline Mode mode_of(int cs, int cg) { return cg % 8 == 0 ? kVec : cs % 8 == 0 ? kWhole : kRagged; }

// The groups and channels a workgroup covers, and its sample.
struct Slab {
    int n, g0, ng, c0, cs;  // sample, first group, groups, first channel, channels
    bool live;
};

// Slab form: XCD x (blockIdx & 7) owns a run of (sample, span) pairs, spans innermost, so spans that
// share 128-byte lines meet in one L2.
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

// Split form: all channels of sample blockIdx / chunks, pixels [p0, p1) of chunk k.
struct Chunk : Slab {
    int k, p0, p1;
};
__device__ __forceinline__ Chunk chunk_of(const GnArgs &a)
{
    Chunk s;
    s.n = (int)(blockIdx.x / (unsigned)a.chunks);
    s.k = (int)(blockIdx.x - (unsigned)s.n * (unsigned)a.chunks);
    s.g0 = s.c0 = 0;
    s.ng = a.groups;
    s.cs = a.c;
    s.live = true;
    s.p0 = s.k * a.px;
    s.p1 = min(a.hw, s.p0 + a.px);
    return s;
}

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
    p.tp = __builtin_amdgcn_readfirstlane(T / tcv);
    p.pl = (int)threadIdx.x / tcv;
    p.vec = (int)threadIdx.x - p.pl * tcv;
    p.active = p.pl < p.tp;
    return p;
}

// A thread's view of a tensor of n * hw pixels: eight channels from channel ch on of the pixels row + i * step, of
// which `valid` are the caller's (WHOLE: all).  The others' values are arbitrary: where memory goes on
// behind them (the next pixel) they are read too, so only a tensor's very last vector is read value by
// value.  The start is one 64-bit product, a pixel's address one addition of a uniform stride.
template <typename E, bool WHOLE>
struct Pixels {
    const E *at, *end;
    long long stride;
    int valid;
    bool past;  // stored past the caches
    __device__ __forceinline__ Pixels(const void *p, const GnArgs &a, long long ld, long long row, int step, int ch, int valid_,
                                      bool past_ = false)
        : at((const E *)p + row * ld + ch), end((const E *)p + ((long long)a.n * a.hw - 1) * ld + a.c), stride(step * ld),
          valid(valid_), past(past_)
    {
    }
    __device__ __forceinline__ Oct<E> get(int i) const
    {
        const E *p = at + i * stride;
        if constexpr (WHOLE)
            return load8(p);
        else
            return load8(p, p + 8 <= end ? 8 : valid);
    }
    __device__ __forceinline__ void put(int i, const float (&f)[8]) const
    {
        E *p = const_cast<E *>(at) + i * stride;
        if constexpr (!WHOLE) {
            store8(p, valid, f);
        } else if (past) {
            keep_apart();
            store8<true>(p, f);
            keep_apart();
        } else {
            store8(p, f);
        }
    }
    // on by i steps
    __device__ __forceinline__ void advance(int i) { at += i * stride; }
};

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

// Sums over each group of the slab of the threads' per-channel values v (VEC: their sum in v[0]); values of
// inactive threads and of channels past the span are not looked at.  out[g] for the slab's groups;
// red holds T * (VEC ? 1 : 8) values.  Barriers: one before the sums, one after; the caller has one
// between two calls with the same arrays.
template <int T, bool VEC>
__device__ __forceinline__ void group_sums(const float *v, const Place &p, const Slab &s, const GnArgs &a, float *red,
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
#pragma unroll 4
        for (int j = sub; j < p.tp * per; j += a.lpg) {
            const int q = fdiv(j, mul, shr);
            f += red[q * width + g * per + (j - q * per)];
        }
        f = lanes_sum(f, a.lpg);
        if (sub == 0) out[g] = f;
    }
    __syncthreads();
}

// weight and bias of the slab's channels (1 and 0 where there is none) into LDS; visible after the next barrier.
template <int T>
__device__ __forceinline__ void stage_params(const Slab &s, const GnArgs &a, float *w, float *b)
{
    for (int i = threadIdx.x; i < s.cs; i += T) {
        w[i] = a.weight ? a.weight[s.c0 + i] : 1.0f;
        b[i] = a.bias ? a.bias[s.c0 + i] : 0.0f;
    }
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
typedef void (*GnKernel)(GnArgs);

// The threads and vectors per thread of the slab kernels, by rising capacity.  Plan and dispatch both walk these
// lists, and an entry is compiled for just the types and modes whose plans may take it (slab_holds).
struct Variant {
    int threads, nv;
};
constexpr Variant kSlab[] = {{256, 2}, {256, 8}, {512, 8}, {512, 16}, {1024, 16}};
constexpr Variant kGradSlab[] = {{256, 2}, {256, 4}, {512, 4}, {1024, 2}, {512, 8}};

// Registers for raw values: 64 of a thread's 128 (x and dy in the gradient), half where a channel's group takes
// registers of its own (vec: it takes none) beside packed values or a second tensor.
constexpr bool slab_holds(Variant v, int type, bool vec, bool grad)
{
    const int most = (type == 0 ? 8 : 16) / (grad ? 2 : 1);
    return v.nv <= (vec || (type == 0 && !grad) ? most : most / 2);
}

// A slab kernel and the block it is compiled for; kernel: null where the entry is not compiled.
struct Instance {
    GnKernel kernel;
    int threads, nv;
};

// f(type, mode) as compile-time constants.
template <typename F>
Instance with_type_mode(int type, Mode mode, F f)
{
    auto modes = [&](auto t) {
        return mode == kVec     ? f(t, std::integral_constant<Mode, kVec>())
               : mode == kWhole ? f(t, std::integral_constant<Mode, kWhole>())
                                : f(t, std::integral_constant<Mode, kRagged>());
    };
    return type == 0 ? modes(Slot0()) : type == 1 ? modes(Slot1()) : modes(Slot2());
}

struct Plan {
    int threads;
    int slab, gs, spans;  // slab: entry of its list, groups of a span, spans; slab = -1: split
    int chunks, px;       // split: chunks of a sample and their pixels
};
Plan gn_plan(int n, int hw, int c, int groups, int type, bool grad, bool mx4);
// Sets up the launcher's fields of `a` for a plan.
void gn_fill(GnArgs &a, const Plan &p);

#define IFX_GN_TYPES(kernel, T, ...)                                                            \
    (a.type == 0 ? kernel<T, 0, ##__VA_ARGS__> : a.type == 1 ? kernel<T, 1, ##__VA_ARGS__> : kernel<T, 2, ##__VA_ARGS__>)

}  // namespace ifx
