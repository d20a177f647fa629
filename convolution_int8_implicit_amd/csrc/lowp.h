// Device helpers of the 4-bit and normalisation kernels: typed loads and stores of eight
// consecutive values, the activation functions and the rounding of a block of 32 values to
// microscaled 4-bit codes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace ifx {

// Element types as include/ifx.h numbers them (IFX_F32, IFX_BF16, IFX_F16).
template <int TYPE>
struct Elem;
template <>
struct Elem<0> {
    typedef float type;
};
template <>
struct Elem<1> {
    typedef __bf16 type;
};
template <>
struct Elem<2> {
    typedef _Float16 type;
};

// Eight consecutive values as they lie in memory: four 32-bit words of a 16-bit type, eight of float.
// Kept packed in registers and widened where they are used.
template <typename E>
struct Oct {
    static constexpr int W = sizeof(E) * 2;
    unsigned w[W];

    __device__ __forceinline__ float get(int e) const
    {
        if constexpr (sizeof(E) == 4)
            return __uint_as_float(w[e]);
        else if constexpr (__is_same(E, __bf16))
            return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        else
            return (float)__builtin_bit_cast(_Float16, (unsigned short)(w[e / 2] >> (16 * (e & 1))));
    }
    // Makes the words opaque to the optimiser, which would otherwise keep the widened values of one
    // use for the next, in twice the registers.
    __device__ __forceinline__ void forget()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) asm volatile("" : "+v"(w[i]));
    }
};

// Words aligned to the element only: one such access is a single 16-byte load or store at any
// element boundary, so odd row pitches and slices need no path of their own.
template <int ALIGN>
struct Words;
template <>
struct Words<2> {
    typedef unsigned type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Words<4> {
    typedef unsigned type __attribute__((ext_vector_type(4), aligned(4)));
};

// ONCE: read once and by one access a line, kept out of the caches that reused data is in.
template <bool ONCE = false, typename E>
__device__ __forceinline__ Oct<E> load8(const E *p)
{
    typedef typename Words<sizeof(E)>::type V;
    Oct<E> o;
#pragma unroll
    for (int i = 0; i < Oct<E>::W / 4; ++i) {
        const V v = ONCE ? __builtin_nontemporal_load((const V *)p + i) : ((const V *)p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) o.w[4 * i + j] = v[j];
    }
    return o;
}

// The first `valid` >= 1 of eight values; those past them are arbitrary (the last one again).
template <bool ONCE = false, typename E>
__device__ __forceinline__ Oct<E> load8(const E *p, int valid)
{
    if (valid >= 8) return load8<ONCE>(p);
    Oct<E> o;
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o.w[e] = ((const unsigned *)p)[min(e, valid - 1)];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o.w[e] = ((const unsigned short *)p)[min(2 * e, valid - 1)] |
                     (unsigned)((const unsigned short *)p)[min(2 * e + 1, valid - 1)] << 16;
    }
    return o;
}

template <typename E>
__device__ __forceinline__ unsigned pack2(float a, float b)
{
    typedef E V __attribute__((ext_vector_type(2)));
    const V v = {(E)a, (E)b};
    return __builtin_bit_cast(unsigned, v);
}

// Beside a store past the caches in one of two branches: without it the compiler joins the two branches' stores
// into one and drops the mark.
__device__ __forceinline__ void keep_apart() { asm volatile(""); }

// PAST: past the caches, for 16-bit results too large to stay there whose rows fill whole lines.
template <bool PAST = false, typename E>
__device__ __forceinline__ void store8(E *p, const float (&f)[8])
{
    typedef typename Words<sizeof(E)>::type V;
    if constexpr (sizeof(E) == 4) {
        ((V *)p)[0] = (V){__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
        ((V *)p)[1] = (V){__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])};
    } else {
        const V v = {pack2<E>(f[0], f[1]), pack2<E>(f[2], f[3]), pack2<E>(f[4], f[5]), pack2<E>(f[6], f[7])};
        if (PAST)
            __builtin_nontemporal_store(v, (V *)p);
        else
            *(V *)p = v;
    }
}

template <typename E>
__device__ __forceinline__ void store8(E *p, int valid, const float (&f)[8])
{
    if (valid >= 8) {
        store8(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < valid) p[e] = (E)f[e];
    }
}

// Activations (include/ifx.h: IFX_ACT_NONE, IFX_ACT_RELU, IFX_ACT_SILU).  A NaN stays a NaN.  The
// sigmoid is one exponential and one reciprocal instruction, each good to a unit in the last place.
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// The activation of z / pre_scale<ACT>(): SiLU takes z log2(e), which spares the exponential's product.
template <int ACT>
__device__ __forceinline__ constexpr float pre_scale()
{
    return ACT == 2 ? 1.44269504f : 1.0f;
}
template <int ACT>
__device__ __forceinline__ float act_scaled(float z)
{
    if (ACT == 1) return z < 0.0f ? 0.0f : z;
    if (ACT == 2) return z * __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(-z), 1.44269504f, 1.44269504f));
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_of(float z)
{
    if (ACT == 1) return z < 0.0f ? 0.0f : z;
    if (ACT == 2) return z * sigmoid(z);
    return z;
}

// f(tag) with the activation as a compile-time constant, so no value's loop chooses one.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    if (act == 2)
        f(Slot2());
    else if (act == 1)
        f(Slot1());
    else
        f(Slot0());
}

// Maximum over the four lanes 4i .. 4i + 3 (every lane of the wave active).
__device__ __forceinline__ unsigned quad_max(unsigned u)
{
    u = max(u, (unsigned)__builtin_amdgcn_mov_dpp((int)u, 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
    return max(u, (unsigned)__builtin_amdgcn_mov_dpp((int)u, 0x4e, 0xf, 0xf, true));  // lanes 2 3 0 1
}

// Microscaled 4-bit codes of a block of 32 values held by four neighbouring lanes, eight each
// (every lane of the wave active).  The scale's exponent is floor(log2 max |x|) - 2, read off the
// largest magnitude's bit pattern; the conversion instruction rounds x / 2^(s - 127) to nearest
// even on the grid 0 .. 6 and saturates.  A block with a NaN or an infinity gets the NaN scale 255
// and zero codes.  Returns the lane's eight codes, the lowest column in the lowest bits.
__device__ __forceinline__ unsigned mx4_codes(const float (&f)[8], unsigned &scale)
{
    // the maximum that keeps a NaN, three operands at a time
    float top = __builtin_elementwise_maximum(fabsf(f[0]), fabsf(f[1]));
    top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(top, fabsf(f[2])), fabsf(f[3]));
    top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(top, fabsf(f[4])), fabsf(f[5]));
    top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(top, fabsf(f[6])), fabsf(f[7]));
    const unsigned u = quad_max(__float_as_uint(top)) >> 23 & 255u;
    const bool bad = u == 255u;
    const unsigned s = (u < 2u ? 2u : u) - 2u;
    scale = bad ? 255u : s;
    const float sf = __uint_as_float(s << 23);  // the instruction reads the exponent field only
    unsigned r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0], f[1], sf, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2], f[3], sf, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4], f[5], sf, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6], f[7], sf, 3);
    return bad ? 0u : r;
}

}  // namespace ifx
