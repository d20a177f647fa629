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

// Eight consecutive values as they lie in memory.  The struct carries the element's alignment
// only, so one copy of it is a single 16-byte access (two for float) at any element boundary:
// odd row pitches and slices need no path of their own.
template <typename E>
struct Oct {
    E v[8];
};

template <typename E>
__device__ __forceinline__ void load8(const E *p, int valid, E (&raw)[8])
{
    if (valid >= 8) {
        const Oct<E> o = *(const Oct<E> *)p;
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] = o.v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] = e < valid ? p[e] : (E)0.0f;
    }
}

template <typename E>
__device__ __forceinline__ void store8(E *p, int valid, const float (&f)[8])
{
    if (valid >= 8) {
        Oct<E> o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = (E)f[e];
        *(Oct<E> *)p = o;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < valid) p[e] = (E)f[e];
    }
}

// Activations (include/ifx.h: IFX_ACT_NONE, IFX_ACT_RELU, IFX_ACT_SILU).  A NaN stays a NaN.
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_of(float z)
{
    if (ACT == 1) return z < 0.0f ? 0.0f : z;
    if (ACT == 2) return z * sigmoid(z);
    return z;
}
__device__ __forceinline__ float act_any(int act, float z)
{
    return act == 1 ? act_of<1>(z) : act == 2 ? act_of<2>(z) : z;
}

// Maximum over the four lanes 4i .. 4i + 3 (every lane of the wave active).
__device__ __forceinline__ unsigned quad_max(unsigned u)
{
    const unsigned a = (unsigned)__builtin_amdgcn_mov_dpp((int)u, 0xb1, 0xf, 0xf, true);  // lanes 1 0 3 2
    u = a > u ? a : u;
    const unsigned b = (unsigned)__builtin_amdgcn_mov_dpp((int)u, 0x4e, 0xf, 0xf, true);  // lanes 2 3 0 1
    return b > u ? b : u;
}

// Microscaled 4-bit codes of a block of 32 values held by four neighbouring lanes, eight each
// (every lane of the wave active).  The scale's exponent is floor(log2 max |x|) - 2, read off the
// largest magnitude's bit pattern; the conversion instruction rounds x / 2^(s - 127) to nearest
// even on the grid 0 .. 6 and saturates.  A block with a NaN or an infinity gets the NaN scale 255
// and zero codes.  Returns the lane's eight codes, the lowest column in the lowest bits.
__device__ __forceinline__ unsigned mx4_codes(const float (&f)[8], unsigned &scale)
{
    unsigned u = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const unsigned a = __float_as_uint(f[e]) & 0x7fffffffu;
        u = a > u ? a : u;
    }
    u = quad_max(u) >> 23;
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
