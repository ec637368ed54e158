// qig_i8_device.h -- element types of the int8 linear layer's inputs and
// outputs on the device.
#pragma once
#include "qig_device.h"
#include "qig_i8.h"

namespace qig {

template <int T> struct Elem;
template <> struct Elem<T_F32> { typedef float type; };
template <> struct Elem<T_BF16> { typedef __bf16 type; };
template <> struct Elem<T_F16> { typedef _Float16 type; };
template <int T> using elem_t = typename Elem<T>::type;

// 16 bytes of elements as fp32 (4 of fp32, 8 of the 16-bit types).
template <int T> constexpr int VEC = T == T_F32 ? 4 : 8;

template <int T>
__device__ __forceinline__ void unpack16(u32x4 v, float (&o)[VEC<T>])
{
    if constexpr (T == T_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(float, (uint32_t)v[i]);
    } else if constexpr (T == T_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = v[i];
            o[2 * i] = __builtin_bit_cast(float, w << 16);
            o[2 * i + 1] = __builtin_bit_cast(float, w & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = v[i];
            o[2 * i] = h2f(w);
            o[2 * i + 1] = h2f(w >> 16);
        }
    }
}

// fp32 to 16 bytes of elements, each rounded once (to nearest even).
template <int T>
__device__ __forceinline__ u32x4 pack16(const float (&f)[VEC<T>])
{
    u32x4 v;
    if constexpr (T == T_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint32_t, f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const elem_t<T> a = (elem_t<T>)f[2 * i], b = (elem_t<T>)f[2 * i + 1];
            v[i] = (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
        }
    }
    return v;
}

// The 16 bytes at any element's address: the hardware takes unaligned vector
// accesses, so rows may start and step anywhere.
template <int T>
__device__ __forceinline__ u32x4 load16(const elem_t<T> *p)
{
    typedef u32x4 u32x4u __attribute__((aligned(2)));
    return *reinterpret_cast<const u32x4u *>(p);
}
template <int T>
__device__ __forceinline__ void store16(elem_t<T> *p, u32x4 v)
{
    typedef u32x4 u32x4u __attribute__((aligned(2)));
    *reinterpret_cast<u32x4u *>(p) = v;
}

// a * sigmoid(a) * b in fp32, for an output of type T, from the hardware's exp2
// and reciprocal (each within an ulp).  t = a * -log2(e) loses up to 2^-18 to its
// rounding, which would be that much of the exponential (59 * 2^-24 of the value
// at a = -63).  For fp32 outputs the product's low part, and that of log2(e), is
// added behind exp2 as the factor 1 + low * ln 2: all roundings together are below
// 10 * 2^-24 of the value, whatever a is.  16-bit outputs, whose own rounding is
// 2^-12 or more, go without (four instructions an output: 2630 tokens of 2 x 18944
// x 3584 to bf16 would take 320 us for 315).  For a far below zero exp2 overflows
// and the reciprocal of infinity gives the limit 0 (below -87.3 it is already below
// the smallest normal number); beyond +-128 the exponential is 0 or infinity, so a
// is held there, where the low part is small.
template <int T>
__device__ __forceinline__ float silu_mul(float a, float b)
{
    constexpr float L = -1.44269502f, L_LOW = -1.92596303e-8f;   // -log2(e) = L + L_LOW
    float e1;
    if constexpr (T == T_F32) {
        const float x = __builtin_amdgcn_fmed3f(a, -128.0f, 128.0f);
        const float t = x * L;
        const float low = __builtin_fmaf(x, L_LOW, __builtin_fmaf(x, L, -t));
        e1 = __builtin_fmaf(__builtin_amdgcn_exp2f(t), __builtin_fmaf(low, 0.693147181f, 1.0f), 1.0f);
    } else {
        e1 = 1.0f + __builtin_amdgcn_exp2f(a * L);
    }
    return a * __builtin_amdgcn_rcpf(e1) * b;
}

}  // namespace qig
