// qig_attend_device.h -- what the attention kernels share on the device.
#pragma once
#include "qig_attend.h"
#include "qig_i8_device.h"

namespace qig {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// The number of i in [0, n) for which f(i) holds, where f holds up to some i and
// from there on no more.  All lanes of a wave must be here with the same n; each
// round they ask 64 places at once, one round for n <= 64 (a bisection would wait
// log2 n times for memory).
template <typename F>
__device__ __forceinline__ int count_first(int n, F f)
{
    int lo = 0;
    const int lane = threadIdx.x & 63;
    while (n > 0) {
        const int step = (n + 63) >> 6;
        const int i = lane * step;
        const int hits = __popcll(__ballot(i < n && f(lo + i)));
        if (step == 1) return lo + hits;
        if (hits == 0) return lo;
        const int base = (hits - 1) * step;          // f holds there
        lo += base + 1;
        n = (base + step < n ? base + step : n) - base - 1;
    }
    return lo;
}

// A packed position as the caller gave it, held inside [0, n]: whatever starts
// holds, no row outside of the tensors is touched.
__device__ __forceinline__ int held(int at, int64_t n)
{
    return at < 0 ? 0 : at > n ? (int)n : at;
}

// One result at element `at` of y, rounded once to y's type.
__device__ __forceinline__ void store1(void *y, int type, int64_t at, float f)
{
    if (type == T_F32) static_cast<float *>(y)[at] = f;
    else if (type == T_BF16) static_cast<__bf16 *>(y)[at] = (__bf16)f;
    else static_cast<_Float16 *>(y)[at] = (_Float16)f;
}

// Four results in a row at element `at` of y, each rounded once to y's type.
__device__ __forceinline__ void store4(void *y, int type, int64_t at, const float (&f)[4])
{
    typedef u32x4 u32x4u __attribute__((aligned(4)));
    typedef u32x2 u32x2u __attribute__((aligned(2)));
    if (type == T_F32) {
        *reinterpret_cast<u32x4u *>(static_cast<float *>(y) + at) = pack16<T_F32>(f);
    } else {
        const float g[8] = {f[0], f[1], f[2], f[3], 0.0f, 0.0f, 0.0f, 0.0f};
        const u32x4 v = type == T_BF16 ? pack16<T_BF16>(g) : pack16<T_F16>(g);
        *reinterpret_cast<u32x2u *>(static_cast<uint16_t *>(y) + at) = u32x2{v[0], v[1]};
    }
}

}  // namespace qig
