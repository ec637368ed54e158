// quantize_i8.hip -- rows of fp32, bf16 or fp16 to int8 with one scale a row.
//
// s = fp32(max|x| / 127), q = the integer nearest x / s, ties away from zero.
// Which integer that is, is decided exactly: the candidate k = rint(|x| * r),
// r an approximate 1 / s, is at most one off, and the sign of an fma is exact
// although its value is rounded, so the two comparisons with the borders
// (2k + 1) s and (2k - 1) s against 2|x| settle it (round_exact).  The quant
// bytes therefore do not depend on how a quotient is rounded.  A row that
// holds a NaN or an infinity gets s = NaN and quants 0, so that every product
// with the row is NaN; the largest magnitude is taken over the bit patterns,
// which order NaN above infinity above all numbers.
#include "qig_i8_device.h"
#include "qig_launch.h"

namespace qig {

// The integer nearest a / s (a >= 0, s > 0, both normal or a = 0), ties up,
// at most 127: r within a few ulps of 1 / s.
__device__ __forceinline__ float round_exact(float a, float s, float r)
{
    float k = __builtin_rintf(a * r);
    // 2a >= (2k + 1) s: one more; 2a < (2k - 1) s: one less
    const float up = __builtin_fmaf(-(2.0f * k + 1.0f), s, 2.0f * a);
    const float dn = __builtin_fmaf(-(2.0f * k - 1.0f), s, 2.0f * a);
    k = up >= 0.0f ? k + 1.0f : (dn < 0.0f ? k - 1.0f : k);
    return __builtin_fminf(k, 127.0f);
}

__device__ __forceinline__ uint32_t max_bits(uint32_t m, float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
    return b > m ? b : m;
}

struct RowScale {
    float s;      // the scale as stored (NaN for a row with NaN or infinity)
    float sc, r;  // scale and reciprocal that the rounding uses
    float up;     // power of two that x is multiplied with before it
    bool zero;    // all quants are 0
};

// Scales below 2^-100 (their reciprocals may overflow, and the exact
// comparison may lose bits below the smallest number) are lifted by 2^64
// together with x, and scales above 2^100 (2 |x| may overflow) lowered by as
// much: no quotient changes, and an x that falls below the smallest number is
// far below s / 2.
__device__ __forceinline__ RowScale row_scale(uint32_t bits)
{
    RowScale o;
    const float big = __builtin_bit_cast(float, bits);
    o.s = big / 127.0f;
    o.zero = bits >= 0x7f800000u || o.s == 0.0f;
    if (bits >= 0x7f800000u) o.s = __builtin_nanf("");
    o.up = o.s < 0x1p-100f ? 0x1p64f : (o.s > 0x1p100f ? 0x1p-64f : 1.0f);
    o.sc = o.zero ? 1.0f : o.s * o.up;
    o.r = __builtin_amdgcn_rcpf(o.sc);
    return o;
}

__device__ __forceinline__ uint32_t quant_byte(float x, const RowScale &c)
{
    const float k = round_exact(__builtin_fabsf(x) * c.up, c.sc, c.r);
    const int q = (int)(c.zero ? 0.0f : __builtin_copysignf(k, x));
    return (uint32_t)q & 0xffu;
}

// One workgroup a row, the row read twice (the second time from the caches).
template <int T>
__global__ __launch_bounds__(256) void quantize_i8_kernel(const elem_t<T> *__restrict__ x, int64_t id, int64_t ldx,
                                                          int8_t *__restrict__ q, int64_t ldq,
                                                          float *__restrict__ s)
{
    const int64_t t = blockIdx.x;
    const elem_t<T> *row = x + t * ldx;
    __shared__ uint32_t part[4];
    uint32_t m = 0;
    for (int64_t i = threadIdx.x; i < id; i += 256) m = max_bits(m, (float)row[i]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = part[w] > m ? part[w] : m;
    const RowScale c = row_scale(m);
    if (threadIdx.x == 0) s[t] = c.s;
    for (int64_t i = threadIdx.x; i < id; i += 256) q[t * ldq + i] = (int8_t)quant_byte((float)row[i], c);
}

template <int T>
static int launch(const void *x, int64_t nt, int64_t id, int64_t ldx, int8_t *q, int64_t ldq, float *s,
                  hipStream_t stream)
{
    return launch_kernel(quantize_i8_kernel<T>, dim3((unsigned)nt), dim3(256), stream,
                         static_cast<const elem_t<T> *>(x), id, ldx, q, ldq, s);
}

int launch_quantize_i8(const void *x, int xtype, int64_t nt, int64_t id, int64_t ldx, int8_t *q, int64_t ldq,
                       float *s, hipStream_t stream)
{
    if (nt > 0x7fffffff) return -1;
    switch (xtype) {
    case T_F32: return launch<T_F32>(x, nt, id, ldx, q, ldq, s, stream);
    case T_BF16: return launch<T_BF16>(x, nt, id, ldx, q, ldq, s, stream);
    default: return launch<T_F16>(x, nt, id, ldx, q, ldq, s, stream);
    }
}

}  // namespace qig
