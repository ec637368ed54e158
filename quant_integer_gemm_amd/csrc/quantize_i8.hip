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

// 16 bytes of elements (fewer than VEC at the end of a row: n) to their quant
// bytes.  x * r rounded to an integer by adding 1.5 * 2^23 (its low byte is
// the quant) is right unless the quotient lies within 2^-13 of a border
// between two integers: x * r is off by less than 2^-15 for quotients up to
// 127.  Only then, and for scales that are lifted or lowered, the exact
// comparison runs.
template <int T>
__device__ __forceinline__ void quant_vec(const float (&x)[VEC<T>], const RowScale &c, uint32_t (&o)[VEC<T> / 4])
{
    constexpr float NEAR = 0.5f - 0x1p-13f;
    uint32_t b[VEC<T>];
    float far = c.up == 1.0f && !c.zero ? 0.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < VEC<T>; ++i) {
        const float y = __builtin_fmaf(x[i], c.r, MAGIC_F);
        far = __builtin_fmaxf(far, __builtin_fabsf(__builtin_fmaf(x[i], c.r, -(y - MAGIC_F))));
        b[i] = __builtin_bit_cast(uint32_t, y);
    }
    if (far > NEAR) {
#pragma unroll
        for (int i = 0; i < VEC<T>; ++i) b[i] = quant_byte(x[i], c);
    }
#pragma unroll
    for (int i = 0; i < VEC<T> / 4; ++i) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000c0cu);
        o[i] = lo | hi;
    }
}

// THR threads a row (64: one wave, four rows a workgroup), the row read once
// into NV vectors of 16 bytes a thread.
//
// Bound by memory: 2630 x 18944 bf16 (149 MB in and out) 26.8 us, 5.6 TB/s;
// 15780 x 2368 bf16 (112 MB) 25 us; 2630 x 3584 bf16 (28 MB) 7 us, where loads
// and the launch show.  256 threads for rows of 65 to 1024 vectors: a wave a
// row, without a barrier, measured the same at 15780 rows and 15% slower at
// 2630, and 512 threads slower at both.
template <int T, int THR, int NV>
__global__ __launch_bounds__(THR < 256 ? 256 : THR) void quantize_i8_kernel(const elem_t<T> *__restrict__ x,
                                                                            int64_t nt, int id, int64_t ldx,
                                                                            int8_t *__restrict__ q, int64_t ldq,
                                                                            float *__restrict__ s)
{
    constexpr int V = VEC<T>;
    constexpr int ROWS = THR == 64 ? 4 : 1;
    const int tid = THR == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t t = (int64_t)blockIdx.x * ROWS + (THR == 64 ? threadIdx.x >> 6 : 0);
    if (THR == 64 && t >= nt) return;
    const elem_t<T> *row = x + t * ldx;
    u32x4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * THR + tid) * V;
        if (at + V <= id) {
            v[i] = load16<T>(row + at);
        } else {
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = at + e < id ? (float)row[at + e] : 0.0f;
            v[i] = pack16<T>(f);
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[V];
        unpack16<T>(v[i], f);
#pragma unroll
        for (int e = 0; e < V; ++e) m = max_bits(m, f[e]);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    if constexpr (THR > 64) {
        __shared__ uint32_t part[THR / 64];
        if ((tid & 63) == 0) part[tid >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THR / 64; ++w) m = part[w] > m ? part[w] : m;
    }
    const RowScale c = row_scale(m);
    if (tid == 0) s[t] = c.s;
    int8_t *out = q + t * ldq;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * THR + tid) * V;
        if (at >= id) break;
        float f[V];
        uint32_t o[V / 4];
        unpack16<T>(v[i], f);
        quant_vec<T>(f, c, o);
        if (at + V <= id) {
            typedef uint32_t u32u __attribute__((aligned(1)));
            typedef uint64_t u64u __attribute__((aligned(1)));
            if constexpr (V == 4)
                *reinterpret_cast<u32u *>(out + at) = o[0];
            else
                *reinterpret_cast<u64u *>(out + at) = (uint64_t)o[0] | ((uint64_t)o[V / 4 - 1] << 32);
        } else {
            for (int e = 0; at + e < id; ++e) out[at + e] = (int8_t)(o[e >> 2] >> (8 * (e & 3)));
        }
    }
}

// Rows longer than the registers of a workgroup: read twice, the second time
// from the caches.
template <int T>
__global__ __launch_bounds__(1024) void quantize_i8_long_kernel(const elem_t<T> *__restrict__ x, int64_t id,
                                                                int64_t ldx, int8_t *__restrict__ q, int64_t ldq,
                                                                float *__restrict__ s)
{
    constexpr int V = VEC<T>;
    const int64_t t = blockIdx.x;
    const elem_t<T> *row = x + t * ldx;
    __shared__ uint32_t part[16];
    uint32_t m = 0;
    const int64_t whole = id / V * V;
    for (int64_t i = (int64_t)threadIdx.x * V; i < whole; i += 1024 * V) {
        float f[V];
        unpack16<T>(load16<T>(row + i), f);
#pragma unroll
        for (int e = 0; e < V; ++e) m = max_bits(m, f[e]);
    }
    if (whole + threadIdx.x < id) m = max_bits(m, (float)row[whole + threadIdx.x]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) m = part[w] > m ? part[w] : m;
    const RowScale c = row_scale(m);
    if (threadIdx.x == 0) s[t] = c.s;
    int8_t *out = q + t * ldq;
    for (int64_t i = (int64_t)threadIdx.x * V; i < whole; i += 1024 * V) {
        float f[V];
        uint32_t o[V / 4];
        unpack16<T>(load16<T>(row + i), f);
        quant_vec<T>(f, c, o);
        typedef uint32_t u32u __attribute__((aligned(1)));
#pragma unroll
        for (int w = 0; w < V / 4; ++w) reinterpret_cast<u32u *>(out + i)[w] = o[w];
    }
    if (whole + threadIdx.x < id) out[whole + threadIdx.x] = (int8_t)quant_byte((float)row[whole + threadIdx.x], c);
}

template <int T, int THR, int NV>
static int launch_rows(const elem_t<T> *x, int64_t nt, int64_t id, int64_t ldx, int8_t *q, int64_t ldq, float *s,
                       hipStream_t stream)
{
    constexpr int BLOCK = THR < 256 ? 256 : THR, ROWS = THR == 64 ? 4 : 1;
    return in_launches(nt, launch_groups(BLOCK) * ROWS, [&](int64_t r, int64_t n) {
        return launch_kernel(quantize_i8_kernel<T, THR, NV>, dim3((unsigned)((n + ROWS - 1) / ROWS)), dim3(BLOCK),
                             stream, x + r * ldx, n, (int)id, ldx, q + r * ldq, ldq, s + r);
    });
}

template <int T>
static int launch(const void *xv, int64_t nt, int64_t id, int64_t ldx, int8_t *q, int64_t ldq, float *s,
                  hipStream_t stream)
{
    const elem_t<T> *x = static_cast<const elem_t<T> *>(xv);
    const int64_t nv = (id + VEC<T> - 1) / VEC<T>;
    if (nv <= 64) return launch_rows<T, 64, 1>(x, nt, id, ldx, q, ldq, s, stream);
    if (nv <= 256) return launch_rows<T, 256, 1>(x, nt, id, ldx, q, ldq, s, stream);
    if (nv <= 512) return launch_rows<T, 256, 2>(x, nt, id, ldx, q, ldq, s, stream);
    if (nv <= 1024) return launch_rows<T, 256, 4>(x, nt, id, ldx, q, ldq, s, stream);
    if (nv <= 2560) return launch_rows<T, 512, 5>(x, nt, id, ldx, q, ldq, s, stream);
    if (nv <= 5120) return launch_rows<T, 1024, 5>(x, nt, id, ldx, q, ldq, s, stream);
    return in_launches(nt, launch_groups(1024), [&](int64_t r, int64_t n) {
        return launch_kernel(quantize_i8_long_kernel<T>, dim3((unsigned)n), dim3(1024), stream, x + r * ldx, id, ldx,
                             q + r * ldq, ldq, s + r);
    });
}

int launch_quantize_i8(const void *x, int xtype, int64_t nt, int64_t id, int64_t ldx, int8_t *q, int64_t ldq,
                       float *s, hipStream_t stream)
{
    switch (xtype) {
    case T_F32: return launch<T_F32>(x, nt, id, ldx, q, ldq, s, stream);
    case T_BF16: return launch<T_BF16>(x, nt, id, ldx, q, ldq, s, stream);
    default: return launch<T_F16>(x, nt, id, ldx, q, ldq, s, stream);
    }
}

}  // namespace qig
