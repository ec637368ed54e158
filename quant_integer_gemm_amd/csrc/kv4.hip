// kv4.hip -- keys and values in 4 bits: into the pages of a cache, and back.
//
// 32 values of a row, lo the lowest and hi the highest of them, are kept as
//   m = the largest bf16 <= lo,  s = the smallest bf16 >= (hi - m) / 15,
//   c = floor((x - m) / s + 1/2), held to 0 .. 15   (0 where s = 0)
// in fp64 arithmetic: hi - m, its 15th part and x - m are each rounded to nearest (exact
// while x and m lie within 2^29 of each other) before s is rounded up and the nearest
// code decided.  They stand for m + s c.  With m rounded down and s up no value lies outside
// of m .. m + 15 s by more than fp64's roundings, 2^-51 of it, so that none is off by more than
// s / 2 and that.  Both as bf16 are one word for 32 values: 5 bits a value, the codes 4 of
// them.
//
// A wave has a token and 512 channels, so that a few tokens are many waves; a group's
// ends are two exchanges among four lanes.  Measured, 4 heads of 128: 2630 tokens from
// fp32 8.0 us to write (12.4 MB: 1.6 TB/s), 7.2 to read back as fp32 (1.7 TB/s); 64 tokens
// 5.0 and 3.8: bound by the launch and by each wave's chain of loads (starts, length,
// page, values).  65536 tokens: 77 us to write (4.0 TB/s), 63 to read (4.9), near a copy's 5.3.
#include "qig_attend_device.h"
#include "qig_launch.h"

namespace qig {
namespace {

// Where a packed token stands.  All lanes of a wave ask for the same one.
struct Place {
    int64_t block;   // byte offset of head 0's block in the pages, -1: nowhere
    int u, h, i;     // token 16 u + 4 h + i of the block
    bool inside;     // it is some sequence's
};

__device__ __forceinline__ Place find_place(const Kv4 &c, int64_t nt, int token)
{
    Place p = {-1, 0, 0, 0, false};
    int seq = token, last = token + 1;
    if (c.starts) {
        const int32_t *starts = c.starts;
        seq = __builtin_amdgcn_readfirstlane(
            count_first((int)c.nseq + 1, [&](int s) { return held(starts[s], nt) <= token; }) - 1);
        if (seq < 0 || seq >= c.nseq) return p;
        last = held(c.starts[seq + 1], nt);
    }
    p.inside = true;
    const int64_t pos = (int64_t)c.lengths[seq] - last + token;
    if (pos < 0 || pos >= c.width * c.page) return p;
    const int col = (int)(pos / c.page), r = (int)(pos - (int64_t)col * c.page);
    const int page = c.tables[(int64_t)seq * c.ld + col];
    if (page < 0 || page >= c.npages) return p;
    p.block = (int64_t)page * c.page_bytes + (int64_t)(r >> 5) * (40 * c.d);
    p.u = (r >> 4) & 1;
    p.h = (r >> 2) & 3;
    p.i = r & 3;
    return p;
}

// A wave takes one token and 512 channels: 512 / D rows of the token's keys' heads and
// then its values' heads, eight channels a lane, so that four lanes have a group.
template <int D>
struct Lane {
    int token, head, c;     // c: the lane's first channel
    bool values, real;
    __device__ __forceinline__ Lane(const Kv4 &k, int64_t wave, int chunks)
    {
        const int lane = threadIdx.x & 63;
        token = __builtin_amdgcn_readfirstlane((int)(wave / chunks));
        const int r = (int)(wave % chunks) * (512 / D) + lane / (D / 8);
        values = r >= k.heads;
        head = values ? r - k.heads : r;
        real = r < 2 * k.heads;
        c = lane % (D / 8) * 8;
    }
};

__device__ __forceinline__ uint32_t floor_bf16(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x), low = b & 0xffffu;
    return b - low + ((b >> 31) != 0 && low != 0 ? 0x10000u : 0u);
}

// The smallest bf16 not below x >= 0.
__device__ __forceinline__ uint32_t ceil_bf16(double x)
{
    const float f = (float)x;
    uint32_t b = __builtin_bit_cast(uint32_t, f);
    if ((double)f < x) ++b;                      // the next one up
    return (b + 0xffffu) & 0xffff0000u;
}

// The scale's word of 32 values: s in its low half, m in its high one.
__device__ __forceinline__ uint32_t scale_word(float lo, float hi, float &s, float &m)
{
    if (lo != lo) {                              // by its bits some NaN would round to 0
        s = m = NAN;
        return 0x7fc07fc0;
    }
    const uint32_t mb = floor_bf16(lo);
    m = __builtin_bit_cast(float, mb);
    const uint32_t sb = ceil_bf16(((double)hi - (double)m) / 15.0);
    s = __builtin_bit_cast(float, sb);
    return mb | (sb >> 16);
}

// The code of x: of d = x - m as fp64 has it, exactly.  The sign of d - (c -+ 1/2) s is (one
// rounding in an fma): c from the product with 1 / s is at most one off and is put right by
// these.
__device__ __forceinline__ uint32_t code4(float x, double m, double s, double inv)
{
    const double d = (double)x - m;
    double c = __builtin_floor(__builtin_fma(d, inv, 0.5));
    c = __builtin_fma(0.5 - c, s, d) < 0.0 ? c - 1.0 : __builtin_fma(-0.5 - c, s, d) >= 0.0 ? c + 1.0 : c;
    return c > 15.0 ? 15u : c > 0.0 ? (uint32_t)c : 0u;
}

// The lowest (or highest) of the four lanes of a group; a NaN stays.
template <bool LOW>
__device__ __forceinline__ float of_group(float v)
{
    const auto pick = [](float a, float b) { return (LOW ? b < a : b > a) || b != b ? b : a; };
    v = pick(v, __shfl_xor(v, 1));
    return pick(v, __shfl_xor(v, 2));
}

template <int T, int D>
__global__ __launch_bounds__(256) void write_kernel(Kv4 c, Kv4Rows r, int64_t first, int64_t count, int chunks)
{
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (wave >= count) return;
    const Lane<D> me(c, first + wave, chunks);
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 0.0f;
    if (me.real) {
        const Heads &from = me.values ? r.v : r.k;
        const elem_t<T> *x = static_cast<const elem_t<T> *>(from.p) + (int64_t)me.token * from.token +
                             (int64_t)me.head * from.head + me.c;
#pragma unroll
        for (int k = 0; k < 8 / VEC<T>; ++k) {
            float t[VEC<T>];
            unpack16<T>(load16<T>(x + k * VEC<T>), t);
#pragma unroll
            for (int i = 0; i < VEC<T>; ++i) f[k * VEC<T> + i] = t[i];
        }
    }
    const Place p = find_place(c, r.nt, me.token);
    if (p.block < 0) return;
    float lo = f[0], hi = f[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        // a NaN stays: the group then stands for NaN
        lo = f[i] < lo || f[i] != f[i] ? f[i] : lo;
        hi = f[i] > hi || f[i] != f[i] ? f[i] : hi;
    }
    float s, m;
    const uint32_t word = scale_word(of_group<true>(lo), of_group<false>(hi), s, m);
    // In 32 bits (x - m) / s + 1/2, at most 16.5, is off by less than 2^-18: what lies 2^-16 from
    // an integer is decided there, and a wave with any other does its codes in 64 bits
    // (65536 tokens of 4 heads of 128: fp32 96 us all in 64 bits, 77 so; 16-bit values lie
    // on such borders too often, 87 either way).
    const float quick = s > 0x1p-100f ? 1.0f / s : INFINITY;
    uint32_t code[8];
    bool near = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float q = __builtin_fmaf(f[k] - m, quick, 0.5f);
        near |= !(__builtin_fabsf(q - __builtin_rintf(q)) > 0x1p-16f);
        code[k] = min((uint32_t)q, 15u);
    }
    if (__any(near && me.real)) {
        const double inv = s > 0.0f ? 1.0 / (double)s : 0.0;
#pragma unroll
        for (int k = 0; k < 8; ++k) code[k] = s > 0.0f ? code4(f[k], m, s, inv) : 0;
    }

    constexpr int G = D / 32;
    const int g = me.c / 32, e = me.c % 32 / 8;
    uint8_t *block = c.pages + p.block + (int64_t)me.head * (c.page / 32) * (40 * D);
    uint32_t *words = reinterpret_cast<uint32_t *>(block);
    if (me.real && e == 0) words[(me.values ? 9 : 8) * D + (p.h * 8 + p.u * 4 + p.i) * G + g] = word;
    // keys: the lane's channels are one word
    if (me.real && !me.values) {
        uint32_t all = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) all |= code[k] << (16 * (k & 1) + 4 * (k >> 1));
        const int w = p.u * G + g;
        words[((w >> 2) * 64 + e * 16 + 4 * p.h + p.i) * 4 + (w & 3)] = all;
    }
    // values: channel 64 n + 16 b + l in bits 4 b of the half word l; the four lanes with the
    // same l have b = 0 .. 3, and each then writes two of their eight
    if (__any(me.values)) {
        const int n = me.c / 64, b = me.c / 16 % 4, l0 = me.c % 16;
        uint32_t two[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            two[k] = (code[2 * k] | code[2 * k + 1] << 16) << (4 * b);
            two[k] |= __shfl_xor(two[k], 2);
            two[k] |= __shfl_xor(two[k], 4);
        }
        const uint32_t out = b == 0 ? two[0] : b == 1 ? two[1] : b == 2 ? two[2] : two[3];
        if (me.real && me.values) {
            const int w = (2 * p.u + (p.i >> 1)) * (D / 64) + n;
            uint16_t *at = reinterpret_cast<uint16_t *>(block) +
                           2 * (4 * D + ((w >> 2) * 64 + p.h * 16 + l0 + 2 * b) * 4 + (w & 3)) + (p.i & 1);
            at[0] = (uint16_t)out;
            at[8] = (uint16_t)(out >> 16);
        }
    }
}

// The same rows back, as the values that they stand for; tokens that stand
// nowhere are zeros.
template <int T, int D>
__global__ __launch_bounds__(256) void read_kernel(Kv4 c, Kv4Rows r, int64_t first, int64_t count, int chunks)
{
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (wave >= count) return;
    const Lane<D> me(c, first + wave, chunks);
    const Place p = find_place(c, r.nt, me.token);
    if (!p.inside || !me.real) return;
    constexpr int G = D / 32;
    const int g = me.c / 32, e = me.c % 32 / 8;
    const uint8_t *block = c.pages + p.block + (int64_t)me.head * (c.page / 32) * (40 * D);
    const uint32_t *words = reinterpret_cast<const uint32_t *>(block);
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 0.0f;
    if (p.block >= 0) {
        const uint32_t sm = words[(me.values ? 9 : 8) * D + (p.h * 8 + p.u * 4 + p.i) * G + g];
        const float s = __builtin_bit_cast(float, sm << 16), m = __builtin_bit_cast(float, sm & 0xffff0000u);
        uint32_t code[8];
        if (!me.values) {
            const int w = p.u * G + g;
            const uint32_t all = words[((w >> 2) * 64 + e * 16 + 4 * p.h + p.i) * 4 + (w & 3)];
#pragma unroll
            for (int k = 0; k < 8; ++k) code[k] = all >> (16 * (k & 1) + 4 * (k >> 1));
        } else {
            const int n = me.c / 64, b = me.c / 16 % 4, l0 = me.c % 16, w = (2 * p.u + (p.i >> 1)) * (D / 64) + n;
            const uint16_t *at = reinterpret_cast<const uint16_t *>(block) +
                                 2 * (4 * D + ((w >> 2) * 64 + p.h * 16 + l0) * 4 + (w & 3)) + (p.i & 1);
#pragma unroll
            for (int k = 0; k < 8; ++k) code[k] = at[k * 8] >> (4 * b);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __builtin_fmaf((float)(code[k] & 15u), s, m);
    }
    const Heads &to = me.values ? r.v : r.k;
    elem_t<T> *y = static_cast<elem_t<T> *>(const_cast<void *>(to.p)) + (int64_t)me.token * to.token +
                   (int64_t)me.head * to.head + me.c;
#pragma unroll
    for (int k = 0; k < 8 / VEC<T>; ++k) {
        float t[VEC<T>];
#pragma unroll
        for (int i = 0; i < VEC<T>; ++i) t[i] = f[k * VEC<T> + i];
        store16<T>(y + k * VEC<T>, pack16<T>(t));
    }
}

template <int D, bool WRITE>
int launch_rows(const Kv4 &c, const Kv4Rows &r, hipStream_t stream)
{
    const int chunks = (2 * c.heads * D + 511) / 512;
    return in_launches(r.nt * chunks, launch_groups(256) * 4, [&](int64_t first, int64_t count) {
        const dim3 grid((unsigned)((count + 3) / 4)), block(256);
        const auto go = [&](auto kernel) { return launch_kernel(kernel, grid, block, stream, c, r, first, count, chunks); };
        if (r.type == T_F32) return WRITE ? go(write_kernel<T_F32, D>) : go(read_kernel<T_F32, D>);
        if (r.type == T_BF16) return WRITE ? go(write_kernel<T_BF16, D>) : go(read_kernel<T_BF16, D>);
        return WRITE ? go(write_kernel<T_F16, D>) : go(read_kernel<T_F16, D>);
    });
}

template <bool WRITE>
int launch_dim(const Kv4 &c, const Kv4Rows &r, hipStream_t stream)
{
    if (c.d == 64) return launch_rows<64, WRITE>(c, r, stream);
    if (c.d == 128) return launch_rows<128, WRITE>(c, r, stream);
    return launch_rows<256, WRITE>(c, r, stream);
}

}  // namespace

int launch_write_kv4(const Kv4 &c, const Kv4Rows &r, hipStream_t stream) { return launch_dim<true>(c, r, stream); }
int launch_read_kv4(const Kv4 &c, const Kv4Rows &r, hipStream_t stream) { return launch_dim<false>(c, r, stream); }

}  // namespace qig
