// kv4.hip -- keys and values in 4 bits: into the pages of a cache, and back.
//
// 32 values of a row, lo the lowest and hi the highest of them, are kept as
//   m = the largest bf16 <= lo,  s = the smallest bf16 >= (hi - m) / 15,
//   c = floor((x - m) / s + 1/2), held to 0 .. 15   (0 where s = 0)
// and stand for m + s c.  With m rounded down and s up no value lies outside of
// m .. m + 15 s, so that none is off by more than s / 2.  Both as bf16 are one word
// for 32 values: 5 bits a value, the codes 4 of them.
#include "qig_attend_device.h"
#include "qig_launch.h"

namespace qig {
namespace {

// Where a packed token stands.
struct Place {
    int64_t block;   // byte offset of head 0's block in the pages, -1: nowhere
    int u, h, i;     // token 16 u + 4 h + i of the block
};

__device__ __forceinline__ Place find_place(const Kv4 &c, int64_t nt, int token)
{
    Place p = {-1, 0, 0, 0};
    int seq = token;
    int64_t pos;
    if (c.starts) {
        int lo = 0, hi = (int)c.nseq + 1;        // starts at or before the token
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (held(c.starts[mid], nt) <= token) lo = mid + 1; else hi = mid;
        }
        seq = lo - 1;
        if (seq < 0 || seq >= c.nseq) return p;
        pos = (int64_t)c.lengths[seq] - held(c.starts[seq + 1], nt) + token;
    } else {
        pos = (int64_t)c.lengths[seq] - 1;
    }
    const int64_t col = pos / c.page;
    if (pos < 0 || col >= c.width) return p;
    const int page = c.tables[(int64_t)seq * c.ld + col];
    if (page < 0 || page >= c.npages) return p;
    const int r = (int)(pos - col * c.page);
    p.block = (int64_t)page * c.page_bytes + (int64_t)(r >> 5) * (40 * c.d);
    p.u = (r >> 4) & 1;
    p.h = (r >> 2) & 3;
    p.i = r & 3;
    return p;
}

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
    const uint32_t mb = floor_bf16(lo);
    m = __builtin_bit_cast(float, mb);
    const uint32_t sb = ceil_bf16(((double)hi - (double)m) / 15.0);
    s = __builtin_bit_cast(float, sb);
    return mb | (sb >> 16);
}

// Which code is nearest is decided in 64 bits.
__device__ __forceinline__ uint32_t code4(float x, float s, float m)
{
    if (!(s > 0.0f)) return 0;
    const double v = __builtin_floor(((double)x - (double)m) / (double)s + 0.5);
    return v > 15.0 ? 15u : v > 0.0 ? (uint32_t)v : 0u;
}

// A thread: 64 channels of one token and head, of its keys or its values.
template <int T>
__global__ __launch_bounds__(256) void write_kernel(Kv4 c, Kv4Rows r, int64_t first, int64_t count)
{
    const int64_t id = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= first + count) return;
    const int part = (int)(id % (c.d / 64));
    const int64_t row = id / (c.d / 64) / 2;
    const bool values = (id / (c.d / 64)) & 1;
    const int head = (int)(row % c.heads), token = (int)(row / c.heads);
    const Place p = find_place(c, r.nt, token);
    if (p.block < 0) return;
    uint8_t *block = c.pages + p.block + (int64_t)head * (c.page / 32) * (40 * c.d);
    const Heads &from = values ? r.v : r.k;
    const elem_t<T> *x = static_cast<const elem_t<T> *>(from.p) + (int64_t)token * from.token +
                         (int64_t)head * from.head + part * 64;
    const int G = c.d / 32;
    uint32_t *scales = reinterpret_cast<uint32_t *>(block) + (values ? 9 : 8) * c.d + (p.h * 8 + p.u * 4 + p.i) * G;
    uint32_t half[16];
#pragma unroll
    for (int l = 0; l < 16; ++l) half[l] = 0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float f[32];
#pragma unroll
        for (int k = 0; k < 32 / VEC<T>; ++k) {
            float t[VEC<T>];
            unpack16<T>(load16<T>(x + g * 32 + k * VEC<T>), t);
#pragma unroll
            for (int i = 0; i < VEC<T>; ++i) f[k * VEC<T> + i] = t[i];
        }
        float lo = f[0], hi = f[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) {
            // a NaN stays: the group then stands for NaN
            lo = f[i] < lo || f[i] != f[i] ? f[i] : lo;
            hi = f[i] > hi || f[i] != f[i] ? f[i] : hi;
        }
        float s, m;
        scales[part * 2 + g] = scale_word(lo, hi, s, m);
        if (!values) {
            const int w = p.u * G + part * 2 + g;
            uint32_t *at = reinterpret_cast<uint32_t *>(block) + ((w >> 2) * 64 + 4 * p.h + p.i) * 4 + (w & 3);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t word = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) word |= code4(f[e * 8 + k], s, m) << (16 * (k & 1) + 4 * (k >> 1));
                at[e * 64] = word;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) half[k & 15] |= code4(f[k], s, m) << (4 * (2 * g + (k >> 4)));
        }
    }
    if (values) {
        const int w = (2 * p.u + (p.i >> 1)) * (c.d / 64) + part;
        uint16_t *at = reinterpret_cast<uint16_t *>(block) +
                       2 * (4 * c.d + ((w >> 2) * 64 + p.h * 16) * 4 + (w & 3)) + (p.i & 1);
#pragma unroll
        for (int l = 0; l < 16; ++l) at[l * 8] = (uint16_t)half[l];
    }
}

// The same rows back, as the values that they stand for; tokens that stand
// nowhere are zeros.
template <int T>
__global__ __launch_bounds__(256) void read_kernel(Kv4 c, Kv4Rows r, int64_t first, int64_t count)
{
    const int64_t id = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= first + count) return;
    const int part = (int)(id % (c.d / 64));
    const int64_t row = id / (c.d / 64) / 2;
    const bool values = (id / (c.d / 64)) & 1;
    const int head = (int)(row % c.heads), token = (int)(row / c.heads);
    if (c.starts && (token < held(c.starts[0], r.nt) || token >= held(c.starts[c.nseq], r.nt))) return;
    const Place p = find_place(c, r.nt, token);
    const Heads &to = values ? r.v : r.k;
    elem_t<T> *y = static_cast<elem_t<T> *>(const_cast<void *>(to.p)) + (int64_t)token * to.token +
                   (int64_t)head * to.head + part * 64;
    const uint8_t *block = c.pages + p.block + (int64_t)head * (c.page / 32) * (40 * c.d);
    const uint32_t *words = reinterpret_cast<const uint32_t *>(block);
    const uint16_t *halves = reinterpret_cast<const uint16_t *>(block);
    const int G = c.d / 32;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float f[32];
        if (p.block < 0) {
#pragma unroll
            for (int k = 0; k < 32; ++k) f[k] = 0.0f;
        } else {
            const uint32_t sm = words[(values ? 9 : 8) * c.d + (p.h * 8 + p.u * 4 + p.i) * G + part * 2 + g];
            const float s = __builtin_bit_cast(float, sm << 16), m = __builtin_bit_cast(float, sm & 0xffff0000u);
            if (!values) {
                const int w = p.u * G + part * 2 + g;
                const uint32_t *at = words + ((w >> 2) * 64 + 4 * p.h + p.i) * 4 + (w & 3);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t word = at[e * 64];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        f[e * 8 + k] = __builtin_fmaf((float)((word >> (16 * (k & 1) + 4 * (k >> 1))) & 15u), s, m);
                }
            } else {
                const int w = (2 * p.u + (p.i >> 1)) * (c.d / 64) + part;
                const uint16_t *at = halves + 2 * (4 * c.d + ((w >> 2) * 64 + p.h * 16) * 4 + (w & 3)) + (p.i & 1);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    f[k] = __builtin_fmaf((float)((at[(k & 15) * 8] >> (4 * (2 * g + (k >> 4)))) & 15u), s, m);
            }
        }
#pragma unroll
        for (int k = 0; k < 32 / VEC<T>; ++k) {
            float t[VEC<T>];
#pragma unroll
            for (int i = 0; i < VEC<T>; ++i) t[i] = f[k * VEC<T> + i];
            store16<T>(y + g * 32 + k * VEC<T>, pack16<T>(t));
        }
    }
}

template <typename K>
int launch_rows(K kernel, const Kv4 &c, const Kv4Rows &r, hipStream_t stream)
{
    const int64_t units = r.nt * c.heads * 2 * (c.d / 64);
    return in_launches(units, launch_groups(256) * 256, [&](int64_t first, int64_t count) {
        return launch_kernel(kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), stream, c, r, first, count);
    });
}

}  // namespace

int launch_write_kv4(const Kv4 &c, const Kv4Rows &r, hipStream_t stream)
{
    if (r.type == T_F32) return launch_rows(write_kernel<T_F32>, c, r, stream);
    if (r.type == T_BF16) return launch_rows(write_kernel<T_BF16>, c, r, stream);
    return launch_rows(write_kernel<T_F16>, c, r, stream);
}

int launch_read_kv4(const Kv4 &c, const Kv4Rows &r, hipStream_t stream)
{
    if (r.type == T_F32) return launch_rows(read_kernel<T_F32>, c, r, stream);
    if (r.type == T_BF16) return launch_rows(read_kernel<T_BF16>, c, r, stream);
    return launch_rows(read_kernel<T_F16>, c, r, stream);
}

}  // namespace qig
