// attend_kv4.hip -- attention over the 4-bit cache: the queries of the newest
// tokens against all tokens of their sequences.
//
//   t_j = c sum_ch q_ch (m_jg + s_jg code_j,ch),  g = ch / 32,  c = scale * log2(e)
//       = c sum_g [ s_jg (sum_ch q code) + m_jg (sum_ch q) ],   P_j = 2^(t_j - ref)
//   y_ch = sum_j P_j (m_jg + s_jg code_j,ch) / sum_j P_j
//        = [ sum_j (P_j s_jg) code_j,ch + sum_j P_j m_jg ] / sum_j P_j
//
// so that both products run on the codes themselves, on v_mfma_f32_16x16x32_f16:
//  * 4 bits put into the mantissa of a 16-bit zero are the f16 subnormal code *
//    2^-24 (or code * 2^-20, four bits further up), which the MFMA multiplies exactly.
//    Eight codes take five instructions and no conversion.
//  * S^T = K Q^T: 16 tokens by 16 rows of queries, one MFMA for each group of 32
//    channels, whose sum then meets its token's scale.  O^T = V^T P^T: 16 channels by
//    16 rows over 32 tokens, with P_j s_jg for the channels' group.  The cache's layout
//    gives every lane its operands in 16-byte pieces, and S^T's registers are P^T's
//    operand as they are.
//  * A row of 16 lanes loads the 8 tokens' scales that its lanes need, a word or a
//    few each; each use takes its word from the lane that has it (a row broadcast
//    within the multiply).
// Rows: (query, head of the group) pairs of one key head, 16 at a time.
//
// Range in f16: a query's row is scaled by a power of two so that its largest
// value lies in [2^14, 2^15); what falls below 2^-24 there is 2^-39 of the largest.
// P s is scaled by 2^(6 - E), E the largest exponent of the group's scales so far:
// with P <= 2^8 it stays below 2^15.  P s is rounded to f16 once where y is bf16 (its
// 2^-12 is small beside y's own 2^-9); for fp32 and f16 results a second MFMA adds
// what the rounding left, 22 bits together, and the same for fp32 queries.
//
// The work, 32 tokens by 16 rows by key head, is split evenly over the workgroups
// whatever the sequences' lengths: they all sum the lengths and take equal runs of
// the list of all blocks.  What does not cover a sequence's row goes to the workspace
// and is joined by a second launch.
#include <utility>

#include "qig_attend_device.h"
#include "qig_launch.h"

namespace qig {
namespace {

constexpr int WAVES = 4, ROWS = 16;
constexpr float LAZY = 8.0f;   // the reference follows the maximum when it is this far behind

template <int... I, typename F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f)
{
    each(std::make_integer_sequence<int, N>(), f);
}

// Lane L's value of each row of 16 lanes.
template <int L>
__device__ __forceinline__ float row_bcast(float v)
{
    const int x = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, x, 0x150 + L, 0xf, 0xf, true));
}

__device__ __forceinline__ f16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __builtin_bit_cast(f16x8, u32x4{a, b, c, d});
}

__device__ __forceinline__ f32x4 mfma_f16(f16x8 a, f16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_f16(_Float16 a, _Float16 b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
}

__device__ __forceinline__ float ldexp_f(float x, int e) { return __builtin_amdgcn_ldexpf(x, e); }

// What exponents are taken against: 0 where nothing has been seen, so that the power is
// 0 there and a NaN stays one.
__device__ __forceinline__ float base_of(float ref) { return ref == -INFINITY ? 0.0f : ref; }

// What a piece of a row leaves in the workspace: m and l of its 16 rows, then O.
template <int D> constexpr int SLOT = 2 * ROWS + ROWS * D;

struct Header { int seq, head, tile, pieces; };   // the row whose first piece a workgroup has, if it has more

struct Job {
    Kv4 c;
    Kv4Attend a;
    int per;            // heads of queries on one key head
    int split;          // 0: every row in one piece
    int groups;         // workgroups
    float *slots;       // [groups][2][SLOT]
    Header *headers;    // [groups]
};

// A sequence's place in the list of all blocks.
struct Seq {
    int q0, n;          // packed queries
    int64_t length;     // tokens, as given (not negative)
    int64_t keys;       // of them, those that the table has room for
    int64_t blocks;     // list entries of one (head, tile): at least one, so that rows without keys get their zeros
    int tiles;
};

__device__ __forceinline__ Seq get_seq(const Job &j, int s)
{
    Seq q;
    if (j.c.starts) {
        q.q0 = held(j.c.starts[s], j.a.nt);
        q.n = held(j.c.starts[s + 1], j.a.nt) - q.q0;
        if (q.n < 0) q.n = 0;
    } else {
        q.q0 = s;
        q.n = 1;
    }
    const int len = j.c.lengths[s];
    q.length = len < 0 ? 0 : len;
    const int64_t room = j.c.width * j.c.page;
    q.keys = q.length < room ? q.length : room;
    q.blocks = !j.split || q.keys == 0 ? 1 : (q.keys + 31) / 32;
    q.tiles = (int)(((int64_t)q.n * j.per + ROWS - 1) / ROWS);
    return q;
}

__device__ __forceinline__ int64_t units(const Job &j, const Seq &q) { return (int64_t)j.c.heads * q.tiles * q.blocks; }

// Sum of a 64-bit value over the lanes before this one, and over all 256 threads.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t *tmp, int64_t &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t up = __shfl_up(s, o);
        if (lane >= o) s += up;
    }
    __syncthreads();
    if (lane == 63) tmp[wave] = s;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < wave; ++w) before += tmp[w];
    total = tmp[0] + tmp[1] + tmp[2] + tmp[3];
    return before + s - v;
}

template <int D> struct Loaded {
    static constexpr int G = D / 32, Q = G / 2;   // groups of channels, and 16-byte pieces a lane has of the codes
    u32x4 k[Q], v[Q];
    uint32_t ks[Q], vs[Q];
};

template <int D>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[D / 64])
{
    if constexpr (D == 64) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (D == 128) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
        w[0] = v[0], w[1] = v[1];
    } else {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
        w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
    }
}

template <int D>
__device__ __forceinline__ void load_block(const uint8_t *block, int lane, Loaded<D> &b)
{
    constexpr int Q = Loaded<D>::Q;
#pragma unroll
    for (int i = 0; i < Q; ++i) b.k[i] = *reinterpret_cast<const u32x4 *>(block + i * 1024 + lane * 16);
    load_words<D>(block + 32 * D + lane * (4 * Q), b.ks);
#pragma unroll
    for (int i = 0; i < Q; ++i) b.v[i] = *reinterpret_cast<const u32x4 *>(block + 16 * D + i * 1024 + lane * 16);
    load_words<D>(block + 36 * D + lane * (4 * Q), b.vs);
}

template <int T, int D, int QP, int PP>
__global__ __launch_bounds__(256) void kv4_kernel(Job j)
{
    typedef elem_t<T> E;
    constexpr int G = D / 32, Q = G / 2, TILES = D / 16;
    __shared__ float joined[WAVES][ROWS * D];
    __shared__ float stats[WAVES][2][ROWS];
    __shared__ int64_t tmp[4];
    __shared__ int64_t found[2];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l = lane & 15, h = lane >> 4;
    const int nseq = (int)j.c.nseq;

    // the list's length, and where this workgroup's run of it begins
    int64_t mine = 0, total, size;
    for (int s = threadIdx.x; s < nseq; s += 256) mine += units(j, get_seq(j, s));
    scan(mine, tmp, total);
    size = (total + j.groups - 1) / j.groups;
    if (j.split && size < WAVES) size = WAVES;
    if (size < 1) size = 1;
    int64_t at = (int64_t)blockIdx.x * size;
    const int64_t end = at + size < total ? at + size : total;
    if (threadIdx.x == 0 && j.split) j.headers[blockIdx.x].pieces = 0;
    if (at >= end) return;
    int64_t ahead = 0;
    for (int s0 = 0; s0 < nseq; s0 += 256) {
        const int s = s0 + threadIdx.x;
        const int64_t u = s < nseq ? units(j, get_seq(j, s)) : 0;
        int64_t sum;
        const int64_t before = ahead + scan(u, tmp, sum);
        if (at >= before && at < before + u) {
            found[0] = s;
            found[1] = before;
        }
        ahead += sum;
        if (ahead > at) break;
    }
    __syncthreads();
    int s = __builtin_amdgcn_readfirstlane((int)found[0]);
    int64_t seq_at = found[1];
    Seq q = get_seq(j, s);

    while (at < end) {
        while (at >= seq_at + units(j, q)) {
            seq_at += units(j, q);
            q = get_seq(j, ++s);
        }
        const int64_t part = (at - seq_at) / q.blocks;
        const int64_t first = (at - seq_at) % q.blocks;             // list entries of this row before the piece
        const int64_t left = q.blocks - first;
        const int64_t entries = left < end - at ? left : end - at;
        const int head = (int)(part / q.tiles), tile = (int)(part % q.tiles);
        // the blocks of tokens: all of them where rows are not split
        const int64_t all = (q.keys + 31) / 32;
        const int64_t b0 = j.split ? first : 0, b1 = j.split ? (first + entries < all ? first + entries : all) : all;

        // this lane's row: its query, scaled into f16, and the sums of its groups
        const int64_t R = (int64_t)tile * ROWS + l;
        const bool real = R < (int64_t)q.n * j.per;
        const int64_t Rq = real ? R : (int64_t)q.n * j.per - 1;
        const int qi = (int)(Rq / j.per), qh = head * j.per + (int)(Rq % j.per);
        const E *qp = static_cast<const E *>(j.a.q.p) + (int64_t)(q.q0 + qi) * j.a.q.token + (int64_t)qh * j.a.q.head;
        f16x8 qv[QP][G];
        float qs[G], F;
        {
            float f[G][8], top = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int x = 0; x < 8 / VEC<T>; ++x) {
                    float t[VEC<T>];
                    unpack16<T>(load16<T>(qp + g * 32 + h * 8 + x * VEC<T>), t);
#pragma unroll
                    for (int i = 0; i < VEC<T>; ++i) f[g][x * VEC<T> + i] = t[i];
                }
                qs[g] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    top = fmaxf(top, fabsf(f[g][i]));
                    qs[g] += f[g][i];
                }
                qs[g] += __shfl_xor(qs[g], 16);
                qs[g] += __shfl_xor(qs[g], 32);
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const int e = top > 0.0f && top < INFINITY ? __builtin_amdgcn_frexp_expf(top) - 15 : 0;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                _Float16 hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = ldexp_f(f[g][i], ((i >> 1) & 1 ? -4 : 0) - e);
                    hi[i] = (_Float16)v;
                    lo[i] = (_Float16)(v - (float)hi[i]);
                }
                qv[0][g] = f16x8{hi[0], hi[1], hi[2], hi[3], hi[4], hi[5], hi[6], hi[7]};
                if constexpr (QP > 1) qv[1][g] = f16x8{lo[0], lo[1], lo[2], lo[3], lo[4], lo[5], lo[6], lo[7]};
                qs[g] = ldexp_f(qs[g], -24 - e);
            }
            F = ldexp_f(j.a.c, 24 + e);
        }
        // the tokens that this row sees: the first `limit` ones
        int64_t lim = q.length - q.n + qi + 1;
        const int64_t limit = lim < 0 ? 0 : lim < q.keys ? lim : q.keys;
        // from this token on some row of the tile sees less than all
        const int q_first = (int)((int64_t)tile * ROWS / j.per);
        int64_t full = q.length - q.n + q_first + 1;
        full = full < q.keys ? full : q.keys;

        f32x4 o[TILES];
        float mm[G], ref = -INFINITY, sum = 0.0f;
        int E[Q];                                   // exponents of the scales' references, in the scales' lanes
#pragma unroll
        for (int x = 0; x < TILES; ++x) o[x] = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) mm[g] = 0.0f;
#pragma unroll
        for (int x = 0; x < Q; ++x) E[x] = -200;

        const int32_t *table = j.c.tables + (int64_t)s * j.c.ld;
        const int page_blocks = j.c.page / 32;
        const auto block_at = [&](int64_t b) -> const uint8_t * {
            const int64_t col = b / page_blocks;
            const int page = __builtin_amdgcn_readfirstlane(table[col]);
            if (page < 0 || page >= j.c.npages) return nullptr;
            return j.c.pages + page * j.c.page_bytes +
                   ((int64_t)head * page_blocks + (b - col * page_blocks)) * (40 * D);
        };

        Loaded<D> now, next;
        int64_t b = b0 + wave;
        const uint8_t *here = b < b1 ? block_at(b) : nullptr;
        if (here) load_block<D>(here, lane, now);
        for (; b < b1; b += WAVES) {
            const uint8_t *then = b + WAVES < b1 ? block_at(b + WAVES) : nullptr;
            if (then) load_block<D>(then, lane, next);
            if (here) {
                const bool tail = b * 32 + 32 > full;
                float ks[Q], km[Q], vs[Q], vm[Q];
#pragma unroll
                for (int x = 0; x < Q; ++x) {
                    uint32_t kw = now.ks[x], vw = now.vs[x];
                    if (tail) {                     // words behind the sequence's end hold anything
                        const int slot = (l * Q + x) / G;
                        if (b * 32 + (slot >> 2) * 16 + h * 4 + (slot & 3) >= q.keys) kw = vw = 0;
                    }
                    ks[x] = __builtin_bit_cast(float, kw << 16);
                    km[x] = __builtin_bit_cast(float, kw & 0xffff0000u);
                    vs[x] = __builtin_bit_cast(float, vw << 16);
                    vm[x] = __builtin_bit_cast(float, vw & 0xffff0000u);
                }
                float t[8];
                each<2>([&](auto uc) {
                    constexpr int u = uc.value;
                    f32x4 acc = 0.0f;
                    each<G>([&](auto gc) {
                        constexpr int g = gc.value, w = u * G + g;
                        const uint32_t c0 = now.k[w / 4][w % 4], c1 = c0 >> 8;
                        const f16x8 kv = operand(c0 & 0x000f000fu, c0 & 0x00f000f0u, c1 & 0x000f000fu, c1 & 0x00f000f0u);
                        f32x4 dot = 0.0f;
                        dot = mfma_f16(kv, qv[0][g], dot);
                        if constexpr (QP > 1) dot = mfma_f16(kv, qv[1][g], dot);
                        each<4>([&](auto rc) {
                            constexpr int r = rc.value, from = (u * 4 + r) * 2 + g / Q;
                            acc[r] = __builtin_fmaf(row_bcast<from>(ks[g % Q]), dot[r], acc[r]);
                            acc[r] = __builtin_fmaf(row_bcast<from>(km[g % Q]), qs[g], acc[r]);
                        });
                    });
#pragma unroll
                    for (int r = 0; r < 4; ++r) t[u * 4 + r] = acc[r] * F;
                });
                bool seen[8];
                if (tail) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        seen[x] = b * 32 + (x >> 2) * 16 + h * 4 + (x & 3) < limit;
                        if (!seen[x]) t[x] = -INFINITY;
                    }
                }
                float top = t[0];
#pragma unroll
                for (int x = 1; x < 8; ++x) top = fmaxf(top, t[x]);
                if (__any(top > ref + LAZY)) {      // also the first time: nothing is above -infinity
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float to = fmaxf(ref, top);
                    const float fix = __builtin_amdgcn_exp2f(ref - base_of(to));
                    ref = to;
                    sum *= fix;
#pragma unroll
                    for (int x = 0; x < TILES; ++x) o[x] *= fix;
#pragma unroll
                    for (int g = 0; g < G; ++g) mm[g] *= fix;
                }
                const float base = base_of(ref);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    t[x] = __builtin_amdgcn_exp2f(t[x] - base);
                    sum += t[x];
                }
                // the references of the values' scales
                bool above = false;
#pragma unroll
                for (int x = 0; x < Q; ++x) above |= vs[x] != 0.0f && __builtin_amdgcn_frexp_expf(vs[x]) > E[x];
                if (__any(above)) {
#pragma unroll
                    for (int x = 0; x < Q; ++x) {
                        // lanes of the same parity hold the same groups
                        int e = vs[x] != 0.0f ? __builtin_amdgcn_frexp_expf(vs[x]) : -200;
#pragma unroll
                        for (int dist = 2; dist < 64; dist <<= 1) {
                            const int other = __shfl_xor(e, dist);
                            e = other > e ? other : e;
                        }
                        e = e > E[x] ? e : E[x];
                        const int shift = E[x] - e;
                        E[x] = e;
#pragma unroll
                        for (int par = 0; par < 2; ++par) {
                            const int sh = __builtin_amdgcn_readlane(shift, par);
                            const int g = par * Q + x;
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                o[2 * g][r] = ldexp_f(o[2 * g][r], sh);
                                o[2 * g + 1][r] = ldexp_f(o[2 * g + 1][r], sh);
                            }
                        }
                    }
                }
                float vn[Q];
#pragma unroll
                for (int x = 0; x < Q; ++x) vn[x] = ldexp_f(vs[x], 6 - E[x]);
                each<G>([&](auto gc) {
                    constexpr int g = gc.value;
                    _Float16 hi[8], lo[8];
                    each<8>([&](auto xc) {
                        constexpr int x = xc.value, from = x * 2 + g / Q;
                        float w = t[x] * row_bcast<from>(vn[g % Q]);
                        float m = t[x] * row_bcast<from>(vm[g % Q]);
                        if (tail && !seen[x]) w = m = 0.0f;   // a token that this row may not see can be anything
                        mm[g] += m;
                        hi[x] = (_Float16)w;
                        if constexpr (PP > 1) lo[x] = (_Float16)(w - (float)hi[x]);
                    });
                    const f16x8 p0 = operand(pack_f16(hi[0], hi[1]), pack_f16(hi[2], hi[3]), pack_f16(hi[4], hi[5]),
                                             pack_f16(hi[6], hi[7]));
                    f16x8 p1;
                    if constexpr (PP > 1)
                        p1 = operand(pack_f16(lo[0], lo[1]), pack_f16(lo[2], lo[3]), pack_f16(lo[4], lo[5]),
                                     pack_f16(lo[6], lo[7]));
                    each<2>([&](auto yc) {
                        constexpr int n = 2 * g + yc.value, bit = n % 4;
                        uint32_t c[4];
                        each<4>([&](auto pc) {
                            constexpr int w = pc.value * (D / 64) + n / 4;
                            const uint32_t word = now.v[w / 4][w % 4];
                            c[pc.value] = (bit & 2 ? word >> 8 : word) & (bit & 1 ? 0x00f000f0u : 0x000f000fu);
                        });
                        const f16x8 vv = operand(c[0], c[1], c[2], c[3]);
                        o[n] = mfma_f16(vv, p0, o[n]);
                        if constexpr (PP > 1) o[n] = mfma_f16(vv, p1, o[n]);
                    });
                });
            }
            now = next;
            here = then;
        }

        // the wave's rows: channels 16 n + 4 h + r of row l in o[n][r]
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        each<G>([&](auto gc) {
            constexpr int g = gc.value;
            mm[g] += __shfl_xor(mm[g], 16);
            mm[g] += __shfl_xor(mm[g], 32);
            const int e = __builtin_amdgcn_readlane(E[g % Q], g / Q);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int n = 2 * g + y;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    o[n][r] = ldexp_f(o[n][r], e + 24 - 6 - (n & 1 ? 4 : 0)) + mm[g];
            }
        });
        __syncthreads();                            // the piece before is out of LDS
        if (h == 0) {
            stats[wave][0][l] = ref;
            stats[wave][1][l] = sum;
        }
        __syncthreads();
        float top = stats[0][0][l];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) top = fmaxf(top, stats[w][0][l]);
        const float fix = __builtin_amdgcn_exp2f(ref - base_of(top));
#pragma unroll
        for (int n = 0; n < TILES; ++n)
            *reinterpret_cast<f32x4 *>(&joined[wave][l * D + 16 * n + 4 * h]) = o[n] * fix;
        __syncthreads();
        const bool whole = entries == q.blocks;
        float *slot = j.slots + (int64_t)(blockIdx.x * 2 + (first == 0 ? 1 : 0)) * SLOT<D>;
        for (int x = threadIdx.x * 4; x < ROWS * D; x += 1024) {
            const int row = x / D;
            f32x4 v = *reinterpret_cast<const f32x4 *>(&joined[0][x]);
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const f32x4 *>(&joined[w][x]);
            float M = stats[0][0][row], lsum = 0.0f;
#pragma unroll
            for (int w = 1; w < WAVES; ++w) M = fmaxf(M, stats[w][0][row]);
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                lsum += stats[w][1][row] * __builtin_amdgcn_exp2f(stats[w][0][row] - base_of(M));
            if (whole) {
                const int64_t Ry = (int64_t)tile * ROWS + row;
                if (Ry < (int64_t)q.n * j.per) {
                    const float inv = lsum != 0.0f ? 1.0f / lsum : 0.0f;
                    const float f[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
                    store4(j.a.y, j.a.ytype, (int64_t)(q.q0 + (int)(Ry / j.per)) * j.a.y_token +
                                                 (int64_t)(head * j.per + (int)(Ry % j.per)) * j.a.y_head + x % D, f);
                }
            } else {
                *reinterpret_cast<f32x4 *>(slot + 2 * ROWS + x) = v;
                if (x % D == 0) {
                    slot[row] = M;
                    slot[ROWS + row] = lsum;
                }
            }
        }
        if (!whole && first == 0 && threadIdx.x == 0) {
            const int64_t last = (at + q.blocks - 1) / size;         // the workgroup with the row's last piece
            j.headers[blockIdx.x] = {s, head, tile, (int)(last - blockIdx.x) + 1};
        }
        at += entries;
    }
}

// The rows of more than one piece: the first is workgroup g's last one (slot 1), the
// others are the first ones of the next workgroups (slot 0).
template <int D>
__global__ __launch_bounds__(256) void kv4_join(Job j)
{
    const int g = blockIdx.x;
    const Header hd = j.headers[g];
    if (hd.pieces == 0) return;
    const Seq q = get_seq(j, hd.seq);
    const auto slot_of = [&](int p) { return j.slots + (int64_t)((g + p) * 2 + (p == 0 ? 1 : 0)) * SLOT<D>; };
    for (int x = threadIdx.x * 4; x < ROWS * D; x += 1024) {
        const int row = x / D;
        float M = -INFINITY, lsum = 0.0f;
        for (int p = 0; p < hd.pieces; ++p) M = fmaxf(M, slot_of(p)[row]);
        f32x4 v = 0.0f;
        for (int p = 0; p < hd.pieces; ++p) {
            const float *slot = slot_of(p);
            const float fix = __builtin_amdgcn_exp2f(slot[row] - base_of(M));
            lsum += slot[ROWS + row] * fix;
            v += *reinterpret_cast<const f32x4 *>(slot + 2 * ROWS + x) * fix;
        }
        const int64_t R = (int64_t)hd.tile * ROWS + row;
        if (R >= (int64_t)q.n * j.per) continue;
        const float inv = lsum != 0.0f ? 1.0f / lsum : 0.0f;
        const float f[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
        store4(j.a.y, j.a.ytype, (int64_t)(q.q0 + (int)(R / j.per)) * j.a.y_token +
                                     (int64_t)(hd.head * j.per + (int)(R % j.per)) * j.a.y_head + x % D, f);
    }
}

template <int T, int D, int QP, int PP>
int launch_typed(Job j, hipStream_t stream)
{
    // rows of 16 over all sequences, and their blocks, are at most
    const int64_t rows = j.c.heads * ((j.a.nt * j.per) / ROWS + j.c.nseq);
    const int64_t blocks = (j.c.width * j.c.page + 31) / 32;
    int64_t groups = rows;
    j.split = j.a.ws != nullptr;
    if (j.split) {
        const int64_t each = 2 * SLOT<D> * 4 + (int64_t)sizeof(Header);
        int64_t most = ATTEND_WS_BYTES / each;
        if (most > 1024) most = 1024;
        const int64_t want = blocks > (int64_t(1) << 40) / rows ? most : (rows * blocks + WAVES - 1) / WAVES;
        groups = want < 1 ? 1 : want < most ? want : most;
        j.headers = static_cast<Header *>(j.a.ws);
        j.slots = reinterpret_cast<float *>(j.headers + groups);
    }
    if (groups > launch_groups(256) || groups >= (int64_t(1) << 31)) return -1;
    j.groups = (int)groups;
    const int rc = launch_kernel(kv4_kernel<T, D, QP, PP>, dim3((unsigned)groups), dim3(256), stream, j);
    if (rc != 0 || !j.split) return rc;
    return launch_kernel(kv4_join<D>, dim3((unsigned)groups), dim3(256), stream, j);
}

template <int D>
int launch_dim(const Job &j, hipStream_t stream)
{
    const bool fine = j.a.ytype != T_BF16;
    if (j.a.type == T_F32)
        return fine ? launch_typed<T_F32, D, 2, 2>(j, stream) : launch_typed<T_F32, D, 2, 1>(j, stream);
    if (j.a.type == T_BF16)
        return fine ? launch_typed<T_BF16, D, 1, 2>(j, stream) : launch_typed<T_BF16, D, 1, 1>(j, stream);
    return fine ? launch_typed<T_F16, D, 1, 2>(j, stream) : launch_typed<T_F16, D, 1, 1>(j, stream);
}

}  // namespace

int launch_attend_kv4(const Kv4 &c, const Kv4Attend &a, hipStream_t stream)
{
    Job j = {c, a, a.hq / c.heads, 0, 0, nullptr, nullptr};
    if (c.d == 64) return launch_dim<64>(j, stream);
    if (c.d == 128) return launch_dim<128>(j, stream);
    return launch_dim<256>(j, stream);
}

}  // namespace qig
