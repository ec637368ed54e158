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
//    2^-24 (or code * 2^-20, four bits further up): eight codes take five instructions and
//    no conversion.  The MFMA aligns a sum's products by their operands' exponents, which
//    for all subnormals is the same one: with the codes in the lowest bits it keeps
//    about 17 bits below the largest product (measured), far more than 16-bit
//    results have.  For fp32 queries or results the codes are put in the highest four bits,
//    code * 2^-18, where it keeps all 24 (eight instructions for eight codes).
//  * S^T = K Q^T: 16 tokens by 16 rows of queries, one MFMA for each group of 32
//    channels, whose sum then meets its token's scale.  O^T = V^T P^T: 16 channels by
//    16 rows over 32 tokens, with P_j s_jg for the channels' group.  The cache's layout
//    gives every lane its operands in 16-byte pieces, and S^T's registers are P^T's
//    operand as they are.
//  * A row of 16 lanes loads the 8 tokens' scales that its lanes need, a word or a
//    few each; each use takes its word from the lane that has it (a row broadcast
//    within the multiply).  The keys' m, bf16 as they stand, meet the queries' sums in an
//    MFMA of their own, the sums in three bf16 parts.
// Rows: (query, head of the group) pairs of one key head, 16 at a time.
//
// Range in f16: a query's row is scaled by a power of two so that its largest
// value lies in [2^14, 2^15); what falls below 2^-24 there is 2^-39 of the largest.  Where the
// largest of some 32 channels is less than 2^-QNEAR of that, each 32 have a power of their own,
// applied to their sums in a copy of the scores' part (the search for it costs 1.3%, 61.0 ->
// 61.8 us for the batch below).
// P s is scaled by 2^(10 - E), scales below 2^E: with P <= 2^LAZY it stays below 2^15.  E is HEAD
// above the largest exponent in the wave's first block.  While all scales of the group that
// the wave has met lie in [2^(E - NEAR - 1), 2^E) a row's largest P s is at least 1/4 there (its
// largest P is at least 1), and f16's smallest step no more than 2^-22 of it.  From the first
// block on that has a scale outside of that, or none (a zero), a wave scales each block's P s, and O for their product,
// by each row's largest one: what a row does not see, or gives no weight, takes no bits from
// the rest however large it is.  (The checks cost 2%, 59.7 -> 60.7 us for the batch below.  64
// requests of 4096 tokens 45 us, with a first token of values 2^20 times the others' 59.)
// P s is rounded to f16 once where y is bf16 (its
// 2^-11 is small beside y's own 2^-8); for fp32 and f16 results a second MFMA adds
// what the rounding left, 22 bits together, and the same for fp32 queries (QP and PP:
// parts of the queries and of P s, PP 3 being two parts for fp32 results).
//
// The work, 32 tokens by 16 rows by key head, is split evenly over the workgroups
// whatever the sequences' lengths: they all sum the lengths and take equal runs of
// the list of all blocks.  What does not cover a sequence's row goes to the workspace,
// and the last workgroup to leave a piece of a row there joins them, in the list's order.
//
// Measured, 28 query heads on 4 of 128, bf16: 64 requests of up to 16384 tokens (209 MB of
// cache) 52-62 us as cards go, 3.4-4.0 TB/s, where a large copy moves 5.3.  Waves wait half of
// their cycles for their blocks, and the vector units are busy half of the time: three waves a
// SIMD with one block each on its way reach neither limit.  (One register copy of a
// block less, the keys' m on an MFMA and a 32-bit list took it from 111 to 75 us, as many
// workgroups as the GPU holds to 64, the lengths summed by each wave and one launch to 50, on
// one card; the checks for scales and queries far apart from 59.7 to 61.8, on another.)  One
// request of 4099 tokens 19 us, 2.6 MB: latency, a chain of the lengths' sum 1.5 us, the
// sequence 1.1, the blocks 2.2, the waves' join 1.8, the piece's write 1.2, the count 0.8, and
// the last one's reads and sums.  A launch of its own for the join: 17.7 for 18.2, but 22.7
// for 21.4 with 16 x 5 drafted tokens.
#include <utility>

#include "qig_attend_device.h"
#include "qig_launch.h"

namespace qig {
namespace {

constexpr int WAVES = 4, ROWS = 16, CUS = 256;
// Blocks of a run: two a wave, so that a long sequence alone is in fewer pieces.  Runs of short
// sequences' rows are as long, one row behind the other: 64 requests on 4 key heads take 44 us
// with 30 tokens each, 13 with 100, 27 with 1000 and 26 with 2000, and without a workspace 8,
// 8, 20 and 33.
constexpr int LEAST = 8;
constexpr float LAZY = 5.0f;   // the reference follows the maximum when it is this far behind
constexpr int NEAR = 16 - (int)LAZY;   // scales of a group from 2^(E - NEAR) on share E
constexpr int HEAD = 3;        // what E is above the first block's largest scale
constexpr int NONE = -1;       // no block yet
constexpr int QNEAR = 16;      // a query's groups of channels within 2^QNEAR of its largest share a power

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

__device__ __forceinline__ f32x4 mfma_bf16_16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The compiler would unpack a block's codes all at once, for 100 registers that three
// waves a SIMD do not have.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// Two values rounded to f16, and what the rounding left.
__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}
__device__ __forceinline__ uint32_t pack_rest(uint32_t hi, float a, float b)
{
    const f16x2 v = __builtin_bit_cast(f16x2, hi);
    return pack_f16(a - (float)v[0], b - (float)v[1]);
}

// m + sum over x of t[x] * (lane 2 x + PAR's value of each row of 16 lanes).  The compiler
// makes two instructions of each of these; the wait is that of a row broadcast
// behind a write of its source (and covers t's last powers).
template <int PAR>
__device__ __forceinline__ float row_dot(float m, float v, const float (&t)[8])
{
#define QIG_ROW_FMA(T, L) "v_fmac_f32_dpp %0, %1, " T " row_newbcast:" L " row_mask:0xf bank_mask:0xf\n"
    if constexpr (PAR == 0) {
        asm("s_nop 1\n" QIG_ROW_FMA("%2", "0") QIG_ROW_FMA("%3", "2") QIG_ROW_FMA("%4", "4") QIG_ROW_FMA("%5", "6")
                QIG_ROW_FMA("%6", "8") QIG_ROW_FMA("%7", "10") QIG_ROW_FMA("%8", "12") QIG_ROW_FMA("%9", "14")
            : "+v"(m) : "v"(v), "v"(t[0]), "v"(t[1]), "v"(t[2]), "v"(t[3]), "v"(t[4]), "v"(t[5]), "v"(t[6]), "v"(t[7]));
    } else {
        asm("s_nop 1\n" QIG_ROW_FMA("%2", "1") QIG_ROW_FMA("%3", "3") QIG_ROW_FMA("%4", "5") QIG_ROW_FMA("%5", "7")
                QIG_ROW_FMA("%6", "9") QIG_ROW_FMA("%7", "11") QIG_ROW_FMA("%8", "13") QIG_ROW_FMA("%9", "15")
            : "+v"(m) : "v"(v), "v"(t[0]), "v"(t[1]), "v"(t[2]), "v"(t[3]), "v"(t[4]), "v"(t[5]), "v"(t[6]), "v"(t[7]));
    }
#undef QIG_ROW_FMA
    return m;
}

__device__ __forceinline__ float ldexp_f(float x, int e) { return __builtin_amdgcn_ldexpf(x, e); }

// A row's sums in group G of its channels.
template <int G, int N, typename F>
__device__ __forceinline__ void for_o(f32x4 (&o)[N], F f)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v = o[2 * G + i / 4][i % 4];
        f(v);
        o[2 * G + i / 4][i % 4] = v;
    }
}

// What exponents are taken against: 0 where nothing has been seen, so that the power is
// 0 there and a NaN stays one.
__device__ __forceinline__ float base_of(float ref) { return ref == -INFINITY ? 0.0f : ref; }

// What a piece of a row leaves in the workspace: m and l of its 16 rows, then O.
template <int D> constexpr int SLOT = 2 * ROWS + ROWS * D;

struct Job {
    Kv4 c;
    Kv4Attend a;
    int per;            // heads of queries on one key head
    int split;          // 0: every row in one piece
    int room;           // tokens that a row of the table has pages for
    int groups;         // workgroups
    float *slots;       // [groups][2][SLOT]
    uint32_t *arrived;  // [groups]: pieces of the row that begins in a workgroup's run; 0 before and after a call
};

// A sequence's place in the list of all blocks.
struct Seq {
    int q0, n;          // packed queries
    int length;         // tokens, as given (not negative)
    int keys;           // of them, those that the table has room for
    uint32_t blocks;    // list entries of one (head, tile): at least one, so that rows without keys get their zeros
    uint32_t tiles;
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
    q.keys = q.length < j.room ? q.length : j.room;
    q.blocks = !j.split || q.keys == 0 ? 1 : (uint32_t)(q.keys - 1) / 32 + 1;
    q.tiles = (uint32_t)q.n * (uint32_t)j.per / ROWS + ((uint32_t)q.n * (uint32_t)j.per % ROWS != 0);
    return q;
}

__device__ __forceinline__ uint32_t units(const Job &j, const Seq &q) { return (uint32_t)j.c.heads * q.tiles * q.blocks; }

// Sums of list entries.  A call's true list is shorter than 2^31; starts that decrease can
// ask for more, and no sum of theirs may wrap: it stops at 2^31 - 1, beyond which the list
// is cut off.
__device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b) { return min(a + b, (uint32_t)INT32_MAX); }

__device__ __forceinline__ uint32_t sum_to_lane(uint32_t s)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t up = __shfl_up(s, o);
        if (lane >= o) s = plus(s, up);
    }
    return s;
}

// Sum of a value over the threads before this one, and over all 256.
__device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t *tmp, uint32_t &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t s = sum_to_lane(v), left = __shfl_up(s, 1);
    __syncthreads();
    if (lane == 63) tmp[wave] = s;
    __syncthreads();
    const uint32_t t0 = tmp[0], t1 = plus(t0, tmp[1]), t2 = plus(t1, tmp[2]);
    total = plus(t2, tmp[3]);
    return plus(lane > 0 ? left : 0, wave == 0 ? 0 : wave == 1 ? t0 : wave == 2 ? t1 : t2);
}

// A lane's operands from a block.  G: groups of channels; Q: the 16-byte pieces that a
// lane has of the codes, and its words of the scales.
template <int D> struct Keys {
    static constexpr int G = D / 32, Q = G / 2;
    u32x4 c[Q];
    uint32_t s[Q], m[2][G];                        // m: the scales of keys l and 16 + l
};
template <int D> struct Values {
    static constexpr int Q = D / 64;
    u32x4 c[Q];
    uint32_t s[Q];
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w)
{
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
        w[0] = v[0], w[1] = v[1];
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(p + 4 * i);
            w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
        }
    }
}

template <int D>
__device__ __forceinline__ void load_keys(const uint8_t *block, int lane, Keys<D> &k)
{
    constexpr int Q = Keys<D>::Q, G = Keys<D>::G;
#pragma unroll
    for (int i = 0; i < Q; ++i) k.c[i] = *reinterpret_cast<const u32x4 *>(block + i * 1024 + lane * 16);
    load_words<Q>(block + 32 * D + lane * (4 * Q), k.s);
    const int l = lane & 15;
#pragma unroll
    for (int u = 0; u < 2; ++u) load_words<G>(block + 32 * D + ((l >> 2) * 8 + u * 4 + (l & 3)) * (4 * G), k.m[u]);
}

template <int D>
__device__ __forceinline__ void load_values(const uint8_t *block, int lane, Values<D> &v)
{
    constexpr int Q = Values<D>::Q;
#pragma unroll
    for (int i = 0; i < Q; ++i) v.c[i] = *reinterpret_cast<const u32x4 *>(block + 16 * D + i * 1024 + lane * 16);
    load_words<Q>(block + 36 * D + lane * (4 * Q), v.s);
}

// Pieces cross XCDs, whose L2s are not coherent: agent-scope accesses, two floats each.
__device__ __forceinline__ void put2(float *p, float a, float b)
{
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), __builtin_bit_cast(uint64_t, f32x2{a, b}), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x2 get2(const float *p)
{
    return __builtin_bit_cast(f32x2, __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED,
                                                       __HIP_MEMORY_SCOPE_AGENT));
}

// A tile whose first piece is workgroup g's last one (slot 1), the others being the
// first ones of the next workgroups (slot 0), by the whole workgroup: 16 threads a row
// form the maximum and the pieces' factors, 64 pieces at a time, then a wave sums its rows,
// two at once and 8 pieces of each on their way.  fix: 64 x 16 floats of LDS.
template <int D>
__device__ __forceinline__ void join_rows(const Job &j, uint32_t g, int pieces, const Seq &q, int head, int tile, int rows,
                                          float *fix, float *total)
{
    constexpr int C = D < 128 ? 1 : D / 128;       // pairs of channels a lane
    const auto slot_of = [&](int p) { return j.slots + (int64_t)(p == 0 ? 2 * g + 1 : 2 * (g + p)) * SLOT<D>; };
    const int here = rows - tile * ROWS < ROWS ? rows - tile * ROWS : ROWS;
    const int row = threadIdx.x >> 4, sub = threadIdx.x & 15;
    f32x2 ml[4];
    float M = -INFINITY, lsum = 0.0f;
    for (int p0 = 0; p0 < pieces; p0 += 64) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 16 * i + sub;
            ml[i] = p < pieces && row < here ? get2(slot_of(p) + 2 * row) : f32x2{-INFINITY, 0.0f};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) M = fmaxf(M, ml[i][0]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
    const float base = base_of(M);

    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int at = 2 * ROWS + (D < 128 ? (lane & 31) * 2 : lane * 2 * C);
    f32x2 v[ROWS / WAVES][C];
#pragma unroll
    for (int r = 0; r < ROWS / WAVES; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) v[r][c] = 0.0f;
    for (int p0 = 0; p0 < pieces; p0 += 64) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 16 * i + sub;
            if (pieces > 64) ml[i] = p < pieces && row < here ? get2(slot_of(p) + 2 * row) : f32x2{-INFINITY, 0.0f};
            const float f = __builtin_amdgcn_exp2f(ml[i][0] - base);
            lsum += ml[i][1] * f;
            fix[(16 * i + sub) * ROWS + row] = f;
        }
        __syncthreads();
        const int n = pieces - p0 < 64 ? pieces - p0 : 64;
#pragma unroll
        for (int r = 0; r < ROWS / WAVES; r += 2) {
            const int r0 = wave + r * WAVES, r1 = r0 + WAVES;
            if (r0 >= here) break;
            constexpr int AHEAD = 8 / C;
            for (int p = 0; p < n; p += AHEAD) {
                f32x2 w[2][AHEAD][C];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float *slot = slot_of(p0 + p + i) + at + 2 * c;
                        w[0][i][c] = p + i < n ? get2(slot + r0 * D) : f32x2(0.0f);
                        w[1][i][c] = p + i < n && r1 < here ? get2(slot + r1 * D) : f32x2(0.0f);
                    }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (p + i >= n) break;
                    const float f0 = fix[(p + i) * ROWS + r0], f1 = fix[(p + i) * ROWS + r1];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        v[r][c] += w[0][i][c] * f0;
                        v[r + 1][c] += w[1][i][c] * f1;
                    }
                }
            }
        }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) lsum += __shfl_xor(lsum, o);
    if (sub == 0) total[row] = lsum;
    __syncthreads();
    if (D < 128 && lane >= 32) return;
#pragma unroll
    for (int r = 0; r < ROWS / WAVES; ++r) {
        const int mine = wave + r * WAVES;
        if (mine >= here) break;
        const float l = total[mine], inv = l != 0.0f ? 1.0f / l : 0.0f;
        const int R = tile * ROWS + mine, i = R / j.per;
        const int64_t y = (int64_t)(q.q0 + i) * j.a.y_token + (int64_t)(head * j.per + (R - i * j.per)) * j.a.y_head;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            store1(j.a.y, j.a.ytype, y + lane * 2 * C + 2 * c, v[r][c][0] * inv);
            store1(j.a.y, j.a.ytype, y + lane * 2 * C + 2 * c + 1, v[r][c][1] * inv);
        }
    }
}

// Workgroups a CU with a workspace, each with its share of the list: no more than its
// registers hold at once, so that none waits for another's end.  (They hold one more for 64
// channels with fp32 queries and for 256 with 16-bit ones.)
template <int D, int QP, int PP> constexpr int RESIDENT = D == 256 ? 1 : QP == 2 ? 2 : 3;

// What the registers are to hold: without a workspace 256 requests of 700 tokens, 16 heads on 2
// of 256, take 31 us with two workgroups a CU and 50 with one.
template <int D, int QP, int PP> constexpr int HELD = D == 256 && QP == 1 ? 2 : RESIDENT<D, QP, PP>;

// Two codes of a word, at bits 4 b of its halves, as f16 subnormals: code * 2^-18 where
// FINE, else code * 2^-24, or 2^-20 for odd b.
template <int B, bool FINE>
__device__ __forceinline__ uint32_t codes(uint32_t w)
{
    if constexpr (FINE) return (B == 0 ? w << 6 : B == 1 ? w << 2 : B == 2 ? w >> 2 : w >> 6) & 0x03c003c0u;
    return (B & 2 ? w >> 8 : w) & (B & 1 ? 0x00f000f0u : 0x000f000fu);
}

template <int T, int D, int QP, int PP>
__global__ __launch_bounds__(256, (HELD<D, QP, PP>)) void kv4_kernel(Job j)
{
    typedef elem_t<T> E;
    constexpr int G = D / 32, Q = G / 2, TILES = D / 16;
    // fp32 queries (QP 2) or results (PP 3): all bits of the products are kept
    constexpr bool FINE_K = QP == 2 || PP == 3, FINE_V = PP == 3;
    constexpr int UP_P = 141 - (int)LAZY;   // P <= 2^LAZY, s < 2^(E - 126) and their product scaled by 2^(UP_P - E) < 2^15
    constexpr int UP_K = FINE_K ? 18 : 24, UP_V = FINE_V ? 18 : 24;   // codes are 2^-UP
    __shared__ float joined[WAVES][ROWS * D];
    __shared__ float stats[WAVES][2][ROWS];
    __shared__ int beyond[WAVES][64];               // each lane's own (a register more spills: 61 -> 63 us)
    __shared__ int16_t apart_q[G][WAVES][64];
    __shared__ uint32_t tmp[4], found[2], arrivals;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, l = lane & 15, h = lane >> 4;
    const int nseq = (int)j.c.nseq;

    // the list's length, and where this workgroup's run of it begins
    uint32_t total, size, at, end, seq_at;
    int s;
    Seq q;
    const auto run_of = [&]() {
        size = (total + j.groups - 1) / j.groups;
        if (j.split && size < LEAST) size = LEAST;
        if (size < 1) size = 1;
        at = blockIdx.x * size;
        end = at + size < total ? at + size : total;
    };
    if (nseq <= 64) {                               // each wave sums them by itself
        Seq mine = {};
        if (lane < nseq) mine = get_seq(j, lane);
        const uint32_t sum = sum_to_lane(lane < nseq ? units(j, mine) : 0);
        total = __builtin_amdgcn_readlane(sum, 63);
        run_of();
        if (at >= end) return;
        s = __popcll(__ballot(sum <= at));           // sequences that end before it
        const auto of = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, s); };
        seq_at = s > 0 ? (uint32_t)__builtin_amdgcn_readlane((int)sum, s - 1) : 0;
        q = {(int)of(mine.q0), (int)of(mine.n), (int)of(mine.length), (int)of(mine.keys), of(mine.blocks), of(mine.tiles)};
    } else {
        uint32_t mine = 0;
        for (int i = threadIdx.x; i < nseq; i += 256) mine = plus(mine, units(j, get_seq(j, i)));
        scan(mine, tmp, total);
        run_of();
        if (at >= end) return;
        uint32_t ahead = 0;
        for (int s0 = 0; s0 < nseq; s0 += 256) {
            const int i = s0 + threadIdx.x;
            const uint32_t u = i < nseq ? units(j, get_seq(j, i)) : 0;
            uint32_t sum;
            const uint32_t before = plus(ahead, scan(u, tmp, sum));
            if (at >= before && at < before + u) {
                found[0] = i;
                found[1] = before;
            }
            ahead = plus(ahead, sum);
            if (ahead > at) break;
        }
        __syncthreads();
        s = __builtin_amdgcn_readfirstlane(found[0]);
        seq_at = __builtin_amdgcn_readfirstlane(found[1]);
        q = get_seq(j, s);
    }

    while (at < end) {
        while (at >= seq_at + units(j, q)) {
            seq_at += units(j, q);
            q = get_seq(j, ++s);
        }
        const uint32_t part = (at - seq_at) / q.blocks;
        const uint32_t first = (at - seq_at) - part * q.blocks;     // list entries of this row before the piece
        const uint32_t left = q.blocks - first;
        const uint32_t entries = left < end - at ? left : end - at;
        const int head = (int)(part / q.tiles), tile = (int)(part - head * q.tiles);
        // the blocks of tokens: all of them where rows are not split
        const int all = q.keys == 0 ? 0 : (q.keys - 1) / 32 + 1;
        const int b0 = j.split ? (int)first : 0;
        const int b1 = j.split && (int)(first + entries) < all ? (int)(first + entries) : all;

        // the pages of this piece's first 64 columns, one a lane
        const int32_t *table = j.c.tables + (int64_t)s * j.c.ld;
        const int page_blocks = j.c.page / 32, width = (int)j.c.width;
        int col = (b0 + wave) / page_blocks, rem = (b0 + wave) - col * page_blocks;
        const int step_col = WAVES / page_blocks, step_rem = WAVES - step_col * page_blocks;
        int col0 = col;
        const auto ids_from = [&](int c) { return c + lane < width ? table[c + lane] : -1; };
        int ids = ids_from(col0);
        const auto next_block = [&]() -> const uint8_t * {
            if (col - col0 >= 64) {
                col0 = col;
                ids = ids_from(col0);
            }
            const int page = __builtin_amdgcn_readlane(ids, col - col0);
            const uint8_t *p = j.c.pages + page * j.c.page_bytes + ((int64_t)head * page_blocks + rem) * (40 * D);
            col += step_col;
            rem += step_rem;
            if (rem >= page_blocks) {
                rem -= page_blocks;
                ++col;
            }
            return page < 0 || page >= j.c.npages ? nullptr : p;
        };

        // this lane's row: its query, scaled into f16, and the sums of its groups
        const int rows = q.n * j.per;
        const int R = tile * ROWS + l;
        const int Rq = R < rows ? R : rows - 1;
        const int qi = Rq / j.per, qh = head * j.per + (Rq - qi * j.per);
        const E *qp = static_cast<const E *>(j.a.q.p) + (int64_t)(q.q0 + qi) * j.a.q.token + (int64_t)qh * j.a.q.head;
        f16x8 qv[QP][G];
        u32x4 qm = {0, 0, 0, 0};                    // the groups' sums in bf16: the first, second, third part in lanes 0.., 16.., 32..
        float F;                                    // t = F times the codes' sums
        bool steep;                                 // and times 2^beyond for some row
        bool uneven;                                // groups of channels have powers of their own, 2^apart_q to the row's
        {
            float f[G][8], qs[G], tops[G], top = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int x = 0; x < 8 / VEC<T>; ++x) {
                    float t[VEC<T>];
                    unpack16<T>(load16<T>(qp + g * 32 + h * 8 + x * VEC<T>), t);
#pragma unroll
                    for (int i = 0; i < VEC<T>; ++i) f[g][x * VEC<T> + i] = t[i];
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                qs[g] = tops[g] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    tops[g] = fmaxf(tops[g], fabsf(f[g][i]));
                    qs[g] += f[g][i];
                }
                qs[g] += __shfl_xor(qs[g], 16);
                qs[g] += __shfl_xor(qs[g], 32);
                tops[g] = fmaxf(tops[g], __shfl_xor(tops[g], 16));
                tops[g] = fmaxf(tops[g], __shfl_xor(tops[g], 32));
                top = fmaxf(top, tops[g]);
            }
            const bool plain = top > 0.0f && top < INFINITY;
            const int e = plain ? __builtin_amdgcn_frexp_expf(top) - 15 : 0;
            int down[G];
            bool far = false;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                down[g] = plain && tops[g] > 0.0f ? e + 15 - __builtin_amdgcn_frexp_expf(tops[g]) : 0;
                far |= down[g] > QNEAR;
            }
            uneven = __any(far);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (!uneven) down[g] = 0;
                else apart_q[g][wave][lane] = (int16_t)-down[g];
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int sh = (!FINE_K && i & 1 ? -4 : 0) - e + down[g];
                    const float v0 = ldexp_f(f[g][2 * i], sh), v1 = ldexp_f(f[g][2 * i + 1], sh);
                    hi[i] = pack_f16(v0, v1);
                    lo[i] = pack_rest(hi[i], v0, v1);
                }
                qv[0][g] = operand(hi[0], hi[1], hi[2], hi[3]);
                if constexpr (QP > 1) qv[1][g] = operand(lo[0], lo[1], lo[2], lo[3]);
                const float v = ldexp_f(qs[g], -UP_K - e);
                const __bf16 p0 = (__bf16)v, p1 = (__bf16)(v - (float)p0), p2 = (__bf16)(v - (float)p0 - (float)p1);
                const __bf16 mine = h == 0 ? p0 : h == 1 ? p1 : p2;
                if (h < 3) qm[g / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, mine) << (16 * (g % 2));
            }
            // F alone may lie beyond fp32 where t does not
            int over = __builtin_amdgcn_frexp_expf(j.a.c) + UP_K + e - 126;
            over = over > 0 ? over : 0;
            F = ldexp_f(j.a.c, UP_K + e - over);
            steep = __any(over > 0);
            if (steep) beyond[wave][lane] = over;
        }
        // the tokens that this row sees: the first `limit` ones; from token `full` on some
        // row of the tile sees less than all
        const int lim = q.length - q.n + qi + 1;
        const int limit = lim < 0 ? 0 : lim < q.keys ? lim : q.keys;
        int full = q.length - q.n + tile * ROWS / j.per + 1;
        full = full < q.keys ? full : q.keys;

        f32x4 o[TILES];
        float mm[G], ref = -INFINITY, sum = 0.0f;
        int E[Q];                                   // what the scales' exponents stay below (biased), in the scales' lanes
        bool apart = false;                         // some scale was outside of E's window
#pragma unroll
        for (int x = 0; x < TILES; ++x) o[x] = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) mm[g] = 0.0f;
#pragma unroll
        for (int x = 0; x < Q; ++x) E[x] = NONE;

        Keys<D> k;
        Values<D> v;
        int b = b0 + wave;
        const uint8_t *here = b < b1 ? next_block() : nullptr;
        if (here) {
            load_keys<D>(here, lane, k);
            load_values<D>(here, lane, v);
        }
        for (; b < b1; b += WAVES) {
            const uint8_t *then = b + WAVES < b1 ? next_block() : nullptr;
            float t[8];
            if (here) {
                const auto scores = [&](auto uneven_c) {
                    constexpr bool UNEVEN = uneven_c.value;
                    each<2>([&](auto uc) {
                        constexpr int u = uc.value;
                        u32x4 m4 = {0, 0, 0, 0};
#pragma unroll
                        for (int g = 0; g < G; g += 2) m4[g / 2] = __builtin_amdgcn_perm(k.m[u][g + 1], k.m[u][g], 0x07060302);
                        f32x4 acc = mfma_bf16_16(m4, qm, f32x4(0.0f));
                        each<G>([&](auto gc) {
                            constexpr int g = gc.value, w = u * G + g;
                            uint32_t c = k.c[w / 4][w % 4];
                            if constexpr (UNEVEN) asm("" : "+v"(c));   // else both ways' codes would be formed ahead of the branch
                            const f16x8 kv = operand(codes<0, FINE_K>(c), codes<1, FINE_K>(c), codes<2, FINE_K>(c), codes<3, FINE_K>(c));
                            f32x4 dot = 0.0f;
                            dot = mfma_f16(kv, qv[0][g], dot);
                            if constexpr (QP > 1) dot = mfma_f16(kv, qv[1][g], dot);
                            if constexpr (UNEVEN) {
                                const int up = apart_q[g][wave][lane];
#pragma unroll
                                for (int r = 0; r < 4; ++r) dot[r] = ldexp_f(dot[r], up);
                            }
                            const float ks = __builtin_bit_cast(float, k.s[g % Q] << 16);
                            each<4>([&](auto rc) {
                                constexpr int r = rc.value, from = (u * 4 + r) * 2 + g / Q;
                                acc[r] += row_bcast<from>(ks) * dot[r];
                            });
                        });
#pragma unroll
                        for (int r = 0; r < 4; ++r) t[u * 4 + r] = acc[r] * F;
                        keep_order();
                    });
                };
                if (__builtin_expect(uneven, false)) scores(std::true_type());
                else scores(std::false_type());
                if (__builtin_expect(steep, false))
#pragma unroll
                    for (int x = 0; x < 8; ++x) t[x] = ldexp_f(t[x], beyond[wave][lane]);
            }
            // the keys' registers are free: the next block's come while this one's values are used
            if (then) load_keys<D>(then, lane, k);
            if (here) {
                const bool tail = b * 32 > full - 32;
                if (tail) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (b * 32 + (x >> 2) * 16 + h * 4 + (x & 3) >= limit) t[x] = -INFINITY;
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
                int skip = 0;                       // words that no row has to do with
                if (tail) {
                    // Words behind the sequence's end hold anything, and a token may stand for NaN that
                    // some rows do not see: such words count as 0, and the groups of the rows that do
                    // see one become NaN.
                    float bad[Q];
                    bool any = false;
#pragma unroll
                    for (int x = 0; x < Q; ++x) {
                        const int slot = (l * Q + x) / G;
                        const uint32_t w = b * 32 + (slot >> 2) * 16 + h * 4 + (slot & 3) < q.keys ? v.s[x] : 0;
                        const bool nan = (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
                        bad[x] = nan ? 1.0f : 0.0f;
                        v.s[x] = nan ? 0 : w;
                        any |= nan;
                        skip |= (nan || b * 32 + (slot >> 2) * 16 + h * 4 + (slot & 3) >= q.keys) << x;
                    }
                    if (__any(any))
                        each<G>([&](auto gc) {
                            constexpr int g = gc.value;
                            each<8>([&](auto xc) {
                                constexpr int x = xc.value;
                                const bool hit = row_bcast<x * 2 + g / Q>(bad[g % Q]) != 0.0f;
                                if (hit && b * 32 + (x >> 2) * 16 + h * 4 + (x & 3) < limit) mm[g] = NAN;
                            });
                        });
                }
                float vs[Q], vm[Q];
                // scales outside of their window
                bool out = false;
#pragma unroll
                for (int x = 0; x < Q; ++x) {
                    vs[x] = __builtin_bit_cast(float, v.s[x] << 16);
                    vm[x] = __builtin_bit_cast(float, v.s[x] & 0xffff0000u);
                    const int e = v.s[x] >> 7 & 0xff;
                    out |= (uint32_t)(E[x] - e) > NEAR && !(skip >> x & 1);
                }
                if (__builtin_expect(__any(out), false)) {
                    bool below = false;
#pragma unroll
                    for (int x = 0; x < Q; ++x) {
                        // lanes of the same parity hold the same groups
                        const int mine = v.s[x] >> 7 & 0xff;
                        int top = mine;
#pragma unroll
                        for (int dist = 2; dist < 64; dist <<= 1) {
                            const int other = __shfl_xor(top, dist);
                            top = other > top ? other : top;
                        }
                        const int was = E[x];
                        if (was < top) E[x] = top + HEAD > NEAR + 1 ? top + HEAD : NEAR + 1;
                        // words before this block may lie anywhere in a window that has moved
                        below |= (was != NONE && E[x] != was) || (E[x] - mine > NEAR && !(skip >> x & 1));
                        const int shift = was - E[x];
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
                    apart |= __any(below);
                }
                float vn[Q];
#pragma unroll
                for (int x = 0; x < Q; ++x) vn[x] = ldexp_f(vs[x], apart ? -8 : UP_P - E[x]);   // apart: P s < 2^126
                each<G>([&](auto gc) {
                    constexpr int g = gc.value;
                    mm[g] = row_dot<g / Q>(mm[g], vm[g % Q], t);
                    float w[8];
                    each<8>([&](auto xc) { w[xc.value] = t[xc.value] * row_bcast<xc.value * 2 + g / Q>(vn[g % Q]); });
                    int back = 0;                   // 2^-back: O's unit to that of these P s, never a larger one
                    if (__builtin_expect(apart, false)) {
                        float most = w[0], held_most = 0.0f;
#pragma unroll
                        for (int x = 1; x < 8; ++x) most = fmaxf(most, w[x]);
                        for_o<g>(o, [&](float &v) { held_most = fmaxf(held_most, fabsf(v)); });
#pragma unroll
                        for (int dist = 16; dist < 64; dist <<= 1) {
                            most = fmaxf(most, __shfl_xor(most, dist));
                            held_most = fmaxf(held_most, __shfl_xor(held_most, dist));
                        }
                        const int unit = UP_P + 8 - __builtin_amdgcn_readlane(E[g % Q], g / Q);
                        back = most > 0.0f ? unit - 15 + __builtin_amdgcn_frexp_expf(most) : 0;
                        // O stays below 2^100: what is that far below it adds nothing
                        const int least = held_most > 0.0f ? __builtin_amdgcn_frexp_expf(held_most) - 100 : back;
                        back = back > least ? back : least;
#pragma unroll
                        for (int x = 0; x < 8; ++x) w[x] = ldexp_f(w[x], unit - back);
                        for_o<g>(o, [&](float &v) { v = ldexp_f(v, -back); });
                    }
                    const uint32_t p0 = pack_f16(w[0], w[1]), p1 = pack_f16(w[2], w[3]), p2 = pack_f16(w[4], w[5]), p3 = pack_f16(w[6], w[7]);
                    const f16x8 hi = operand(p0, p1, p2, p3);
                    f16x8 lo;
                    if constexpr (PP > 1)
                        lo = operand(pack_rest(p0, w[0], w[1]), pack_rest(p1, w[2], w[3]), pack_rest(p2, w[4], w[5]), pack_rest(p3, w[6], w[7]));
                    each<2>([&](auto yc) {
                        constexpr int n = 2 * g + yc.value, bit = n % 4;
                        uint32_t c[4];
                        each<4>([&](auto pc) {
                            constexpr int i = pc.value * (D / 64) + n / 4;
                            c[pc.value] = codes<bit, FINE_V>(v.c[i / 4][i % 4]);
                        });
                        const f16x8 vv = operand(c[0], c[1], c[2], c[3]);
                        o[n] = mfma_f16(vv, hi, o[n]);
                        if constexpr (PP > 1) o[n] = mfma_f16(vv, lo, o[n]);
                    });
                    if (__builtin_expect(apart, false)) for_o<g>(o, [&](float &v) { v = ldexp_f(v, back); });
                    keep_order();
                });
            }
            if (then) load_values<D>(then, lane, v);
            here = then;
        }

        // the wave's rows: channels 16 n + 4 h + r of row l in o[n][r]
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        each<G>([&](auto gc) {
            constexpr int g = gc.value;
            mm[g] += __shfl_xor(mm[g], 16);
            mm[g] += __shfl_xor(mm[g], 32);
            const int e = __builtin_amdgcn_readlane(E[g % Q], g / Q) - UP_P;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int n = 2 * g + y;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    o[n][r] = ldexp_f(o[n][r], e + UP_V - (!FINE_V && n & 1 ? 4 : 0)) + mm[g];
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
        // this piece is the row's first one in its workgroup's second slot, or in the first slot a later one
        float *slot = j.slots + (int64_t)(blockIdx.x * 2 + (first == 0 ? 1 : 0)) * SLOT<D>;
        for (int x = threadIdx.x * 4; x < ROWS * D; x += 1024) {
            const int row = x / D, Ry = tile * ROWS + row;
            if (Ry >= rows) break;
            f32x4 v4 = *reinterpret_cast<const f32x4 *>(&joined[0][x]);
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v4 += *reinterpret_cast<const f32x4 *>(&joined[w][x]);
            float M = stats[0][0][row], lsum = 0.0f;
#pragma unroll
            for (int w = 1; w < WAVES; ++w) M = fmaxf(M, stats[w][0][row]);
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                lsum += stats[w][1][row] * __builtin_amdgcn_exp2f(stats[w][0][row] - base_of(M));
            if (whole) {
                const float inv = lsum != 0.0f ? 1.0f / lsum : 0.0f;
                const float f[4] = {v4[0] * inv, v4[1] * inv, v4[2] * inv, v4[3] * inv};
                const int i = Ry / j.per;
                store4(j.a.y, j.a.ytype, (int64_t)(q.q0 + i) * j.a.y_token +
                                             (int64_t)(head * j.per + (Ry - i * j.per)) * j.a.y_head + x % D, f);
            } else {
                put2(slot + 2 * ROWS + x, v4[0], v4[1]);
                put2(slot + 2 * ROWS + x + 2, v4[2], v4[3]);
                if (x % D == 0) put2(slot + 2 * row, M, lsum);
            }
        }
        if (!whole) {
            const uint32_t row_at = at - first, owner = row_at / size;
            const uint32_t row_end = min(row_at + q.blocks, total);   // where the list is cut off as well
            const int pieces = (int)((row_end - 1) / size - owner) + 1;
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the piece is at the coherence point
            __syncthreads();
            if (threadIdx.x == 0)
                arrivals = __hip_atomic_fetch_add(j.arrived + owner, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (arrivals == (uint32_t)pieces - 1) {
                join_rows<D>(j, owner, pieces, q, head, tile, rows, &joined[0][0], &stats[0][0][0]);
                if (threadIdx.x == 0)
                    __hip_atomic_store(j.arrived + owner, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        at += entries;
    }
}

template <int T, int D, int QP, int PP>
int launch_typed(Job j, hipStream_t stream)
{
    // rows of 16 over all sequences, and their blocks, are at most
    const int64_t rows = j.c.heads * ((j.a.nt * j.per) / ROWS + j.c.nseq);
    const int64_t room = j.c.width * j.c.page, blocks = room / 32 + 1;
    int64_t groups = rows;
    j.split = j.a.ws != nullptr;
    j.room = room < INT32_MAX ? (int)room : INT32_MAX;
    // the list is counted in 32 bits
    const int64_t most_blocks = blocks < (int64_t(1) << 26) ? blocks : int64_t(1) << 26;   // of 2^31 tokens
    if (j.a.nt * j.per >= (int64_t(1) << 31) || rows > ((int64_t(1) << 31) - 1) / (j.split ? most_blocks : 1)) return -1;
    if (j.split) {
        int64_t most = ATTEND_WS_BYTES / (2 * SLOT<D> * 4);
        if (most > CUS * RESIDENT<D, QP, PP>) most = CUS * RESIDENT<D, QP, PP>;
        const int64_t want = (rows * most_blocks + WAVES - 1) / WAVES;
        groups = want < 1 ? 1 : want < most ? want : most;
        j.slots = static_cast<float *>(j.a.ws);
        j.arrived = reinterpret_cast<uint32_t *>(static_cast<char *>(j.a.ws) + ATTEND_WS_BYTES);
    }
    if (groups > launch_groups(256) || groups >= (int64_t(1) << 31)) return -1;
    j.groups = (int)groups;
    return launch_kernel(kv4_kernel<T, D, QP, PP>, dim3((unsigned)groups), dim3(256), stream, j);
}

template <int D>
int launch_dim(const Job &j, hipStream_t stream)
{
    const auto by_result = [&](auto t) {
        constexpr int T = t.value, QP = T == T_F32 ? 2 : 1;
        if (j.a.ytype == T_BF16) return launch_typed<T, D, QP, 1>(j, stream);
        if (j.a.ytype == T_F16) return launch_typed<T, D, QP, 2>(j, stream);
        return launch_typed<T, D, QP, 3>(j, stream);
    };
    if (j.a.type == T_F32) return by_result(std::integral_constant<int, T_F32>());
    if (j.a.type == T_BF16) return by_result(std::integral_constant<int, T_BF16>());
    return by_result(std::integral_constant<int, T_F16>());
}

}  // namespace

int launch_attend_kv4(const Kv4 &c, const Kv4Attend &a, hipStream_t stream)
{
    Job j = {c, a, a.hq / c.heads, 0, 0, 0, nullptr, nullptr};
    if (c.d == 64) return launch_dim<64>(j, stream);
    if (c.d == 128) return launch_dim<128>(j, stream);
    return launch_dim<256>(j, stream);
}

}  // namespace qig
