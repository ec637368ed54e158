// attend_prompt.hip -- attention over whole prompts, packed one behind the other.
//
//   y_i = sum_j p_ij v_j,  p_ij = exp(scale q_i . k_j) / sum_j exp(scale q_i . k_j)
//
// over the keys j that query i sees.  One pass over the keys: with t_ij =
// c q_i . k_j, c = scale * log2(e), and the running maximum m of t,
//   P = 2^(t - m),  l = l * 2^(m_old - m) + sum P,  O = O * 2^(m_old - m) + P V,
// y = O / l; l, m and O are fp32.
//
// Both products are formed transposed: S^T = K Q^T has a query a lane, so that its
// maximum and sum need one exchange between the wave's halves, its correction is
// a factor a lane, and S^T's registers are P^T's operand for O^T = V^T P^T as
// they are: which keys a lane holds decides only which keys of V it must be
// given.
#include "qig_attend_device.h"
#include "qig_launch.h"

namespace qig {
namespace {

// Which sequence a workgroup works on.  With `per` rows a query, sequence i's tiles of
// BM rows have the slots from starts[i] * per / BM + i on: those of the next begin
// behind its last one, whatever its length, so that nt * per / BM + nseq slots are
// enough and no sum over the sequences before is needed.  Some slots stay empty.
struct Tile {
    int q0, nq;      // first packed query of the sequence, queries
    int k0, nk;
    int rows, row0;  // (query, head) rows of the sequence, the first one of the tile
};

template <int BM>
__device__ __forceinline__ bool find_rows(const PromptArgs &a, int slot, int per, Tile &t)
{
    const int32_t *starts = a.starts;
    const int64_t nt = a.nt;
    const auto first_slot = [&](int s) { return held(starts[s], nt) * per / BM + s; };   // nt * per < 2^31
    const int i = __builtin_amdgcn_readfirstlane(
        count_first((int)a.nseq, [&](int s) { return first_slot(s) <= slot; }) - 1);
    if (i < 0) return false;
    t.q0 = held(a.starts[i], a.nt);
    t.nq = held(a.starts[i + 1], a.nt) - t.q0;
    t.k0 = held(a.k_starts[i], a.nk);
    t.nk = held(a.k_starts[i + 1], a.nk) - t.k0;
    if (t.nk < 0) t.nk = 0;
    t.rows = t.nq * per;
    const int64_t row0 = (int64_t)(slot - first_slot(i)) * BM;
    t.row0 = (int)row0;
    return row0 >= 0 && row0 < t.rows;   // below 0: starts that decrease
}

__device__ __forceinline__ bool finite(float v) { return __builtin_fabsf(v) < INFINITY; }

// Values of a 16-byte unit that are not finite go (and whether there was one is returned).
template <int T>
__device__ __forceinline__ int clean(u32x4 &v)
{
    uint32_t bad = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        constexpr uint32_t EXP = T == T_F32 ? 0x7f800000 : T == T_F16 ? 0x7c00 : 0x7f80;
        const uint32_t w = v[j], lo = (w & EXP) == EXP, hi = T != T_F32 && ((w >> 16) & EXP) == EXP;
        bad |= lo | hi;
        v[j] = w & ~((lo ? T == T_F32 ? ~0u : 0xffffu : 0u) | (hi ? 0xffff0000u : 0u));
    }
    return (int)bad;
}

// A value that is not finite must reach the queries that see it and no other one; in the
// product its 0 * NaN would reach them all.  So in steps where some query does not
// see some key such values are 0 in LDS, and if there were any the sums that saw one
// become NaN here: sums over the keys (seen) * (not finite), on the fp32 MFMA, whose
// operands and results lie as S^T's and O^T's.
template <int D, typename E>
__device__ __forceinline__ void poison_tile(f32x16 &o, const E *vp, int64_t step, int k0, int nk, int c, int d,
                                                      int end, int h)
{
    f32x16 hits = 0.0f;
#pragma unroll 1
    for (int r = 0; r < 16; ++r) {   // a loop: it hardly ever runs, and its registers would be the kernel's
        const int key = k0 + mfma_row(r, h);
        const bool bad = key < nk && c < d && !finite((float)vp[(int64_t)key * step + c]);
        hits = __builtin_amdgcn_mfma_f32_32x32x2f32(bad ? 1.0f : 0.0f, key < end ? 1.0f : 0.0f, hits, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r)
        if (hits[r] > 0.0f) o[r] = NAN;
}

template <int D, typename E>
__device__ __forceinline__ void poison(f32x16 (&o)[D / 32], const E *vp, int64_t step, int k0, int nk, int d, int end,
                                       int n, int h)
{
#pragma unroll
    for (int x = 0; x < D / 32; ++x) poison_tile<D, E>(o[x], vp, step, k0, nk, 32 * x + n, d, end, h);
}

// A workgroup's tile in the list of (tile, key head) pairs, from the last sequence's last tile
// on: within a causal sequence the longest come first; across sequences nothing orders
// them, so that a batch may end on its longest one.  Of the first 512 workgroups a CU gets one of the first and one of the second 256: the second
// are taken in reverse, so that a CU with a long tile has a short one beside it; later ones
// go where there is room.  2630 fp32 tokens, 28 heads on 4 of 128 (576 tiles): 507 us in the
// list's order, 436 so.  Every other 256 in reverse: the same there, but 388 for 367 with
// 4 x 1000 tokens of 32 heads on 8, and 63 for 58 in fp16.
__device__ __forceinline__ uint32_t place(uint32_t block, uint32_t groups)
{
    return block >> 8 == 1 && groups >= 512 ? 256 + 255 - (block & 255) : block;
}

// One 1 KB copy of 16 bytes a lane, from base + off to LDS byte address lds + 16 lane.
// The compiler does not see it: what it brings is read behind landed() and a barrier.
// s_nop 4 covers the waits behind writes of the scalar base and of M0.
__device__ __forceinline__ void copy16(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_nop 4\n\t"
                 "global_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(base), "{m0}"(lds)
                 : "memory");
}
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// How keys and values reach LDS: through registers, for rows at any address; copied
// straight into it, for rows of d = D elements at multiples of 16 bytes; and the same with
// d < D (PADDED), where the lanes of units behind d copy none of the keys, whose places are
// zeroed once, and any of the values, whose sums are not written.  1024 causal tokens, 32
// heads on 8 of 96: fp32 175 us through registers, 155 so; fp16 32 and 29.5.
enum { REGISTERS, STRAIGHT, PADDED };

// fp32 operands on v_mfma_f32_32x32x2_f32.  Rows are (query, head of the group) pairs of
// one key head, heads fastest: all heads that share a key head read one copy of it
// from LDS, and a tile spans few queries, so that little of its last steps is masked.  A
// wave holds 32 rows, a workgroup 4 waves; 32 keys a step.
//   S^T: lane (n = lane % 32, h = lane / 32) gives key n's and row n's channels
//   8 j + 4 h + i: MFMA i of chunk j then sums channels 8 j + i and 8 j + 4 + i, and
//   four of them need one 16-byte read.
//   S^T register r of lane (n, h): row n, key 8 (r / 4) + 4 h + r % 4; MFMA r of
//   O^T sums these two keys.
// LDS: 16-byte unit u of row r of K stands at u ^ (r & 15) (rows of 256 bytes), so that 16
// lanes reading one unit of 16 rows meet in no bank, and of V at u ^ 8 (r / 4 & 1), so
// that the two keys of a read do not.
// Measured, 2630 causal tokens, 28 heads on 4 of 128: 438 us, 113 TFLOP/s; a large fp32
// matrix product reaches 154.  The MFMAs are 75% of the time: they have the rate of the
// vector units here, and the softmax's instructions come on top.  With a head a tile
// and keys through registers it took 592.
template <int D, int COPY>
__global__ __launch_bounds__(256, D > 128 ? 1 : 2) void prompt_f32(PromptArgs a, int slots, int per)
{
    constexpr int CH = D / 4, N = 32 * CH / 256, BM = 128;   // 16-byte units of a row; of a thread
    constexpr bool DIRECT = COPY != REGISTERS, PAD = COPY == PADDED;
    __shared__ __align__(16) float lds_k[2][32 * D], lds_v[2][32 * D];
    const uint32_t work = place(blockIdx.x, gridDim.x);
    const int kvh = (int)(work % (uint32_t)a.hkv);
    Tile t;
    if (!find_rows<BM>(a, slots - 1 - (int)(work / (uint32_t)a.hkv), per, t)) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
    const int d = a.d;
    const float *kp = static_cast<const float *>(a.k.p) + (int64_t)t.k0 * a.k.token + (int64_t)kvh * a.k.head;
    const float *vp = static_cast<const float *>(a.v.p) + (int64_t)t.k0 * a.v.token + (int64_t)kvh * a.v.head;

    const uint32_t rows = t.rows, mine = t.row0 + wave * 32 + n;
    const auto query_of = [&](uint32_t r) { return (int)((r < rows ? r : rows - 1) / (uint32_t)per); };
    const int query = query_of(mine), head = kvh * per + (int)((mine < rows ? mine : rows - 1) - (uint32_t)query * per);
    const float *qp = static_cast<const float *>(a.q.p) + (int64_t)(t.q0 + query) * a.q.token + (int64_t)head * a.q.head;
    f32x4 q[D / 8];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
        const int c = 8 * j + 4 * h;
        q[j] = c < d ? __builtin_bit_cast(f32x4, load16<T_F32>(qp + c)) : f32x4(0.0f);
    }

    // the keys that this lane's, its wave's and its workgroup's rows see
    const int off = t.nk - t.nq;
    const auto end_of = [&](int i) {
        const int e = a.causal ? off + i + 1 : t.nk;
        return e < 0 ? 0 : e > t.nk ? t.nk : e;
    };
    const int end = end_of(query);
    const int kend = end_of(query_of(t.row0 + BM - 1)), all_full = end_of(query_of(t.row0));
    const int wave_end = __builtin_amdgcn_readfirstlane(end_of(query_of(t.row0 + wave * 32 + 31)));
    const int wave_full = __builtin_amdgcn_readfirstlane(end_of(query_of(t.row0 + wave * 32)));
    const auto masks_at = [&](int k0) { return k0 + 32 > all_full; };
    const auto at_k = [](int r, int c) { return r * CH + (c ^ (r & 15)); };
    const auto at_v = [](int r, int c) { return r * CH + (c ^ (r & 4) << 1); };

    uint32_t k_off[DIRECT ? N : 1], v_off[DIRECT ? N : 1], k_in = 0;
    const auto offsets = [&](int keys) {           // of the copies, keys beyond the last one being that again
#pragma unroll
        for (int i = 0; i < (DIRECT ? N : 0); ++i) {
            const int u = i * 256 + threadIdx.x, r = u / CH, c = u % CH, at = r < keys ? r : keys - 1;
            const int ck = c ^ (r & 15), cv = c ^ (r & 4) << 1;
            k_off[i] = (uint32_t)at * (uint32_t)a.k.token * 4u + ck * 16;
            v_off[i] = (uint32_t)at * (uint32_t)a.v.token * 4u + (!PAD || 4 * cv < d ? cv : 0) * 16;
            k_in |= (uint32_t)(4 * ck < d) << i;
        }
    };
    offsets(32);
    if constexpr (PAD) {
        for (int i = threadIdx.x; i < 2 * 32 * D; i += 256) (&lds_k[0][0])[i] = 0.0f;
        __syncthreads();
    }
    const uint32_t k_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float *)&lds_k[0][0];
    const uint32_t v_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float *)&lds_v[0][0];
    const int first_wave = __builtin_amdgcn_readfirstlane(threadIdx.x & ~63);
    const auto load = [&](int k0, int buf) {
        if constexpr (DIRECT) {
            if (t.nk - k0 < 32) offsets(t.nk - k0);
            const float *kb = kp + (int64_t)k0 * a.k.token, *vb = vp + (int64_t)k0 * a.v.token;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (!PAD || k_in >> i & 1) copy16(kb, k_off[i], k_lds + (uint32_t)(buf * 32 * CH + i * 256 + first_wave) * 16);
#pragma unroll
            for (int i = 0; i < N; ++i) copy16(vb, v_off[i], v_lds + (uint32_t)(buf * 32 * CH + i * 256 + first_wave) * 16);
        } else {
#pragma unroll 2
            for (int i = 0; i < N; ++i) {
                const int u = i * 256 + threadIdx.x, r = u / CH, c = u % CH;
                u32x4 kv = {0, 0, 0, 0}, vv = kv;
                if (k0 + r < t.nk && 4 * c < d) {
                    kv = load16<T_F32>(kp + (int64_t)(k0 + r) * a.k.token + 4 * c);
                    vv = load16<T_F32>(vp + (int64_t)(k0 + r) * a.v.token + 4 * c);
                }
                reinterpret_cast<u32x4 *>(lds_k[buf])[at_k(r, c)] = kv;
                reinterpret_cast<u32x4 *>(lds_v[buf])[at_v(r, c)] = vv;
            }
        }
    };
    // The step's keys and values are in LDS for all waves; with masks whether there was a
    // value that is not finite.
    const auto arrive = [&](int buf, bool masks) {
        if constexpr (DIRECT) landed();
        __syncthreads();
        if (!masks) return 0;
        int bad = 0;
        for (int i = threadIdx.x; i < 32 * D; i += 256) {
            if (!finite(lds_v[buf][i])) {
                lds_v[buf][i] = 0.0f;
                bad = 1;
            }
        }
        return __syncthreads_or(bad);
    };

    f32x16 o[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x) o[x] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    int bad = 0;
    if (kend > 0) {
        load(0, 0);
        bad = arrive(0, masks_at(0));
    }
    for (int k0 = 0, buf = 0; k0 < kend; k0 += 32, buf ^= 1) {
        const bool more = k0 + 32 < kend;
        if (more) load(k0 + 32, buf ^ 1);
        if (k0 < wave_end) {
            f32x16 s = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                const f32x4 k4 = reinterpret_cast<const f32x4 *>(lds_k[buf])[at_k(n, 2 * j + h)];
#pragma unroll
                for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_32x32x2f32(k4[i], q[j][i], s, 0, 0, 0);
            }
            if (k0 + 32 > wave_full) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (k0 + mfma_row(r, h) >= end) s[r] = -INFINITY;
            }
            float top = s[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
            top = fmaxf(top, __shfl_xor(top, 32));
            const float mn = fmaxf(m, top * a.c);
            const float ref = mn == -INFINITY ? 0.0f : mn;
            const float fix = __builtin_amdgcn_exp2f(m - ref);
            m = mn;
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], a.c, -ref));
                sum += s[r];
            }
            l = l * fix + sum;
            if (__any(fix != 1.0f)) {
#pragma unroll
                for (int x = 0; x < D / 32; ++x) o[x] *= fix;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r)
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const int key = mfma_row(r, h);
                    const float v = lds_v[buf][at_v(key, 8 * x + (n >> 2)) * 4 + (n & 3)];
                    o[x] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, s[r], o[x], 0, 0, 0);
                }
            if (bad) poison<D, float>(o, vp, a.v.token, k0, t.nk, d, end, n, h);
        }
        bad = more ? arrive(buf ^ 1, masks_at(k0 + 32)) : 0;
    }
    l += __shfl_xor(l, 32);
    if (mine >= rows) return;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    const int64_t at = (int64_t)(t.q0 + query) * a.y_token + (int64_t)head * a.y_head;
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const int c = 32 * x + mfma_row(r, h);   // four channels in a row
            const float f[4] = {o[x][r] * inv, o[x][r + 1] * inv, o[x][r + 2] * inv, o[x][r + 3] * inv};
            if (c < d) store4(a.y, a.ytype, at + c, f);
        }
}

// 16-bit operands on v_mfma_f32_32x32x16 (bf16 or f16).  Rows are (query, head of the
// group) pairs of one key head, heads fastest, 32 a wave: all heads that share a key
// head read one copy of it from LDS, and a tile of 32 W rows spans few queries, so
// that little of its last steps is masked.
//   S^T: lane (n, h) gives key n's and row n's channels 16 x + 8 h .. + 7.
//   S^T's registers 8 y .. 8 y + 7 of lane (n, h), rounded, are row n's operand for the
//   keys 16 y + {4 h + i, 8 + 4 h + i}, i < 4; V's, four keys of a channel at a time, come
//   from ds_read_b64_tr_b16, which turns 4 keys by 16 channels in each 16 lanes.
// LDS: 16-byte units of a row of K stand at unit ^ (row & 15) (rows of 128 bytes: ^ (row /
// 2 & 7)), so that 16 lanes reading one unit of 16 rows meet in no bank; those of V at
// unit ^ 4 (row & 3) (^ 4 (row / 2 & 1)), so that the four keys' 64 bytes of a
// transposing read do not either.
// The reference of a row's exponents follows its maximum only when that is 2^LAZY above
// it: most steps then correct nothing.  P <= 2^LAZY, times 2^6 in f16, where it
// then loses bits only below 2^-20 of the reference (and no more than 2^-31 of it).
// Measured, causal, 28 heads on 4 of 128, bf16: 8191 tokens 455-490 us, 980-1060 TFLOP/s; a
// large bf16 matrix product reaches 1407.  MFMAs take 49% of a SIMD's cycles, vector
// instructions (a power, a conversion and a sum for each score) 44%, at 2.0 GHz; LDS
// 25%, without conflicts: the two kinds of instructions hardly run beside each other, so
// that their sum bounds it.  Slower: the next scores' product beside this one's values
// (467 to 454, and 70 to 55 us for 24 ragged prompts of 64 channels, for registers),
// 32 keys a step (531 to 475), eight waves a workgroup (480 to 463, 76 to 56), 16 rows a
// wave (twice the LDS reads: 67 to 55), 64 rows a workgroup (67 to 58).
constexpr float LAZY = 8.0f;

template <int T> struct Mfma16;
template <> struct Mfma16<T_BF16> {
    typedef bf16x8 type;
    static constexpr float UP = 0.0f;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
    }
    static __device__ __forceinline__ f32x16 mul(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(type, a), __builtin_bit_cast(type, b), c, 0, 0,
                                                       0);
    }
};
template <> struct Mfma16<T_F16> {
    typedef f16x8 type;
    static constexpr float UP = 6.0f;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
    }
    static __device__ __forceinline__ f32x16 mul(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(type, a), __builtin_bit_cast(type, b), c, 0, 0, 0);
    }
};

// Four keys of one channel: 16 lanes hand in the addresses of 4 keys' 16 channels.
__device__ __forceinline__ u32x2 read_turned(const uint16_t *p)
{
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p)));
}

template <int D> __device__ __forceinline__ int swz_k(int row) { return D == 64 ? (row >> 1) & 7 : row & 15; }
template <int D> __device__ __forceinline__ int swz_v(int row) { return D == 64 ? (row >> 1 & 1) << 2 : (row & 3) << 2; }

// The lane that copies a unit asks for the one that belongs there.
template <int T, int D, int W, int KT, int COPY>
__global__ __launch_bounds__(64 * W, D > 128 ? 1 : 2) void prompt_16(PromptArgs a, int slots, int per)
{
    typedef elem_t<T> E;
    typedef Mfma16<T> M;
    constexpr int NT = 64 * W, BM = 32 * W, CH = D / 8, N = KT * CH / NT;
    constexpr bool DIRECT = COPY != REGISTERS, PAD = COPY == PADDED;
    __shared__ __align__(16) uint16_t lds_k[2][KT * D], lds_v[2][KT * D];
    const uint32_t work = place(blockIdx.x, gridDim.x);
    const int kvh = (int)(work % (uint32_t)a.hkv);
    Tile t;
    if (!find_rows<BM>(a, slots - 1 - (int)(work / (uint32_t)a.hkv), per, t)) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
    const int d = a.d;
    const E *kp = static_cast<const E *>(a.k.p) + (int64_t)t.k0 * a.k.token + (int64_t)kvh * a.k.head;
    const E *vp = static_cast<const E *>(a.v.p) + (int64_t)t.k0 * a.v.token + (int64_t)kvh * a.v.head;

    const uint32_t rows = t.rows, mine = t.row0 + wave * 32 + n;
    const auto query_of = [&](uint32_t r) { return (int)((r < rows ? r : rows - 1) / (uint32_t)per); };
    const int query = query_of(mine), head = kvh * per + (int)((mine < rows ? mine : rows - 1) - (uint32_t)query * per);
    const E *qp = static_cast<const E *>(a.q.p) + (int64_t)(t.q0 + query) * a.q.token + (int64_t)head * a.q.head;
    u32x4 q[D / 16];
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
        const int c = 16 * x + 8 * h;
        q[x] = c < d ? load16<T>(qp + c) : u32x4{0, 0, 0, 0};
    }

    const int off = t.nk - t.nq;
    const auto end_of = [&](int i) {
        const int e = a.causal ? off + i + 1 : t.nk;
        return e < 0 ? 0 : e > t.nk ? t.nk : e;
    };
    const int end = end_of(query);
    const int kend = end_of(query_of(t.row0 + BM - 1)), all_full = end_of(query_of(t.row0));
    const int wave_end = __builtin_amdgcn_readfirstlane(end_of(query_of(t.row0 + wave * 32 + 31)));
    const int wave_full = __builtin_amdgcn_readfirstlane(end_of(query_of(t.row0 + wave * 32)));

    u32x4 ks[DIRECT ? 1 : N], vs[DIRECT ? 1 : N];
    uint32_t k_off[DIRECT ? N : 1], v_off[DIRECT ? N : 1], k_in = 0;
    const auto offsets = [&](int rows) {         // of the copies, keys beyond the last one being that again
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = i * NT + threadIdx.x, r = u / CH, c = u % CH, at = r < rows ? r : rows - 1;
            const int ck = c ^ swz_k<D>(r), cv = c ^ swz_v<D>(r);
            k_off[i] = (uint32_t)at * (uint32_t)a.k.token * 2u + ck * 16;
            v_off[i] = (uint32_t)at * (uint32_t)a.v.token * 2u + (!PAD || 8 * cv < d ? cv : 0) * 16;
            k_in |= (uint32_t)(8 * ck < d) << i;
        }
    };
    if constexpr (DIRECT) offsets(KT);
    if constexpr (PAD) {
        for (int i = threadIdx.x; i < 2 * KT * D / 2; i += NT) reinterpret_cast<uint32_t *>(&lds_k[0][0])[i] = 0;
        __syncthreads();
    }
    const uint32_t k_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t *)&lds_k[0][0];
    const uint32_t v_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t *)&lds_v[0][0];
    const int first_wave = __builtin_amdgcn_readfirstlane(threadIdx.x & ~63);
    const auto load = [&](int k0, int buf) {
        if constexpr (DIRECT) {
            if (t.nk - k0 < KT) offsets(t.nk - k0);
            const E *kb = kp + (int64_t)k0 * a.k.token, *vb = vp + (int64_t)k0 * a.v.token;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (!PAD || k_in >> i & 1) copy16(kb, k_off[i], k_lds + (uint32_t)(buf * KT * CH + i * NT + first_wave) * 16);
#pragma unroll
            for (int i = 0; i < N; ++i) copy16(vb, v_off[i], v_lds + (uint32_t)(buf * KT * CH + i * NT + first_wave) * 16);
            return;
        }
#pragma unroll
        for (int i = 0; i < (DIRECT ? 0 : N); ++i) {
            const int u = i * NT + threadIdx.x, r = u / CH, c = (u % CH) * 8;
            ks[i] = vs[i] = u32x4{0, 0, 0, 0};
            if (k0 + r < t.nk && c < d) {
                ks[i] = load16<T>(kp + (int64_t)(k0 + r) * a.k.token + c);
                vs[i] = load16<T>(vp + (int64_t)(k0 + r) * a.v.token + c);
            }
        }
    };
    // The step's keys and values are in LDS for all waves; with masks whether there was a
    // value that is not finite.
    const auto arrive = [&](int buf, bool masks) {
        int bad = 0;
        if constexpr (DIRECT) {
            landed();
            __syncthreads();
            if (!masks) return 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {        // all in place: no step with masks is before another without
                u32x4 *at = reinterpret_cast<u32x4 *>(&lds_v[buf][(i * NT + threadIdx.x) * 8]);
                u32x4 v = *at;
                if (clean<T>(v)) {
                    *at = v;
                    bad = 1;
                }
            }
            return __syncthreads_or(bad);
        }
#pragma unroll
        for (int i = 0; i < (DIRECT ? 0 : N); ++i) {
            const int u = i * NT + threadIdx.x, r = u / CH, c = u % CH;
            *reinterpret_cast<u32x4 *>(&lds_k[buf][(r * CH + (c ^ swz_k<D>(r))) * 8]) = ks[i];
            if (masks) bad |= clean<T>(vs[i]);
            *reinterpret_cast<u32x4 *>(&lds_v[buf][(r * CH + (c ^ swz_v<D>(r))) * 8]) = vs[i];
        }
        if (masks) return __syncthreads_or(bad);
        __syncthreads();
        return 0;
    };
    const auto masks_at = [&](int k0) { return k0 + KT > all_full; };

    f32x16 o[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x) o[x] = 0.0f;
    float ref = -INFINITY, l = 0.0f;
    const int turned = ((lane >> 5) * 4 + ((lane & 15) >> 2)) * D;         // this lane's key in a transposing read
    const int turned_c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);         // its unit within 32 channels
    const int turned_x = swz_v<D>((lane & 15) >> 2);

    int bad = 0;
    if (kend > 0) {
        load(0, 0);
        bad = arrive(0, masks_at(0));
    }
    for (int k0 = 0, buf = 0; k0 < kend; k0 += KT, buf ^= 1) {
        const bool more = k0 + KT < kend;
        if (more) load(k0 + KT, buf ^ 1);
        if (k0 < wave_end) {
            f32x16 s[KT / 32];
#pragma unroll
            for (int y = 0; y < KT / 32; ++y) s[y] = 0.0f;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {     // two sums in turn: none waits for its own last product
#pragma unroll
                for (int y = 0; y < KT / 32; ++y) {
                    const u32x4 kv = *reinterpret_cast<const u32x4 *>(
                        &lds_k[buf][((y * 32 + n) * CH + ((2 * x + h) ^ swz_k<D>(n))) * 8]);
                    s[y] = M::mul(kv, q[x], s[y]);
                }
            }
            if (k0 + KT > wave_full) {
#pragma unroll
                for (int y = 0; y < KT / 32; ++y)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (k0 + y * 32 + mfma_row(r, h) >= end) s[y][r] = -INFINITY;
            }
            float top = s[0][0];
#pragma unroll
            for (int y = 0; y < KT / 32; ++y)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, s[y][r]);
            top *= a.c;
            if (__any(top > ref + LAZY)) {          // also the first time
                top = fmaxf(top, __shfl_xor(top, 32));
                const float to = fmaxf(ref, top);
                const float fix = __builtin_amdgcn_exp2f(ref - (to == -INFINITY ? 0.0f : to));
                ref = to;
                l *= fix;
#pragma unroll
                for (int x = 0; x < D / 32; ++x) o[x] *= fix;
            }
            const float base = ref == -INFINITY ? 0.0f : ref - M::UP;
            u32x4 p[KT / 16];
#pragma unroll
            for (int y = 0; y < KT / 16; ++y) {
                float f[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    f[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[y / 2][8 * (y % 2) + r], a.c, -base));
                    l += f[r];
                }
                p[y] = u32x4{M::pack(f[0], f[1]), M::pack(f[2], f[3]), M::pack(f[4], f[5]), M::pack(f[6], f[7])};
            }
#pragma unroll
            for (int y = 0; y < KT / 16; ++y)
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint16_t *at = &lds_v[buf][turned + 16 * y * D + (((4 * x + turned_c) ^ turned_x) * 8) + (lane & 1) * 4];
                    const u32x2 v0 = read_turned(at), v1 = read_turned(at + 8 * D);
                    o[x] = M::mul(u32x4{v0[0], v0[1], v1[0], v1[1]}, p[y], o[x]);
                }
            if (bad) {
#pragma unroll
                for (int y = 0; y < KT / 32; ++y) poison<D, E>(o, vp, a.v.token, k0 + 32 * y, t.nk, d, end, n, h);
            }
        }
        bad = more ? arrive(buf ^ 1, masks_at(k0 + KT)) : 0;
    }
    l += __shfl_xor(l, 32);
    if (mine >= rows) return;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    const int64_t at = (int64_t)(t.q0 + query) * a.y_token + (int64_t)head * a.y_head;
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const int c = 32 * x + mfma_row(r, h);
            const float f[4] = {o[x][r] * inv, o[x][r + 1] * inv, o[x][r + 2] * inv, o[x][r + 3] * inv};
            if (c < d) store4(a.y, a.ytype, at + c, f);
        }
}

// Few rows against many keys: a workgroup has 32 rows, and its four waves each every
// fourth step of the keys, in LDS of their own and without a barrier; their sums are
// joined at the end.  A quarter of the serial steps, for four times the reads of keys
// and values from the caches.
//   Waits: keys i and values i are N copies each (where all lanes take part in all of
// them, else each product waits for all); keys i + 1 are asked for when S^T has
//   read keys i, values i + 1 when O^T has read values i; so before either product the
//   N youngest copies may still be on their way.
// One workgroup has a CU (128 KB of LDS at 128 channels), so it is taken while the tiles of
// 128 rows would leave CUs or their second places empty.  Tiles of 128 rows against this,
// 128 channels, us: fp32 with 16 queries on 4096 keys 576 / 166, 1024 causal ones (32 heads
// on 8) 152 / 116, 1536 267 / 233, 2048 314 / 388; fp16 85 / 40 with 16 queries, 8 x 32 queries
// on 1024 keys 32 / 19, 512 causal ones 18 / 21.  fp32 at 256 channels, two waves a workgroup:
// 16 queries on 4096 keys 1090 / 592, 512 causal ones 148 / 109, 768 218 / 229.
template <int T, int D> struct Split {
    static constexpr int KT = D == 256 || T == T_F32 ? 32 : 64;
    static constexpr int W = D == 256 && T == T_F32 ? 2 : 4;     // as many as have room in LDS
    static constexpr int64_t GROUPS = T != T_F32 ? 128 : D == 256 ? 160 : 400;   // tiles of 128 rows, over all key heads
};

template <int N>
__device__ __forceinline__ void all_but(bool more)
{
    if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}
__device__ __forceinline__ void lds_read() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int T, int D, int COPY>
__global__ __launch_bounds__((64 * Split<T, D>::W), 1) void prompt_split(PromptArgs a, int slots, int per)
{
    typedef elem_t<T> E;
    constexpr int B = sizeof(E), KT = Split<T, D>::KT, W = Split<T, D>::W, CH = D * B / 16, N = KT * CH / 64, V = VEC<T>;
    constexpr int TILE = KT * D * B;
    constexpr bool PAD = COPY == PADDED;
    __shared__ __align__(16) uint8_t lds[W][2][TILE];
    __shared__ float stats[W][2][32];
    const int kvh = (int)(blockIdx.x % (uint32_t)a.hkv);
    Tile t;
    if (!find_rows<32>(a, slots - 1 - (int)(blockIdx.x / (uint32_t)a.hkv), per, t)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
    const int d = a.d;
    const E *kp = static_cast<const E *>(a.k.p) + (int64_t)t.k0 * a.k.token + (int64_t)kvh * a.k.head;
    const E *vp = static_cast<const E *>(a.v.p) + (int64_t)t.k0 * a.v.token + (int64_t)kvh * a.v.head;
    const uint32_t rows = t.rows, mine = t.row0 + n;
    const auto query_of = [&](uint32_t r) { return (int)((r < rows ? r : rows - 1) / (uint32_t)per); };
    const int query = query_of(mine), head = kvh * per + (int)((mine < rows ? mine : rows - 1) - (uint32_t)query * per);
    const E *qp = static_cast<const E *>(a.q.p) + (int64_t)(t.q0 + query) * a.q.token + (int64_t)head * a.q.head;
    constexpr int QU = CH / 2;                     // 16-byte units of a row in a lane: every other one
    u32x4 q[QU];
#pragma unroll
    for (int x = 0; x < QU; ++x) {
        const int c = (2 * x + h) * V;
        q[x] = c < d ? load16<T>(qp + c) : u32x4{0, 0, 0, 0};
    }
    const int off = t.nk - t.nq;
    const auto end_of = [&](int i) {
        const int e = a.causal ? off + i + 1 : t.nk;
        return e < 0 ? 0 : e > t.nk ? t.nk : e;
    };
    const int end = end_of(query);
    const int kend = __builtin_amdgcn_readfirstlane(end_of(query_of(t.row0 + 31)));
    const int full = __builtin_amdgcn_readfirstlane(end_of(query_of(t.row0)));

    uint8_t *lk = lds[wave][0], *lv = lds[wave][1];
    // Layouts decide how keys come, not which kernel: results are the same bits at any address.
    const auto unit_k = [](int r, int c) { return r * CH + (c ^ (T == T_F32 ? r & 15 : swz_k<D>(r))); };
    const auto unit_v = [](int r, int c) { return r * CH + (c ^ (T == T_F32 ? (r & 4) << 1 : swz_v<D>(r))); };
    const auto load = [&](bool values, int k0) {
        const E *p = (values ? vp : kp) + (int64_t)k0 * (values ? a.v.token : a.k.token);
        const int64_t step = values ? a.v.token : a.k.token;
        uint8_t *to = values ? lv : lk;
        const int keys = t.nk - k0;
        if constexpr (COPY == REGISTERS) {
#pragma unroll 8
            for (int i = 0; i < N; ++i) {
                const int u = i * 64 + lane, r = u / CH, c = u % CH;
                const u32x4 w = r < keys && c * V < d ? load16<T>(p + (int64_t)r * step + c * V) : u32x4{0, 0, 0, 0};
                reinterpret_cast<u32x4 *>(to)[values ? unit_v(r, c) : unit_k(r, c)] = w;
            }
            return;
        }
        const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)to;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = i * 64 + lane, r = u / CH, pc = u % CH, row = r < keys ? r : keys - 1;
            int c = (values ? unit_v(r, pc) : unit_k(r, pc)) - r * CH;
            if (PAD && values && c * V >= d) c = 0;
            if (!PAD || c * V < d) copy16(p, (uint32_t)row * (uint32_t)step * (uint32_t)B + c * 16, at + i * 1024);
        }
    };

    f32x16 o[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x) o[x] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    int k0 = wave * KT;
    if constexpr (PAD) {
#pragma unroll 4
        for (int i = lane; i < TILE / 16; i += 64) reinterpret_cast<u32x4 *>(lk)[i] = u32x4{0, 0, 0, 0};
        lds_read();
    }
    if (k0 < kend) {
        load(false, k0);
        load(true, k0);
    }
    for (; k0 < kend; k0 += W * KT) {
        const bool more = k0 + W * KT < kend;
        if constexpr (COPY == REGISTERS) lds_read();
        else all_but<N>(!PAD);
        f32x16 s[KT / 32];
#pragma unroll
        for (int y = 0; y < KT / 32; ++y) s[y] = 0.0f;
#pragma unroll
        for (int x = 0; x < QU; ++x)
#pragma unroll
            for (int y = 0; y < KT / 32; ++y) {
                const u32x4 kv = reinterpret_cast<const u32x4 *>(lk)[unit_k(32 * y + n, 2 * x + h)];
                if constexpr (T == T_F32) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[y] = __builtin_amdgcn_mfma_f32_32x32x2f32(__builtin_bit_cast(f32x4, kv)[i], __builtin_bit_cast(f32x4, q[x])[i],
                                                                    s[y], 0, 0, 0);
                } else {
                    s[y] = Mfma16<T>::mul(kv, q[x], s[y]);
                }
            }
        lds_read();
        if (more) load(false, k0 + W * KT);
        if (k0 + KT > full) {
#pragma unroll
            for (int y = 0; y < KT / 32; ++y)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (k0 + 32 * y + mfma_row(r, h) >= end) s[y][r] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int y = 0; y < KT / 32; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[y][r]);
        top = fmaxf(top, __shfl_xor(top, 32));
        const float mn = fmaxf(m, top * a.c), ref = mn == -INFINITY ? 0.0f : mn;
        const float fix = __builtin_amdgcn_exp2f(m - ref);
        m = mn;
        float sum = 0.0f;
        constexpr float UP = T == T_F16 ? 6.0f : 0.0f;
#pragma unroll
        for (int y = 0; y < KT / 32; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[y][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[y][r], a.c, UP - ref));
                sum += s[y][r];
            }
        l = l * fix + sum;
        if (__any(fix != 1.0f)) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x) o[x] *= fix;
        }
        if constexpr (COPY != REGISTERS) all_but<N>(more && !PAD);
        bool bad = false;
        if (k0 + KT > full) {                      // values that are not finite go, as in the other kernels
#pragma unroll
            for (int i = 0; i < N; ++i) {
                u32x4 *at = reinterpret_cast<u32x4 *>(lv) + i * 64 + lane;
                u32x4 v = *at;
                if (clean<T>(v)) {
                    *at = v;
                    bad = true;
                }
            }
            lds_read();
            bad = __any(bad);
        }
        if constexpr (T == T_F32) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const float v = reinterpret_cast<const float *>(lv)[unit_v(mfma_row(r, h), 8 * x + (n >> 2)) * 4 + (n & 3)];
                    o[x] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, s[0][r], o[x], 0, 0, 0);
                }
        } else {
            typedef Mfma16<T> M;
            const int turned = (h * 4 + ((lane & 15) >> 2)) * D, turned_x = swz_v<D>((lane & 15) >> 2);
            const int turned_c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
#pragma unroll
            for (int y = 0; y < KT / 16; ++y) {
                const f32x16 &f = s[y / 2];
                const int b = 8 * (y % 2);
                const u32x4 p = {M::pack(f[b], f[b + 1]), M::pack(f[b + 2], f[b + 3]), M::pack(f[b + 4], f[b + 5]),
                                 M::pack(f[b + 6], f[b + 7])};
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint16_t *at = reinterpret_cast<const uint16_t *>(lv) + turned + 16 * y * D +
                                         (((4 * x + turned_c) ^ turned_x) * 8) + (lane & 1) * 4;
                    const u32x2 v0 = read_turned(at), v1 = read_turned(at + 8 * D);
                    o[x] = M::mul(u32x4{v0[0], v0[1], v1[0], v1[1]}, p, o[x]);
                }
            }
        }
        lds_read();
        if (more) load(true, k0 + W * KT);
        if (bad) {
#pragma unroll
            for (int y = 0; y < KT / 32; ++y) poison<D, E>(o, vp, a.v.token, k0 + 32 * y, t.nk, d, end, n, h);
        }
    }

    l += __shfl_xor(l, 32);
    if (h == 0) {
        stats[wave][0][n] = m;
        stats[wave][1][n] = l;
    }
    __syncthreads();                               // all waves are done with their keys and values
    float top = stats[0][0][n];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, stats[w][0][n]);
    const float mine_fix = __builtin_amdgcn_exp2f(m - (top == -INFINITY ? 0.0f : top));
    constexpr int PITCH = D + (D < 256 ? 4 : 0);   // a row's four channels of 16 lanes meet in no bank
    static_assert(W * 32 * PITCH * 4 <= (int)sizeof(lds), "the waves' sums stand where their keys and values were");
    float *sums = reinterpret_cast<float *>(&lds[0][0][0]);
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const f32x4 f = {o[x][r] * mine_fix, o[x][r + 1] * mine_fix, o[x][r + 2] * mine_fix, o[x][r + 3] * mine_fix};
            *reinterpret_cast<f32x4 *>(&sums[(wave * 32 + n) * PITCH + 32 * x + mfma_row(r, h)]) = f;
        }
    __syncthreads();
    for (int i = threadIdx.x * 4; i < 32 * D; i += 256 * W) {
        const int row = i / D, c = i % D;
        const uint32_t R = t.row0 + row;
        if (R >= rows) break;
        if (c >= d) continue;
        float M = stats[0][0][row], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < W; ++w) M = fmaxf(M, stats[w][0][row]);
        f32x4 v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            sum += stats[w][1][row] * __builtin_amdgcn_exp2f(stats[w][0][row] - (M == -INFINITY ? 0.0f : M));
            v += *reinterpret_cast<const f32x4 *>(&sums[(w * 32 + row) * PITCH + c]);
        }
        const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
        const float f[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
        const int i_q = (int)(R / (uint32_t)per);
        store4(a.y, a.ytype, (int64_t)(t.q0 + i_q) * a.y_token + (int64_t)(kvh * per + (int)(R - (uint32_t)i_q * per)) * a.y_head + c, f);
    }
}

// Whether the rows of x can be copied straight into LDS, `step` keys at a time: 16-byte
// units, and offsets of a step's rows in 32 bits.
bool direct(const Heads &x, int64_t elem, int step)
{
    return (((uintptr_t)x.p | (uintptr_t)(x.token * elem) | (uintptr_t)(x.head * elem)) & 15) == 0 &&
           x.token * elem < (int64_t(1) << 31) / step;
}

int copy_of(const PromptArgs &a, int64_t elem, int step, int D)
{
    if (!direct(a.k, elem, step) || !direct(a.v, elem, step)) return REGISTERS;
    return a.d == D ? STRAIGHT : PADDED;
}

// kernel(grid, slots, rows a query) for tiles of bm rows.
template <typename F>
int by_tiles(const PromptArgs &a, int bm, int threads, F launch)
{
    const int per = a.hq / a.hkv;
    const int64_t slots = a.nt * per / bm + a.nseq, groups = slots * a.hkv;
    if (a.nt * per >= (int64_t(1) << 31) || slots >= (int64_t(1) << 31) || groups > launch_groups(threads)) return -1;
    return launch(dim3((unsigned)groups), (int)slots, per);
}

template <int T, int D>
bool split(const PromptArgs &a)
{
    const int64_t groups = (a.nt * (a.hq / a.hkv) / 128 + a.nseq) * a.hkv;
    return groups <= Split<T, D>::GROUPS && a.nk > 2 * Split<T, D>::KT;
}

template <int T, int D>
int launch_split(const PromptArgs &a, hipStream_t stream)
{
    constexpr int KT = Split<T, D>::KT, threads = 64 * Split<T, D>::W;
    return by_tiles(a, 32, threads, [&](dim3 grid, int slots, int per) {
        const int copy = copy_of(a, sizeof(elem_t<T>), KT, D);
        if (copy == STRAIGHT) return launch_kernel(prompt_split<T, D, STRAIGHT>, grid, dim3(threads), stream, a, slots, per);
        if (copy == PADDED) return launch_kernel(prompt_split<T, D, PADDED>, grid, dim3(threads), stream, a, slots, per);
        return launch_kernel(prompt_split<T, D, REGISTERS>, grid, dim3(threads), stream, a, slots, per);
    });
}

template <int T, int D, int W, int KT>
int launch_16_dim(const PromptArgs &a, hipStream_t stream)
{
    if (split<T, D>(a)) return launch_split<T, D>(a, stream);
    return by_tiles(a, 32 * W, 64 * W, [&](dim3 grid, int slots, int per) {
        const int copy = copy_of(a, 2, KT, D);
        if (copy == STRAIGHT) return launch_kernel(prompt_16<T, D, W, KT, STRAIGHT>, grid, dim3(64 * W), stream, a, slots, per);
        if (copy == PADDED) return launch_kernel(prompt_16<T, D, W, KT, PADDED>, grid, dim3(64 * W), stream, a, slots, per);
        return launch_kernel(prompt_16<T, D, W, KT, REGISTERS>, grid, dim3(64 * W), stream, a, slots, per);
    });
}

template <int T>
int launch_16(const PromptArgs &a, hipStream_t stream)
{
    if (a.d <= 64) return launch_16_dim<T, 64, 4, 64>(a, stream);
    if (a.d <= 128) return launch_16_dim<T, 128, 4, 64>(a, stream);
    return launch_16_dim<T, 256, 4, 32>(a, stream);
}

template <int D>
int launch_f32_dim(const PromptArgs &a, hipStream_t stream)
{
    if (split<T_F32, D>(a)) return launch_split<T_F32, D>(a, stream);
    return by_tiles(a, 128, 256, [&](dim3 grid, int slots, int per) {
        const int copy = copy_of(a, 4, 32, D);
        if (copy == STRAIGHT) return launch_kernel(prompt_f32<D, STRAIGHT>, grid, dim3(256), stream, a, slots, per);
        if (copy == PADDED) return launch_kernel(prompt_f32<D, PADDED>, grid, dim3(256), stream, a, slots, per);
        return launch_kernel(prompt_f32<D, REGISTERS>, grid, dim3(256), stream, a, slots, per);
    });
}

int launch_f32(const PromptArgs &a, hipStream_t stream)
{
    return a.d <= 64 ? launch_f32_dim<64>(a, stream) : a.d <= 128 ? launch_f32_dim<128>(a, stream) : launch_f32_dim<256>(a, stream);
}

}  // namespace

int launch_attend_prompt(const PromptArgs &a, hipStream_t stream)
{
    if (a.type == T_F32) return launch_f32(a, stream);
    if (a.type == T_BF16) return launch_16<T_BF16>(a, stream);
    return launch_16<T_F16>(a, stream);
}

}  // namespace qig
