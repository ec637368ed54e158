// gemm_i8.hip -- y = (q . W^T) * sq * sw + bias for int8 rows q (one scale a
// row) and int8 weights W (one scale an output channel), and the same product
// for rows sorted by expert.
//
// The sum over id is a plain int32 sum, so the whole contraction stays on the
// int8 MFMA and both scales are applied once per output.  A workgroup owns a
// BM x BN tile (tokens x weight rows) and walks id in steps of 128 bytes: both
// operands are copied straight into LDS (global_load_lds), the next steps'
// copies in flight while this one is multiplied, one barrier a step, the LDS
// reads and the copies spread between the MFMAs.
//
// What bounds it, and what it reaches: large products are held by the card's
// power (the clock falls from 2.4 to 1.75 GHz; zeros as data run at 2.4).  8192^3
// 420 us, 2610 TOPS, above the vendor library's product on the same card (2500);
// 2630 tokens, 2 x 18944 x 3584 gated to bf16 306 us, 2330 TOPS (317 on another
// card); 18944 -> 3584 to fp32 148 us, 2420 TOPS (157 us with operands from HBM).  Of the 8192^3 time, an
// earlier build without its copies took 16% less, one without the LDS reads 12%,
// one with neither 27%.  Small products: launch, first loads and epilogue, 5 us,
// then 0.25 us a step (3584 x 3584, 512 tokens 14.5 us).  Experts' products: the
// weights' bytes up to about 50 rows an expert (5.0 TB/s), above that bytes and
// power together (64 experts of 2 x 2368 x 3584, 15780 rows: 349 us; 300 us with
// the weights of two experts for all, which stay in the caches).
//
// LDS rows are 128 bytes, eight 16-byte granules; granule g of row r is kept
// at slot g ^ (r & 7), so that the eight lanes of a read phase (eight rows,
// one granule) touch eight different bank groups.  The copy writes lane l's
// bytes at 16 l of each 1 KB piece (eight rows), so the swizzle is done by
// choosing which granule a lane loads.
//
// id need not be a multiple of 128: granules past the last one of the row are
// not read (the lane reads the step's first granule instead), and the bytes
// past id are zeroed in the activations' LDS rows before the multiplication,
// which makes the weights' bytes there irrelevant.
#include "qig_i8_device.h"
#include "qig_launch.h"

#include <algorithm>
#include <type_traits>

namespace qig {

constexpr int BK = 128;
// Bands of the tile order (tile_of).
constexpr unsigned BAND = 8, EXPERT_BAND = 1;

struct I8Args {
    const uint8_t *W, *q;
    const float *sw, *sq, *bias;
    void *y;
    const int32_t *plan;
    int32_t *part;    // split sums: one BM x BN slot of int32 a workgroup
    uint32_t *cnt;    // and one arrival counter a tile
    int64_t ldw, ldq, ldy, od, nt;
    int id, nbt, nbj, ne, slots, splits;
};

__device__ __forceinline__ uint64_t uniform64(const void *p)
{
    const uint64_t b = reinterpret_cast<uintptr_t>(p);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    return (uint64_t)lo | ((uint64_t)hi << 32);
}

// 16 x 16 x 64: lane l supplies row l % 16 and 16 bytes (l / 16) of the 64 of
// both operands; the result's column (b's row) is l % 16, its rows (a's)
// 4 (l / 16) + i.
__device__ __forceinline__ i32x4 mfma16(i32x4 a, i32x4 b, i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// One 1 KB copy, 16 bytes a lane, to LDS byte address lds + 16 lane.  Issued
// from inline assembly, unseen by the compiler's wait counts: its data is
// read only after an explicit vmcnt wait and a barrier.  s_nop 4 covers the
// wait states after a VALU write of the scalar base and an M0 write.
__device__ __forceinline__ void copy16(uint64_t base, uint32_t voff, uint32_t lds)
{
    const uint32_t m0v = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds);
    asm volatile("s_nop 4\n\t"
                 "global_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(voff), "s"(base), "{m0}"(m0v)
                 : "memory");
}

// The same with a 64-bit address per lane (rows anywhere in memory).
__device__ __forceinline__ void copy16_at(uint64_t addr, uint32_t lds)
{
    const uint32_t m0v = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds);
    asm volatile("s_nop 4\n\t"
                 "global_load_lds_dwordx4 %0, off"
                 :
                 : "v"(addr), "{m0}"(m0v)
                 : "memory");
}

// Tile i of the tile order: bands of BAND token tiles, the tiles of a band
// fastest, so that the tiles in work at one time share both weight rows and
// tokens.
template <unsigned BAND>
__device__ __forceinline__ void tile_of(unsigned i, unsigned nbt, unsigned nbj, int &mt, int &jt)
{
    const unsigned band = BAND * nbj;
    const unsigned bi = i / band, in = i - bi * band;
    const unsigned left = nbt - bi * BAND, h = left < BAND ? left : BAND;
    jt = (int)(in / h);
    mt = (int)(bi * BAND + in % h);
}

// Workgroup b's place in the order of `total` tiles.  Workgroups go round-robin
// over the eight XCDs, each with its own L2: XCD x takes a contiguous run.
// False: more workgroups than tiles, and this one has none.
__device__ __forceinline__ bool place_of(unsigned b, unsigned total, unsigned &i)
{
    const unsigned per = total / 8, rem = total % 8, x = b % 8;
    i = x * per + (x < rem ? x : rem) + b / 8;
    return b / 8 < per + (x < rem);
}

// The experts' token tiles, counted in order, the dropped rows' tiles last
// (expert ne).  One wave's lanes hold 64 experts at a time.
struct Rows {
    int e, first, count;   // expert, first position in the order, rows of the tile
};

// Token tiles of all experts, at most the `most` that the grid was made for.
template <int BM>
__device__ __forceinline__ int count_tiles(const int32_t *plan, int ne, int most)
{
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e = lane; e <= ne; e += 64) n += (plan[e + 1] - plan[e] + BM - 1) / BM;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
    n = __builtin_amdgcn_readfirstlane(n);
    return n < 0 ? 0 : (n < most ? n : most);
}

// Flat row number i of the order, for a tile of `count` rows.  The host cannot
// see whether a plan belongs to the call: one made for other rows gives wrong
// rows here, but none outside [0, nrows).
__device__ __forceinline__ int row_of(const int32_t *plan, int ne, const Rows &r, int i, int nrows)
{
    int at = r.first + (i < r.count ? i : r.count - 1);
    at = at < 0 ? 0 : (at < nrows ? at : nrows - 1);
    const int row = plan[ne + 2 + at];
    return (unsigned)row < (unsigned)nrows ? row : nrows - 1;
}

// Token tile mt, which exists.
template <int BM>
__device__ __forceinline__ Rows find_rows(const int32_t *plan, int ne, int mt)
{
    const int lane = threadIdx.x & 63;
    Rows r = {0, 0, 0};
    int before = 0;
    for (int e0 = 0; e0 <= ne; e0 += 64) {
        const int e = e0 + lane;
        const int lo = e <= ne ? plan[e] : 0;
        const int n = e <= ne ? plan[e + 1] - lo : 0;
        const int tiles = (n + BM - 1) / BM;
        int incl = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
        const int excl = before + incl - tiles;
        const uint64_t hit = __ballot(mt >= excl && mt < excl + tiles);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int m = mt - __builtin_amdgcn_readlane(excl, src);
            r.e = e0 + src;
            r.first = __builtin_amdgcn_readlane(lo, src) + m * BM;
            const int left = __builtin_amdgcn_readlane(n, src) - m * BM;
            r.count = left < BM ? left : BM;
            break;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return r;
}

// BM x BN tile, WM x WN waves, each BM/WM x BN/WN.
// GLU: of every 32 of the tile's weight rows the first 16 are gate rows and
// the last 16 the up rows of the same outputs, so a wave holds both halves of
// an output in the same lane and register.
template <int BM, int BN, int WM, int WN, int S, int SB, bool SPLIT, bool GLU, bool EXPERTS, int YT>
__global__ __launch_bounds__(WM *WN * 64) void gemm_i8_kernel(I8Args g)
{
    constexpr int NW = WM * WN;
    constexpr int TMAX = BM / WM / 32, TN = BN / WN / 32;
    constexpr int PAMAX = BM / 8 / NW, PB = BN / 8 / NW;   // 1 KB pieces a wave copies each step
    constexpr int LDS = (S * BM + SB * BN) * BK;
    constexpr int BJ = GLU ? BN / 2 : BN;               // outputs of a tile
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && TMAX >= 1 && TMAX <= 4 && TN >= 1, "tile");
    static_assert((S == 2 && (SB == 2 || SB == 3)) || (S >= 4 && SB == S), "stages");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
    static_assert(BM <= NW * 64 && BN <= NW * 64, "a thread a row");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int jt, mt, split = 0;
    unsigned block = blockIdx.x;
    if constexpr (SPLIT) {
        split = (int)(block % (unsigned)g.splits);
        block /= (unsigned)g.splits;
    }
    if constexpr (EXPERTS) {
        unsigned i;
        const unsigned nbt = (unsigned)count_tiles<BM>(g.plan, g.ne, g.nbt);
        if (!place_of(block, nbt * (unsigned)g.nbj, i)) return;
        tile_of<EXPERT_BAND>(i, nbt, (unsigned)g.nbj, mt, jt);
    } else {
        unsigned i;
        place_of(block, (unsigned)g.nbt * (unsigned)g.nbj, i);
        tile_of<BAND>(i, (unsigned)g.nbt, (unsigned)g.nbj, mt, jt);
    }
    const int64_t j0 = (int64_t)jt * BJ;
    const uint8_t *W = g.W;
    const float *sw = g.sw, *bias = g.bias;
    int64_t t0 = (int64_t)mt * BM;
    int count;
    elem_t<YT> *y = static_cast<elem_t<YT> *>(g.y);
    [[maybe_unused]] Rows rows = {0, 0, 0};

    if constexpr (EXPERTS) {
        rows = find_rows<BM>(g.plan, g.ne, mt);
        const Rows &r = rows;
        count = r.count;
        if (r.e == g.ne) {
            // dropped rows: zeros
            for (int i = wave; i < count; i += NW) {
                elem_t<YT> *row = y + (int64_t)row_of(g.plan, g.ne, r, i, (int)g.nt) * g.ldy;
                for (int64_t j = j0 + lane; j < j0 + BJ && j < g.od; j += 64) row[j] = (elem_t<YT>)0.0f;
            }
            return;
        }
        const int64_t wrows = GLU ? 2 * g.od : g.od;
        W += (int64_t)r.e * wrows * g.ldw;
        sw += (int64_t)r.e * wrows;
        if (bias) bias += (int64_t)r.e * wrows;
    } else {
        count = (int)(g.nt - t0 < BM ? g.nt - t0 : BM);
    }

    // The rows that this lane copies: piece p of the wave holds rows
    // 8 (NW p + wave) .. + 7, lane l row l / 8 and slot l % 8.
    const int lr = lane >> 3;
    const uint32_t gran = (uint32_t)((lane & 7) ^ lr);   // the granule that belongs in this lane's slot
    uint32_t aoff[EXPERTS ? 1 : PAMAX], boff[PB];
    uint64_t aptr[EXPERTS ? PAMAX : 1];
#pragma unroll
    for (int p = 0; p < PAMAX; ++p) {
        const int r = 8 * (NW * p + wave) + lr;
        if constexpr (EXPERTS)
            aptr[p] = reinterpret_cast<uintptr_t>(
                g.q + (int64_t)(row_of(g.plan, g.ne, rows, r, (int)g.nt) / g.slots) * g.ldq);
        else
            aoff[p] = (uint32_t)(r < count ? r : count - 1) * (uint32_t)g.ldq;
    }
    uint64_t bbase = uniform64(W + (GLU ? j0 : (int64_t)jt * BN) * g.ldw);
    [[maybe_unused]] const uint64_t uphalf = GLU ? (uint64_t)(g.od * g.ldw) : 0;
    bool bup[PB];
#pragma unroll
    for (int p = 0; p < PB; ++p) {
        // a piece's eight rows lie in one block of 16, so gate or up is the
        // same for the whole piece
        const int r = 8 * (NW * p + wave) + lr;
        int j = GLU ? (r >> 5) * 16 + (r & 15) : r;
        bup[p] = GLU && ((8 * (NW * p + wave)) & 16) != 0;
        const int64_t last = g.od - 1 - j0;
        if (j > last) j = (int)last;
        boff[p] = (uint32_t)j * (uint32_t)g.ldw;
    }
    const uint64_t abase0 = EXPERTS ? 0 : uniform64(g.q + t0 * g.ldq);
    const uint32_t l0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

    int nk = (g.id + BK - 1) / BK;
    int tail = g.id - (nk - 1) * BK;   // bytes of the last step, 1 .. 128
    int kfirst = 0;
    if constexpr (SPLIT) {
        // this workgroup's share of the steps (at least one)
        const int all = nk;
        kfirst = (int)((int64_t)all * split / g.splits);
        nk = (int)((int64_t)all * (split + 1) / g.splits) - kfirst;
        if (kfirst + nk < all) tail = BK;
    }

    // Scales, biases and rows for the epilogue, one of each a thread: loaded
    // before the last step and put into LDS behind it, since the stages may take
    // all of the LDS.  Weight rows in the order of their LDS rows.
    float e_sq = 0.0f, e_sw = 0.0f, e_bias = 0.0f;
    [[maybe_unused]] int e_row = 0;
    auto fetch = [&]() {
        if (tid < BM) {
            if constexpr (EXPERTS) {
                e_row = row_of(g.plan, g.ne, rows, tid, (int)g.nt);
                e_sq = g.sq[e_row / g.slots];
            } else {
                e_sq = g.sq[t0 + (tid < count ? tid : count - 1)];
            }
        }
        if (tid < BN) {
            int64_t j = j0 + (GLU ? (tid >> 5) * 16 + (tid & 15) : tid);
            j = j < g.od ? j : g.od - 1;
            if (GLU && (tid & 16)) j += g.od;
            e_sw = sw[j];
            if (bias) e_bias = bias[j];
        }
    };

    const int wm = wave / WN, wn = wave % WN;
    const int l16 = lane & 15, quad = lane >> 4;

    // The tile with TM x 32 of every wave's rows: only as many as have tokens
    // (the last tile of the tokens, or of an expert's rows, is mostly smaller).
    auto run = [&](auto frags) {
        constexpr int TM = frags;
        constexpr int PA = TM * WM * 32 / 8 / NW;   // pieces of the activations a wave copies
        static_assert(PA * 8 * NW == TM * WM * 32, "whole pieces");
        // Where step kt's activations and weights are kept: S and SB stages.
        auto a_at = [&](int kt) -> uint32_t { return (uint32_t)kt % S * (BM * BK); };
        auto b_at = [&](int kt) -> uint32_t { return S * BM * BK + (uint32_t)kt % SB * (BN * BK); };
        // Copy piece p of step kt: first the wave's PA pieces of the activations,
        // then its PB pieces of the weights.
        auto copy = [&](int kt, int p) {
            const uint64_t k0 = (uint64_t)(kfirst + kt) * BK;
            uint32_t go = 16 * gran;
            if (kt == nk - 1 && (int)go >= tail) go = 0;
            if (p < PA) {
                const uint32_t d = l0 + a_at(kt) + 1024 * (NW * p + wave);
                if constexpr (EXPERTS)
                    copy16_at(aptr[p] + k0 + go, d);
                else
                    copy16(abase0 + k0, aoff[p] + go, d);
            } else {
                p -= PA;
                copy16(bbase + k0 + (bup[p] ? uphalf : 0), boff[p] + go, l0 + b_at(kt) + 1024 * (NW * p + wave));
            }
        };
        // Step kt's bytes past id become zero in the activations' rows.
        auto clear_tail = [&](uint8_t *st) {
            for (int i = tid; i < TM * WM * 32 * 8; i += NW * 64) {
                const int r = i >> 3, slot = i & 7;
                const int left = tail - 16 * (slot ^ (r & 7));   // valid bytes of the granule
                if (left >= 16) continue;
                u32x4 *p = reinterpret_cast<u32x4 *>(st + 16 * i);
                u32x4 v = *p;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int b = left - 4 * w;
                    v[w] = b >= 4 ? v[w] : (b <= 0 ? 0u : v[w] & ((1u << (8 * b)) - 1u));
                }
                *p = v;
            }
            __syncthreads();
        };

        // 16 x 16 x 64 MFMAs: FM blocks of 16 tokens, FN of 16 weight rows.  (The
        // 32 x 32 x 32 form moves more accumulator bytes an operation and, where
        // the card's power is the limit, is slower: from registers alone, random
        // data, 3550 against 4150 TOPS.)
        constexpr int FM = 2 * TM, FN = 2 * TN;
        i32x4 acc[FM][FN];
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
            for (int n = 0; n < FN; ++n) acc[m][n] = i32x4{0, 0, 0, 0};

        // Chunk c of a step is 64 bytes of every row: granules 4 c .. 4 c + 3,
        // one for each quarter of the wave.  Rows of one lane differ by multiples
        // of 16, so its slot is the same in all of them.
        constexpr int NC = BK / 64, NP = PA + PB, P3 = SB == 3 ? PA : NP / 2;
        uint32_t aat[NC], bat[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint32_t slot = 16 * ((4 * c + quad) ^ (l16 & 7));
            aat[c] = (wm * FM * 16 + l16) * BK + slot;
            bat[c] = (wn * FN * 16 + l16) * BK + slot;
        }
        auto read_a = [&](int kt, int c, int m) {
            return *reinterpret_cast<const i32x4 *>(lds + a_at(kt) + aat[c] + m * 16 * BK);
        };
        auto read_b = [&](int kt, int c, int n) {
            return *reinterpret_cast<const i32x4 *>(lds + b_at(kt) + bat[c] + n * 16 * BK);
        };
        constexpr std::true_type yes;
        constexpr std::false_type no;

        if constexpr (S == 2) {
            // A step is MS row steps: one block of tokens against the FN blocks of
            // weights, chunk after chunk.  Token blocks are read LA row steps
            // ahead into a ring of four, weight blocks while the chunk before
            // theirs is multiplied.  In the last LA row steps all of this step's
            // blocks have been read, the next step has landed and its first blocks
            // are read; the copies go out one by one there (pieces up to P3 of the
            // step after the next, whose stage is free then) and in the first
            // quarter, FIRST row steps (the others).
            // With three stages of weights (SB) they are copied two steps ahead
            // in the first quarter, and the activations at the end: weights
            // come from HBM, whose latency is longer than a step (18944 -> 3584,
            // 2630 tokens, operands not in the caches: 192 us with two stages,
            // 157 us with three; touching the lines ahead of the copies instead
            // cost more than it hid).
            constexpr int MS = NC * FM, FIRST = MS / 4, LA = FIRST < 3 ? FIRST : 3;
            i32x4 ra[4], rb[NC][FN];
            auto step = [&](auto late, auto early, auto next, int kt) {
#pragma unroll
                for (int s = 0; s < MS; ++s) {
                    const int c = s / FM, m = s % FM;
                    const int in = s - (MS - LA);   // row step of the last part
                    if (next && in == 0) {
                        // the next step has landed (all but the weights of the step
                        // after it, issued last), and nobody reads this one any more
                        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(SB == 3 && late ? PB : 0) : "memory");
                        __syncthreads();
                        if constexpr (!early)
                            if (tail < BK) clear_tail(lds + a_at(kt + 1));
                    }
#pragma unroll
                    for (int n = 0; n < FN; ++n) {
                        acc[m][n] = mfma16(rb[c][n], ra[s & 3], acc[m][n]);
                        if (n == 0) {
                            const int t = s + LA;
                            if (t < MS)
                                ra[t & 3] = read_a(kt, t / FM, t % FM);
                            else if (next)
                                ra[t & 3] = read_a(kt + 1, 0, t - MS);
                        }
                        // the weight blocks of the coming chunk, evenly spread
                        if (s < FIRST) {
#pragma unroll
                            for (int i = 0; i < FN; ++i)
                                if (i * FIRST == s * FN + n) rb[1][i] = read_b(kt, 1, i);
                        } else if (next && in >= 0) {
#pragma unroll
                            for (int i = 0; i < FN; ++i)
                                if (i * LA == in * FN + n) rb[0][i] = read_b(kt + 1, 0, i);
                        }
                        if (late && s < FIRST) {
#pragma unroll
                            for (int i = 0; i < NP - P3; ++i)
                                if (i * FIRST * FN / (NP - P3) == s * FN + n) copy(kt + SB - 1, P3 + i);
                        } else if (early && in >= 0) {
#pragma unroll
                            for (int i = 0; i < P3; ++i)
                                if (i * LA * FN / P3 == in * FN + n) copy(kt + 2, i);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            };
#pragma unroll
            for (int p = 0; p < NP; ++p) copy(0, p);
            if (SB == 3 && nk > 1) {
#pragma unroll
                for (int p = 0; p < NP; ++p) copy(1, p);
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NP) : "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
            __syncthreads();
            if (nk == 1 && tail < BK) clear_tail(lds);
#pragma unroll
            for (int i = 0; i < FN; ++i) rb[0][i] = read_b(0, 0, i);
#pragma unroll
            for (int t = 0; t < LA; ++t) ra[t] = read_a(0, 0, t);
            if (nk > 1) {
                if constexpr (SB == 2) {
#pragma unroll
                    for (int p = 0; p < P3; ++p) copy(1, p);
                }
                for (int kt = 0; kt < nk - 2; ++kt) step(yes, yes, yes, kt);
                step(std::bool_constant<SB == 2>{}, no, yes, nk - 2);
            }
            fetch();
            step(no, no, no, nk - 1);
        } else {
            // Body kt multiplies step kt, held in registers, and reads step
            // kt + 1 block by block into the registers as they come free, so
            // nearly a whole step lies between a read and its use; it copies step
            // kt + S - 1 into the stage of step kt - 1, whose reads every wave
            // has used by then.
            i32x4 fa[NC][FM], fb[NC][FN];
            constexpr int ALL = NC * FM * FN;
            auto body = [&](auto copies, auto next, int kt) {
                constexpr int N = copies ? NP : 0;
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int m = 0; m < FM; ++m)
#pragma unroll
                        for (int n = 0; n < FN; ++n) {
                            acc[m][n] = mfma16(fb[c][n], fa[c][m], acc[m][n]);
                            if constexpr (next) {
                                if (m == FM - 1) fb[c][n] = read_b(kt + 1, c, n);
                                if (n == FN - 1) fa[c][m] = read_a(kt + 1, c, m);
                            }
#pragma unroll
                            for (int j = 0; j < N; ++j)
                                if (j * ALL / N == (c * FM + m) * FN + n) copy(kt + S - 1, j);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                if constexpr (next) {
                    if constexpr (copies)
                        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 3) * NP) : "memory");
                    else
                        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                }
            };
#pragma unroll
            for (int k = 0; k < S - 1; ++k)
                if (k < nk)
#pragma unroll
                    for (int p = 0; p < NP; ++p) copy(k, p);
            if (nk >= S - 1)
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 3) * NP) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (nk <= 2 && tail < BK) clear_tail(lds + a_at(nk - 1));
#pragma unroll
            for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int n = 0; n < FN; ++n) fb[c][n] = read_b(0, c, n);
#pragma unroll
                for (int m = 0; m < FM; ++m) fa[c][m] = read_a(0, c, m);
            }
            int kt = 0;
            for (; kt <= nk - S; ++kt) body(yes, yes, kt);
            for (; kt < nk - 1; ++kt) {
                body(no, yes, kt);
                if (kt + 2 == nk - 1 && tail < BK) clear_tail(lds + a_at(nk - 1));
            }
            fetch();
            body(no, no, kt);
        }

        if constexpr (SPLIT) {
            // Every share leaves its sums in its slot; the last to arrive at the
            // tile adds the others' to its own (integers: in any order the same)
            // and finishes.  Slots and counter go through agent-scope accesses:
            // the shares run on XCDs whose L2s are not coherent.
            constexpr int LANES = NW * 64;
            const int tile = (int)(blockIdx.x / (unsigned)g.splits);
            int32_t *slot = g.part + (int64_t)tile * g.splits * (BM * BN);
            int32_t *mine = slot + (int64_t)split * (BM * BN) + tid;
#pragma unroll
            for (int m = 0; m < FM; ++m)
#pragma unroll
                for (int n = 0; n < FN; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        __hip_atomic_store(mine + ((m * FN + n) * 4 + i) * LANES, acc[m][n][i], __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the sums are at the coherence point
            __syncthreads();
            __shared__ uint32_t s_before;
            if (tid == 0)
                s_before = __hip_atomic_fetch_add(g.cnt + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (s_before != (uint32_t)g.splits - 1) return;
            for (int o = 0; o < g.splits; ++o) {
                if (o == split) continue;
                int32_t *other = slot + (int64_t)o * (BM * BN) + tid;
#pragma unroll
                for (int m = 0; m < FM; ++m)
#pragma unroll
                    for (int n = 0; n < FN; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[m][n][i] += __hip_atomic_load(other + ((m * FN + n) * 4 + i) * LANES, __ATOMIC_RELAXED,
                                                              __HIP_MEMORY_SCOPE_AGENT);
            }
            if (tid == 0) __hip_atomic_store(g.cnt + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }

        // The weights are the rows of the result: lane l, register i holds token
        // l % 16 and weight row 4 (l / 16) + i, four neighbouring outputs of one
        // token.  Every wave turns 32 tokens at a time through its own part of
        // the stages' LDS, so that its stores are whole rows of 64 to 256 bytes
        // (stored straight from the registers, 16 bytes a row, fp32 outputs cost
        // 12% of the time at 8192^3).
        constexpr int NO = GLU ? FN / 2 : FN;              // blocks of 16 outputs
        constexpr int EB = YT == T_F32 ? 4 : 2;            // bytes of an output
        constexpr int PITCH = NO * 16 * EB + 16;           // 16 more: the rows' writes on different banks
        constexpr int CH = NO * EB;                        // 16-byte chunks a row
        constexpr int PER = 16 / EB;                       // outputs of a chunk
        float *s_sq = reinterpret_cast<float *>(lds + NW * 32 * PITCH);
        float *s_sw = s_sq + BM, *s_bias = s_sw + BN;
        int32_t *s_row = reinterpret_cast<int32_t *>(s_bias + BN);
        static_assert(NW * 32 * PITCH + (2 * BM + 2 * BN) * 4 <= LDS, "the waves' parts and the scales");
        __syncthreads();   // nobody reads the stages any more
        if (tid < BM) {
            s_sq[tid] = e_sq;
            if constexpr (EXPERTS) s_row[tid] = e_row;
        }
        if (tid < BN) {
            s_sw[tid] = e_sw;
            s_bias[tid] = e_bias;
        }
        __syncthreads();
        uint8_t *mine = lds + wave * (32 * PITCH);
        const int64_t jw = j0 + wn * NO * 16;
#pragma unroll
        for (int m2 = 0; m2 < TM; ++m2) {
            const int r0 = (wm * TM + m2) * 32;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = 2 * m2 + h;
                const float s = s_sq[r0 + 16 * h + l16];
#pragma unroll
                for (int n = 0; n < NO; ++n) {
                    const int at = (wn * FN + (GLU ? 2 * n : n)) * 16 + 4 * quad;
                    const f32x4 w = *reinterpret_cast<const f32x4 *>(s_sw + at);
                    const f32x4 b = *reinterpret_cast<const f32x4 *>(s_bias + at);
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (GLU) {
                            const f32x4 w1 = *reinterpret_cast<const f32x4 *>(s_sw + at + 16);
                            const f32x4 b1 = *reinterpret_cast<const f32x4 *>(s_bias + at + 16);
                            const float ga = (float)acc[m][2 * n][i] * s * w[i] + b[i];
                            const float up = (float)acc[m][2 * n + 1][i] * s * w1[i] + b1[i];
                            v[i] = silu_mul<YT>(ga, up);
                        } else {
                            v[i] = (float)acc[m][n][i] * s * w[i] + b[i];
                        }
                    }
                    uint8_t *to = mine + (16 * h + l16) * PITCH + (n * 16 + 4 * quad) * EB;
                    if constexpr (EB == 4) {
                        *reinterpret_cast<f32x4 *>(to) = f32x4{v[0], v[1], v[2], v[3]};
                    } else {
                        typedef elem_t<YT> four __attribute__((ext_vector_type(4)));
                        *reinterpret_cast<four *>(to) =
                            four{(elem_t<YT>)v[0], (elem_t<YT>)v[1], (elem_t<YT>)v[2], (elem_t<YT>)v[3]};
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < CH / 2; ++c) {
                const int i = c * 64 + lane, row = i / CH, ch = i % CH;
                const u32x4 v = *reinterpret_cast<const u32x4 *>(mine + row * PITCH + 16 * ch);
                const int r = r0 + row;
                const int64_t j = jw + ch * PER;
                if (r >= count || j >= g.od) continue;
                elem_t<YT> *out = y + (EXPERTS ? (int64_t)s_row[r] : t0 + r) * g.ldy + j;
                if (j + PER <= g.od) {
                    store16<YT>(out, v);
                } else {
                    const int left = (int)(g.od - j);
#pragma unroll
                    for (int i = 0; i < PER - 1; ++i) {
                        if (i >= left) break;
                        if constexpr (EB == 4)
                            out[i] = __builtin_bit_cast(float, (uint32_t)v[i]);
                        else
                            out[i] = __builtin_bit_cast(elem_t<YT>, (uint16_t)(v[i / 2] >> (16 * (i & 1))));
                    }
                }
            }
        }
    };
    if constexpr (TMAX >= 2)
        if (count <= WM * 32) return run(std::integral_constant<int, 1>{});
    if constexpr (TMAX >= 3)
        if (count <= WM * 64) return run(std::integral_constant<int, 2>{});
    if constexpr (TMAX >= 4)
        if (count <= WM * 96) return run(std::integral_constant<int, 3>{});
    run(std::integral_constant<int, TMAX>{});
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------
// The weights' bytes are what counts here: each is used for a few products, and
// a tile in LDS would only delay it.  A workgroup owns 16 weight rows (gated:
// 16 gate and 16 up rows) and 16 tokens; its waves take the 128-byte pieces of
// id in turn, load both operands straight into the registers of the
// 16 x 16 x 64 MFMA (lane l: row l % 16, 16 bytes l / 16 of each 64), DEPTH
// pieces before the first product, and their sums meet in LDS at the end.  The
// weights are the rows of the result, so a lane holds four neighbouring
// outputs of one token.  Bound by the weights' bytes: one token, 2 x 18944 x 3584
// gated 24.6 us (5.5 TB/s), 3584 x 3584 5.0 us (2.6 TB/s: the launch and one
// memory latency).
constexpr int GEMV_WAVES = 8, GEMV_ROWS = 16;

template <bool GLU, bool EXPERTS, int YT>
__global__ __launch_bounds__(GEMV_WAVES * 64) void gemv_i8_kernel(I8Args g)
{
    constexpr int NW = GEMV_WAVES, BM = 16;
    constexpr int NB = GLU ? 2 : 1;   // blocks of 16 weight rows
    constexpr int DEPTH = 4;          // pieces in flight a wave
    __shared__ i32x4 s_sum[NW][NB][64];
    __shared__ float s_sq[BM];
    __shared__ int32_t s_row[EXPERTS ? BM : 1];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int jt = (int)(blockIdx.x % (unsigned)g.nbj), mt = (int)(blockIdx.x / (unsigned)g.nbj);
    if constexpr (EXPERTS)
        if (mt >= count_tiles<BM>(g.plan, g.ne, g.nbt)) return;
    const int64_t j0 = (int64_t)jt * GEMV_ROWS;
    const uint8_t *W = g.W;
    const float *sw = g.sw, *bias = g.bias;
    const int64_t t0 = (int64_t)mt * BM;
    int count;
    elem_t<YT> *y = static_cast<elem_t<YT> *>(g.y);
    if constexpr (EXPERTS) {
        const Rows r = find_rows<BM>(g.plan, g.ne, mt);
        count = r.count;
        if (r.e == g.ne) {
            // dropped rows: zeros
            for (int i = tid; i < count * GEMV_ROWS; i += NW * 64)
                if (j0 + i % GEMV_ROWS < g.od)
                    y[(int64_t)row_of(g.plan, g.ne, r, i / GEMV_ROWS, (int)g.nt) * g.ldy + j0 + i % GEMV_ROWS] =
                        (elem_t<YT>)0.0f;
            return;
        }
        const int64_t rows = GLU ? 2 * g.od : g.od;
        W += (int64_t)r.e * rows * g.ldw;
        sw += (int64_t)r.e * rows;
        if (bias) bias += (int64_t)r.e * rows;
        if (tid < BM) {
            const int row = row_of(g.plan, g.ne, r, tid, (int)g.nt);
            s_row[tid] = row;
            s_sq[tid] = g.sq[row / g.slots];
        }
        __syncthreads();
    } else {
        count = (int)(g.nt - t0 < BM ? g.nt - t0 : BM);
        if (tid < BM) s_sq[tid] = g.sq[t0 + (tid < count ? tid : count - 1)];
    }
    const int l16 = lane & 15, quad = lane >> 4;
    const int64_t j = j0 + l16 < g.od ? j0 + l16 : g.od - 1;
    const uint8_t *wp[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wp[b] = W + (j + b * g.od) * g.ldw + 16 * quad;
    const int64_t xrow = EXPERTS ? (int64_t)(s_row[l16] / g.slots) : t0 + (l16 < count ? l16 : count - 1);
    const uint8_t *xp = g.q + xrow * g.ldq + 16 * quad;
    i32x4 acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = i32x4{0, 0, 0, 0};

    struct Piece {
        i32x4 w[NB][2], x[2];
    };
    auto load = [&](Piece &p, int64_t k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int b = 0; b < NB; ++b) p.w[b][h] = *reinterpret_cast<const i32x4 *>(wp[b] + k + 64 * h);
            p.x[h] = *reinterpret_cast<const i32x4 *>(xp + k + 64 * h);
        }
    };
    auto multiply = [&](const Piece &p) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                acc[b] = mfma16(p.w[b][h], p.x[h], acc[b]);
    };
    const int full = g.id / BK;
    Piece p[DEPTH];
    int c = wave;
    for (; c + (DEPTH - 1) * NW < full; c += DEPTH * NW) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(p[d], (int64_t)(c + d * NW) * BK);
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) multiply(p[d]);
    }
    // fewer than DEPTH pieces left: still all loads before the products (a
    // piece that is not there is read as the first, and zeroed in x)
    if (c < full) {
#pragma unroll
        for (int d = 0; d < DEPTH - 1; ++d) {
            const bool there = c + d * NW < full;
            load(p[d], there ? (int64_t)(c + d * NW) * BK : 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) p[d].x[h] = there ? p[d].x[h] : i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int d = 0; d < DEPTH - 1; ++d) multiply(p[d]);
    }
    if (full % NW == wave && g.id % BK != 0) {
        // the last, partial piece: granules past id are not read, and the
        // tokens' bytes past id are zeros
        const int64_t k = (int64_t)full * BK;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int left = g.id - (int)k - 64 * h - 16 * quad;   // valid bytes of this lane's granule
            const int64_t at = left > 0 ? k + 64 * h : -16 * quad;
#pragma unroll
            for (int b = 0; b < NB; ++b) p[0].w[b][h] = *reinterpret_cast<const i32x4 *>(wp[b] + at);
            i32x4 v = *reinterpret_cast<const i32x4 *>(xp + at);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int b = left - 4 * w;
                v[w] = b >= 4 ? v[w] : (b <= 0 ? 0 : (int)((uint32_t)v[w] & ((1u << (8 * b)) - 1u)));
            }
            p[0].x[h] = v;
        }
        multiply(p[0]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) s_sum[wave][b][lane] = acc[b];
    __syncthreads();
    // waves 0 .. 3 finish one of a lane's four outputs each
    if (wave >= 4) return;
    int v[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        v[b] = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) v[b] += reinterpret_cast<const int32_t *>(&s_sum[w][b][lane])[wave];
    }
    const int64_t o = j0 + 4 * quad + wave;
    if (l16 >= count || o >= g.od) return;
    const float s = s_sq[l16];
    float r = (float)v[0] * s * sw[o] + (bias ? bias[o] : 0.0f);
    if constexpr (GLU) r = silu_mul<YT>(r, (float)v[NB - 1] * s * sw[g.od + o] + (bias ? bias[g.od + o] : 0.0f));
    const int64_t row = EXPERTS ? (int64_t)s_row[l16] : t0 + l16;
    y[row * g.ldy + o] = (elem_t<YT>)r;
}

template <bool GLU, bool EXPERTS, int YT>
static int launch_gemv(I8Args a, hipStream_t stream)
{
    const int64_t nbj = (a.od + GEMV_ROWS - 1) / GEMV_ROWS;
    const int64_t nbt = EXPERTS ? a.nt / 16 + (a.nt < a.ne + 1 ? a.nt : a.ne + 1) : (a.nt + 15) / 16;
    if (nbt * nbj > 0x7fffffff) return -1;
    a.nbt = (int)nbt;
    a.nbj = (int)nbj;
    return launch_kernel(gemv_i8_kernel<GLU, EXPERTS, YT>, dim3((unsigned)(nbt * nbj)), dim3(GEMV_WAVES * 64), stream,
                         a);
}

template <int BM, int BN, int WM, int WN, int S, int SB, bool SPLIT, bool GLU, bool EXPERTS, int YT>
static int launch_tile(I8Args a, int64_t od, int64_t nt, hipStream_t stream)
{
    constexpr int BJ = GLU ? BN / 2 : BN;
    const int64_t nbj = (od + BJ - 1) / BJ;
    // experts: every expert, and the dropped rows, may end in a partial tile
    const int64_t nbt = EXPERTS ? nt / BM + (nt < a.ne + 1 ? nt : a.ne + 1) : (nt + BM - 1) / BM;
    const int64_t n = nbt * nbj * (SPLIT ? a.splits : 1);
    if (n > 0x7fffffff) return -1;
    a.nbt = (int)nbt;
    a.nbj = (int)nbj;
    return launch_kernel(gemm_i8_kernel<BM, BN, WM, WN, S, SB, SPLIT, GLU, EXPERTS, YT>, dim3((unsigned)n),
                         dim3(WM * WN * 64), stream, a);
}

// What a tile shape costs, in us per 128-byte step of one tile: `alone` in a
// round of tiles that leaves CUs without one, `full` as a CU's share when all
// are busy, where the card's power holds the clock down (1.75 GHz under the
// 256 x 256 tiles against 2.4); `ends` are a round's first loads and epilogue.
// Measured at 8192^3 (full: 420 us with 256 x 256, 452 with 192 x 256, 740 with
// 64 x 128), and with 2630 tokens of 18944 -> 3584 (167, 148 and 244 us) and 64
// to 512 of 3584 -> 3584 (alone).
struct TileCost {
    int bm, bn, per_cu;
    double alone, full, ends;
};
constexpr TileCost COST_256 = {256, 256, 1, 1.05, 1.55, 6.0};
constexpr TileCost COST_192 = {192, 256, 1, 0.84, 1.21, 6.0};
constexpr TileCost COST_64 = {64, 128, 1, 0.30, 0.32, 3.0};
constexpr TileCost COST_64S = {64, 128, 3, 0.54, 0.32, 3.0};   // two stages: three workgroups a CU

template <bool GLU>
static double cost(const TileCost &c, const I8Args &a)
{
    const int64_t bj = GLU ? c.bn / 2 : c.bn;
    const double tiles = (double)((a.od + bj - 1) / bj) * (double)((a.nt + c.bm - 1) / c.bm);
    const double rounds = __builtin_ceil(tiles / (256.0 * c.per_cu));
    const double busy = tiles / 256.0 * c.full, alone = rounds * c.alone;
    return (double)((a.id + BK - 1) / BK) * (busy > alone ? busy : alone) + rounds * c.ends;
}

// The few-token kernel is taken for up to 16 tokens, and up to this many bytes
// of weights (times passes over them) for up to 64: 3584 x 3584 with 16 tokens
// 7.5 us against the tiles' 11 us, level with them at 64 tokens; at 68 MB and 32
// tokens 38 us against 21 us.
constexpr int64_t GEMV_BYTES = int64_t(40) << 20;
// For experts: weights of the experts that have rows, and rows of each.  Above
// it tiles keep more of the weights' loads in flight: 6 experts' 4736 x 3584
// with one row each 23.8 us against 19.4 us, but 6 experts' 1024 x 2048 8.5 us
// against 9.3 us, 4 experts' 700 x 5000 8.4 us against 13.7 us.
constexpr int64_t EXPERTS_GEMV_BYTES = int64_t(24) << 20, EXPERTS_GEMV_ROWS = 16;
// Rows of an expert, on average (the host knows no more: where routing is skewed,
// a few experts with most rows walk small tiles), from which the larger tiles are
// faster, and the tiles it takes for that.  With few rows what counts is how evenly the
// weights' bytes spread over the CUs and how many are in flight: 32 x 128 tiles
// with four stages, two workgroups a CU.  64 experts' 4736 x 3584, us for
// 32 x 128, 64 x 128, 128 x 256 and 256 x 256: 24 rows (23 experts) 73, 88, 85, -;
// 4.5 rows each 175, 173, 184, 208; 15 rows 192, 205, 194, -; 48 rows -, 220, 206,
// 221; 246 rows -, 599, 396, 349.  3584 x 2368, 6 rows: 98, 106, 111, -.  Where
// 64 x 128 tiles are no more than the CUs (TILES_64) their deep form: 8 experts'
// 2048 x 4096, 64 rows each 19.5 against 24.4 us; 2000 x 2048, 128 rows, 320 tiles,
// 20.5 against 17.2.
constexpr double ROWS_64 = 16, ROWS_256 = 96, TILES_64 = 256, TILES_128 = 256, TILES_256 = 192;
// Split sums: shares of at least SPLIT_STEPS steps, a workgroup a CU, and at
// most SPLIT_MOST shares: the last share to arrive reads the others' sums one
// after the other (18944 -> 3584, 32 tokens: 45 us whole, 21 us in four, 28 us
// in nine).  SPLIT_SLOTS and SPLIT_TILES are what the workspace holds.
constexpr int SPLIT_STEPS = 16, SPLIT_MOST = 4, SPLIT_SLOTS = 1024, SPLIT_TILES = 4096, SPLIT_CUS = 256;

// The kernels' forms: 100 * token rows of a tile + 10 * stages of activations
// (0: the few-token kernel).
enum Form { FEW = 1600, T32 = 3240, T64S = 6420, T64 = 6440, T128 = 12820, T192 = 19220, T256 = 25620 };

// The form of a product, and into how many shares its sums are split.
template <bool GLU>
static Form dense_form(const I8Args &a, int &splits)
{
    splits = 1;
    const int64_t wbytes = (GLU ? 2 : 1) * a.od * (int64_t)a.id;
    // (more weight rows than a launch of it holds, from 2^27 on, go to the tiles)
    if ((a.nt <= 16 && (a.od + GEMV_ROWS - 1) / GEMV_ROWS <= launch_groups(GEMV_WAVES * 64)) ||
        (a.nt <= 64 && (a.nt + 15) / 16 * wbytes <= GEMV_BYTES))
        return FEW;
    const double c256 = cost<GLU>(COST_256, a), c192 = cost<GLU>(COST_192, a);
    const double c64 = cost<GLU>(COST_64, a), c64s = cost<GLU>(COST_64S, a);
    if (std::min(c64, c64s) >= std::min(c192, c256)) return c192 < c256 ? T192 : T256;
    if (c64s < c64) return T64S;
    const int64_t tiles = (a.nt + 63) / 64 * ((a.od + (GLU ? 63 : 127)) / (GLU ? 64 : 128));
    const int64_t nk = (a.id + BK - 1) / BK;
    const int64_t most = std::min<int64_t>(std::min<int64_t>(nk / SPLIT_STEPS, SPLIT_MOST), SPLIT_CUS / tiles);
    if (a.part && most >= 2 && tiles * most <= SPLIT_SLOTS && tiles <= SPLIT_TILES) splits = (int)most;
    return T64;
}

template <bool GLU, int YT>
static int pick_dense(I8Args a, hipStream_t stream)
{
    switch (dense_form<GLU>(a, a.splits)) {
    case FEW: return launch_gemv<GLU, false, YT>(a, stream);
    case T192: return launch_tile<192, 256, 2, 4, 2, 3, false, GLU, false, YT>(a, a.od, a.nt, stream);
    case T256: return launch_tile<256, 256, 2, 4, 2, 3, false, GLU, false, YT>(a, a.od, a.nt, stream);
    case T64S: return launch_tile<64, 128, 2, 2, 2, 2, false, GLU, false, YT>(a, a.od, a.nt, stream);
    default: break;
    }
    if (a.splits > 1) return launch_tile<64, 128, 2, 2, 4, 4, true, GLU, false, YT>(a, a.od, a.nt, stream);
    return launch_tile<64, 128, 2, 2, 4, 4, false, GLU, false, YT>(a, a.od, a.nt, stream);
}

template <bool GLU>
static Form experts_form(const I8Args &a)
{
    const int64_t used = a.nt < a.ne ? a.nt : a.ne, rows = (GLU ? 2 : 1) * a.od;
    const double each = (double)a.nt / (double)used;
    if (each <= EXPERTS_GEMV_ROWS && used * rows * a.id <= EXPERTS_GEMV_BYTES) return FEW;
    auto tiles = [&](int bm, int bn) {   // half a tile lost in each expert
        return ((double)a.nt / bm + 0.5 * (double)used) * (double)((rows + bn - 1) / bn);
    };
    if (each >= ROWS_256 && tiles(256, 256) >= TILES_256) return T256;
    if (each < ROWS_64) return T32;
    if (tiles(128, 256) >= TILES_128) return T128;
    return tiles(64, 128) > TILES_64 ? T64S : T64;
}

template <bool GLU, int YT>
static int pick_experts(const I8Args &a, hipStream_t stream)
{
    switch (experts_form<GLU>(a)) {
    case FEW: return launch_gemv<GLU, true, YT>(a, stream);
    case T256: return launch_tile<256, 256, 2, 4, 2, 3, false, GLU, true, YT>(a, a.od, a.nt, stream);
    case T32: return launch_tile<32, 128, 1, 4, 4, 4, false, GLU, true, YT>(a, a.od, a.nt, stream);
    case T128: return launch_tile<128, 256, 2, 4, 2, 3, false, GLU, true, YT>(a, a.od, a.nt, stream);
    case T64S: return launch_tile<64, 128, 2, 2, 2, 2, false, GLU, true, YT>(a, a.od, a.nt, stream);
    default: return launch_tile<64, 128, 2, 2, 4, 4, false, GLU, true, YT>(a, a.od, a.nt, stream);
    }
}

template <int YT>
static int pick_form(const I8Args &a, bool glu, hipStream_t stream)
{
    if (a.plan) return glu ? pick_experts<true, YT>(a, stream) : pick_experts<false, YT>(a, stream);
    return glu ? pick_dense<true, YT>(a, stream) : pick_dense<false, YT>(a, stream);
}

static I8Args args_of(const I8Gemm &g)
{
    I8Args a;
    a.W = reinterpret_cast<const uint8_t *>(g.W);
    a.q = reinterpret_cast<const uint8_t *>(g.q);
    a.sw = g.sw;
    a.sq = g.sq;
    a.bias = g.bias;
    a.y = g.y;
    a.plan = g.plan;
    a.part = static_cast<int32_t *>(g.ws);
    a.cnt = g.ws ? reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(g.ws) + mmq_ws_partial_bytes(MMQ_MAX_WORKERS))
                 : nullptr;
    a.splits = 1;
    a.ldw = g.ldw;
    a.ldq = g.ldq;
    a.ldy = g.ldy;
    a.od = g.od;
    a.nt = g.nt;
    a.id = (int)g.id;
    a.nbt = a.nbj = 0;
    a.ne = (int)g.ne;
    a.slots = (int)g.slots;
    return a;
}

int launch_i8_gemm(const I8Gemm &g, hipStream_t stream)
{
    const I8Args a = args_of(g);
    switch (g.ytype) {
    case T_F32: return pick_form<T_F32>(a, g.glu != 0, stream);
    case T_BF16: return pick_form<T_BF16>(a, g.glu != 0, stream);
    default: return pick_form<T_F16>(a, g.glu != 0, stream);
    }
}

int i8_form(const I8Gemm &g)
{
    const I8Args a = args_of(g);
    if (g.ne > 0) return (g.glu ? experts_form<true>(a) : experts_form<false>(a)) + 1;
    int splits;
    const Form f = g.glu ? dense_form<true>(a, splits) : dense_form<false>(a, splits);
    return f + splits;
}

}  // namespace qig
