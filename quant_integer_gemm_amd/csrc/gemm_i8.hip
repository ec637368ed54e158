// gemm_i8.hip -- y = (q . W^T) * sq * sw + bias for int8 rows q (one scale a
// row) and int8 weights W (one scale an output channel), and the same product
// for rows sorted by expert.
//
// The sum over id is a plain int32 sum, so the whole contraction stays on the
// int8 MFMA and both scales are applied once per output.  A workgroup owns a
// BM x BN tile (tokens x weight rows) and walks id in steps of 128 bytes: both
// operands are copied straight into LDS (global_load_lds), the next step's
// copies in flight while this one is multiplied, one barrier a step.
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

namespace qig {

constexpr int BK = 128;

struct I8Args {
    const uint8_t *W, *q;
    const float *sw, *sq, *bias;
    void *y;
    const int32_t *plan;
    int64_t ldw, ldq, ldy, od, nt;
    int id, nbt, nbj, ne, slots;
};

__device__ __forceinline__ uint64_t uniform64(const void *p)
{
    const uint64_t b = reinterpret_cast<uintptr_t>(p);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    return (uint64_t)lo | ((uint64_t)hi << 32);
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

// Which expert and rows a workgroup's token tile covers: tile number mt
// counts the experts' tiles in order, the dropped rows' tiles last (e == ne).
struct Rows {
    int e, first, count;   // expert, first position in the order, rows of the tile (0: no such tile)
};

template <int BM>
__device__ __forceinline__ Rows find_rows(const int32_t *plan, int ne, int mt)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 <= ne; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, n = 0;
        if (e <= ne) {
            lo = plan[e];
            n = plan[e + 1] - lo;
        }
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
            const int m = mt - __shfl(excl, src);
            Rows r;
            r.e = e0 + src;
            r.first = __shfl(lo, src) + m * BM;
            const int left = __shfl(n, src) - m * BM;
            r.count = left < BM ? left : BM;
            return r;
        }
        before += __shfl(incl, 63);
    }
    return Rows{0, 0, 0};
}

// BM x BN tile, WM x WN waves, each BM/WM x BN/WN in 32 x 32 MFMA tiles.
// GLU: of every 64 of the tile's weight rows the first 32 are gate rows and
// the last 32 the up rows of the same outputs, so a wave holds both halves of
// an output in the same lane and register.
template <int BM, int BN, int WM, int WN, bool GLU, bool EXPERTS, int YT>
__global__ __launch_bounds__(WM *WN * 64) void gemm_i8_kernel(I8Args g)
{
    constexpr int NW = WM * WN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr int PA = BM / 8 / NW, PB = BN / 8 / NW;   // 1 KB pieces a wave copies each step
    constexpr int STAGE = (BM + BN) * BK;
    constexpr int BJ = GLU ? BN / 2 : BN;               // outputs of a tile
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && TM >= 1 && TN >= 1, "tile");
    static_assert(!GLU || TN % 2 == 0, "gate and up rows of an output in one wave");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];
    __shared__ float s_sq[BM];
    __shared__ int32_t s_row[EXPERTS ? BM : 1];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int jt = (int)(blockIdx.x % (unsigned)g.nbj), mt = (int)(blockIdx.x / (unsigned)g.nbj);
    const int64_t j0 = (int64_t)jt * BJ;
    const uint8_t *W = g.W;
    const float *sw = g.sw, *bias = g.bias;
    int64_t t0 = (int64_t)mt * BM;
    int count;
    elem_t<YT> *y = static_cast<elem_t<YT> *>(g.y);

    if constexpr (EXPERTS) {
        const Rows r = find_rows<BM>(g.plan, g.ne, mt);
        if (r.count == 0) return;
        count = r.count;
        const int32_t *order = g.plan + g.ne + 2 + r.first;
        if (r.e == g.ne) {
            // dropped rows: zeros
            for (int i = wave; i < count; i += NW) {
                elem_t<YT> *row = y + (int64_t)order[i] * g.ldy;
                for (int64_t j = j0 + lane; j < j0 + BJ && j < g.od; j += 64) row[j] = (elem_t<YT>)0.0f;
            }
            return;
        }
        const int64_t rows = GLU ? 2 * g.od : g.od;
        W += (int64_t)r.e * rows * g.ldw;
        sw += (int64_t)r.e * rows;
        if (bias) bias += (int64_t)r.e * rows;
        for (int i = tid; i < BM; i += NW * 64) {
            const int32_t row = order[i < count ? i : count - 1];
            s_row[i] = row;
            s_sq[i] = g.sq[row / g.slots];
        }
        __syncthreads();
    } else {
        count = (int)(g.nt - t0 < BM ? g.nt - t0 : BM);
        for (int i = tid; i < BM; i += NW * 64) s_sq[i] = g.sq[t0 + (i < count ? i : count - 1)];
    }

    // The rows that this lane copies: piece p of the wave holds rows
    // 8 (PA wave + p) .. + 7, lane l row l / 8 and slot l % 8.
    const int lr = lane >> 3;
    const uint32_t gran = (uint32_t)((lane & 7) ^ lr);   // the granule that belongs in this lane's slot
    uint32_t aoff[EXPERTS ? 1 : PA], boff[PB];
    uint64_t aptr[EXPERTS ? PA : 1];
#pragma unroll
    for (int p = 0; p < PA; ++p) {
        const int r = 8 * (PA * wave + p) + lr;
        if constexpr (EXPERTS)
            aptr[p] = reinterpret_cast<uintptr_t>(g.q + (int64_t)(s_row[r] / g.slots) * g.ldq);
        else
            aoff[p] = (uint32_t)(r < count ? r : count - 1) * (uint32_t)g.ldq;
    }
    uint64_t bbase = uniform64(W + (GLU ? j0 : (int64_t)jt * BN) * g.ldw);
    [[maybe_unused]] const uint64_t uphalf = GLU ? (uint64_t)(g.od * g.ldw) : 0;
    bool bup[PB];
#pragma unroll
    for (int p = 0; p < PB; ++p) {
        // a piece's eight rows lie in one block of 32, so gate or up is the
        // same for the whole piece
        const int r = 8 * (PB * wave + p) + lr;
        int j = GLU ? (r >> 6) * 32 + (r & 31) : r;
        bup[p] = GLU && ((8 * (PB * wave + p)) & 32) != 0;
        const int64_t last = g.od - 1 - j0;
        if (j > last) j = (int)last;
        boff[p] = (uint32_t)j * (uint32_t)g.ldw;
    }
    const uint64_t abase0 = EXPERTS ? 0 : uniform64(g.q + t0 * g.ldq);
    const uint32_t l0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

    const int nk = (g.id + BK - 1) / BK;
    const int tail = g.id - (nk - 1) * BK;   // bytes of the last step, 1 .. 128

    auto issue = [&](int kt) {
        const uint32_t dst = l0 + (kt & 1) * STAGE;
        const uint64_t k0 = (uint64_t)kt * BK;
        uint32_t go = 16 * gran;
        if (kt == nk - 1 && (int)go >= tail) go = 0;
#pragma unroll
        for (int p = 0; p < PA; ++p) {
            const uint32_t d = dst + 1024 * (PA * wave + p);
            if constexpr (EXPERTS)
                copy16_at(aptr[p] + k0 + go, d);
            else
                copy16(abase0 + k0, aoff[p] + go, d);
        }
#pragma unroll
        for (int p = 0; p < PB; ++p)
            copy16(bbase + k0 + (bup[p] ? uphalf : 0), boff[p] + go, dst + BM * BK + 1024 * (PB * wave + p));
    };

    const int wm = wave / WN, wn = wave % WN;
    const int lrow = lane & 31, lhalf = lane >> 5;
    i32x16 acc[TM][TN];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0;

    issue(0);
    for (int kt = 0; kt < nk; ++kt) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        uint8_t *st = lds + (kt & 1) * STAGE;
        if (kt + 1 < nk) {
            issue(kt + 1);
        } else if (tail < BK) {
            // zero the activations' bytes past id
            for (int i = tid; i < BM * 8; i += NW * 64) {
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
        }
#pragma unroll
        for (int c = 0; c < BK / 32; ++c) {
            i32x4 a[TM], b[TN];
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const int r = (wm * TM + m) * 32 + lrow;
                a[m] = *reinterpret_cast<const i32x4 *>(st + r * BK + 16 * ((2 * c + lhalf) ^ (r & 7)));
            }
#pragma unroll
            for (int n = 0; n < TN; ++n) {
                const int r = (wn * TN + n) * 32 + lrow;
                b[n] = *reinterpret_cast<const i32x4 *>(st + BM * BK + r * BK + 16 * ((2 * c + lhalf) ^ (r & 7)));
            }
#pragma unroll
            for (int m = 0; m < TM; ++m)
#pragma unroll
                for (int n = 0; n < TN; ++n) acc[m][n] = mfma_i8(a[m], b[n], acc[m][n]);
        }
    }

    // Lane l, register i: token 8 (i / 4) + 4 (l / 32) + i % 4, weight row l % 32.
    constexpr int NO = GLU ? TN / 2 : TN;
#pragma unroll
    for (int n = 0; n < NO; ++n) {
        const int64_t j = j0 + (wn * NO + n) * 32 + lrow;
        const bool jok = j < g.od;
        const int64_t jc = jok ? j : 0;
        const float w0 = sw[jc], b0 = bias ? bias[jc] : 0.0f;
        float w1 = 0.0f, b1 = 0.0f;
        if constexpr (GLU) {
            w1 = sw[g.od + jc];
            b1 = bias ? bias[g.od + jc] : 0.0f;
        }
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = (wm * TM + m) * 32 + mfma_row(i, lhalf);
                const float s = s_sq[r];
                float v;
                if constexpr (GLU) {
                    const float a = (float)acc[m][2 * n][i] * s * w0 + b0;
                    const float b = (float)acc[m][2 * n + 1][i] * s * w1 + b1;
                    v = silu_mul(a, b);
                } else {
                    v = (float)acc[m][n][i] * s * w0 + b0;
                }
                if (r < count && jok) {
                    const int64_t row = EXPERTS ? (int64_t)s_row[r] : t0 + r;
                    y[row * g.ldy + j] = (elem_t<YT>)v;
                }
            }
    }
}

template <int BM, int BN, int WM, int WN, bool GLU, bool EXPERTS, int YT>
static int launch_tile(I8Args a, int64_t od, int64_t nt, hipStream_t stream)
{
    constexpr int BJ = GLU ? BN / 2 : BN;
    const int64_t nbj = (od + BJ - 1) / BJ;
    // experts: every expert, and the dropped rows, may end in a partial tile
    const int64_t nbt = EXPERTS ? nt / BM + (nt < a.ne + 1 ? nt : a.ne + 1) : (nt + BM - 1) / BM;
    if (nbt * nbj > 0x7fffffff) return -1;
    a.nbt = (int)nbt;
    a.nbj = (int)nbj;
    return launch_kernel(gemm_i8_kernel<BM, BN, WM, WN, GLU, EXPERTS, YT>, dim3((unsigned)(nbt * nbj)),
                         dim3(WM * WN * 64), stream, a);
}

template <bool GLU, bool EXPERTS, int YT>
static int pick(const I8Args &a, hipStream_t stream)
{
    return launch_tile<128, 128, 2, 2, GLU, EXPERTS, YT>(a, a.od, a.nt, stream);
}

template <int YT>
static int pick_form(const I8Args &a, bool glu, hipStream_t stream)
{
    if (a.plan) return glu ? pick<true, true, YT>(a, stream) : pick<false, true, YT>(a, stream);
    return glu ? pick<true, false, YT>(a, stream) : pick<false, false, YT>(a, stream);
}

int launch_i8_gemm(const I8Gemm &g, hipStream_t stream)
{
    I8Args a;
    a.W = reinterpret_cast<const uint8_t *>(g.W);
    a.q = reinterpret_cast<const uint8_t *>(g.q);
    a.sw = g.sw;
    a.sq = g.sq;
    a.bias = g.bias;
    a.y = g.y;
    a.plan = g.plan;
    a.ldw = g.ldw;
    a.ldq = g.ldq;
    a.ldy = g.ldy;
    a.od = g.od;
    a.nt = g.nt;
    a.id = (int)g.id;
    a.nbt = a.nbj = 0;
    a.ne = (int)g.ne;
    a.slots = (int)g.slots;
    switch (g.ytype) {
    case T_F32: return pick_form<T_F32>(a, g.glu != 0, stream);
    case T_BF16: return pick_form<T_BF16>(a, g.glu != 0, stream);
    default: return pick_form<T_F16>(a, g.glu != 0, stream);
    }
}

}  // namespace qig
