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

// Which sequence a workgroup works on.  Sequence i's tiles of BM queries have the
// slots from starts[i] / BM + i on: those of the next begin behind its last one,
// whatever its length, so that nt / BM + nseq slots are enough and no sum over the
// sequences before is needed.  Some slots stay empty.
struct Tile {
    int q0, nq;      // first packed query of the sequence, queries
    int k0, nk;
    int first;       // first query of the tile in its sequence
};

template <int BM>
__device__ __forceinline__ bool find_tile(const PromptArgs &a, int slot, Tile &t)
{
    const int32_t *starts = a.starts;
    const int64_t nt = a.nt;
    const int i = __builtin_amdgcn_readfirstlane(
        count_first((int)a.nseq, [&](int s) { return held(starts[s], nt) / BM + s <= slot; }) - 1);
    if (i < 0) return false;
    t.q0 = held(a.starts[i], a.nt);
    t.nq = held(a.starts[i + 1], a.nt) - t.q0;
    t.k0 = held(a.k_starts[i], a.nk);
    t.nk = held(a.k_starts[i + 1], a.nk) - t.k0;
    if (t.nk < 0) t.nk = 0;
    const int64_t first = (int64_t)(slot - (t.q0 / BM + i)) * BM;
    if (first < 0 || first >= t.nq) return false;   // below 0: starts that decrease
    t.first = (int)first;
    return true;
}

__device__ __forceinline__ bool finite(float v) { return __builtin_fabsf(v) < INFINITY; }

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
#pragma unroll
    for (int r = 0; r < 16; ++r) {
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

// fp32 products on v_mfma_f32_32x32x2_f32 for operands of every type (16-bit ones
// are widened on their way into LDS).  A wave holds 32 queries, a workgroup 4
// waves; 32 keys a step.
//   S^T: lane (n = lane % 32, h = lane / 32) gives key n's and query n's channels
//   8 j + 4 h + i: MFMA i of chunk j then sums channels 8 j + i and 8 j + 4 + i, and
//   four of them need one 16-byte read.
//   S^T register r of lane (n, h): query n, key 8 (r / 4) + 4 h + r % 4; MFMA r of
//   O^T sums these two keys.
template <int D>
struct F32Lds {
    static constexpr int KS = D + 4;             // row step of K: 16-byte reads of 8 rows meet in no bank
    float k[32 * KS];
    float v[32 * D];
};

template <int T, int D>
__global__ __launch_bounds__(256, D > 128 ? 1 : 2) void prompt_f32(PromptArgs a, int slots, int per)
{
    typedef elem_t<T> E;
    __shared__ F32Lds<D> lds;
    constexpr int V = VEC<T>, CH = D / V;        // elements and units of 16 bytes in a row
    const int head = blockIdx.x % a.hq;
    Tile t;
    if (!find_tile<128>(a, slots - 1 - (int)(blockIdx.x / a.hq), t)) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
    const int kvh = head / per, d = a.d;
    const E *kp = static_cast<const E *>(a.k.p) + (int64_t)t.k0 * a.k.token + (int64_t)kvh * a.k.head;
    const E *vp = static_cast<const E *>(a.v.p) + (int64_t)t.k0 * a.v.token + (int64_t)kvh * a.v.head;

    const int mine = t.first + wave * 32 + n;    // this lane's query in its sequence
    const int row = mine < t.nq ? mine : t.nq - 1;
    const E *qp = static_cast<const E *>(a.q.p) + (int64_t)(t.q0 + row) * a.q.token + (int64_t)head * a.q.head;
    float q[D / 2];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 8 * j + 4 * h + i;
            q[4 * j + i] = c < d ? (float)qp[c] : 0.0f;
        }

    // the keys that this lane's, its wave's and its workgroup's queries see
    const int off = t.nk - t.nq;
    const auto end_of = [&](int query) {
        const int e = a.causal ? off + query + 1 : t.nk;
        return e < 0 ? 0 : e > t.nk ? t.nk : e;
    };
    const int end = end_of(row);
    const int last = t.first + 127 < t.nq ? t.first + 127 : t.nq - 1;
    const int kend = end_of(last);
    const int wave_last = t.first + wave * 32 + 31 < t.nq ? t.first + wave * 32 + 31 : t.nq - 1;
    const int wave_end = end_of(wave_last), wave_full = end_of(t.first + wave * 32 < t.nq ? t.first + wave * 32 : t.nq - 1);

    f32x16 o[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x) o[x] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    const int all_full = end_of(t.first);
    for (int k0 = 0; k0 < kend; k0 += 32) {
        const bool masks = k0 + 32 > all_full;   // some query of the workgroup does not see some key
        int bad = 0;
        __syncthreads();
        for (int u = threadIdx.x; u < 32 * CH; u += 256) {
            const int r = u / CH, c = (u % CH) * V;
            float kf[V], vf[V];
            if (k0 + r < t.nk && c < d) {
                const int64_t key = k0 + r;
                unpack16<T>(load16<T>(kp + key * a.k.token + c), kf);
                unpack16<T>(load16<T>(vp + key * a.v.token + c), vf);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) kf[i] = vf[i] = 0.0f;
            }
            if (masks) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const bool fine = finite(vf[i]);
                    bad |= !fine;
                    vf[i] = fine ? vf[i] : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                lds.k[r * F32Lds<D>::KS + c + i] = kf[i];
                lds.v[r * D + c + i] = vf[i];
            }
        }
        if (masks) bad = __syncthreads_or(bad);
        else __syncthreads();
        if (k0 >= wave_end) continue;
        f32x16 s = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            const f32x4 k4 = *reinterpret_cast<const f32x4 *>(&lds.k[n * F32Lds<D>::KS + 8 * j + 4 * h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_32x32x2f32(k4[i], q[4 * j + i], s, 0, 0, 0);
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
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            o[x] *= fix;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                o[x] = __builtin_amdgcn_mfma_f32_32x32x2f32(lds.v[mfma_row(r, h) * D + 32 * x + n], s[r], o[x], 0, 0, 0);
        }
        if (bad) poison<D, E>(o, vp, a.v.token, k0, t.nk, d, end, n, h);
    }
    l += __shfl_xor(l, 32);
    if (mine >= t.nq) return;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    const int64_t at = (int64_t)(t.q0 + mine) * a.y_token + (int64_t)head * a.y_head;
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const int c = 32 * x + mfma_row(r, h);   // four channels in a row
            const float f[4] = {o[x][r] * inv, o[x][r + 1] * inv, o[x][r + 2] * inv, o[x][r + 3] * inv};
            if (c < d) store4(a.y, a.ytype, at + c, f);
        }
}

template <int T>
int launch_f32(const PromptArgs &a, hipStream_t stream)
{
    const int64_t slots = a.nt / 128 + a.nseq;
    const int64_t groups = slots * a.hq;
    if (slots >= (int64_t(1) << 31) || groups > launch_groups(256)) return -1;
    const dim3 grid((unsigned)groups), block(256);
    const int per = a.hq / a.hkv;
    if (a.d <= 64) return launch_kernel(prompt_f32<T, 64>, grid, block, stream, a, (int)slots, per);
    if (a.d <= 128) return launch_kernel(prompt_f32<T, 128>, grid, block, stream, a, (int)slots, per);
    return launch_kernel(prompt_f32<T, 256>, grid, block, stream, a, (int)slots, per);
}

}  // namespace

int launch_attend_prompt(const PromptArgs &a, hipStream_t stream)
{
    if (a.type == T_F32) return launch_f32<T_F32>(a, stream);
    if (a.type == T_BF16) return launch_f32<T_BF16>(a, stream);
    return launch_f32<T_F16>(a, stream);
}

}  // namespace qig
