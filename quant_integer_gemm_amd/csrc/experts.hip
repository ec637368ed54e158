// experts.hip -- routing of tokens to experts, the order of rows by expert,
// and the weighted sum of the experts' outputs.
#include "qig_i8_device.h"
#include "qig_launch.h"

#include <math.h>

namespace qig {

// ---------------------------------------------------------------------------
// routing
// ---------------------------------------------------------------------------
// Scores: p = softmax(l) or sigmoid(l); the choice is by c = p + bias, the k
// largest among the experts of the topk_groups best groups (a group's score:
// the sum of its group_top largest c), equal values to the lower index.  Which
// expert wins is a comparison of near values: it is decided in 64 bits, since
// in 32 the rounding of exp would decide about one row in ten thousand.
// Softmax without a bias keeps the order of the logits, so there the choice
// compares the logits themselves (also where the scores underflow), unless groups
// are ranked by the sum of two scores: then groups and experts go by the scores.
// A logit of -infinity or NaN is an expert that may not be chosen; +infinity
// counts as the largest finite number.
//
// Only rows that need 64 bits pay for them: route_kernel first chooses by c in
// 32 bits with a bound on its error.  Where neighbours among the first k + 1 are
// nearer than that bound, those are put in order by their c in 64 bits; where
// that cannot settle it (three values at the border of the chosen, two groups at
// theirs), the whole row is chosen again by route_exact.  The weights of the k
// chosen are formed in 64 bits either way (one expert a lane).

constexpr float LARGEST = 3.402823466e38f;

// Order-preserving integer of a finite or infinite fp32 (never 0).
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);   // -0 to +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Largest of the wave's values, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
#define QIG_STEP(ctrl, rows)                                                                                   \
    {                                                                                                          \
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false);           \
        v = o > v ? o : v;                                                                                     \
    }
    QIG_STEP(0x111, 0xf)   // from the lane 1 before, in rows of 16
    QIG_STEP(0x112, 0xf)
    QIG_STEP(0x114, 0xf)
    QIG_STEP(0x118, 0xf)
    QIG_STEP(0x142, 0xa)   // last lane of row 0 to row 1, of 2 to 3
    QIG_STEP(0x143, 0xc)   // last lane of row 1 to rows 2 and 3
#undef QIG_STEP
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

__device__ __forceinline__ void lds_order()
{
    // one wave's LDS accesses are executed in order: only the compiler must
    // keep theirs
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// A logit as the routing takes it: whether the expert may be chosen.
__device__ __forceinline__ bool take_logit(bool there, float v, float &x)
{
    x = there ? v : -INFINITY;
    const bool ok = x > -INFINITY;   // false for NaN
    x = ok ? __builtin_fminf(x, LARGEST) : 0.0f;
    return ok;
}

// A lane's NS neighbouring values, n of them there (0 for the others).
template <int NS, typename E>
__device__ __forceinline__ void load_run(const E *p, int n, float (&o)[NS])
{
    if (n >= NS) {
        struct __attribute__((packed, aligned(2))) Run {
            E v[NS];
        };
        const Run r = *reinterpret_cast<const Run *>(p);
#pragma unroll
        for (int i = 0; i < NS; ++i) o[i] = (float)r.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) o[i] = i < n ? (float)p[i] : 0.0f;
    }
}

// The group of expert e.  e < 512, so the rounding of by_size adds less than
// 2^-11 to e / size, which is at least 2^-9 below the next integer.
__device__ __forceinline__ int group_of(const RouteArgs &a, int e)
{
    return (int)(((uint32_t)e * a.by_size) >> 20);
}

// One wave chooses a token's experts in 64 bits: lane l holds experts l,
// l + 64, ...  Returns the expert of slot `lane` (-1: none).
template <int NS, int T>
__device__ int route_exact(const RouteArgs &a, const elem_t<T> *l, double *s_c, double *s_g, uint8_t *s_keep)
{
    const int lane = threadIdx.x & 63;
    double c[NS];
    bool ok[NS];
    double top = -INFINITY, sum = 0.0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        float x;
        const int e = lane + 64 * i;
        ok[i] = take_logit(e < a.ne, e < a.ne ? (float)l[e] : 0.0f, x);
        c[i] = (double)x;
        if (ok[i]) top = fmax(top, c[i]);
    }
    const bool by_logit = a.score == 0 && !a.bias && (a.groups == 1 || a.group_top == 1);
    if (!by_logit) {
        if (a.score == 0) {
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) top = fmax(top, __shfl_xor(top, d));
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                c[i] = ok[i] ? exp(c[i] - top) : 0.0;
                sum += c[i];
            }
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
            const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
            for (int i = 0; i < NS; ++i) c[i] *= inv;
        } else {
#pragma unroll
            for (int i = 0; i < NS; ++i) c[i] = ok[i] ? 1.0 / (1.0 + exp(-c[i])) : 0.0;
        }
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (a.bias && lane + 64 * i < a.ne) c[i] += (double)a.bias[lane + 64 * i];
    }
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (!ok[i] || !(c[i] > -INFINITY)) {
            ok[i] = false;
            c[i] = -INFINITY;
        }
    if (a.groups > 1) {
        const int size = (int)a.size;
#pragma unroll
        for (int i = 0; i < NS; ++i) s_c[lane + 64 * i] = c[i];
        lds_order();
        if (lane < a.groups) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const double x = s_c[e];
                b2 = fmax(b2, fmin(b1, x));
                b1 = fmax(b1, x);
            }
            // a group's missing second score adds nothing
            s_g[lane] = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
        }
        lds_order();
        if (lane < a.groups) {
            int better = 0;
            for (int o = 0; o < a.groups; ++o) better += s_g[o] > s_g[lane] || (s_g[o] == s_g[lane] && o < lane);
            s_keep[lane] = better < a.topk_groups;
        }
        lds_order();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int e = lane + 64 * i;
            if (e < a.ne && !s_keep[group_of(a, e)]) ok[i] = false;
        }
    }
    int my_id = -1;
    for (int r = 0; r < a.k; ++r) {
        double best = -INFINITY;
        int be = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (ok[i] && c[i] > best) {
                best = c[i];
                be = lane + 64 * i;
            }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const double ob = __shfl_xor(best, d);
            const int oe = __shfl_xor(be, d);
            if (ob > best || (ob == best && oe < be)) {
                best = ob;
                be = oe;
            }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (lane + 64 * i == be) ok[i] = false;
        if (lane == r && be != 0x7fffffff) my_id = be;
    }
    return my_id;
}

constexpr int ROUTE_WAVES = 4;

// One wave a token, four a workgroup; lane l holds the NS experts from l NS on,
// sorted by falling key, so that each of the k rounds compares one key a lane:
// a DPP maximum over the wave, then the first lane that has it (the lowest
// expert among equals, since a lane's equals stay in order).
//
// Error bounds of the 32-bit scores (u = 2^-24): sigmoid(x) is off by at most
// p (1 - p) (|x| + 2) u + 3 p u < 4 u; softmax, its sum of up to 512 terms added
// in a tree of 15 levels, by less than 20 u times the row's largest p; the sum
// with the bias adds u |c|.  A comparison of two group scores takes four of
// them.  So values further apart than 2^-20 (sigmoid) or 2^-17 p_max (softmax)
// plus 2^-21 |c| (a group's score: the sum of its |c|) are in their exact order.
//
// Bound by its instructions and their latencies, not by the logits' bytes:
// 16384 tokens, 256 experts in 8 groups, k = 8 (17 MB) 20 us, 610 vector
// instructions a token; without groups 16 us (450), and 11 for k = 1 (300).  With
// the weights formed by every wave 22 us (670).  Eight waves a SIMD (64
// registers) against six, then: 26 and 30.
template <int NS, int T>
__global__ __launch_bounds__(ROUTE_WAVES * 64, NS <= 4 ? 8 : 1) void route_kernel(RouteArgs a)
{
    __shared__ double s_all[ROUTE_WAVES][NS * 64 + 64];
    __shared__ uint8_t s_keeps[ROUTE_WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __shared__ float s_x[ROUTE_WAVES][ROUTE_MAX_K], s_top[ROUTE_WAVES];
    __shared__ double s_sum[ROUTE_WAVES];
    const int64_t t0 = (int64_t)blockIdx.x * ROUTE_WAVES, t = t0 + wave < a.nt ? t0 + wave : a.nt - 1;
    const elem_t<T> *l = static_cast<const elem_t<T> *>(a.logits) + t * a.ldl;
    float x[NS], c[NS];
    bool ok[NS];
    float top = -INFINITY;
    const int here = a.ne - lane * NS;   // experts of this lane (any number)
    load_run<NS>(l + lane * NS, here, x);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        ok[i] = take_logit(i < here, x[i], x[i]);
        if (ok[i]) top = __builtin_fmaxf(top, x[i]);
    }
    if (a.score == 0) top = key_value(wave_max(order_key(top)));
    const bool by_logit = a.score == 0 && !a.bias && (a.groups == 1 || a.group_top == 1);
    float tol = 0.0f;   // nearer values than tol + 2^-21 |c| are not told apart here
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < NS; ++i) c[i] = x[i];
    } else {
        if (a.score == 0) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                c[i] = ok[i] ? __builtin_amdgcn_exp2f((x[i] - top) * 1.4426950408889634f) : 0.0f;
                sum += c[i];
            }
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
            for (int i = 0; i < NS; ++i) c[i] *= inv;
            tol = 0x1p-17f * inv;   // the largest p is inv
        } else {
#pragma unroll
            for (int i = 0; i < NS; ++i)
                c[i] = ok[i] ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[i] * -1.4426950408889634f)) : 0.0f;
            tol = 0x1p-20f;
        }
        if (a.bias) {
            float b[NS];
            load_run<NS>(a.bias + lane * NS, here, b);
#pragma unroll
            for (int i = 0; i < NS; ++i) c[i] += b[i];
        }
    }
    // key 0: not to be chosen
    uint32_t key[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) key[i] = ok[i] && c[i] > -INFINITY ? order_key(c[i]) : 0u;
    bool near_groups = false;
    if (a.groups > 1) {
        const int size = (int)a.size;
        uint32_t *s_k = reinterpret_cast<uint32_t *>(s_all[wave]);
        uint8_t *s_keep = s_keeps[wave];
#pragma unroll
        for (int i = 0; i < NS; ++i) s_k[lane * NS + i] = key[i];
        lds_order();
        // `lanes` lanes a group (a power of two), each over every lanes-th expert
        const int lanes = 1 << a.lane_bits, g = lane >> a.lane_bits, in = lane & (lanes - 1);
        uint32_t b1 = 0, b2 = 0;
        if (g < a.groups)
            for (int e = g * size + in; e < (g + 1) * size; e += lanes) {
                const uint32_t v = s_k[e];
                const uint32_t low = b1 < v ? b1 : v;
                b2 = low > b2 ? low : b2;
                b1 = b1 > v ? b1 : v;
            }
        for (int d = 1; d < lanes; d *= 2) {
            const int from = (lane ^ d) * 4;
            const uint32_t o1 = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)b1);
            const uint32_t o2 = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)b2);
            const uint32_t low = b1 < o1 ? b1 : o1;
            b2 = b2 > o2 ? b2 : o2;
            b2 = low > b2 ? low : b2;
            b1 = b1 > o1 ? b1 : o1;
        }
        // a group's missing second score adds nothing; -infinity: nothing to choose
        float score = b1 ? key_value(b1) : -INFINITY;
        float size12 = __builtin_fabsf(score);   // of the terms that the score is rounded from
        if (a.group_top == 2 && b2) {
            score += key_value(b2);
            size12 += __builtin_fabsf(key_value(b2));
        }
        int rank = 64;   // of the group, in its first lane
        if (in == 0 && g < a.groups) rank = 0;
        for (int o = 0; o < a.groups; ++o) {
            const float other = lane_value(score, o * lanes);
            rank += other > score || (other == score && o < g);
        }
        if (in == 0 && g < a.groups) s_keep[g] = rank < a.topk_groups;
        if (!by_logit && a.topk_groups < a.groups) {
            // the last group that stays against the first that goes
            const int w0 = __ffsll((unsigned long long)__ballot(rank == a.topk_groups - 1)) - 1;
            const int w1 = __ffsll((unsigned long long)__ballot(rank == a.topk_groups)) - 1;
            const float size12s = __builtin_fmaxf(lane_value(size12, w0), lane_value(size12, w1));
            // (sums that overflow 32 bits need 64, too: their difference is NaN)
            near_groups = !(lane_value(score, w0) - lane_value(score, w1) > tol + 0x1p-21f * size12s);
        }
        lds_order();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int e = lane * NS + i;
            if (e < a.ne && !s_keep[group_of(a, e)]) key[i] = 0;
        }
    }
    // the lane's keys by falling value, equals in order
    int slot[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) slot[i] = i;
#pragma unroll
    for (int i = 1; i < NS; ++i)
#pragma unroll
        for (int j = i; j > 0; --j) {
            const bool swap = key[j] > key[j - 1];
            const uint32_t k0 = swap ? key[j] : key[j - 1], k1 = swap ? key[j - 1] : key[j];
            const int s0 = swap ? slot[j] : slot[j - 1], s1 = swap ? slot[j - 1] : slot[j];
            key[j - 1] = k0;
            key[j] = k1;
            slot[j - 1] = s0;
            slot[j] = s1;
        }
    // round r puts its key and expert into lane r; two rounds more than k show
    // what the last ones won against
    int my_id = -1;
    uint32_t my_key = 0;
    const int rounds = by_logit ? a.k : a.k + 2;
    for (int r = 0; r < rounds; ++r) {
        const uint32_t best = wave_max(key[0]);
        const int w = __ffsll((unsigned long long)__ballot(key[0] == best)) - 1;
        const int id = w * NS + __builtin_amdgcn_readlane(slot[0], w);
        my_id = lane == r ? id : my_id;
        my_key = lane == r ? best : my_key;
        const bool mine = lane == w;
#pragma unroll
        for (int i = 0; i + 1 < NS; ++i) {
            key[i] = mine ? key[i + 1] : key[i];
            slot[i] = mine ? slot[i + 1] : slot[i];
        }
        key[NS - 1] = mine ? 0u : key[NS - 1];
    }
    if (!by_logit) {
        // nearer to the next (or the one after it) than the bound?
        const uint32_t k1 = (uint32_t)__shfl_down((int)my_key, 1), k2 = (uint32_t)__shfl_down((int)my_key, 2);
        const float v = key_value(my_key), n1 = key_value(k1), n2 = key_value(k2);
        const bool near1 = k1 != 0 && v - n1 <= tol + 0x1p-21f * __builtin_fabsf(n1);
        const bool near2 = k2 != 0 && v - n2 <= tol + 0x1p-21f * __builtin_fabsf(n2);
        if (near_groups || __any(lane == a.k - 1 && near2)) {
            my_id = route_exact<NS, T>(a, l, s_all[wave], s_all[wave] + NS * 64, s_keeps[wave]);
            my_key = my_id >= 0 ? 1u : 0u;
        } else if (__any(lane < a.k && near1)) {
            // the k + 1 first hold the k chosen: put them in order in 64 bits
            double e = -INFINITY, sum = 1.0;
            if (a.score == 0) {
                sum = 0.0;
#pragma unroll
                for (int i = 0; i < NS; ++i) sum += ok[i] ? exp((double)x[i] - (double)top) : 0.0;
#pragma unroll
                for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
            }
            if (lane <= a.k && my_key != 0) {
                float xi;
                take_logit(true, (float)l[my_id], xi);
                e = a.score == 0 ? exp((double)xi - (double)top) * (1.0 / sum) : 1.0 / (1.0 + exp(-(double)xi));
                if (a.bias) e += (double)a.bias[my_id];
            }
            int rank = 0;
            for (int o = 0; o <= a.k; ++o) {
                const double oe = __shfl(e, o);
                const int oid = __shfl(my_id, o);
                rank += oe > e || (oe == e && (e == -INFINITY ? o < lane : oid < my_id));
            }
            if (lane > a.k) rank = lane;
            my_id = __builtin_amdgcn_ds_permute(4 * rank, my_id);
            my_key = (uint32_t)__builtin_amdgcn_ds_permute(4 * rank, (int)my_key);
        }
    }
    if (lane >= a.k || my_key == 0) my_id = -1;

    if (lane < a.k && t0 + wave < a.nt) a.ids[t * a.k + lane] = my_id;

    // Weights in 64 bits, a third of the instructions if every wave formed its
    // own: the first waves form those of all four tokens, 16 or 32 lanes a token.
    if (lane < ROUTE_MAX_K) {
        float xi = -INFINITY;   // none
        if (my_id >= 0) take_logit(true, (float)l[my_id], xi);
        s_x[wave][lane] = xi;
    }
    if (a.score == 0) {
        double sum = 1.0;
        if (!a.renorm) {
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < NS; ++i) sum += ok[i] ? exp((double)x[i] - (double)top) : 0.0;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
        }
        if (lane == 0) {
            s_top[wave] = top;
            s_sum[wave] = sum;
        }
    }
    __syncthreads();
    const int bits = a.k <= 16 ? 4 : 5;   // log2 of the lanes a token
    const int mine = (wave << (6 - bits)) + (lane >> bits), at = lane & ((1 << bits) - 1);
    if (mine >= ROUTE_WAVES) return;   // the whole wave
    const float xi = s_x[mine][at];
    double p = 0.0;
    if (xi > -INFINITY) {
        if (a.score == 0) {
            p = exp((double)xi - (double)s_top[mine]);
            if (!a.renorm) p /= s_sum[mine];
        } else {
            p = 1.0 / (1.0 + exp(-(double)xi));
        }
    }
    double scale = (double)a.scale;
    if (a.renorm) {
        double sum = p;
        if (bits == 5) sum += __shfl_xor(sum, 16);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
        scale = sum > 0.0 ? scale / sum : 0.0;
    }
    if (at < a.k && t0 + mine < a.nt) a.w[(t0 + mine) * a.k + at] = (float)(p * scale);
}

template <int T>
static int route_typed(const RouteArgs &args, hipStream_t stream)
{
    return in_launches(args.nt, launch_groups(ROUTE_WAVES * 64) * ROUTE_WAVES, [&](int64_t r, int64_t n) {
        RouteArgs a = args;
        a.logits = static_cast<const elem_t<T> *>(args.logits) + r * args.ldl;
        a.ids += r * a.k;
        a.w += r * a.k;
        a.nt = n;
        const dim3 grid((unsigned)((n + ROUTE_WAVES - 1) / ROUTE_WAVES)), block(ROUTE_WAVES * 64);
        if (a.ne <= 64) return launch_kernel(route_kernel<1, T>, grid, block, stream, a);
        if (a.ne <= 128) return launch_kernel(route_kernel<2, T>, grid, block, stream, a);
        if (a.ne <= 256) return launch_kernel(route_kernel<4, T>, grid, block, stream, a);
        return launch_kernel(route_kernel<8, T>, grid, block, stream, a);
    });
}

int launch_route(const RouteArgs &args, hipStream_t stream)
{
    RouteArgs a = args;
    a.size = (uint32_t)(a.ne / a.groups);
    a.by_size = ((1u << 20) + a.size - 1) / a.size;
    while ((2 << a.lane_bits) * a.groups <= 64) ++a.lane_bits;
    switch (a.ltype) {
    case T_F32: return route_typed<T_F32>(a, stream);
    case T_BF16: return route_typed<T_BF16>(a, stream);
    default: return route_typed<T_F16>(a, stream);
    }
}

// ---------------------------------------------------------------------------
// the order of rows by expert
// ---------------------------------------------------------------------------
// A stable counting sort in one launch.  Every workgroup counts all rows per
// expert, those before its own share apart (LDS counters; the ids come from the
// caches), which gives it the first position of its rows of each expert without
// waiting for another workgroup; then each wave places its part of the share,
// 64 rows at a time, a row's rank among the 64 being the number of lower lanes
// with the same expert.  The placing is what costs (a ballot a bit of the
// expert's number), and it is what the workgroups share out: 15780 rows of 64
// experts 7 us, 25 us with one workgroup.  Ids outside [0, ne) count as expert
// ne (dropped rows).
constexpr int PLAN_WAVES = 16, PLAN_THREADS = PLAN_WAVES * 64, PLAN_BATCH = 16, PLAN_GROUPS = 64;

__global__ __launch_bounds__(PLAN_THREADS) void plan_kernel(const int32_t *__restrict__ ids, int nrows, int ne,
                                                            int share, int32_t *__restrict__ plan)
{
    __shared__ int32_t s_count[2][EXPERTS_MAX + 1];   // rows before the share, and the others
    __shared__ int32_t s_at[EXPERTS_MAX + 1][PLAN_WAVES];   // next position of a wave's rows
    __shared__ int32_t part[PLAN_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int lo = (int)blockIdx.x * share;   // a multiple of PLAN_THREADS
    const int per = share / PLAN_WAVES;       // a wave's rows, a multiple of 64
    const int wlo = lo + wave * per;
    const int whi = wlo + per < nrows ? wlo + per : nrows;
    int e[PLAN_BATCH];
    auto load = [&](int i0) {
#pragma unroll
        for (int b = 0; b < PLAN_BATCH; ++b) {
            const int64_t i = (int64_t)i0 + PLAN_THREADS * b + tid;
            e[b] = i < nrows ? ids[i] : -1;
        }
#pragma unroll
        for (int b = 0; b < PLAN_BATCH; ++b) e[b] = (unsigned)e[b] < (unsigned)ne ? e[b] : ne;
    };
    load(0);
    for (int i = tid; i <= ne; i += PLAN_THREADS) {
        s_count[0][i] = 0;
        s_count[1][i] = 0;
    }
    for (int i = tid; i < (ne + 1) * PLAN_WAVES; i += PLAN_THREADS) s_at[i / PLAN_WAVES][i % PLAN_WAVES] = 0;
    __syncthreads();
    for (int64_t i0 = 0; i0 < nrows; i0 += PLAN_THREADS * PLAN_BATCH) {
        if (i0 > 0) load((int)i0);
#pragma unroll
        for (int b = 0; b < PLAN_BATCH; ++b) {
            const int64_t i = i0 + PLAN_THREADS * b;
            if (i + tid < nrows) atomicAdd(&s_count[i >= lo][e[b]], 1);
        }
    }
    for (int i = wlo + lane; i < whi; i += 64) {
        const int x = ids[i];
        atomicAdd(&s_at[(unsigned)x < (unsigned)ne ? x : ne][wave], 1);
    }
    __syncthreads();
    // thread i: expert i (ne <= 512 < 1024)
    const int before = tid <= ne ? s_count[0][tid] : 0;
    const int all = tid <= ne ? before + s_count[1][tid] : 0;
    int incl = all;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    int first = incl - all;
    for (int w = 0; w < wave; ++w) first += part[w];
    if (tid <= ne) {
        int at = first + before;
#pragma unroll
        for (int w = 0; w < PLAN_WAVES; ++w) {
            const int c = s_at[tid][w];
            s_at[tid][w] = at;
            at += c;
        }
        if (blockIdx.x == 0) plan[tid] = first;
    }
    if (blockIdx.x == 0 && tid == 0) plan[ne + 1] = nrows;
    __syncthreads();
    int32_t *order = plan + ne + 2;
    const int bits = 32 - __builtin_clz(ne);
    for (int i0 = wlo; i0 < whi; i0 += 64) {
        const int i = i0 + lane;
        const bool live = i < whi;
        int x = live ? ids[i] : ne;
        x = (unsigned)x < (unsigned)ne ? x : ne;
        uint64_t same = __ballot(live);   // lanes with the same expert, by its bits
        for (int bit = 0; bit < bits; ++bit) {
            const bool mine = (x >> bit) & 1;
            const uint64_t set = __ballot(mine);
            same &= mine ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (live) {
            const int base = s_at[x][wave];
            order[base + rank] = i;
            if (rank == 0) s_at[x][wave] = base + __popcll(same);
        }
    }
}

int launch_plan(const int32_t *ids, int64_t nrows, int64_t ne, int32_t *plan, hipStream_t stream)
{
    // shares of a multiple of PLAN_THREADS rows, at most PLAN_GROUPS of them
    int64_t share = (nrows + PLAN_GROUPS - 1) / PLAN_GROUPS;
    share = (share + PLAN_THREADS - 1) / PLAN_THREADS * PLAN_THREADS;
    if (share == 0) share = PLAN_THREADS;
    const int64_t groups = nrows > 0 ? (nrows + share - 1) / share : 1;
    return launch_kernel(plan_kernel, dim3((unsigned)groups), dim3(PLAN_THREADS), stream, ids, (int)nrows, (int)ne,
                         (int)share, plan);
}

// ---------------------------------------------------------------------------
// the weighted sum
// ---------------------------------------------------------------------------
// y[t] = sum over s of w[t][s] h[t k + s], in fp32 and in the order of s.  A
// thread owns V neighbouring outputs of one token and reads BATCH slots' values
// before it adds them.  Bound by memory: 2630 tokens, k = 6, od = 3584, bf16
// (132 MB) 22 us, 6 TB/s; from fp32 rows (245 MB) 36 us, 6.8 TB/s.
template <int TH, int TY>
__global__ __launch_bounds__(256) void combine_kernel(const elem_t<TH> *__restrict__ h, int64_t ldh,
                                                      const float *__restrict__ w, int k, int64_t od, int64_t per,
                                                      int64_t total, elem_t<TY> *__restrict__ y, int64_t ldy)
{
    constexpr int V = VEC<TH>, BATCH = 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t t = i / per, j = (i - t * per) * V;
    const elem_t<TH> *row = h + t * k * ldh + j;
    const float *wt = w + t * k;
    elem_t<TY> *out = y + t * ldy + j;
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.0f;
    if (j + V <= od) {
        int s = 0;
        for (; s + BATCH <= k; s += BATCH) {
            u32x4 r[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) r[b] = load16<TH>(row + (s + b) * ldh);
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                float f[V];
                unpack16<TH>(r[b], f);
                const float g = wt[s + b];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] += g * f[e];
            }
        }
        for (; s < k; ++s) {
            float f[V];
            unpack16<TH>(load16<TH>(row + s * ldh), f);
            const float g = wt[s];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] += g * f[e];
        }
        if constexpr (VEC<TY> <= V) {
#pragma unroll
            for (int p = 0; p < V / VEC<TY>; ++p) {
                float o[VEC<TY>];
#pragma unroll
                for (int e = 0; e < VEC<TY>; ++e) o[e] = v[p * VEC<TY> + e];
                store16<TY>(out + p * VEC<TY>, pack16<TY>(o));
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) out[e] = (elem_t<TY>)v[e];
        }
    } else {
        for (int e = 0; j + e < od; ++e) {
            float a = 0.0f;
            for (int s = 0; s < k; ++s) a += wt[s] * (float)row[s * ldh + e];
            out[e] = (elem_t<TY>)a;
        }
    }
}

template <int TH, int TY>
static int combine(const void *h, int64_t ldh, const float *w, int64_t nt, int64_t k, int64_t od, void *y,
                   int64_t ldy, hipStream_t stream)
{
    const int64_t per = (od + VEC<TH> - 1) / VEC<TH>, most = launch_groups(256) * 256 / per;
    if (most == 0) return -1;
    return in_launches(nt, most, [&](int64_t r, int64_t n) {
        return launch_kernel(combine_kernel<TH, TY>, dim3((unsigned)((n * per + 255) / 256)), dim3(256), stream,
                             static_cast<const elem_t<TH> *>(h) + r * k * ldh, ldh, w + r * k, (int)k, od, per,
                             n * per, static_cast<elem_t<TY> *>(y) + r * ldy, ldy);
    });
}

template <int TH>
static int combine_to(const void *h, int64_t ldh, const float *w, int64_t nt, int64_t k, int64_t od, void *y,
                      int ytype, int64_t ldy, hipStream_t stream)
{
    switch (ytype) {
    case T_F32: return combine<TH, T_F32>(h, ldh, w, nt, k, od, y, ldy, stream);
    case T_BF16: return combine<TH, T_BF16>(h, ldh, w, nt, k, od, y, ldy, stream);
    default: return combine<TH, T_F16>(h, ldh, w, nt, k, od, y, ldy, stream);
    }
}

int launch_combine(const void *h, int htype, int64_t ldh, const float *w, int64_t nt, int64_t k, int64_t od,
                   void *y, int ytype, int64_t ldy, hipStream_t stream)
{
    switch (htype) {
    case T_F32: return combine_to<T_F32>(h, ldh, w, nt, k, od, y, ytype, ldy, stream);
    case T_BF16: return combine_to<T_BF16>(h, ldh, w, nt, k, od, y, ytype, ldy, stream);
    default: return combine_to<T_F16>(h, ldh, w, nt, k, od, y, ytype, ldy, stream);
    }
}

}  // namespace qig
