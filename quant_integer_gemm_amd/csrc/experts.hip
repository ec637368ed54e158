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
// the sum of its group_top largest c), equal values to the lower index.  The
// scores are formed and compared in 64 bits: which expert wins is a
// comparison of near values, and in 32 bits the rounding of exp would decide
// about one row in ten thousand.  Softmax without a bias keeps the order of
// the logits, so there the choice compares the logits themselves (also where
// the scores underflow).  A logit of -infinity or NaN is an expert that may
// not be chosen; +infinity counts as the largest finite number.

// One wave a token, lane l holding experts l, l + 64, ...
template <int NS, int T>
__global__ __launch_bounds__(64) void route_kernel(RouteArgs a)
{
    __shared__ double s_c[NS * 64];
    __shared__ double s_g[64];
    __shared__ uint8_t s_keep[64];
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    const elem_t<T> *l = static_cast<const elem_t<T> *>(a.logits) + t * a.ldl;
    double v[NS], p[NS], c[NS];
    bool ok[NS];
    double top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int e = lane + 64 * i;
        float x = e < a.ne ? (float)l[e] : -INFINITY;
        ok[i] = x > -INFINITY;   // false for NaN
        x = ok[i] ? __builtin_fminf(x, 3.402823466e38f) : 0.0f;
        v[i] = (double)x;
        if (ok[i]) top = fmax(top, v[i]);
    }
    if (a.score == 0) {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmax(top, __shfl_xor(top, d));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            p[i] = ok[i] ? exp(v[i] - top) : 0.0;
            sum += p[i];
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
        const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int i = 0; i < NS; ++i) p[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) p[i] = ok[i] ? 1.0 / (1.0 + exp(-v[i])) : 0.0;
    }
    const bool by_logit = a.score == 0 && !a.bias && (a.groups == 1 || a.group_top == 1);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int e = lane + 64 * i;
        c[i] = by_logit ? v[i] : p[i] + (a.bias && e < a.ne ? (double)a.bias[e] : 0.0);
        if (!ok[i] || !(c[i] > -INFINITY)) {
            ok[i] = false;
            c[i] = -INFINITY;
        }
    }
    if (a.groups > 1) {
        const int size = a.ne / a.groups;
#pragma unroll
        for (int i = 0; i < NS; ++i) s_c[lane + 64 * i] = c[i];
        __syncthreads();
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
        __syncthreads();
        if (lane < a.groups) {
            int better = 0;
            for (int o = 0; o < a.groups; ++o)
                better += s_g[o] > s_g[lane] || (s_g[o] == s_g[lane] && o < lane);
            s_keep[lane] = better < a.topk_groups;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int e = lane + 64 * i;
            if (e < a.ne && !s_keep[e / size]) ok[i] = false;
        }
    }
    // k rounds of the largest remaining (value, then lowest index)
    double wsum = 0.0, mine = 0.0;
    int my_id = -1;
    for (int r = 0; r < a.k; ++r) {
        double best = -INFINITY, bp = 0.0;
        int be = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (ok[i] && c[i] > best) {
                best = c[i];
                be = lane + 64 * i;
                bp = p[i];
            }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const double ob = __shfl_xor(best, d), op = __shfl_xor(bp, d);
            const int oe = __shfl_xor(be, d);
            if (ob > best || (ob == best && oe < be)) {
                best = ob;
                be = oe;
                bp = op;
            }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (lane + 64 * i == be) ok[i] = false;
        const bool found = be != 0x7fffffff;
        if (lane == r) {
            my_id = found ? be : -1;
            mine = found ? bp : 0.0;
        }
        wsum += found ? bp : 0.0;
    }
    if (lane < a.k) {
        const double scale = a.renorm ? (wsum > 0.0 ? (double)a.scale / wsum : 0.0) : (double)a.scale;
        a.ids[t * a.k + lane] = my_id;
        a.w[t * a.k + lane] = (float)(mine * scale);
    }
}

template <int T>
static int route_typed(const RouteArgs &a, hipStream_t stream)
{
    const dim3 grid((unsigned)a.nt), block(64);
    if (a.ne <= 64) return launch_kernel(route_kernel<1, T>, grid, block, stream, a);
    if (a.ne <= 128) return launch_kernel(route_kernel<2, T>, grid, block, stream, a);
    if (a.ne <= 256) return launch_kernel(route_kernel<4, T>, grid, block, stream, a);
    return launch_kernel(route_kernel<8, T>, grid, block, stream, a);
}

int launch_route(const RouteArgs &a, hipStream_t stream)
{
    if (a.nt > 0x7fffffff) return -1;
    switch (a.ltype) {
    case T_F32: return route_typed<T_F32>(a, stream);
    case T_BF16: return route_typed<T_BF16>(a, stream);
    default: return route_typed<T_F16>(a, stream);
    }
}

// ---------------------------------------------------------------------------
// the order of rows by expert
// ---------------------------------------------------------------------------
// A stable counting sort by one workgroup: every wave counts a contiguous
// share of the rows per expert, the counts become first positions (expert
// major, wave minor), and every wave places its rows in order.  Ids outside
// [0, ne) count as expert ne (dropped rows).
constexpr int PLAN_WAVES = 16;

__global__ __launch_bounds__(PLAN_WAVES * 64) void plan_kernel(const int32_t *__restrict__ ids, int nrows, int ne,
                                                               int32_t *__restrict__ plan)
{
    extern __shared__ int32_t hist[];   // [ne + 1][PLAN_WAVES]
    __shared__ int32_t part[PLAN_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = (ne + 1) * PLAN_WAVES;
    for (int i = tid; i < n; i += PLAN_WAVES * 64) hist[i] = 0;
    __syncthreads();
    const int per = (nrows + PLAN_WAVES * 64 - 1) / (PLAN_WAVES * 64) * 64;
    const int lo = wave * per, hi = lo + per < nrows ? lo + per : nrows;
    for (int i = lo + lane; i < hi; i += 64) {
        const int e = ids[i];
        atomicAdd(&hist[((unsigned)e < (unsigned)ne ? e : ne) * PLAN_WAVES + wave], 1);
    }
    __syncthreads();
    // exclusive scan of hist in its order
    const int chunk = (n + PLAN_WAVES * 64 - 1) / (PLAN_WAVES * 64);
    const int a = tid * chunk, b = a + chunk < n ? a + chunk : n;
    int sum = 0;
    for (int i = a; i < b; ++i) sum += hist[i];
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < wave; ++w) at += part[w];
    for (int i = a; i < b; ++i) {
        const int c = hist[i];
        hist[i] = at;
        at += c;
    }
    __syncthreads();
    for (int e = tid; e <= ne; e += PLAN_WAVES * 64) plan[e] = hist[e * PLAN_WAVES];
    if (tid == 0) plan[ne + 1] = nrows;
    __syncthreads();
    int32_t *order = plan + ne + 2;
    for (int i0 = lo; i0 < hi; i0 += 64) {
        const int i = i0 + lane;
        const bool live = i < hi;
        int e = live ? ids[i] : ne;
        e = (unsigned)e < (unsigned)ne ? e : ne;
        // lanes with the same expert, by its bits
        uint64_t same = __ballot(live);
        for (int bit = 0; (1 << bit) <= ne; ++bit) {
            const uint64_t set = __ballot((e >> bit) & 1);
            same &= ((e >> bit) & 1) ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int base = 0;
        if (live) base = hist[e * PLAN_WAVES + wave];
        if (live) order[base + rank] = i;
        if (live && rank == 0) hist[e * PLAN_WAVES + wave] = base + __popcll(same);
    }
}

int launch_plan(const int32_t *ids, int64_t nrows, int64_t ne, int32_t *plan, hipStream_t stream)
{
    int n = (int)nrows, e = (int)ne;
    void *args[] = {&ids, &n, &e, &plan};
    const hipError_t r = hipLaunchKernel(reinterpret_cast<const void *>(plan_kernel), dim3(1), dim3(PLAN_WAVES * 64),
                                         args, (size_t)(ne + 1) * PLAN_WAVES * 4, stream);
    return r == hipSuccess ? 0 : -3;
}

// ---------------------------------------------------------------------------
// the weighted sum
// ---------------------------------------------------------------------------
// y[t] = sum over s of w[t][s] h[t k + s], in fp32 and in the order of s.
template <int TH, int TY>
__global__ __launch_bounds__(256) void combine_kernel(const elem_t<TH> *__restrict__ h, int64_t ldh,
                                                      const float *__restrict__ w, int k, int64_t od,
                                                      elem_t<TY> *__restrict__ y, int64_t ldy)
{
    const int64_t t = blockIdx.x;
    for (int64_t j = threadIdx.x; j < od; j += 256) {
        float v = 0.0f;
        for (int s = 0; s < k; ++s) v += w[t * k + s] * (float)h[(t * k + s) * ldh + j];
        y[t * ldy + j] = (elem_t<TY>)v;
    }
}

template <int TH, int TY>
static int combine(const void *h, int64_t ldh, const float *w, int64_t nt, int64_t k, int64_t od, void *y,
                   int64_t ldy, hipStream_t stream)
{
    return launch_kernel(combine_kernel<TH, TY>, dim3((unsigned)nt), dim3(256), stream,
                         static_cast<const elem_t<TH> *>(h), ldh, w, (int)k, od, static_cast<elem_t<TY> *>(y), ldy);
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
    if (nt > 0x7fffffff) return -1;
    switch (htype) {
    case T_F32: return combine_to<T_F32>(h, ldh, w, nt, k, od, y, ytype, ldy, stream);
    case T_BF16: return combine_to<T_BF16>(h, ldh, w, nt, k, od, y, ytype, ldy, stream);
    default: return combine_to<T_F16>(h, ldh, w, nt, k, od, y, ytype, ldy, stream);
    }
}

}  // namespace qig
