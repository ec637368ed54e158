// abi_i8.hip -- the C ABI of the int8 linear layer and the experts' operators:
// argument checks, then the launches on the caller's stream.  The full
// contract is in include/qig.h.
#include <qig.h>

#include "qig_i8.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int rc_from_launch(int r) { return r == 0 ? QIG_OK : (r == -1 ? QIG_EINVAL : QIG_ELAUNCH); }

bool bad_type(int t) { return t != QIG_F32 && t != QIG_BF16 && t != QIG_F16; }

uintptr_t elem_bytes(int t) { return t == QIG_F32 ? 4 : 2; }

constexpr int64_t INT_LIM = int64_t(1) << 31;

// rows: outputs' rows of W in the weights of one expert
int check_product(const int8_t *W, int64_t ldw, const float *sw, int64_t od, int64_t id, const int8_t *q, int64_t ldq,
                  const float *sq, int64_t nt, const float *bias, int glu, const void *y, int ytype, int64_t ldy)
{
    if (nt < 0 || od < 0 || id <= 0 || id > qig::I8_MAX_ID || bad_type(ytype)) return QIG_EINVAL;
    if (ldw < id || ldq < id || ldy < od || ldw > qig::I8_MAX_LD || ldq > qig::I8_MAX_LD) return QIG_EINVAL;
    if (nt >= INT_LIM || od >= INT_LIM / 2 || (glu != 0 && glu != 1)) return QIG_EINVAL;
    if (ldw % 16 != 0 || ldq % 16 != 0) return QIG_EALIGN;
    if (nt == 0 || od == 0) return QIG_OK;
    if (!W || !sw || !q || !sq || !y) return QIG_EINVAL;
    if (!aligned(W, 16) || !aligned(q, 16) || !aligned(sw, 4) || !aligned(sq, 4) || !aligned(bias, 4) ||
        !aligned(y, elem_bytes(ytype)))
        return QIG_EALIGN;
    return QIG_OK;
}

}  // namespace

extern "C" {

int quantize_i8(const void *x, int xtype, int64_t nt, int64_t id, int64_t ldx, int8_t *q, int64_t ldq, float *s,
                hipStream_t stream)
{
    if (bad_type(xtype) || nt < 0 || nt >= INT_LIM || id <= 0 || id >= INT_LIM || ldx < id || ldq < id)
        return QIG_EINVAL;
    if (nt == 0) return QIG_OK;
    if (!x || !q || !s) return QIG_EINVAL;
    if (!aligned(x, elem_bytes(xtype)) || !aligned(s, 4)) return QIG_EALIGN;
    return rc_from_launch(qig::launch_quantize_i8(x, xtype, nt, id, ldx, q, ldq, s, stream));
}

int mm_i8(const int8_t *W, int64_t ldw, const float *sw, int64_t od, int64_t id, const int8_t *q, int64_t ldq,
          const float *sq, int64_t nt, const float *bias, int glu, void *y, int ytype, int64_t ldy, void *ws,
          hipStream_t stream)
{
    int rc = check_product(W, ldw, sw, od, id, q, ldq, sq, nt, bias, glu, y, ytype, ldy);
    if (rc != QIG_OK || nt == 0 || od == 0) return rc;
    if (ws && !aligned(ws, 16)) return QIG_EALIGN;
    qig::I8Gemm g = {W, sw, q, sq, bias, y, ldw, ldq, ldy, od, id, nt, glu, ytype};
    g.ws = ws;
    return rc_from_launch(qig::launch_i8_gemm(g, stream));
}

int route_experts(const void *logits, int ltype, int64_t nt, int64_t ne, int64_t ldl, const float *bias, int score,
                  int64_t groups, int64_t topk_groups, int64_t group_top, int64_t k, int renorm, float scale,
                  int32_t *ids, float *w, hipStream_t stream)
{
    if (bad_type(ltype) || nt < 0 || nt >= INT_LIM || ne <= 0 || ne > qig::EXPERTS_MAX || ldl < ne) return QIG_EINVAL;
    if ((score != QIG_SOFTMAX && score != QIG_SIGMOID) || groups < 1 || groups > 64 || ne % groups != 0)
        return QIG_EINVAL;
    if (topk_groups < 1 || topk_groups > groups || (group_top != 1 && group_top != 2)) return QIG_EINVAL;
    if (k < 1 || k > qig::ROUTE_MAX_K || k > topk_groups * (ne / groups)) return QIG_EINVAL;
    if (nt == 0) return QIG_OK;
    if (!logits || !ids || !w) return QIG_EINVAL;
    if (!aligned(logits, elem_bytes(ltype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(w, 4))
        return QIG_EALIGN;
    qig::RouteArgs a = {logits, bias, ids, w, nt, ldl, ltype, (int)ne, score, (int)groups, (int)topk_groups,
                        (int)group_top, (int)k, renorm, scale};
    return rc_from_launch(qig::launch_route(a, stream));
}

size_t expert_plan_bytes(int64_t nrows, int64_t ne)
{
    if (nrows < 0 || nrows >= INT_LIM / 4 || ne <= 0 || ne > qig::EXPERTS_MAX) return 0;
    return (size_t)qig::plan_words(nrows, ne) * 4u;
}

int plan_experts(const int32_t *ids, int64_t nrows, int64_t ne, void *plan, hipStream_t stream)
{
    if (expert_plan_bytes(nrows, ne) == 0) return QIG_EINVAL;
    if (!plan || (!ids && nrows > 0)) return QIG_EINVAL;
    if (!aligned(ids, 4) || !aligned(plan, 4)) return QIG_EALIGN;
    return rc_from_launch(qig::launch_plan(ids, nrows, ne, static_cast<int32_t *>(plan), stream));
}

int mm_i8_experts(const int8_t *W, int64_t ldw, const float *sw, int64_t ne, int64_t od, int64_t id, const int8_t *q,
                  int64_t ldq, const float *sq, int64_t nrows, int64_t slots, const void *plan, const float *bias,
                  int glu, void *y, int ytype, int64_t ldy, hipStream_t stream)
{
    int rc = check_product(W, ldw, sw, od, id, q, ldq, sq, nrows, bias, glu, y, ytype, ldy);
    if (rc != QIG_OK) return rc;
    if (expert_plan_bytes(nrows, ne) == 0 || slots < 1 || slots >= INT_LIM || nrows % slots != 0) return QIG_EINVAL;
    if (nrows == 0 || od == 0) return QIG_OK;
    if (!plan) return QIG_EINVAL;
    if (!aligned(plan, 4)) return QIG_EALIGN;
    qig::I8Gemm g = {W, sw, q, sq, bias, y, ldw, ldq, ldy, od, id, nrows, glu, ytype};
    g.plan = static_cast<const int32_t *>(plan);
    g.ne = ne;
    g.slots = slots;
    return rc_from_launch(qig::launch_i8_gemm(g, stream));
}

int combine_experts(const void *h, int htype, int64_t ldh, const float *w, int64_t nt, int64_t k, int64_t od, void *y,
                    int ytype, int64_t ldy, hipStream_t stream)
{
    if (bad_type(htype) || bad_type(ytype) || nt < 0 || od < 0 || k < 1 || k >= INT_LIM || ldh < od || ldy < od ||
        nt >= INT_LIM / k)
        return QIG_EINVAL;
    if (nt == 0 || od == 0) return QIG_OK;
    if (!h || !w || !y) return QIG_EINVAL;
    if (!aligned(h, elem_bytes(htype)) || !aligned(w, 4) || !aligned(y, elem_bytes(ytype))) return QIG_EALIGN;
    return rc_from_launch(qig::launch_combine(h, htype, ldh, w, nt, k, od, y, ytype, ldy, stream));
}

int mm_i8_form(int64_t ne, int64_t od, int64_t id, int64_t nt, int glu, int ws)
{
    if (ne < 0 || ne > qig::EXPERTS_MAX || od < 1 || od >= INT_LIM / 2 || id < 1 || id > qig::I8_MAX_ID || nt < 1 ||
        nt >= INT_LIM || (glu != 0 && glu != 1))
        return QIG_EINVAL;
    qig::I8Gemm g = {nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, id, id, od, od, id, nt, glu, QIG_F32};
    g.ne = ne;
    int held = 0;
    g.ws = ws ? &held : nullptr;   // there or not: never read
    return qig::i8_form(g);
}

}  // extern "C"
