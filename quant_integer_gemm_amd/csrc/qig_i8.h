// qig_i8.h -- internal launchers of the int8 linear layer and the experts'
// operators behind the C ABI (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qig {

// Element types of the ABI (QIG_F32, QIG_BF16, QIG_F16).
enum { T_F32 = 0, T_BF16 = 1, T_F16 = 2 };

// An int32 sum of id products of int8 values (at most 128 * 128 each) must
// stay below 2^31.
constexpr int64_t I8_MAX_ID = 131071;
// The GEMM addresses the rows of one tile (at most 256) with 32-bit offsets.
constexpr int64_t I8_MAX_LD = (int64_t(1) << 31) / 256 - 256;
constexpr int64_t EXPERTS_MAX = 512;
constexpr int64_t ROUTE_MAX_K = 32;

struct I8Gemm {
    const int8_t *W;       // [od or 2 od][ldw], per expert
    const float *sw;       // [od or 2 od], per expert
    const int8_t *q;       // [rows of x][ldq]
    const float *sq;       // [rows of x]
    const float *bias;     // as sw, or nullptr
    void *y;               // [nt][ldy] of type ytype
    int64_t ldw, ldq, ldy, od, id, nt;
    int glu, ytype;
    // experts: nt flat rows in the plan's order, x row = flat row / slots
    const int32_t *plan = nullptr;
    int64_t ne = 0, slots = 1;
    void *ws = nullptr;
};

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *w;
    int64_t nt, ldl;
    int ltype, ne, score, groups, topk_groups, group_top, k, renorm;
    float scale;
    // set by launch_route: experts of a group, 2^20 over that (rounded up), and
    // log2 of the lanes that share a group
    uint32_t size = 0, by_size = 0;
    int lane_bits = 0;
};

// Plan: int32 words.  [0 .. ne] first position of each expert's rows in the
// order, [ne] being the number of kept rows; [ne + 1] all rows; then the
// order itself: flat rows sorted by expert, dropped rows last.
constexpr int64_t plan_words(int64_t nrows, int64_t ne) { return ne + 2 + nrows; }

// All return 0, -1 (grid too large) or -3 (launch error).
int launch_quantize_i8(const void *x, int xtype, int64_t nt, int64_t id, int64_t ldx, int8_t *q, int64_t ldq,
                       float *s, hipStream_t stream);
int launch_i8_gemm(const I8Gemm &g, hipStream_t stream);
// The kernel that launch_i8_gemm takes (ne > 0: experts), as mm_i8_form codes it.
int i8_form(const I8Gemm &g);
int launch_route(const RouteArgs &a, hipStream_t stream);
int launch_plan(const int32_t *ids, int64_t nrows, int64_t ne, int32_t *plan, hipStream_t stream);
int launch_combine(const void *h, int htype, int64_t ldh, const float *w, int64_t nt, int64_t k, int64_t od,
                   void *y, int ytype, int64_t ldy, hipStream_t stream);

}  // namespace qig
