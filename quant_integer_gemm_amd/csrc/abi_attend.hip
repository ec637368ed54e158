// abi_attend.hip -- the C ABI of the attention operators, the 4-bit cache and its
// pages: argument checks, then the launches on the caller's stream.  The full
// contract is in include/qig.h.
#include <math.h>
#include <string.h>
#include <qig.h>

#include "qig_attend.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int rc_from_launch(int r) { return r == 0 ? QIG_OK : (r == -1 ? QIG_EINVAL : QIG_ELAUNCH); }

bool bad_type(int t) { return t != QIG_F32 && t != QIG_BF16 && t != QIG_F16; }

uintptr_t elem_bytes(int t) { return t == QIG_F32 ? 4 : 2; }

constexpr int64_t INT_LIM = int64_t(1) << 31;
constexpr int64_t MAX_HEADS = 1024;

bool bad_strides(int64_t token, int64_t head) { return token < 0 || head < 0; }

// c = scale * log2(e); 0 asks for 1 / sqrt(d).
bool exponent(float scale, int64_t d, float &c)
{
    if (!(scale >= 0.0f) || scale > 1e30f) return false;
    c = (float)((scale == 0.0f ? 1.0 / sqrt((double)d) : (double)scale) * 1.4426950408889634);
    return c > 0.0f;
}

bool bad_heads(int64_t hq, int64_t hkv) { return hkv < 1 || hkv > MAX_HEADS || hq < 1 || hq > MAX_HEADS || hq % hkv != 0; }

bool cache_dim(int64_t d) { return d == 64 || d == 128 || d == 256; }

// The cache's own arguments; tokens: whether the call has work.
int check_cache(const void *pages, int64_t npages, int64_t page_stride, int64_t hkv, int64_t d, int64_t page,
                const int32_t *tables, int64_t ld, int64_t width, const int32_t *lengths, const int32_t *starts,
                int64_t nseq, int64_t nt)
{
    if (!cache_dim(d) || hkv < 1 || hkv > MAX_HEADS || npages < 0 || npages >= INT_LIM) return QIG_EINVAL;
    if (page < 32 || page > 65536 || page % 32 != 0) return QIG_EINVAL;
    if (nseq < 0 || nseq >= INT_LIM - 1 || nt < 0 || nt >= INT_LIM || width < 0 || width >= INT_LIM || ld < width)
        return QIG_EINVAL;
    if (!starts && nt != nseq) return QIG_EINVAL;
    if (npages > 1 && page_stride < hkv * (page / 32) * 40 * d) return QIG_EINVAL;
    if (page_stride % 16 != 0) return QIG_EALIGN;
    if (nt == 0 || nseq == 0) return QIG_OK;
    if ((!pages && npages > 0) || (!tables && width > 0) || !lengths) return QIG_EINVAL;
    if (!aligned(pages, 16) || !aligned(tables, 4) || !aligned(lengths, 4) || !aligned(starts, 4)) return QIG_EALIGN;
    return QIG_OK;
}

qig::Kv4 cache_of(const void *pages, int64_t npages, int64_t page_stride, int64_t hkv, int64_t d, int64_t page,
                  const int32_t *tables, int64_t ld, int64_t width, const int32_t *lengths, const int32_t *starts,
                  int64_t nseq)
{
    return {static_cast<uint8_t *>(const_cast<void *>(pages)), page_stride, tables, lengths, starts, npages, nseq,
            width, ld, (int)page, (int)hkv, (int)d};
}

int check_pool(const int32_t *tables, int64_t rows, int64_t ld, int64_t width, const int32_t *refs, int64_t npages)
{
    if (rows < 0 || width < 0 || ld < width || npages < 1 || npages > qig::POOL_MAX) return QIG_EINVAL;
    if (rows >= INT_LIM || width >= INT_LIM || (width > 0 && rows >= INT_LIM / width)) return QIG_EINVAL;
    if ((!tables && rows > 0 && width > 0) || !refs) return QIG_EINVAL;
    if (!aligned(tables, 4) || !aligned(refs, 4)) return QIG_EALIGN;
    return QIG_OK;
}

int check_pages(const void *pages, int64_t npages, int64_t page_bytes, int64_t page_stride)
{
    if (npages < 0 || npages >= INT_LIM || page_bytes < 1 || (npages > 1 && page_stride < page_bytes)) return QIG_EINVAL;
    if (page_bytes % 16 != 0 || page_stride % 16 != 0) return QIG_EALIGN;
    if (!pages && npages > 0) return QIG_EINVAL;
    return aligned(pages, 16) ? QIG_OK : QIG_EALIGN;
}

}  // namespace

extern "C" {

int attend_prompt(const void *q, int64_t q_token, int64_t q_head, const void *k, int64_t k_token, int64_t k_head,
                  const void *v, int64_t v_token, int64_t v_head, int type, int64_t nt, int64_t nk, int64_t hq,
                  int64_t hkv, int64_t d, const int32_t *starts, const int32_t *k_starts, int64_t nseq, int causal,
                  float scale, void *y, int64_t y_token, int64_t y_head, int ytype, hipStream_t stream)
{
    float c;
    if (bad_type(type) || bad_type(ytype) || bad_heads(hq, hkv) || d < 8 || d > 256 || d % 8 != 0) return QIG_EINVAL;
    // the kernels count keys in ints, up to 256 at a step and one step ahead
    if (nt < 0 || nt >= INT_LIM || nk < 0 || nk > INT_LIM - 1024 || nseq < 0 || nseq >= INT_LIM - 1) return QIG_EINVAL;
    if ((causal != 0 && causal != 1) || !exponent(scale, d, c)) return QIG_EINVAL;
    if (bad_strides(q_token, q_head) || bad_strides(k_token, k_head) || bad_strides(v_token, v_head) ||
        bad_strides(y_token, y_head))
        return QIG_EINVAL;
    if (nt == 0 || nseq == 0) return QIG_OK;
    if (!q || (nk > 0 && (!k || !v)) || !starts || !k_starts || !y) return QIG_EINVAL;
    const uintptr_t e = elem_bytes(type);
    if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(y, elem_bytes(ytype)) || !aligned(starts, 4) ||
        !aligned(k_starts, 4))
        return QIG_EALIGN;
    const qig::PromptArgs a = {{q, q_token, q_head}, {k, k_token, k_head}, {v, v_token, v_head}, y, y_token, y_head,
                               nt, nk, nseq, starts, k_starts, type, ytype, (int)hq, (int)hkv, (int)d, causal, c};
    return rc_from_launch(qig::launch_attend_prompt(a, stream));
}

size_t kv4_page_bytes(int64_t page, int64_t hkv, int64_t d)
{
    if (!cache_dim(d) || hkv < 1 || hkv > MAX_HEADS || page < 32 || page > 65536 || page % 32 != 0) return 0;
    return (size_t)(hkv * (page / 32) * 40 * d);
}

int write_kv4(const void *k, int64_t k_token, int64_t k_head, const void *v, int64_t v_token, int64_t v_head, int type,
              int64_t nt, int64_t hkv, int64_t d, void *pages, int64_t npages, int64_t page_stride, int64_t page,
              const int32_t *tables, int64_t ld, int64_t width, const int32_t *lengths, const int32_t *starts,
              int64_t nseq, hipStream_t stream)
{
    const int rc = check_cache(pages, npages, page_stride, hkv, d, page, tables, ld, width, lengths, starts, nseq, nt);
    if (rc != QIG_OK) return rc;
    if (bad_type(type) || bad_strides(k_token, k_head) || bad_strides(v_token, v_head)) return QIG_EINVAL;
    if (nt == 0 || nseq == 0) return QIG_OK;
    if (!k || !v) return QIG_EINVAL;
    if (!aligned(k, elem_bytes(type)) || !aligned(v, elem_bytes(type))) return QIG_EALIGN;
    const qig::Kv4Rows r = {{k, k_token, k_head}, {v, v_token, v_head}, nt, type};
    return rc_from_launch(qig::launch_write_kv4(
        cache_of(pages, npages, page_stride, hkv, d, page, tables, ld, width, lengths, starts, nseq), r, stream));
}

int read_kv4(void *k, int64_t k_token, int64_t k_head, void *v, int64_t v_token, int64_t v_head, int type, int64_t nt,
             int64_t hkv, int64_t d, const void *pages, int64_t npages, int64_t page_stride, int64_t page,
             const int32_t *tables, int64_t ld, int64_t width, const int32_t *lengths, const int32_t *starts,
             int64_t nseq, hipStream_t stream)
{
    const int rc = check_cache(pages, npages, page_stride, hkv, d, page, tables, ld, width, lengths, starts, nseq, nt);
    if (rc != QIG_OK) return rc;
    if (bad_type(type) || bad_strides(k_token, k_head) || bad_strides(v_token, v_head)) return QIG_EINVAL;
    if (nt == 0 || nseq == 0) return QIG_OK;
    if (!k || !v) return QIG_EINVAL;
    if (!aligned(k, elem_bytes(type)) || !aligned(v, elem_bytes(type))) return QIG_EALIGN;
    const qig::Kv4Rows r = {{k, k_token, k_head}, {v, v_token, v_head}, nt, type};
    return rc_from_launch(qig::launch_read_kv4(
        cache_of(pages, npages, page_stride, hkv, d, page, tables, ld, width, lengths, starts, nseq), r, stream));
}

int attend_kv4(const void *q, int64_t q_token, int64_t q_head, int type, int64_t nt, int64_t hq, int64_t hkv, int64_t d,
               const void *pages, int64_t npages, int64_t page_stride, int64_t page, const int32_t *tables, int64_t ld,
               int64_t width, const int32_t *lengths, const int32_t *starts, int64_t nseq, float scale, void *y,
               int64_t y_token, int64_t y_head, int ytype, void *ws, hipStream_t stream)
{
    float c;
    const int rc = check_cache(pages, npages, page_stride, hkv, d, page, tables, ld, width, lengths, starts, nseq, nt);
    if (rc != QIG_OK) return rc;
    if (bad_type(type) || bad_type(ytype) || bad_heads(hq, hkv) || !exponent(scale, d, c)) return QIG_EINVAL;
    if (bad_strides(q_token, q_head) || bad_strides(y_token, y_head)) return QIG_EINVAL;
    if (nt == 0 || nseq == 0) return QIG_OK;
    if (!q || !y) return QIG_EINVAL;
    if (!aligned(q, elem_bytes(type)) || !aligned(y, elem_bytes(ytype)) || !aligned(ws, 16)) return QIG_EALIGN;
    const qig::Kv4Attend a = {{q, q_token, q_head}, y, y_token, y_head, nt, type, ytype, (int)hq, c, ws};
    return rc_from_launch(qig::launch_attend_kv4(
        cache_of(pages, npages, page_stride, hkv, d, page, tables, ld, width, lengths, starts, nseq), a, stream));
}

int copy_pages(void *pages, int64_t npages, int64_t page_bytes, int64_t page_stride, const int32_t *src,
               const int32_t *dst, int64_t n, hipStream_t stream)
{
    const int rc = check_pages(pages, npages, page_bytes, page_stride);
    if (rc != QIG_OK) return rc;
    if (n < 0 || n >= INT_LIM) return QIG_EINVAL;
    if (n == 0 || npages == 0) return QIG_OK;
    if (!src || !dst) return QIG_EINVAL;
    if (!aligned(src, 4) || !aligned(dst, 4)) return QIG_EALIGN;
    return rc_from_launch(qig::launch_copy_pages(pages, npages, page_bytes, page_stride, src, dst, n, stream));
}

size_t pages_scratch_bytes(int64_t npages, int64_t rows)
{
    if (npages < 1 || npages > qig::POOL_MAX || rows < 0 || rows >= INT_LIM) return 0;
    return (size_t)qig::pool_scratch_bytes(npages, rows);
}

int free_pages(int32_t *tables, int64_t rows, int64_t ld, int64_t width, int32_t *lengths, int32_t *refs,
               int64_t npages, const int32_t *which, int64_t n, hipStream_t stream)
{
    const int rc = check_pool(tables, rows, ld, width, refs, npages);
    if (rc != QIG_OK) return rc;
    if (n < 0 || n >= INT_LIM) return QIG_EINVAL;
    if (n == 0 || rows == 0) return QIG_OK;
    if (!lengths || !which) return QIG_EINVAL;
    if (!aligned(lengths, 4) || !aligned(which, 4)) return QIG_EALIGN;
    const qig::Pool p = {tables, lengths, refs, rows, width, ld, npages, 0};
    return rc_from_launch(qig::launch_free_pages(p, which, n, stream));
}

int take_pages(int32_t *tables, int64_t rows, int64_t ld, int64_t width, const int32_t *lengths, int32_t *refs,
               int64_t npages, int64_t page, int32_t *missing, void *scratch, hipStream_t stream)
{
    const int rc = check_pool(tables, rows, ld, width, refs, npages);
    if (rc != QIG_OK) return rc;
    if (page < 1 || page >= INT_LIM || !missing || !scratch || (!lengths && rows > 0)) return QIG_EINVAL;
    if (!aligned(lengths, 4) || !aligned(missing, 4) || !aligned(scratch, 8)) return QIG_EALIGN;
    const qig::Pool p = {tables, const_cast<int32_t *>(lengths), refs, rows, width, ld, npages, (int)page};
    return rc_from_launch(qig::launch_take_pages(p, missing, scratch, stream));
}

int fork_pages(void *pages, int64_t page_bytes, int64_t page_stride, int32_t *tables, int64_t rows, int64_t ld,
               int64_t width, int32_t *lengths, int32_t *refs, int64_t npages, int64_t page, const int32_t *parents,
               const int32_t *children, int64_t n, int32_t *missing, void *scratch, hipStream_t stream)
{
    int rc = check_pool(tables, rows, ld, width, refs, npages);
    if (rc != QIG_OK) return rc;
    rc = check_pages(pages, npages, page_bytes, page_stride);
    if (rc != QIG_OK) return rc;
    if (page < 1 || page >= INT_LIM || n < 0 || n >= INT_LIM || !missing || !scratch || (!lengths && rows > 0) ||
        (n > 0 && (!parents || !children)))
        return QIG_EINVAL;
    if (!aligned(lengths, 4) || !aligned(parents, 4) || !aligned(children, 4) || !aligned(missing, 4) ||
        !aligned(scratch, 8))
        return QIG_EALIGN;
    const qig::Pool p = {tables, lengths, refs, rows, width, ld, npages, (int)page};
    return rc_from_launch(qig::launch_fork_pages(p, pages, page_bytes, page_stride, parents, children, n, missing,
                                                 scratch, stream));
}

int compact_pages(void *pages, int64_t page_bytes, int64_t page_stride, int32_t *tables, int64_t rows, int64_t ld,
                  int64_t width, int32_t *refs, int64_t npages, int32_t *used, int32_t *to, void *scratch,
                  hipStream_t stream)
{
    int rc = check_pool(tables, rows, ld, width, refs, npages);
    if (rc != QIG_OK) return rc;
    rc = check_pages(pages, npages, page_bytes, page_stride);
    if (rc != QIG_OK) return rc;
    if (!used || !scratch) return QIG_EINVAL;
    if (!aligned(used, 4) || !aligned(to, 4) || !aligned(scratch, 8)) return QIG_EALIGN;
    const qig::Pool p = {tables, nullptr, refs, rows, width, ld, npages, 0};
    return rc_from_launch(qig::launch_compact_pages(p, pages, page_bytes, page_stride, used, to, scratch, stream));
}

int qig_attend_packed(int op, const void *words, hipStream_t stream)
{
    int64_t w[24];
    constexpr int COUNT[] = {24, 20, 20, 24, 7, 9, 10, 16, 12};
    if (op < 0 || op > 8 || !words) return QIG_EINVAL;
    memcpy(w, words, COUNT[op] * 8);
    const auto p = [&](int i) { return reinterpret_cast<void *>(w[i]); };
    const auto n = [&](int i) { return reinterpret_cast<int32_t *>(w[i]); };
    const auto small = [&](int i) { return w[i] < INT32_MIN || w[i] > INT32_MAX ? -1 : (int)w[i]; };
    const auto real = [&](int i) {
        double d;
        memcpy(&d, &w[i], 8);
        return d != 0.0 && (float)d == 0.0f ? -1.0f : (float)d;   // too small a scale does not ask for the default
    };
    switch (op) {
    case 0:
        return attend_prompt(p(0), w[1], w[2], p(3), w[4], w[5], p(6), w[7], w[8], small(9), w[10], w[11], w[12], w[13],
                             w[14], n(15), n(16), w[17], small(18), real(19), p(20), w[21], w[22], small(23), stream);
    case 1:
        return write_kv4(p(0), w[1], w[2], p(3), w[4], w[5], small(6), w[7], w[8], w[9], p(10), w[11], w[12], w[13], n(14),
                         w[15], w[16], n(17), n(18), w[19], stream);
    case 2:
        return read_kv4(p(0), w[1], w[2], p(3), w[4], w[5], small(6), w[7], w[8], w[9], p(10), w[11], w[12], w[13], n(14),
                        w[15], w[16], n(17), n(18), w[19], stream);
    case 3:
        return attend_kv4(p(0), w[1], w[2], small(3), w[4], w[5], w[6], w[7], p(8), w[9], w[10], w[11], n(12), w[13],
                          w[14], n(15), n(16), w[17], real(18), p(19), w[20], w[21], small(22), p(23), stream);
    case 4:
        return copy_pages(p(0), w[1], w[2], w[3], n(4), n(5), w[6], stream);
    case 5:
        return free_pages(n(0), w[1], w[2], w[3], n(4), n(5), w[6], n(7), w[8], stream);
    case 6:
        return take_pages(n(0), w[1], w[2], w[3], n(4), n(5), w[6], w[7], n(8), p(9), stream);
    case 7:
        return fork_pages(p(0), w[1], w[2], n(3), w[4], w[5], w[6], n(7), n(8), w[9], w[10], n(11), n(12), w[13], n(14),
                          p(15), stream);
    default:
        return compact_pages(p(0), w[1], w[2], n(3), w[4], w[5], w[6], n(7), w[8], n(9), n(10), p(11), stream);
    }
}

}  // extern "C"
