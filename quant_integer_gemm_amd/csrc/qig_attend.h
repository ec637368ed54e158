// qig_attend.h -- internal launchers of the attention operators, the 4-bit
// cache and its pages behind the C ABI (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qig {

// A tensor [tokens][heads][d] with unit stride in d; strides in elements.
struct Heads {
    const void *p;
    int64_t token, head;
};

struct PromptArgs {
    Heads q, k, v;
    void *y;
    int64_t y_token, y_head;
    int64_t nt, nk, nseq;
    const int32_t *starts, *k_starts;   // [nseq + 1]
    int type, ytype, hq, hkv, d, causal;
    float c;                            // scale * log2(e): probabilities are powers of two
};

// The 4-bit cache.  A block is 32 tokens of one head, 10 d words:
//   keys' codes 4 d, values' codes 4 d, keys' scales d, values' scales d.
struct Kv4 {
    uint8_t *pages;          // [npages][heads][page / 32][40 d]
    int64_t page_bytes;      // from page to page
    const int32_t *tables;   // [nseq][ld], -1 (or anything outside [0, npages)): no page
    const int32_t *lengths;  // [nseq]
    const int32_t *starts;   // [nseq + 1] packed tokens, or nullptr: token s is sequence s's only one
    int64_t npages, nseq, width, ld;
    int page, heads, d;
};

struct Kv4Rows {
    Heads k, v;              // read for writing, written for reading
    int64_t nt;
    int type;
};

struct Kv4Attend {
    Heads q;
    void *y;
    int64_t y_token, y_head, nt;
    int type, ytype, hq;
    float c;
    void *ws;                // or nullptr
};

// Bytes of the workspace (the stream-K one) that may hold partial results; 4096 arrival
// counters of 32 bits, all zero between calls, follow them.
constexpr int64_t ATTEND_WS_BYTES = int64_t(1024) * 2 * 64 * 64 * 4;

struct Pool {
    int32_t *tables, *lengths, *refs;
    int64_t rows, width, ld, npages;
    int page;
};

// Scratch of the calls that look for free pages: a bit a page, then a count a row.
constexpr int64_t POOL_MAX = int64_t(1) << 20;
constexpr int64_t pool_scratch_bytes(int64_t npages, int64_t rows) { return (npages + 63) / 64 * 8 + rows * 4; }

// All return 0, -1 (grid too large) or -3 (launch error).
int launch_attend_prompt(const PromptArgs &a, hipStream_t stream);
int launch_write_kv4(const Kv4 &c, const Kv4Rows &r, hipStream_t stream);
int launch_read_kv4(const Kv4 &c, const Kv4Rows &r, hipStream_t stream);
int launch_attend_kv4(const Kv4 &c, const Kv4Attend &a, hipStream_t stream);
int launch_copy_pages(void *pages, int64_t npages, int64_t bytes, int64_t stride, const int32_t *src,
                      const int32_t *dst, int64_t n, hipStream_t stream);
int launch_free_pages(const Pool &p, const int32_t *which, int64_t n, hipStream_t stream);
int launch_take_pages(const Pool &p, int32_t *missing, void *scratch, hipStream_t stream);
int launch_fork_pages(const Pool &p, void *pages, int64_t bytes, int64_t stride, const int32_t *parents,
                      const int32_t *children, int64_t n, int32_t *missing, void *scratch, hipStream_t stream);
int launch_compact_pages(const Pool &p, void *pages, int64_t bytes, int64_t stride, int32_t *used, int32_t *to,
                         void *scratch, hipStream_t stream);

}  // namespace qig
