// pages.hip -- the pages of a cache: copied, taken for sequences that grow, given
// up, shared by forked sequences, and packed to the front of the pool.
//
// refs[p] counts the rows of the table that hold page p; a page is free where it is
// 0.  Free pages go lowest first to those that need one, in their order, so that
// every call's result is one and the same however its workgroups run.  A call that
// gives pages has two launches: the first notes a bit for each page and what each
// row needs; the second's workgroups each sum those notes (a bit a page, 2 KB for
// 16384 pages) and so know their own rows' pages with no wait for one another.  The
// notes stay as they are meanwhile: refs and tables change in the second launch
// alone.
//
// Measured: every launch 2-5 us where few pages move, latency alone; 16384 pages of 40 KB,
// of which 4100 move to the front, 65 us (336 MB read and written, 5.2 TB/s, as a large
// copy).  One launch that waits for its own notes would need all workgroups resident.
#include "qig_attend_device.h"
#include "qig_launch.h"

namespace qig {
namespace {

constexpr int CHUNK = 16384;   // bytes of a page that one workgroup of 256 copies

__device__ __forceinline__ bool valid(int p, int64_t n) { return p >= 0 && p < n; }

// 16-byte units [first, first + 1024) of a page.
__device__ __forceinline__ void copy_chunk(const char *src, char *dst, int64_t bytes, int64_t chunk)
{
    const int64_t at = chunk * CHUNK + threadIdx.x * 16;
    u32x4 v[CHUNK / 4096];
#pragma unroll
    for (int i = 0; i < CHUNK / 4096; ++i)
        if (at + i * 4096 < bytes) v[i] = *reinterpret_cast<const u32x4 *>(src + at + i * 4096);
#pragma unroll
    for (int i = 0; i < CHUNK / 4096; ++i)
        if (at + i * 4096 < bytes) *reinterpret_cast<u32x4 *>(dst + at + i * 4096) = v[i];
}

__global__ __launch_bounds__(256) void copy_kernel(char *pages, int64_t npages, int64_t bytes, int64_t stride,
                                                   const int32_t *src, const int32_t *dst, int64_t first, int chunks)
{
    const int64_t i = first + blockIdx.x / chunks;
    const int s = src[i], d = dst[i];
    if (!valid(s, npages) || !valid(d, npages) || s == d) return;
    copy_chunk(pages + s * stride, pages + d * stride, bytes, blockIdx.x % chunks);
}

// --- notes ---------------------------------------------------------------------------------------------------------

// 64 pages a wave: bit p of word p / 64 is set where refs[p] > 0.
__device__ __forceinline__ void note_pages(const int32_t *refs, int64_t npages, uint64_t *notes, int64_t wave)
{
    const int lane = threadIdx.x & 63;
    const int64_t p = wave * 64 + lane;
    if (wave * 64 >= npages) return;
    const uint64_t live = __ballot(p < npages && refs[p] > 0);
    if (lane == 0) notes[wave] = live;
}

__device__ __forceinline__ int64_t words_of(int64_t npages) { return (npages + 63) / 64; }

// Whether page p of word w is wanted: the free ones (FREE), or those in use.
template <bool FREE>
__device__ __forceinline__ uint64_t wanted(const uint64_t *notes, int64_t w, int64_t npages)
{
    const uint64_t live = notes[w];
    if (!FREE) return live;
    const int64_t left = npages - w * 64;
    return ~live & (left >= 64 ? ~uint64_t(0) : (uint64_t(1) << left) - 1);
}

// Sums of a workgroup of 256: the value before this thread's, and the total.
__device__ __forceinline__ int sum_before(int v, int *tmp, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(s, o);
        if (lane >= o) s += up;
    }
    __syncthreads();
    if (lane == 63) tmp[wave] = s;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wave; ++w) before += tmp[w];
    total = tmp[0] + tmp[1] + tmp[2] + tmp[3];
    return before + s - v;
}

// before[w]: wanted pages in the words ahead of w, for all words; returns their
// number.  All 256 threads; W: the most words.
template <bool FREE, int W>
__device__ __forceinline__ int sum_notes(const uint64_t *notes, int64_t npages, int *before, int *tmp)
{
    const int words = (int)words_of(npages);
    const int each = (words + 255) / 256, from = threadIdx.x * each;
    int mine = 0;
    for (int w = from; w < from + each && w < words; ++w) mine += __popcll(wanted<FREE>(notes, w, npages));
    int total;
    int at = sum_before(mine, tmp, total);
    for (int w = from; w < from + each && w < words; ++w) {
        before[w] = at;
        at += __popcll(wanted<FREE>(notes, w, npages));
    }
    __syncthreads();
    return total;
}

// The k-th wanted page (k below their number).
template <bool FREE>
__device__ __forceinline__ int page_at(const uint64_t *notes, int64_t npages, const int *before, int k)
{
    int lo = 0, hi = (int)words_of(npages) - 1;   // the last word with before[w] <= k
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= k) lo = mid; else hi = mid - 1;
    }
    uint64_t bits = wanted<FREE>(notes, lo, npages);
    int left = k - before[lo], at = 0;
#pragma unroll
    for (int half = 32; half > 0; half >>= 1) {
        const int low = __popcll(bits & ((uint64_t(1) << half) - 1));
        if (left >= low) {
            left -= low;
            bits >>= half;
            at += half;
        }
    }
    return lo * 64 + at;
}

// --- giving up ------------------------------------------------------------------------------------------------------

// A row gives up its pages.  The exchange makes a row that is named twice give them
// up once, and a count never falls below 0.
__device__ __forceinline__ void release_row(const Pool &p, int row)
{
    for (int64_t c = threadIdx.x; c < p.width; c += 256) {
        const int page = atomicExch(&p.tables[row * p.ld + c], -1);
        if (valid(page, p.npages) && atomicSub(&p.refs[page], 1) <= 0) atomicAdd(&p.refs[page], 1);
    }
    if (threadIdx.x == 0) p.lengths[row] = 0;
}

__global__ __launch_bounds__(256) void free_kernel(Pool p, const int32_t *which)
{
    const int row = which[blockIdx.x];
    if (valid(row, p.rows)) release_row(p, row);
}

// --- taking ---------------------------------------------------------------------------------------------------------

__device__ __forceinline__ int64_t pages_for(int length, int page)
{
    return length <= 0 ? 0 : ((int64_t)length + page - 1) / page;
}

// First launch: the first groups note the pages, the others a row a wave.
__global__ __launch_bounds__(256) void take_notes(Pool p, uint64_t *notes, int32_t *need, int page_groups)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if ((int)blockIdx.x < page_groups) return note_pages(p.refs, p.npages, notes, (int64_t)blockIdx.x * 4 + wave);
    const int64_t row = (int64_t)(blockIdx.x - page_groups) * 4 + wave;
    if (row >= p.rows) return;
    int64_t n = pages_for(p.lengths[row], p.page);
    if (n > p.width) n = p.width;
    int count = 0;
    for (int64_t c = 0; c < n; c += 64)
        count += __popcll(__ballot(c + lane < n && !valid(p.tables[row * p.ld + c + lane], p.npages)));
    if (lane == 0) need[row] = count;
}

template <int W>
__global__ __launch_bounds__(256) void take_kernel(Pool p, const uint64_t *notes, const int32_t *need,
                                                   int32_t *missing)
{
    __shared__ int before[W], tmp[4];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t row0 = (int64_t)blockIdx.x * 4;
    // what the rows ahead of this group's four need, and these
    int sum = 0;
    const int64_t until = blockIdx.x == 0 ? p.rows : row0;
    for (int64_t r = threadIdx.x; r < until; r += 256) sum += need[r];
    int ahead;
    sum_before(sum, tmp, ahead);
    int mine[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[i] = row0 + i < p.rows ? need[row0 + i] : 0;
    if (blockIdx.x != 0 && mine[0] + mine[1] + mine[2] + mine[3] == 0) return;
    const int free = sum_notes<true, W>(notes, p.npages, before, tmp);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *missing = ahead > free ? ahead - free : 0;
        ahead = 0;
    }
    const int64_t row = row0 + wave;
    if (row >= p.rows) return;
    int k = ahead;
    for (int i = 0; i < wave; ++i) k += mine[i];
    int64_t n = pages_for(p.lengths[row], p.page);
    if (n > p.width) n = p.width;
    if (mine[wave] == 0) return;
    for (int64_t c = 0; c < n; c += 64) {
        const bool lacks = c + lane < n && !valid(p.tables[row * p.ld + c + lane], p.npages);
        const uint64_t all = __ballot(lacks);
        const int rank = k + __popcll(all & ((uint64_t(1) << lane) - 1));
        if (lacks) {
            int page = -1;
            if (rank < free) {
                page = page_at<true>(notes, p.npages, before, rank);
                p.refs[page] = 1;
            }
            p.tables[row * p.ld + c + lane] = page;
        }
        k += __popcll(all);
    }
}

// --- forking --------------------------------------------------------------------------------------------------------

// First launch: which pairs count, and their children's rows given up.
__global__ __launch_bounds__(256) void fork_release(Pool p, const int32_t *parents, const int32_t *children,
                                                    int64_t n, int32_t *state)
{
    const int i = blockIdx.x;
    const int from = parents[i], to = children[i];
    bool bad = !valid(from, p.rows) || !valid(to, p.rows);
    for (int64_t j = threadIdx.x; j < n; j += 256) bad |= children[j] == from || (j > i && children[j] == to);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) state[i] = bad ? -1 : 0;
    if (!bad) release_row(p, to);
}

// Second launch: the first groups note the pages (shared ones are in use before
// and after), the others give a child its parent's full pages.  state: 1 + the
// page to be copied, 0 for none, -1 for a pair that does not count.
__global__ __launch_bounds__(256) void fork_share(Pool p, const int32_t *parents, const int32_t *children,
                                                  int32_t *state, uint64_t *notes, int page_groups)
{
    if ((int)blockIdx.x < page_groups)
        return note_pages(p.refs, p.npages, notes, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6));
    const int i = blockIdx.x - page_groups;
    if (state[i] < 0) return;
    const int64_t from = parents[i], to = children[i];
    const int length = p.lengths[from];
    const int64_t full = length > 0 ? length / p.page : 0;
    for (int64_t c = threadIdx.x; c < p.width && c < full; c += 256) {
        const int page = p.tables[from * p.ld + c];
        if (!valid(page, p.npages)) continue;
        atomicAdd(&p.refs[page], 1);
        p.tables[to * p.ld + c] = page;
    }
    if (threadIdx.x == 0) {
        p.lengths[to] = length;
        int last = -1;
        if (length > 0 && length % p.page != 0 && full < p.width) last = p.tables[from * p.ld + full];
        state[i] = valid(last, p.npages) ? last + 1 : 0;
    }
}

// No pairs: nothing is missing.
__global__ void fork_none(int32_t *missing) { *missing = 0; }

// Third launch: pair i's workgroups find its page and copy a chunk each.
template <int W>
__global__ __launch_bounds__(256) void fork_copy(Pool p, char *pages, int64_t bytes, int64_t stride,
                                                 const int32_t *children, int64_t n, const int32_t *state,
                                                 const uint64_t *notes, int32_t *missing, int chunks)
{
    __shared__ int before[W], tmp[4];
    const int i = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    if (blockIdx.x != 0 && state[i] <= 0) return;
    int ahead = 0, all = 0;
    for (int64_t j = threadIdx.x; j < n; j += 256) {
        const int need = state[j] > 0;
        all += need;
        if (j < i) ahead += need;
    }
    int rank, total;
    sum_before(ahead, tmp, rank);
    sum_before(all, tmp, total);
    const int free = sum_notes<true, W>(notes, p.npages, before, tmp);
    if (blockIdx.x == 0 && threadIdx.x == 0) *missing = total > free ? total - free : 0;
    if (state[i] <= 0 || rank >= free) return;
    const int src = state[i] - 1, dst = page_at<true>(notes, p.npages, before, rank);
    copy_chunk(pages + src * stride, pages + dst * stride, bytes, chunk);
    if (chunk == 0 && threadIdx.x == 0) {
        p.refs[dst] = 1;
        const int to = children[i];
        p.tables[to * p.ld + p.lengths[to] / p.page] = dst;
    }
}

// --- compacting -----------------------------------------------------------------------------------------------------

__global__ __launch_bounds__(256) void compact_notes(const int32_t *refs, int64_t npages, uint64_t *notes)
{
    note_pages(refs, npages, notes, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6));
}

// With U pages in use, the k-th of them from U on goes to the k-th free page below U.
// Sources and targets are different pages, so the copies need no order.  The first
// `movers` workgroups move pages, the others rewrite the table and the map; both
// read the notes alone.
template <int W>
__global__ __launch_bounds__(256) void compact_kernel(Pool p, char *pages, int64_t bytes, int64_t stride,
                                                      const uint64_t *notes, int32_t *used, int32_t *to, int movers,
                                                      int chunks)
{
    __shared__ int before[W], tmp[4];
    const int U = sum_notes<false, W>(notes, p.npages, before, tmp);
    // pages in use below U: the first of those that move is the one with this rank
    int stay = 0;
    if (U < p.npages) {
        const int w = U >> 6;
        stay = before[w] + __popcll(notes[w] & ((uint64_t(1) << (U & 63)) - 1));
    } else {
        stay = U;
    }
    const int moves = U - stay;
    // the k-th free page: the words' free pages ahead are 64 w - before[w]
    const auto hole = [&](int k) {
        int lo = 0, hi = (U - 1) >> 6;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (64 * mid - before[mid] <= k) lo = mid; else hi = mid - 1;
        }
        uint64_t bits = ~notes[lo];
        int left = k - (64 * lo - before[lo]), at = 0;
#pragma unroll
        for (int half = 32; half > 0; half >>= 1) {
            const int low = __popcll(bits & ((uint64_t(1) << half) - 1));
            if (left >= low) {
                left -= low;
                bits >>= half;
                at += half;
            }
        }
        return lo * 64 + at;
    };
    if ((int)blockIdx.x < movers) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *used = U;
        for (int64_t job = blockIdx.x; job < (int64_t)moves * chunks; job += movers) {
            const int k = (int)(job / chunks), chunk = (int)(job % chunks);
            const int src = page_at<false>(notes, p.npages, before, stay + k), dst = hole(k);
            copy_chunk(pages + src * stride, pages + dst * stride, bytes, chunk);
            if (chunk == 0 && threadIdx.x == 0) {
                p.refs[dst] = p.refs[src];
                p.refs[src] = 0;
            }
        }
        return;
    }
    const auto moved = [&](int page) {
        const int w = page >> 6, b = page & 63;
        if (page < U || !((notes[w] >> b) & 1)) return page;
        return hole(before[w] + __popcll(notes[w] & ((uint64_t(1) << b) - 1)) - stay);
    };
    const int64_t step = (int64_t)(gridDim.x - movers) * 256;
    const int64_t self = (int64_t)(blockIdx.x - movers) * 256 + threadIdx.x;
    for (int64_t e = self; e < p.rows * p.width; e += step) {
        int32_t *at = p.tables + e / p.width * p.ld + e % p.width;
        const int page = *at;
        if (valid(page, p.npages) && page >= U) *at = moved(page);
    }
    if (to)
        for (int64_t e = self; e < p.npages; e += step) to[e] = moved((int)e);
}

// f with the most words that npages has: 1024 words (65536 pages) fit in 4 KB of LDS.
template <typename F>
int by_words(int64_t npages, F f)
{
    return npages <= 65536 ? f(std::integral_constant<int, 1024>()) : f(std::integral_constant<int, POOL_MAX / 64>());
}

int64_t chunks_of(int64_t bytes) { return (bytes + CHUNK - 1) / CHUNK; }

uint64_t *notes_of(void *scratch) { return static_cast<uint64_t *>(scratch); }
int32_t *counts_of(void *scratch, int64_t npages)
{
    return reinterpret_cast<int32_t *>(notes_of(scratch) + (npages + 63) / 64);
}

int page_groups(int64_t npages) { return (int)((npages + 255) / 256); }

}  // namespace

int launch_copy_pages(void *pages, int64_t npages, int64_t bytes, int64_t stride, const int32_t *src,
                      const int32_t *dst, int64_t n, hipStream_t stream)
{
    const int64_t chunks = chunks_of(bytes);
    if (chunks > launch_groups(256)) return -1;
    return in_launches(n, launch_groups(256) / chunks, [&](int64_t first, int64_t count) {
        return launch_kernel(copy_kernel, dim3((unsigned)(count * chunks)), dim3(256), stream,
                             static_cast<char *>(pages), npages, bytes, stride, src, dst, first, (int)chunks);
    });
}

int launch_free_pages(const Pool &p, const int32_t *which, int64_t n, hipStream_t stream)
{
    return in_launches(n, launch_groups(256), [&](int64_t first, int64_t count) {
        return launch_kernel(free_kernel, dim3((unsigned)count), dim3(256), stream, p, which + first);
    });
}

int launch_take_pages(const Pool &p, int32_t *missing, void *scratch, hipStream_t stream)
{
    uint64_t *notes = notes_of(scratch);
    int32_t *need = counts_of(scratch, p.npages);
    const int groups = page_groups(p.npages);
    const int64_t rows = (p.rows + 3) / 4;
    if (rows + groups > launch_groups(256)) return -1;
    const int rc = launch_kernel(take_notes, dim3((unsigned)(groups + rows)), dim3(256), stream, p, notes, need, groups);
    if (rc != 0) return rc;
    return by_words(p.npages, [&](auto w) {
        return launch_kernel(take_kernel<w.value>, dim3((unsigned)(rows > 0 ? rows : 1)), dim3(256), stream, p, notes,
                             need, missing);
    });
}

int launch_fork_pages(const Pool &p, void *pages, int64_t bytes, int64_t stride, const int32_t *parents,
                      const int32_t *children, int64_t n, int32_t *missing, void *scratch, hipStream_t stream)
{
    if (n == 0) return launch_kernel(fork_none, dim3(1), dim3(1), stream, missing);
    uint64_t *notes = notes_of(scratch);
    int32_t *state = counts_of(scratch, p.npages);
    const int groups = page_groups(p.npages);
    const int64_t chunks = chunks_of(bytes);
    if (n + groups > launch_groups(256) || n > launch_groups(256) / chunks) return -1;
    int rc = launch_kernel(fork_release, dim3((unsigned)n), dim3(256), stream, p, parents, children, n, state);
    if (rc != 0) return rc;
    rc = launch_kernel(fork_share, dim3((unsigned)(groups + n)), dim3(256), stream, p, parents, children, state, notes,
                       groups);
    if (rc != 0) return rc;
    return by_words(p.npages, [&](auto w) {
        return launch_kernel(fork_copy<w.value>, dim3((unsigned)(n * chunks)), dim3(256), stream, p,
                             static_cast<char *>(pages), bytes, stride, children, n, state, notes, missing, (int)chunks);
    });
}

int launch_compact_pages(const Pool &p, void *pages, int64_t bytes, int64_t stride, int32_t *used, int32_t *to,
                         void *scratch, hipStream_t stream)
{
    uint64_t *notes = notes_of(scratch);
    const int64_t chunks = chunks_of(bytes);
    const int rc = launch_kernel(compact_notes, dim3((unsigned)page_groups(p.npages)), dim3(256), stream, p.refs,
                                 p.npages, notes);
    if (rc != 0) return rc;
    // at most half of the pages move
    const int64_t jobs = p.npages / 2 * chunks;
    const int movers = (int)(jobs < 1 ? 1 : jobs > 4096 ? 4096 : jobs);
    const int64_t entries = p.rows * p.width > p.npages ? p.rows * p.width : p.npages;
    const int64_t rest = (entries + 255) / 256;
    const int writers = (int)(rest > 512 ? 512 : rest);
    return by_words(p.npages, [&](auto w) {
        return launch_kernel(compact_kernel<w.value>, dim3((unsigned)(movers + writers)), dim3(256), stream, p,
                             static_cast<char *>(pages), bytes, stride, notes, used, to, movers, (int)chunks);
    });
}

}  // namespace qig
