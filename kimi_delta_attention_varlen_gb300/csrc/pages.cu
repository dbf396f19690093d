// Page upkeep of a paged cache: fork, release, reserve (with copy on write),
// compaction, page copies, and the append of new latent rows.
//
// The tables are small (a few hundred KB), so every call here but the copies
// is bound by launch and memory latency, not by bandwidth: each takes one or two
// launches, no host round trip and no atomics whose order matters.  The page
// numbers handed out are a function of the tables alone: one cluster of eight
// CTAs counts the free pages of every 4096-page block, keeps one bit a page (so
// that refcounts may change while others still rank pages), meets at its
// barrier, and then sums the counts below its own blocks and ranks their pages
// by popcount.  As two kernels, counting and ranking, kda_pages_reserve took
// 8.4 us of the host's time in a serving step and takes 6.5 us so (2,048 pages,
// and 68,000), kda_pages_compact 10.2 and 8.3 us.
// The copies move whole page payloads in 16-byte vectors at the HBM rate.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kBlockPages = 4096;            // pages ranked at once by one CTA
constexpr int kThreads = 1024;
constexpr int kWords = kBlockPages / 32;     // bitmap words of one block
constexpr int kCluster = 8;                  // CTAs that count and rank together
constexpr int kCopyThreads = 256;
constexpr int kMostVecs = 10;                // 16-byte vectors in flight per thread, at most

// Workspace: a header of four words, then the arrays below (4-byte elements).
struct Plan {
    int32_t *header;    // [0] pages asked for (INT32_MAX: more), [1] copy-on-write moves, [2] a row is too short
    int32_t *free_cnt;  // [blocks] free pages of each block
    uint32_t *bits;     // [blocks * kWords] 1: free
    int32_t *prefix;    // [count + 1] pages asked for by the requests before this one
    int32_t *first;     // [count] table position of the request's first new page; bit 31: it replaces a shared one
    int32_t *rank;      // [n_pages] compaction: which move takes this page (overlays prefix / first)
};

int64_t blocks_of(int64_t n_pages) { return (n_pages + kBlockPages - 1) / kBlockPages; }

Plan plan_of(void *ws, int64_t n_pages, int64_t count)
{
    int32_t *w = static_cast<int32_t *>(ws);
    const int64_t nb = blocks_of(n_pages);
    Plan p{};
    p.header = w;
    p.free_cnt = w + 64;
    p.bits = reinterpret_cast<uint32_t *>(p.free_cnt + nb);
    p.prefix = p.free_cnt + nb + nb * kWords;
    p.first = p.prefix + count + 1;
    p.rank = p.prefix;
    return p;
}

__device__ __forceinline__ int64_t load_index(const void *p, int32_t itype, int64_t i)
{
    return itype == KDA_I32 ? static_cast<int64_t>(static_cast<const int32_t *>(p)[i]) : static_cast<const int64_t *>(p)[i];
}

__device__ __forceinline__ int32_t warp_sum(int32_t x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Sum over the CTA (every thread gets it); `sh` holds 32 words.
__device__ __forceinline__ int32_t block_sum(int32_t x, int32_t *sh)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    x = warp_sum(x);
    __syncthreads();
    if (lane == 0) sh[warp] = x;
    __syncthreads();
    return warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? sh[lane] : 0);
}

// Exclusive prefix sum over the CTA's threads; *total gets the sum.  64-bit: a request may ask for 2^31 tokens.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *sh, int64_t *total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = s;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
        if (w < warp) before += sh[w];
        all += sh[w];
    }
    *total = all;
    return before + s - x;
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int64_t page) { return (tokens + page - 1) / page; }

// Length of a request as the table can hold it.
__device__ __forceinline__ int64_t length_of(const kda_page_table &t, int64_t r)
{
    const int64_t n = t.seq_lens[r], most = t.width * t.page_size;
    return n < 0 ? 0 : n > most ? most : n;
}

__global__ void __launch_bounds__(128) fork_kernel(kda_page_table t, const void *src, const void *dst, int32_t itype,
                                                   int64_t count)
{
    before_next();
    after_previous();
    for (int64_t i = blockIdx.x; i < count; i += gridDim.x) {
        const int64_t s = load_index(src, itype, i), d = load_index(dst, itype, i);
        if (s < 0 || s >= t.requests || d < 0 || d >= t.requests || s == d) continue;
        const int64_t n = pages_of(length_of(t, s), t.page_size);
        for (int64_t j = threadIdx.x; j < t.width; j += blockDim.x) {
            const int32_t e = j < n ? t.block_table[s * t.table_stride + j] : -1;
            t.block_table[d * t.table_stride + j] = e;
            if (e >= 0 && e < t.n_pages) atomicAdd(&t.refcount[e], 1);
        }
        if (threadIdx.x == 0) t.seq_lens[d] = t.seq_lens[s];
    }
}

__global__ void __launch_bounds__(128) release_kernel(kda_page_table t, const void *req, int32_t itype,
                                                      const int32_t *keep, int64_t count)
{
    before_next();
    after_previous();
    for (int64_t i = blockIdx.x; i < count; i += gridDim.x) {
        const int64_t r = load_index(req, itype, i);
        if (r < 0 || r >= t.requests) continue;
        const int64_t n = length_of(t, r);
        int64_t k = keep != nullptr ? keep[i] : 0;
        k = k < 0 ? 0 : k > n ? n : k;
        for (int64_t j = pages_of(k, t.page_size) + threadIdx.x; j < pages_of(n, t.page_size); j += blockDim.x) {
            const int32_t e = t.block_table[r * t.table_stride + j];
            t.block_table[r * t.table_stride + j] = -1;
            if (e >= 0 && e < t.n_pages) atomicSub(&t.refcount[e], 1);
        }
        __syncthreads();  // every thread has read the length
        if (threadIdx.x == 0) t.seq_lens[r] = static_cast<int32_t>(k);
    }
}

// A CTA's stretch of the blocks, the same number for all but the last ones with any.
__device__ __forceinline__ void stretch(int nb, int *from, int *to)
{
    const int per = (nb + kCluster - 1) / kCluster, c = static_cast<int>(blockIdx.x);
    *from = c * per < nb ? c * per : nb;
    *to = *from + per < nb ? *from + per : nb;
}

// Free pages of blocks from .. to-1 and their bitmaps.
__device__ __forceinline__ void count_free(const kda_page_table &t, const Plan &p, int from, int to, int32_t *sh)
{
    const int tid = threadIdx.x;
    for (int block = from; block < to; ++block) {
        int32_t free_pages = 0;
#pragma unroll
        for (int k = 0; k < kBlockPages / kThreads; ++k) {
            const int64_t page = static_cast<int64_t>(block) * kBlockPages + k * kThreads + tid;
            const uint32_t w = __ballot_sync(0xffffffffu, page < t.n_pages && t.refcount[page] == 0);
            if ((tid & 31) == 0) {
                p.bits[block * kWords + k * (kThreads / 32) + (tid >> 5)] = w;
                free_pages += __popc(w);
            }
        }
        free_pages = block_sum(free_pages, sh);
        if (tid == 0) p.free_cnt[block] = free_pages;
    }
}

// What every request asks for, in list order.
__device__ __forceinline__ void count_wanted(const kda_page_table &t, const Plan &p, const void *req, int32_t itype,
                                             const int32_t *new_tokens, int64_t count, int32_t *sh32, int64_t *sh64)
{
    const int tid = threadIdx.x;
    int64_t before = 0;  // pages asked for so far
    int32_t moves = 0, too_short = 0;
    for (int64_t i0 = 0; i0 < count; i0 += kThreads) {
        const int64_t i = i0 + tid;
        int64_t want = 0, have = 0;
        bool cow = false;
        if (i < count) {
            const int64_t r = load_index(req, itype, i);
            const int64_t add = new_tokens[i];
            if (r >= 0 && r < t.requests && add > 0) {
                const int64_t n = length_of(t, r), need = pages_of(n + add, t.page_size);
                have = pages_of(n, t.page_size);
                if (n % t.page_size != 0) {
                    const int32_t last = t.block_table[r * t.table_stride + have - 1];
                    cow = last >= 0 && last < t.n_pages && t.refcount[last] > 1;
                }
                want = need - have + (cow ? 1 : 0);
                if (need > t.width) too_short = 1;
            }
        }
        int64_t total;
        const int64_t mine = before + block_scan(want, sh64, &total);
        if (i < count) {
            p.prefix[i] = static_cast<int32_t>(mine < INT32_MAX ? mine : INT32_MAX);
            p.first[i] = static_cast<int32_t>(have - (cow ? 1 : 0)) | (cow ? INT32_MIN : 0);
        }
        moves += cow ? 1 : 0;
        before += total;
    }
    moves = block_sum(moves, sh32);
    too_short = block_sum(too_short, sh32);
    if (tid == 0) {
        p.prefix[count] = p.header[0] = static_cast<int32_t>(before < INT32_MAX ? before : INT32_MAX);
        p.header[1] = moves;
        p.header[2] = too_short;
    }
}

// Free pages in all blocks and in those below `block`, the same in every thread.
__device__ __forceinline__ void free_totals(const Plan &p, int nb, int block, int32_t *sh, int32_t *all, int32_t *below)
{
    int32_t a = 0, b = 0;
    for (int j = threadIdx.x; j < nb; j += blockDim.x) {
        const int32_t c = p.free_cnt[j];
        a += c;
        b += j < block ? c : 0;
    }
    *all = block_sum(a, sh);
    *below = block_sum(b, sh);
}

// Free pages of this block before its word w, for every w: `words` [kWords], `pre` [kWords].
__device__ __forceinline__ void word_prefix(const Plan &p, int block, uint32_t *words, int32_t *pre)
{
    const int tid = threadIdx.x;
    if (tid < kWords) words[tid] = p.bits[block * kWords + tid];
    __syncthreads();
    if (tid < 32) {  // four words a lane
        int32_t c[4], sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = sum;
            sum += __popc(words[4 * tid + k]);
        }
        int32_t s = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (tid >= o) s += y;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) pre[4 * tid + k] = s - sum + c[k];
    }
    __syncthreads();
}

// Meets the cluster's other CTAs; what they wrote to global memory before is visible after.
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}

// After the barrier each CTA hands out its blocks' free pages: the page of rank k goes where the k-th wanted page is
// wanted.  All together advance the lengths and fill the moves of requests that copy nothing.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads)
reserve_kernel(kda_page_table t, Plan p, int nb, const void *req, int32_t itype, const int32_t *new_tokens, int64_t count,
               int32_t *move_src, int32_t *move_dst, int32_t *info)
{
    before_next();
    after_previous();
    __shared__ int32_t sh[32];
    __shared__ int64_t sh64[32];
    __shared__ uint32_t words[kWords];
    __shared__ int32_t pre[kWords];
    const int tid = threadIdx.x;
    int from, to;
    stretch(nb, &from, &to);
    if (blockIdx.x == kCluster - 1) count_wanted(t, p, req, itype, new_tokens, count, sh, sh64);  // the CTA with fewest blocks
    count_free(t, p, from, to, sh);
    cluster_barrier();
    int32_t all, below;
    free_totals(p, nb, from, sh, &all, &below);
    const int32_t demand = p.header[0], too_short = p.header[2];
    const bool ok = too_short == 0 && demand <= all;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + tid; i < count; i += kCluster * kThreads) {
        const bool cow = p.first[i] < 0;
        if (!ok || !cow) move_src[i] = move_dst[i] = -1;
        const int64_t r = load_index(req, itype, i);
        if (ok && r >= 0 && r < t.requests && new_tokens[i] > 0)
            t.seq_lens[r] = static_cast<int32_t>(length_of(t, r) + new_tokens[i]);
    }
    if (blockIdx.x == 0 && tid == 0) {
        info[0] = too_short ? 2 : demand <= all ? 0 : 1;
        info[1] = ok ? p.header[1] : 0;
        info[2] = demand;
        info[3] = all;
    }
    if (!ok) return;
    for (int block = from; block < to && below < demand; ++block) {
        word_prefix(p, block, words, pre);
        for (int k = 0; k < kBlockPages / kThreads; ++k) {
            const int w = k * (kThreads / 32) + (tid >> 5);
            if (below + pre[w] >= demand) break;  // uniform in the warp; later words rank higher
            const uint32_t word = words[w], bit = 1u << (tid & 31);
            const int32_t rank = below + pre[w] + __popc(word & (bit - 1));
            if (!(word & bit) || rank >= demand) continue;
            const int32_t page = block * kBlockPages + k * kThreads + tid;
            int64_t lo = 0, hi = count;  // the request i with prefix[i] <= rank < prefix[i + 1]
            while (lo + 1 < hi) {
                const int64_t mid = (lo + hi) >> 1;
                if (p.prefix[mid] <= rank) lo = mid;
                else hi = mid;
            }
            const int32_t e = rank - p.prefix[lo], f = p.first[lo];
            int32_t *slot = t.block_table + load_index(req, itype, lo) * t.table_stride + (f & INT32_MAX) + e;
            if (f < 0 && e == 0) {
                const int32_t old = *slot;
                move_src[lo] = old;
                move_dst[lo] = page;
                atomicSub(&t.refcount[old], 1);
            }
            *slot = page;
            t.refcount[page] = 1;
        }
        below += p.free_cnt[block];
        __syncthreads();  // words and pre are written again
    }
}

// Compaction, ranks: the k-th free page below `live` is the k-th destination, the k-th live page at or
// above it the k-th source.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads)
compact_rank_kernel(kda_page_table t, Plan p, int nb, int32_t *move_src, int32_t *move_dst, int32_t *info)
{
    before_next();
    after_previous();
    __shared__ int32_t sh[32];
    __shared__ uint32_t words[kWords];
    __shared__ int32_t pre[kWords];
    const int tid = threadIdx.x;
    const int32_t n_pages = static_cast<int32_t>(t.n_pages);
    int from, to;
    stretch(nb, &from, &to);
    count_free(t, p, from, to, sh);
    cluster_barrier();
    int32_t all, below;
    free_totals(p, nb, from, sh, &all, &below);
    const int32_t live = n_pages - all;
    // free pages below `live`: whole blocks below it, then the words of its own block
    const int lb = live / kBlockPages, left = live % kBlockPages;
    int32_t holes = 0;
    for (int j = tid; j < lb; j += kThreads) holes += p.free_cnt[j];
    if (tid < kWords && lb < nb) {
        const int bits = left - 32 * tid;
        if (bits > 0) holes += __popc(p.bits[lb * kWords + tid] & (bits >= 32 ? 0xffffffffu : (1u << bits) - 1));
    }
    holes = block_sum(holes, sh);
    if (blockIdx.x == 0 && tid == 0) {
        info[0] = 0;
        info[1] = p.header[1] = holes;
        info[2] = p.header[0] = live;
        info[3] = all;
    }
    for (int block = from; block < to; ++block) {
        word_prefix(p, block, words, pre);
#pragma unroll
        for (int k = 0; k < kBlockPages / kThreads; ++k) {
            const int32_t page = block * kBlockPages + k * kThreads + tid;
            if (page >= n_pages) break;
            const int w = k * (kThreads / 32) + (tid >> 5);
            const uint32_t word = words[w], bit = 1u << (tid & 31);
            const int32_t free_rank = below + pre[w] + __popc(word & (bit - 1));
            if (word & bit) {
                if (page < live) move_dst[free_rank] = page;
            } else if (page >= live) {
                const int32_t m = page - free_rank - (live - holes);
                move_src[m] = page;
                p.rank[page] = m;
            }
        }
        below += p.free_cnt[block];
        __syncthreads();
    }
}

// Compaction, tables: every entry that names a moved page follows it; the refcounts move.
__global__ void __launch_bounds__(256) compact_apply_kernel(kda_page_table t, Plan p, int32_t *move_src,
                                                            int32_t *move_dst, int64_t capacity)
{
    before_next();
    after_previous();
    const int32_t live = p.header[0], moves = p.header[1];
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = i0; i < capacity; i += step) {
        if (i < moves) {
            const int32_t s = move_src[i];
            t.refcount[move_dst[i]] = t.refcount[s];
            t.refcount[s] = 0;
        } else {
            move_src[i] = move_dst[i] = -1;
        }
    }
    for (int64_t i = i0; i < t.requests * t.width; i += step) {
        int32_t *slot = t.block_table + (i / t.width) * t.table_stride + i % t.width;
        const int32_t e = *slot;
        if (e >= live && e < t.n_pages && !(p.bits[e >> 5] >> (e & 31) & 1u)) *slot = move_dst[p.rank[e]];
    }
}

// Page copies, one tile of one page per CTA step: the page in as few equal tiles as kMostVecs vectors a thread allow
// (a page of 64 latent rows, 73,728 bytes: two tiles of nine).  The call on 6000 such pages with its plan: 152.6 us
// (6.2 TB/s in the copy); at most 8 vectors (three tiles of six) 158, 12 (two of nine, fewer CTAs an SM) 154, 16 162,
// four with a half-empty last tile 170; a warp an SM with bulk copies through shared memory 168.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_v16(uint4 *cache, int64_t n_rows, int64_t stride_v16,
                                                               int64_t payload_v16, int32_t vecs, const void *src, const void *dst,
                                                               int32_t itype, int64_t count)
{
    before_next();
    after_previous();
    const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kCopyThreads * vecs) + threadIdx.x;
    for (int64_t i = blockIdx.y; i < count; i += gridDim.y) {
        const int64_t s = load_index(src, itype, i), d = load_index(dst, itype, i);
        if (s < 0 || s >= n_rows || d < 0 || d >= n_rows) continue;
        const uint4 *from = cache + s * stride_v16 + v0;
        uint4 *to = cache + d * stride_v16 + v0, buf[kMostVecs];
#pragma unroll
        for (int u = 0; u < kMostVecs; ++u)
            if (u < vecs && v0 + u * kCopyThreads < payload_v16) buf[u] = ld_v4(from + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < kMostVecs; ++u)
            if (u < vecs && v0 + u * kCopyThreads < payload_v16) st_cs_v4(to + u * kCopyThreads, buf[u]);
    }
}

// Layouts that are not 16-byte aligned.
template <typename T>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_scalar(T *cache, int64_t n_rows, int64_t stride, int64_t payload,
                                                                  const void *src, const void *dst, int32_t itype,
                                                                  int64_t count)
{
    before_next();
    after_previous();
    const int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
    if (e >= payload) return;
    for (int64_t i = blockIdx.y; i < count; i += gridDim.y) {
        const int64_t s = load_index(src, itype, i), d = load_index(dst, itype, i);
        if (s >= 0 && s < n_rows && d >= 0 && d < n_rows) cache[d * stride + e] = cache[s * stride + e];
    }
}

// New latent rows into their pages: one warp a token, V elements (16 bytes or one element) at a time.
template <typename V>
__global__ void __launch_bounds__(256) append_kernel(const V *x, int64_t x_stride, int64_t total, const int32_t *cu,
                                                     const void *req, int32_t itype, int64_t count, kda_page_table t,
                                                     V *cache, int64_t row_stride, int64_t width_v)
{
    before_next();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (tok >= total || tok < cu[0] || tok >= cu[count]) return;
    // the request i with cu[i] <= tok < cu[i + 1], by 33-way steps of the warp: two looks for a thousand requests
    int64_t lo = 0, hi = count;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + step * lane;
        const uint32_t below = __ballot_sync(0xffffffffu, at < hi && cu[at] <= tok);  // lane 0 always
        const int64_t from = lo + step * (below != 0 ? __popc(below) - 1 : 0);  // 0 only if the offsets fall somewhere
        hi = from + step < hi ? from + step : hi;
        lo = from;
    }
    const int64_t r = load_index(req, itype, lo);
    if (r < 0 || r >= t.requests || tok >= cu[lo + 1]) return;
    const int64_t pos = length_of(t, r) - cu[lo + 1] + tok;
    if (pos < 0) return;
    const int32_t page = t.block_table[r * t.table_stride + pos / t.page_size];
    if (page < 0 || page >= t.n_pages) return;
    V *to = cache + page * row_stride + (pos % t.page_size) * width_v;
    const V *from = x + tok * x_stride;
    for (int64_t e = lane; e < width_v; e += 32) to[e] = from[e];
}

unsigned row_grid(int64_t n) { return static_cast<unsigned>(n < 65535 ? n : 65535); }

}  // namespace

size_t pages_workspace(int64_t n_pages, int64_t count)
{
    const int64_t nb = blocks_of(n_pages), plan = 2 * count + 1;
    return static_cast<size_t>(64 + nb + nb * kWords + (plan > n_pages ? plan : n_pages)) * 4;
}

cudaError_t launch_pages_fork(const kda_page_table &t, const void *src, const void *dst, int32_t itype, int64_t count,
                              cudaStream_t st)
{
    return launch_overlapped(fork_kernel, dim3(row_grid(count)), dim3(128), 0, st, t, src, dst, itype, count);
}

cudaError_t launch_pages_release(const kda_page_table &t, const void *req, int32_t itype, const int32_t *keep,
                                 int64_t count, cudaStream_t st)
{
    return launch_overlapped(release_kernel, dim3(row_grid(count)), dim3(128), 0, st, t, req, itype, keep, count);
}

cudaError_t launch_pages_reserve(const kda_page_table &t, const void *req, int32_t itype, const int32_t *new_tokens,
                                 int64_t count, int32_t *move_src, int32_t *move_dst, int32_t *info, void *ws,
                                 cudaStream_t st)
{
    const Plan p = plan_of(ws, t.n_pages, count);
    const int nb = static_cast<int>(blocks_of(t.n_pages));
    return launch_overlapped(reserve_kernel, dim3(kCluster), dim3(kThreads), 0, st, t, p, nb, req, itype, new_tokens, count, move_src,
                             move_dst, info);
}

cudaError_t launch_pages_compact(const kda_page_table &t, int32_t *move_src, int32_t *move_dst, int64_t capacity,
                                 int32_t *info, void *ws, cudaStream_t st)
{
    const Plan p = plan_of(ws, t.n_pages, 0);
    const int nb = static_cast<int>(blocks_of(t.n_pages));
    const cudaError_t e = launch_overlapped(compact_rank_kernel, dim3(kCluster), dim3(kThreads), 0, st, t, p, nb, move_src, move_dst, info);
    if (e != cudaSuccess) return e;
    const int64_t work = t.requests * t.width > capacity ? t.requests * t.width : capacity;
    const int64_t grid = (work + 255) / 256, most = sm_count() * 8;
    return launch_overlapped(compact_apply_kernel, dim3(static_cast<unsigned>(grid < most ? grid : most)), dim3(256), 0, st, t, p,
                             move_src, move_dst, capacity);
}

cudaError_t launch_pages_copy(const CacheDesc &c, const void *src, const void *dst, int32_t itype, int64_t count,
                              cudaStream_t st)
{
    const int64_t es = c.dtype == KDA_F32 ? 4 : 2, payload = c.h * c.v * c.k;
    const bool vec = (reinterpret_cast<uintptr_t>(c.data) & 15u) == 0 && c.row_stride * es % 16 == 0 && payload * es % 16 == 0;
    const int64_t units = vec ? payload * es / 16 : payload;
    const int64_t tiles = vec ? (units + kCopyThreads * kMostVecs - 1) / (kCopyThreads * kMostVecs) : (units + kCopyThreads - 1) / kCopyThreads;
    const int32_t vecs = static_cast<int32_t>((units + kCopyThreads * tiles - 1) / (kCopyThreads * tiles));
    const dim3 grid(static_cast<unsigned>(tiles), row_grid(count), 1);
    if (vec)
        return launch_overlapped(copy_pages_v16, grid, dim3(kCopyThreads), 0, st, static_cast<uint4 *>(c.data), c.n_rows,
                                 c.row_stride * es / 16, units, vecs, src, dst, itype, count);
    if (c.dtype == KDA_F32)
        return launch_overlapped(copy_pages_scalar<float>, grid, dim3(kCopyThreads), 0, st, static_cast<float *>(c.data), c.n_rows,
                                 c.row_stride, units, src, dst, itype, count);
    return launch_overlapped(copy_pages_scalar<uint16_t>, grid, dim3(kCopyThreads), 0, st, static_cast<uint16_t *>(c.data), c.n_rows,
                             c.row_stride, units, src, dst, itype, count);
}

cudaError_t launch_latent_append(const void *x, int64_t x_stride, int64_t total, const int32_t *cu, const void *req,
                                 int32_t itype, int64_t count, const kda_page_table &t, const CacheDesc &c, cudaStream_t st)
{
    const int64_t es = c.dtype == KDA_F32 ? 4 : 2;
    const unsigned grid = static_cast<unsigned>((total + 7) / 8);
    const bool vec = ((reinterpret_cast<uintptr_t>(c.data) | reinterpret_cast<uintptr_t>(x)) & 15u) == 0 &&
                     c.row_stride * es % 16 == 0 && c.k * es % 16 == 0 && x_stride * es % 16 == 0;
    if (vec)
        return launch_overlapped(append_kernel<uint4>, dim3(grid), dim3(256), 0, st, static_cast<const uint4 *>(x), x_stride * es / 16,
                                 total, cu, req, itype, count, t, static_cast<uint4 *>(c.data), c.row_stride * es / 16, c.k * es / 16);
    if (c.dtype == KDA_F32)
        return launch_overlapped(append_kernel<float>, dim3(grid), dim3(256), 0, st, static_cast<const float *>(x), x_stride, total, cu,
                                 req, itype, count, t, static_cast<float *>(c.data), c.row_stride, c.k);
    return launch_overlapped(append_kernel<uint16_t>, dim3(grid), dim3(256), 0, st, static_cast<const uint16_t *>(x), x_stride, total, cu,
                             req, itype, count, t, static_cast<uint16_t *>(c.data), c.row_stride, c.k);
}

}  // namespace kda
