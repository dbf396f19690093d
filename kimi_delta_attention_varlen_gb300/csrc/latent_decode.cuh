// What the forms of absorbed latent decode have in common: the line of tiles that the CTAs share out, the walk along it,
// and the join of the parts of items that fell into several shares.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_common.cuh"
#include "kda_internal.h"
#include "tcgen05.cuh"

namespace kda {
namespace prefill {
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // chunk_prep.cu
}
namespace latent {
namespace {  // each unit that includes this has its own

constexpr int T = 64;  // tokens a tile
constexpr int kItemUnits = 3;  // see the share below; 2, 3 and 4 measure alike
constexpr int kSumTiles = 256;  // tiles that the accumulator takes before it is set aside, a power of two
constexpr int kSoftThreads = 128;
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kStatusExpired = 6;
constexpr int kJoinCtas = 6;  // a SM, of which the registers let two or three be resident at once

struct Params {
    LatentDecodeArgs a;
    int32_t rows, groups, box_rows;  // L * h; row groups; rows of a TMA box (divides the page size)
    float scale_log2;
    int32_t *status, *item0, *item1;  // [grid]: first row (of all entries' rows) of the item whose part is in slot 0 / 1 of the CTA, or -1
    float4 *ml;                       // [grid][2][N]: m, l, l of the rounded probabilities
    float *part;                      // [grid][2][N][dl]; also what a segment sets aside, in its slot
    // Prefixes that groups share: what was computed for them, of all entries' rows, and the token that each entry's own
    // part begins with.
    const int32_t *base;              // [batch]
    float4 *pre_ml;                   // [rows of all entries]: m, l, l of the rounded probabilities
    float *pre;                       // [rows of all entries][dl], relative to m
    int32_t *item_rows;               // [grid]: rows of the item in slot 1 (of the prefixes' items)
    const int32_t *shares_any;        // 0: no group has a prefix that is shared
};

__device__ __forceinline__ int64_t slot_of(const LatentDecodeArgs &a, int64_t r)
{
    if (a.req == nullptr) return r;
    return a.idx_type == KDA_I32 ? static_cast<int64_t>(static_cast<const int32_t *>(a.req)[r])
                                 : static_cast<const int64_t *>(a.req)[r];
}

__device__ __forceinline__ int32_t length_of(const LatentDecodeArgs &a, int64_t slot)
{
    if (slot < 0 || slot >= a.requests) return 0;
    const int32_t most = static_cast<int32_t>(a.width * a.page), n = a.seq_lens[slot];
    return n < 0 ? 0 : n > most ? most : n;
}

__device__ __forceinline__ int32_t tiles_of(int32_t n) { return n > T ? (n - 1) / T + 1 : 1; }

// A row that saw nothing has the sum 0: output 0, log-sum-exp -inf.  A NaN stays one.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
// What a sum relative to the maximum `from` is worth relative to `to`.
__device__ __forceinline__ float rebase(float from, float to) { return from == to ? 1.f : ex2_approx(from - to); }
__device__ __forceinline__ float log_sum(float m, float sum) { return sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2; }

__host__ __device__ constexpr uint32_t idesc(int M, int n, bool a_mn)  // bf16 operands, fp32 accumulator, B K-major
{
    return tc::idesc_bf16(M, n, false) | ((a_mn ? 1u : 0u) << 15);
}

struct Edge {
    int64_t r, tiles_before;
    int32_t group, tile;
};

// Token that entry r's line begins with, and the end of its tokens.
template <bool Shared> __device__ __forceinline__ int32_t base_of(const Params &p, int64_t r)
{
    if (!Shared) return 0;
    const int32_t b = p.base[r];  // anything where the groups' offsets break their contract
    return b < 0 || b > p.a.width * p.a.page ? 0 : b;
}
template <bool Shared> __device__ __forceinline__ int32_t end_of(const Params &p, int64_t slot, int32_t base)
{
    const int32_t n = length_of(p.a, slot);
    return Shared && n < base ? base : n;
}

// Position on the line of tiles (Shared: of the tokens behind a shared prefix).
template <bool Shared> struct WalkOf {
    int64_t r, slot;
    int32_t group, tile, base, n, tiles;

    __device__ void load(const Params &p)
    {
        slot = slot_of(p.a, r);
        base = base_of<Shared>(p, r);
        n = end_of<Shared>(p, slot, base);
        tiles = tiles_of(n - base);
    }
    __device__ int32_t token(int32_t t) const { return Shared ? base + t * T : t * T; }  // a tile's first
    __device__ bool first() const { return tile == 0; }
    __device__ bool last() const { return tile + 1 == tiles; }
    // the first query token of the request sees this tile alone
    __device__ bool twice(const Params &p) const { return tile == 0 && n - (p.a.L - 1) <= T; }
    __device__ void next(const Params &p)
    {
        if (++tile < tiles) return;
        tile = 0;
        if (++group < p.groups) return;
        group = 0;
        if (++r < p.a.batch) load(p);
    }
};
using Walk = WalkOf<false>;

// 32 columns of 16 lanes: registers 4 j + {0, 1} are row lane / 4, columns 8 j + 2 (lane % 4) + {0, 1}, and
// 4 j + {2, 3} the same columns of row lane / 4 + 8.
__device__ __forceinline__ void ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                   "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}

__device__ __forceinline__ void ld1(uint32_t taddr, uint32_t &r)  // this thread's lane, one column
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n" : "=r"(r) : "r"(taddr));
}
__device__ __forceinline__ void st1(uint32_t taddr, uint32_t r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n" ::"r"(taddr), "r"(r) : "memory");
}

template <int Threads = kSoftThreads>
__device__ __forceinline__ bool soft_any(bool v)  // the softmax warps (named barrier 1)
{
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"(v ? 1u : 0u), "n"(Threads)
                 : "memory");
    return r != 0;
}

// One lane of the (converged) warp.  Copies and MMAs are issued under this test and not under a test
// of the lane number: after elect.sync the compiler knows that one thread runs and keeps addresses and
// descriptors in uniform registers (measured per MMA: 32 to 48 cycles, the operands' shared memory
// time, instead of 54 to 112).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r)::"memory");
    return r != 0;
}

// The ends edge[0], edge[1] of this CTA's share of the line.  By all threads (Threads of them); `sums` holds a word a warp.
// Synchronises the CTA.
template <int Threads, bool Shared = false>
__device__ __forceinline__ void find_share(const Params &p, int64_t *sums, Edge *edge)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    auto tiles_at = [&](int64_t r) {
        const int32_t base = base_of<Shared>(p, r);
        return tiles_of(end_of<Shared>(p, slot_of(p.a, r), base) - base);
    };
    // A share is [w0, w1) of the line, on which a (request, group) takes its tiles and kItemUnits more: the
    // work that comes with it whatever its length (queries, first tile's latency, epilogue).
    const int64_t per = (p.a.batch + Threads - 1) / Threads, r_lo = per * tid;
    const int64_t r_hi = r_lo + per < p.a.batch ? r_lo + per : p.a.batch;
    int64_t mine = 0;  // units of this thread's slice of the requests, of one group
    for (int64_t r = r_lo; r < r_hi; ++r) mine += tiles_at(r) + kItemUnits;
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
    }
    if (lane == 31) sums[warp] = scan;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    int64_t before = scan - mine, all = 0;
#pragma unroll
    for (int w = 0; w < Threads / 32; ++w) {
        before += w < warp ? sums[w] : 0;
        all += sums[w];
    }
    all *= p.groups;
    before *= p.groups;
    const int64_t shares = all < gridDim.x ? all : gridDim.x;
    // the ends of the share as (request, group, tile) and as a count of tiles before it
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t at = cta + e <= shares ? all * (cta + e) / shares : all;
        if (tid == 0 && at == all) edge[e] = Edge{0, all - kItemUnits * p.groups * p.a.batch, 0, 0};
        if (at >= before && at < before + mine * p.groups) {
            int64_t left = at - before, r = r_lo;
            int32_t tiles;
            for (;; ++r) {
                tiles = tiles_at(r);
                const int64_t u = static_cast<int64_t>(tiles + kItemUnits) * p.groups;
                if (left < u) break;
                left -= u;
            }
            const int32_t group = static_cast<int32_t>(left / (tiles + kItemUnits)), x = static_cast<int32_t>(left % (tiles + kItemUnits));
            const int32_t tile = x > kItemUnits ? x - kItemUnits : 0;
            edge[e] = Edge{r, at - left - kItemUnits * p.groups * r + static_cast<int64_t>(group) * tiles + tile, group, tile};
        }
    }
    __syncthreads();
}

// Joins the parts of the items that fell into several shares: an item's first part is in slot 1 of some share
// c, the next ones are in slot 0 of the shares behind.  Every CTA lists those items (a look at two words a
// share), then takes every grid-th unit of work: eight rows of an item of few parts, one row a warp (a loaded
// batch: about 150 items of two or three parts), or one row of an item of many, the parts dealt out to the
// whole CTA (one long request: 32 rows of 152 parts).
constexpr int kFewParts = 8;

//
// kOwn: the items are entries' own tokens behind a prefix, what was computed for that joins in; kPrefix: the items are
// blocks of rows of the prefixes, and what comes out is not normalised.
enum JoinForm { kPlain, kOwn, kPrefix };

template <int DL, int N, JoinForm Form = kPlain>
__global__ void __launch_bounds__(256) latent_join_kernel(Params p, int32_t shares)
{
    constexpr int kLanes = DL / 4, kSubs = 256 / kLanes, kAhead = 8;  // a row's float4s; parts at once; in flight per thread
    extern __shared__ float weight[];  // [shares] weights, then per listed item: share of its first part, parts, units before it
    int32_t *const first = reinterpret_cast<int32_t *>(weight + shares), *const parts_of = first + shares, *const before = parts_of + shares;
    __shared__ float4 acc[kSubs][kLanes];
    __shared__ float sum[2], top;
    __shared__ int32_t listed, units;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t per = Form != kPrefix && p.rows < N ? p.rows : N;
    before_next();
    after_previous();
    if (Form == kPrefix && *p.shares_any == 0) return;
    int32_t *const head_of = before, *const more_of = reinterpret_cast<int32_t *>(weight);  // until they are needed
    for (int32_t j = tid; j < shares; j += 256) {
        parts_of[j] = 1;
        head_of[j] = p.item1[j];
        more_of[j] = p.item0[j];
    }
    __syncthreads();
    if (warp == 0) {
        int32_t n = 0;
        for (int32_t j0 = 0; j0 < shares; j0 += 32) {
            const int32_t j = j0 + lane;
            const bool head = j < shares && head_of[j] >= 0;
            const uint32_t all = __ballot_sync(0xffffffffu, head);
            const int32_t rank = n + __popc(all & ((1u << lane) - 1));  // items begun before share j
            if (head) first[rank] = j;
            if (j < shares && more_of[j] >= 0) atomicAdd(&parts_of[rank - 1], 1);
            n += __popc(all);
        }
        __syncwarp();
        int32_t sum_u = 0;
        for (int32_t k0 = 0; k0 < n; k0 += 32) {
            const int32_t k = k0 + lane, u = k >= n ? 0 : parts_of[k] > kFewParts ? per : (per + 7) / 8;
            int32_t s = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            if (k < n) before[k] = sum_u + s - u;
            sum_u += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) listed = n, units = sum_u;
    }
    __syncthreads();
    for (int32_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        int32_t lo = 0, hi = listed;  // the item with before[lo] <= unit
        while (lo + 1 < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (before[mid] <= unit) lo = mid;
            else hi = mid;
        }
        const int32_t c = first[lo], parts = parts_of[lo], item = p.item1[c];
        const int32_t left = Form == kPrefix ? p.item_rows[c] : p.rows - item % p.rows;  // rows from the item's first on
        auto at = [&](int32_t j, int32_t row) { return (static_cast<int64_t>(2) * (c + j) + (j == 0 ? 1 : 0)) * N + row; };
        // A row's sum o relative to m, with the sums l and lr, to where it goes; (kOwn) y and ml: the prefix's part.
        const bool joined = Form == kOwn && p.base[item / p.rows] > 0;
        struct Weights {
            float own, prefix;
        };
        auto prefix_sums = [&](int32_t row) { return joined ? p.pre_ml[item + row] : make_float4(-INFINITY, 0.f, 0.f, 0.f); };
        auto prefix_part = [&](int32_t row, int32_t d) {
            return joined ? reinterpret_cast<const float4 *>(p.pre + (static_cast<int64_t>(item) + row) * DL)[d] : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        auto weigh = [&](int32_t row, bool first, float m, float l, float lr, float4 ml) {
            Weights w{1.f, 0.f};
            if (Form == kPrefix) {
                if (first) p.pre_ml[item + row] = make_float4(m, l, lr, 0.f);
                w.own = lr == 0.f ? 0.f : 1.f;
                return w;
            }
            if (joined) {
                const float top = fmaxf(m, ml.x);
                w.own = rebase(m, top), w.prefix = rebase(ml.x, top);
                l = l * w.own + ml.y * w.prefix, lr = lr * w.own + ml.z * w.prefix, m = top;
            }
            const float inv = inverse(lr);
            w.own *= inv, w.prefix *= inv;
            if (first && p.a.lse != nullptr) p.a.lse[item + row] = log_sum(m, l);
            return w;
        };
        auto store = [&](int32_t row, int32_t d, float4 o, Weights w, float4 y) {
            const int64_t at = static_cast<int64_t>(item) + row;
            if (Form == kPrefix) {
                if (w.own == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);  // nothing is seen: 0 times what is not finite
                reinterpret_cast<float4 *>(p.pre + at * DL)[d] = o;
                return;
            }
            o.x *= w.own, o.y *= w.own, o.z *= w.own, o.w *= w.own;
            if (joined) o.x = fmaf(y.x, w.prefix, o.x), o.y = fmaf(y.y, w.prefix, o.y), o.z = fmaf(y.z, w.prefix, o.z), o.w = fmaf(y.w, w.prefix, o.w);
            reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.a.out) + at * DL)[d] = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        };
        if (parts <= kFewParts) {
            const int32_t row = (unit - before[lo]) * 8 + warp;
            if (row >= per || row >= left) continue;
            const float4 prefix = prefix_sums(row);
            float4 y[kLanes / 32];
#pragma unroll
            for (int q = 0; q < kLanes / 32; ++q) y[q] = prefix_part(row, lane + 32 * q);
            float4 ml = make_float4(-INFINITY, 0.f, 0.f, 0.f);
            if (lane < parts) ml = p.ml[at(lane, row)];
            float m = ml.x;
#pragma unroll
            for (int o = kFewParts / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = __shfl_sync(0xffffffffu, m, 0);
            const float f = lane < parts ? ex2_approx(ml.x - (m == -INFINITY ? 0.f : m)) : 0.f;
            float l = f * ml.y, lr = f * ml.z;
#pragma unroll
            for (int o = kFewParts / 2; o; o >>= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, o);
                lr += __shfl_xor_sync(0xffffffffu, lr, o);
            }
            l = __shfl_sync(0xffffffffu, l, 0), lr = __shfl_sync(0xffffffffu, lr, 0);
            float4 o[kLanes / 32];
#pragma unroll
            for (int q = 0; q < kLanes / 32; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int32_t j = 0; j < parts; ++j) {
                const float4 *x = reinterpret_cast<const float4 *>(p.part + at(j, row) * DL) + lane;
                const float fj = __shfl_sync(0xffffffffu, f, j);
#pragma unroll
                for (int q = 0; q < kLanes / 32; ++q) {
                    const float4 y = x[32 * q];
                    o[q].x += fj * y.x, o[q].y += fj * y.y, o[q].z += fj * y.z, o[q].w += fj * y.w;
                }
            }
            const Weights w = weigh(row, lane == 0, m, l, lr, prefix);
#pragma unroll
            for (int q = 0; q < kLanes / 32; ++q) store(row, lane + 32 * q, o[q], w, y[q]);
            continue;
        }
        const int32_t row = unit - before[lo], sub = tid / kLanes, d = tid % kLanes;
        if (row >= left) continue;
        if (warp == 0) {
            float m = -INFINITY, l = 0.f, lr = 0.f;
            for (int32_t j = lane; j < parts; j += 32) m = fmaxf(m, p.ml[at(j, row)].x);
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float base = m == -INFINITY ? 0.f : m;
            for (int32_t j = lane; j < parts; j += 32) {
                const float4 ml = p.ml[at(j, row)];
                const float f = ex2_approx(ml.x - base);
                weight[j] = f;
                l += f * ml.y;
                lr += f * ml.z;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, o);
                lr += __shfl_xor_sync(0xffffffffu, lr, o);
            }
            if (lane == 0) sum[0] = l, sum[1] = lr, top = m;
        }
        __syncthreads();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t j0 = sub; j0 < parts; j0 += kSubs * kAhead) {
            float4 x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (j0 + kSubs * u < parts) x[u] = *reinterpret_cast<const float4 *>(p.part + at(j0 + kSubs * u, row) * DL + 4 * d);
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (j0 + kSubs * u < parts) {
                    const float f = weight[j0 + kSubs * u];
                    o.x += f * x[u].x, o.y += f * x[u].y, o.z += f * x[u].z, o.w += f * x[u].w;
                }
        }
        acc[sub][d] = o;
        __syncthreads();
        if (sub == 0) {
#pragma unroll
            for (int q = 1; q < kSubs; ++q) {
                const float4 y = acc[q][d];
                o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
            }
            store(row, d, o, weigh(row, d == 0, top, sum[0], sum[1], prefix_sums(row)), prefix_part(row, d));
        }
        __syncthreads();  // weight, sum and acc may be written again
    }
}

// Box of 64 columns x `rows` rows of a bf16 matrix [n2][n1][n0], strides in elements, 128-byte swizzle.
inline bool encode(CUtensorMap *m, const void *base, int64_t n0, int64_t n1, int64_t n2, int64_t s1, int64_t s2, int rows)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = prefill::tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(n0), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows), 1}, elem[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a box of a page: the largest power of two that divides it, at most a tile.
inline int box_rows(int64_t page)
{
    int rows = T;
    while (page % rows != 0) rows >>= 1;
    return rows;
}

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace
}  // namespace latent
}  // namespace kda
