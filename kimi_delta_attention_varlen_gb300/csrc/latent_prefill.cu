// Expanded latent attention over a varlen batch (kda_latent_prefill).
//
//   S = scale (Q_nope K_nope^T + Q_rope K_rope^T),  P = e^{S - m},  out = P V / l
// per sequence and head, causal with the queries at the end of the keys, the keys visited in tiles
// of 128 with a running maximum m and sum l a row.
//
// plan_kernel (one CTA; for few blocks a warp of every CTA) lists the query blocks (256 queries of one
// sequence) and decides how one persistent CTA per SM shares the (block, head) pairs; a scheduling warp per
// CTA hands them to the others.
//   From kTurnRounds pairs a CTA on: in turn, by an atomic counter, in order of sequence, head and block,
//     so that blocks of one sequence and head run side by side and their keys and values come from the
//     L2 cache (a block reads 80 KB a key tile for 21 MFLOP: at the tensor cores' rate that is the HBM's);
//     the first quarter of each sequence's blocks, the short ones, come last and even out the end.
//     In turn / longest first: 16 prompts of 512..8192 tokens, 32 heads (68 pairs a CTA) 3.47 / 4.05 ms; two of
//     8192, 32 heads (13 pairs) 0.98 / 1.02 ms; four of 4096, 32 heads (13 pairs) 549 / 571 us; twelve of 300..3000
//     on 2000, 16 heads (9 pairs) 496 / 535 us; four of 2000, 32 heads (7 pairs) 193 / 186 us; one of 4096, 32 heads
//     (3 pairs) 195 / 142 us.
//   Fewer: whole rounds of one pair a CTA, longest first and in turn from either end; of the last, partial
//     round all key tiles lie on one line, of which each CTA takes the stretch that fills its sum of key tiles up
//     to a level common to all.  A pair that falls into several stretches leaves unnormalised parts in the
//     workspace, which join_kernel puts together in order of their keys.  Parts cost about what kCutTiles key
//     tiles do (queries loaded again, parts written and joined: 10 us), so the last round runs whole where its
//     longest pair is not that much longer than an equal stretch.  Cut / whole: 1000 queries on 16000 keys, 4 heads
//     57 / 203 us; 8192 queries, 2 heads 75 / 116 us; three of 578..777 on 7000..9000, 32 heads 285 / 317 us; four
//     prompts of up to 2000, 8 heads 46 / 38 us, one of 4096, 32 heads 147 / 125 us (these run whole).
// Which CTA takes a pair never changes what is computed, and where pairs are cut depends on the lengths alone.
// A block is two query tiles s = 0, 1 of 128 rows that share the key and value tiles:
//   S_s   = Q_s K^T     M = 128, N = 128, K = 192 (two nope panels and the shared rope panel)
//   O_s  += P_s V       M = 128, N = 64 twice, K = 128, P_s in tensor memory
// Tensor memory holds S_0, S_1, O_0, O_1 (128 columns each); P_s (bf16) overlays S_s.  While the
// softmax of one tile runs, the tensor cores do the other tile's two products.  Warps: one issues the
// TMA copies, one the MMAs of each query tile; two warpgroups a query tile do the softmax (two threads a
// row) and the epilogue.
// Key and value panels (128 tokens x 64, 16 KB, 128-byte swizzle) pass through one ring of eight: per
// key tile three key panels (K-major B), then two value panels (MN-major B).
//
// The probabilities of a tile are handed to the second product in two parts, so that it runs on the first while the
// exponentials of the second are taken (16 prompts 3.80 -> 3.56 ms when it was brought in).
//
// The softmax warps' registers (104 after the split, 64 of them a row's scores) do not hold everything: 60 bytes a
// thread are spilled and 84 loaded again.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the last rescale.  The
// probabilities are rounded to bf16, the tensor cores' operand type; the output is normalised by the
// sum of the rounded weights, the log-sum-exp taken from the sum before rounding.  So each weight is off by 2^-8 at
// most, relative to the others, and the output by 2^-7 sum p |v| beside its own rounding; that takes two or three
// weights that outweigh all others and round to opposite sides, else the errors average out.  A query that sees few
// keys has no more weights than that, so for those that see one key tile nothing is left off: in the first key tile of
// a query tile whose first query sees no second one, what the rounding leaves off goes through a second product (the
// other half of S_s holds it).
// The tensor cores cut every product off at 2^-25 of the sum that it joins (the bits of a 26-bit window), so a sum of N
// may lack N 2^-25 of its size: 1.3 % after a million keys behind one that holds half of the weight.  After kSumTiles
// key tiles O, l and lr are therefore added to fp32 sums in the workspace and begin again (16,384 keys: 2^-11 at the
// most).
// A key that a query must not see enters its product with weight 0, and 0 times an infinity or NaN is not 0.
// So in the tiles that not every query of the block sees whole, values that are not finite are taken out
// (set to 0 in shared memory) before the product, and where there were any, the epilogue adds them to the
// queries that do see them.  Value rows behind the sequence's end are set to 0 likewise.
// Every wait is bounded; an expired one sets the workspace's status word (7).  A warp may wait for as long as a pair
// takes: the scheduling warp for the one before the next to be read by all, a query tile without keys for the other
// one's.  So the bound grows with the keys, a second for every 65,536 key tiles (they take 0.12 s).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "kda_common.cuh"
#include "kda_internal.h"
#include "tcgen05.cuh"

namespace kda {
namespace prefill {
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // chunk_prep.cu
}
namespace {

constexpr int DN = 128, DR = 64, DV = 128, DQ = DN + DR;
constexpr int T = 128;                     // queries and keys of a tile
constexpr int kBlock = 2 * T;              // queries of a block
constexpr int PB = T * 128;                // bytes of a panel
constexpr int kRing = 8;                   // panels in flight
constexpr int kQBytes = DQ / 64 * PB;      // of one query tile
constexpr int OFF_RING = 2 * kQBytes, OFF_SHARED = OFF_RING + kRing * PB;
constexpr int kThreads = 640;              // four service warps, two softmax warpgroups a query tile
constexpr int kServiceRegs = 64, kSoftRegs = 104;  // 128 x 64 + 512 x 104 = 61,440 = 640 x 96 registers
constexpr int kHalf = T / 2;               // keys of a softmax thread
constexpr uint32_t kColO = 256;            // S_s at 128 s, O_s at 256 + 128 s
constexpr uint32_t kWaitLimit = 0xffffffffu;  // polls: the time bounds the waits
constexpr int kTilesPerSecond = 1 << 16;
constexpr float kLazy = 8.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kStatusExpired = 7;
constexpr int kBuckets = 1024;
constexpr int kCutTiles = 10;
constexpr int kSumTiles = 128;             // key tiles that O takes before it is set aside, a power of two
constexpr int kTurnRounds = 8, kInTurn = -1;
constexpr int kMostCtas = 256;             // of the grid (one per SM)
constexpr int kFewBlocks = 32;             // up to these every CTA makes its own list
constexpr int kJoinCtas = 6;               // a SM: as many as stay resident
constexpr int kReaders = 3 + 16;           // warps that read a segment

enum Order { kHeadsFirst = 0, kTokensFirst = 1, kOneHead = 2 };  // (x, head, token), (x, token, head), (x, 0, token)

struct Params {
    LatentPrefillArgs a;
    float scale_log2;
    int32_t kn_order, v_order;  // of the map's coordinates: Order
    int32_t *status;
    int32_t *n_blocks, *whole;   // blocks listed; pairs that are taken whole (a multiple of the grid, or all), kInTurn: see Walk
    int32_t *taken;              // pairs taken in turn
    bool few;                    // at most kFewBlocks blocks, and fewer than kTurnRounds pairs a CTA: no plan_kernel
    int64_t *before;             // [max_blocks + 1] key tiles (of one head) before each block of the list, and in all
    int2 *table;                 // [max_blocks] (sequence, block of the sequence)
    int32_t *seq_off, *short_off;  // [num_seqs + 1] blocks before each sequence; of them those in the first quarter of theirs
    int64_t max_blocks;
    int32_t grid;
    uint32_t seconds;            // that a wait may take
    int32_t *item0, *item1;      // [grid] pair whose part is in slot 0 / 1 of the CTA, or -1
    float4 *ml;                  // [grid][2][256] m, l, l of the rounded weights
    float *part;                 // [grid][2][256][DV]; also what a pair sets aside: in its slot, a whole pair's in slot 1
    float4 *kept;                // [grid][512] by softmax thread: the maximum that it is relative to; l, lr set aside
};

struct Maps {
    CUtensorMap q, kn, kr, v;
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t most) { return x < 0 ? 0 : x > most ? most : x; }

// One block's sizes, from offsets held to the tensors' extents.
struct Item {
    int32_t q0, k0;        // first query row of the block, first key of the sequence
    int32_t nk, n;         // keys of the sequence; key tiles of the block
    int32_t rows0, rows1;  // valid queries of each query tile
    int32_t see0;          // keys that the block's first query sees (may be negative)
    int32_t tiles0, tiles1;

    __device__ static int32_t hold(int32_t x, int32_t most) { return x < 0 ? 0 : x > most ? most : x; }
    __device__ void load(const LatentPrefillArgs &a, int32_t b, int32_t blk)
    {
        const int32_t tq = static_cast<int32_t>(a.total_q), tk = static_cast<int32_t>(a.total_k);
        const int32_t qb = hold(a.cu_q[b], tq), qe = hold(a.cu_q[b + 1], tq), kb = hold(a.cu_k[b], tk), ke = hold(a.cu_k[b + 1], tk);
        const int32_t nq = qe > qb ? qe - qb : 0, r0 = blk * kBlock;
        nk = ke > kb ? ke - kb : 0;
        k0 = kb;
        q0 = qb + r0;
        see0 = r0 + nk - nq + 1;
        rows0 = hold(nq - r0, T);
        rows1 = hold(nq - r0 - T, T);
        tiles0 = tiles_of(see0, rows0);
        tiles1 = tiles_of(see0 + T, rows1);
        n = tiles0 > tiles1 ? tiles0 : tiles1;
    }
    // the tile's last query sees the most
    static __device__ int32_t tiles_of(int32_t see, int32_t rows) { return rows > 0 && see + rows > 1 ? (see + rows - 2) / T + 1 : 0; }
    __device__ int32_t rows(int s) const { return s ? rows1 : rows0; }
    __device__ int32_t tiles(int s) const { return s ? tiles1 : tiles0; }
    __device__ int32_t see(int s) const { return see0 + s * T; }
};

// The list of blocks, longest first: in global memory, or in a CTA's own shared memory.
struct List {
    const int2 *table;      // [blocks] (sequence, block of the sequence)
    const int64_t *before;  // [blocks + 1]
    int32_t blocks, whole;  // as n_blocks and whole of Params
};

// Pairs that are taken whole, of a list that is not taken in turn: all, or (a multiple of the grid) all but the last round's.
__device__ __forceinline__ int32_t whole_pairs(const int64_t *before, int32_t blocks, int32_t heads, int32_t grid)
{
    const int32_t items = blocks * heads, whole = items / grid * grid;
    if (whole == items) return items;
    const int32_t b = whole / heads;
    const int64_t longest = before[b + 1] - before[b];
    const int64_t rest = before[blocks] * heads - before[b] * heads - whole % heads * longest;
    return longest > rest / grid + kCutTiles ? whole : items;
}

// The work of one CTA in order: (block, head) pairs, and a stretch [j0, j1) of the key tiles of others.
struct Walk {
    int32_t round, whole;   // rounds of whole pairs taken so far; pairs that are taken whole
    bool cut;                   // the stretch is known
    int32_t next_pair, next_j;  // where it goes on
    int64_t left;               // key tiles of the stretch to come
    int32_t head, pair;
    int32_t j0, j1, slot;   // slot: where a part goes, 0 if it is not its pair's first; -1: the pair is whole
    Item it;

    __device__ void begin(const List &l) { round = 0, whole = l.whole, left = 0, cut = false; }
    // How much of the line's `all` key tiles this CTA takes, and what those before it take.
    __device__ void share(const List &l, int32_t H, int64_t all, int64_t *start)
    {
        const int32_t grid = gridDim.x, lane = threadIdx.x & 31;
        auto sum = [&](int64_t x) {
#pragma unroll
            for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            return x;
        };
        int32_t load[kMostCtas / 32];  // key tiles of CTA 32 k + lane so far; -1: none for it here
#pragma unroll
        for (int k = 0; k < kMostCtas / 32; ++k) {
            const int32_t c = 32 * k + lane;
            load[k] = c < grid ? 0 : -1;
            for (int32_t r = 0; r < whole / grid && c < grid; ++r) {
                const int32_t b = (r * grid + (r & 1 ? grid - 1 - c : c)) / H;
                load[k] += static_cast<int32_t>(l.before[b + 1] - l.before[b]);
            }
        }
        int64_t level, over;  // the sum that all are filled up to, and one more for the first `over`
        for (int32_t n_before = 0;;) {
            int64_t have = 0, n = 0;
#pragma unroll
            for (int k = 0; k < kMostCtas / 32; ++k) have += load[k] >= 0 ? load[k] : 0, n += load[k] >= 0 ? 1 : 0;
            have = sum(have), n = sum(n);
            level = (all + have) / n, over = (all + have) % n;
            if (n == n_before) break;
            n_before = static_cast<int32_t>(n);
#pragma unroll
            for (int k = 0; k < kMostCtas / 32; ++k)
                if (load[k] > level) load[k] = -1;
        }
        int64_t before = 0, mine = 0;
        int32_t rank = 0;
#pragma unroll
        for (int k = 0; k < kMostCtas / 32; ++k) {
            const uint32_t takes = __ballot_sync(0xffffffffu, load[k] >= 0);
            const int64_t x = load[k] < 0 ? 0 : level - load[k] + (rank + __popc(takes & ((1u << lane) - 1)) < over ? 1 : 0);
            rank += __popc(takes);
            if (32 * k + lane < static_cast<int32_t>(blockIdx.x)) before += x;
            if (32 * k + lane == static_cast<int32_t>(blockIdx.x)) mine = x;
        }
        *start = sum(before), left = sum(mine);
    }
    // This CTA's stretch of the line that begins with pair `whole`, by a whole warp: CTAs whose pairs were shorter take
    // more of it, so that all have the same sum of key tiles (but for those whose pairs alone are more).
    __device__ void stretch(const Params &p, const List &l)
    {
        cut = true;
        const int32_t H = p.a.h, blocks = l.blocks, items = blocks * H, grid = gridDim.x;
        if (whole >= items) return;
        const int64_t base = l.before[whole / H] * H + whole % H * (l.before[whole / H + 1] - l.before[whole / H]);
        const int64_t all = l.before[blocks] * H - base;
        int64_t w0 = 0;
        if (whole == 0) {  // no pair yet: equal stretches
            const int64_t n = all < grid ? all : grid, c = static_cast<int32_t>(blockIdx.x) < n ? blockIdx.x : n;
            w0 = all * c / n;
            left = c < n ? all * (c + 1) / n - w0 : 0;
        } else {
            share(l, H, all, &w0);
        }
        if (left == 0) return;
        int32_t lo = whole / H, hi = blocks;  // the block with before[lo] * H <= base + w0 < before[lo + 1] * H
        while (lo + 1 < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (l.before[mid] * H <= base + w0) lo = mid;
            else hi = mid;
        }
        const int64_t rest = base + w0 - l.before[lo] * H, units = l.before[lo + 1] - l.before[lo];
        next_pair = lo * H + static_cast<int32_t>(rest / units);
        next_j = static_cast<int32_t>(rest % units);
    }
    // The next pair or stretch; false: none.  By a whole warp.
    __device__ bool next(const Params &p, const List &l)
    {
        const int32_t items = l.blocks * p.a.h;  // below 2^31: checked on the host
        if (whole == kInTurn) {
            // whoever comes, in order of sequence, head and block, the longest first; the first quarter of each
            // sequence's blocks, the short ones, in a second pass that evens out the end
            pair = 0;
            if ((threadIdx.x & 31) == 0) pair = atomicAdd(p.taken, 1);
            pair = __shfl_sync(0xffffffffu, pair, 0);
            if (pair >= items) return false;
            const int32_t H = p.a.h, seqs = static_cast<int32_t>(p.a.num_seqs);
            const int32_t many = (p.seq_off[seqs] - p.short_off[seqs]) * H;
            const bool second = pair >= many;
            const int32_t at = second ? pair - many : pair;
            auto before = [&](int32_t b) { return (second ? p.short_off[b] : p.seq_off[b] - p.short_off[b]) * H; };
            int32_t lo = 0, hi = seqs;
            while (lo + 1 < hi) {
                const int32_t mid = (lo + hi) >> 1;
                if (before(mid) <= at) lo = mid;
                else hi = mid;
            }
            const int32_t in_seq = at - before(lo), n = (before(lo + 1) - before(lo)) / H;
            head = in_seq / n;
            it.load(p.a, lo, (second ? n : p.seq_off[lo + 1] - p.seq_off[lo]) - 1 - in_seq % n);
            j0 = 0, j1 = it.n, slot = -1;
            return true;
        }
        const int32_t grid = gridDim.x, at = round * grid + (round & 1 ? grid - 1 - static_cast<int32_t>(blockIdx.x) : blockIdx.x);
        const bool entire = round * grid < whole;
        if (entire) {
            ++round;
            if (at >= items) return false;  // beyond the end of a last round that runs whole
            pair = at;
        } else {
            if (!cut) stretch(p, l);
            if (left <= 0) return false;
            pair = next_pair;
        }
        head = pair % p.a.h;
        const int2 e = l.table[pair / p.a.h];
        it.load(p.a, e.x, e.y);
        j0 = 0, j1 = it.n, slot = -1;
        if (!entire) {
            const int32_t units = it.n > 0 ? it.n : 1;  // a block that sees nothing is still written
            const int32_t end = left < units - next_j ? next_j + static_cast<int32_t>(left) : units;
            if (next_j > 0 || end < units) j0 = next_j, j1 = end, slot = j0 > 0 ? 0 : 1;
            left -= end - next_j;
            next_j = 0;
            ++next_pair;
        }
        return true;
    }
    // key tiles of query tile s in this stretch
    __device__ int32_t tiles(int s) const
    {
        const int32_t t = it.tiles(s) < j1 ? it.tiles(s) : j1;
        return t > j0 ? t - j0 : 0;
    }
};

// A row that saw nothing has the sum 0: output 0, log-sum-exp -inf.  A NaN stays one.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
// What a sum relative to the maximum `from` is worth relative to `to`.
__device__ __forceinline__ float rebase(float from, float to) { return from == to ? 1.f : ex2_approx(from - to); }
__device__ __forceinline__ float log_sum(float m, float sum) { return sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2; }

__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r)::"memory");
    return r != 0;
}

// A value that is the same in all lanes, in a form in which the compiler knows it: branches and
// addresses that depend on it then stay uniform, and the MMA takes its descriptors from uniform registers
// (with descriptors from vector registers an MMA took about 100 cycles to issue).
__device__ __forceinline__ int32_t uniform(int32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

__host__ __device__ constexpr int64_t blocks_bound(int64_t total_q, int64_t num_seqs) { return total_q / kBlock + num_seqs; }

// ------------------------------------------------------------------ the plan --
// Place in the list by key tiles: the longest first (beyond kBuckets in order).
__device__ __forceinline__ int32_t bucket(int32_t n) { return n < kBuckets ? kBuckets - 1 - n : 0; }

__global__ void __launch_bounds__(1024) plan_kernel(Params p)
{
    __shared__ int32_t hist[kBuckets];
    __shared__ int64_t sums[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const LatentPrefillArgs &a = p.a;
    before_next();
    after_previous();
    auto scan = [&](int64_t x, int64_t *total) {  // exclusive prefix over the CTA
        int64_t s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        int64_t before = 0, all = 0;
        for (int w = 0; w < 32; ++w) {
            before += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        *total = all;
        return before + s - x;
    };
    if (tid == 0) *p.status = 0;
    hist[tid] = 0;
    int64_t base = 0, short_base = 0;
    for (int64_t b0 = 0; b0 < a.num_seqs; b0 += 1024) {
        const int64_t b = b0 + tid;
        int32_t nb = 0;
        if (b < a.num_seqs) {
            const int64_t n = clamp64(a.cu_q[b + 1], a.total_q) - clamp64(a.cu_q[b], a.total_q);
            nb = n > 0 ? static_cast<int32_t>((n + kBlock - 1) / kBlock) : 0;
        }
        int64_t total, shorts;
        const int64_t at = base + scan(nb, &total), short_at = short_base + scan(nb / 4, &shorts);
        if (b < a.num_seqs) p.seq_off[b] = static_cast<int32_t>(at), p.short_off[b] = static_cast<int32_t>(short_at);
        base += total;
        short_base += shorts;
    }
    // more blocks than the bound only if the offsets are not what the contract says: then nothing is done
    const int32_t blocks = static_cast<int32_t>(base <= p.max_blocks ? base : 0);
    if (tid == 0) p.seq_off[a.num_seqs] = blocks, p.short_off[a.num_seqs] = static_cast<int32_t>(short_base);
    if (tid == 0) *p.n_blocks = blocks;
    __syncthreads();
    auto locate = [&](int32_t i, int2 *e) {  // block i in order of the sequences; its key tiles
        int32_t lo = 0, hi = static_cast<int32_t>(a.num_seqs);
        while (lo + 1 < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (p.seq_off[mid] <= i) lo = mid;
            else hi = mid;
        }
        *e = make_int2(lo, i - p.seq_off[lo]);
        Item it;
        it.load(a, e->x, e->y);
        return it.n;
    };
    // counting sort by key tiles, longest first; blocks of one length stay in order, so that the list, and with it
    // the places where pairs are cut, does not depend on the order of the atomics
    int2 e;
    for (int32_t i = tid; i < blocks; i += 1024) atomicAdd(&hist[bucket(locate(i, &e))], 1);
    __syncthreads();
    int64_t total;
    const int32_t first = static_cast<int32_t>(scan(hist[tid], &total));
    __syncthreads();
    hist[tid] = first;
    __syncthreads();
    for (int32_t i0 = 0; i0 < blocks; i0 += 1024) {
        const int32_t i = i0 + tid, b = i < blocks ? bucket(locate(i, &e)) : -1;
        for (int w = 0; w < 32 && i0 + 32 * w < blocks; ++w) {  // warp after warp
            if (w == warp) {
                const uint32_t same = __match_any_sync(0xffffffffu, b);
                const int32_t rank = __popc(same & ((1u << lane) - 1));
                const int32_t at = b >= 0 ? hist[b] : 0;
                __syncwarp();
                if (b >= 0) {
                    p.table[at + rank] = e;
                    if (rank == 0) hist[b] = at + __popc(same);
                }
            }
            __syncthreads();
        }
    }
    // key tiles before each block of the list
    int64_t units = 0;
    for (int32_t i0 = 0; i0 < blocks; i0 += 1024) {
        const int32_t i = i0 + tid;
        int32_t u = 0;
        if (i < blocks) {
            const int2 b = p.table[i];
            Item it;
            it.load(a, b.x, b.y);
            u = it.n > 0 ? it.n : 1;
        }
        const int64_t at = scan(u, &total);
        if (i < blocks) p.before[i] = units + at;
        units += total;
    }
    __syncthreads();
    if (tid == 0) {
        p.before[blocks] = units;
        *p.taken = 0;
        *p.whole = blocks * a.h >= kTurnRounds * p.grid ? kInTurn : whole_pairs(p.before, blocks, a.h, p.grid);
    }
    for (int32_t c = tid; c < p.grid; c += 1024) p.item0[c] = p.item1[c] = -1;
}

// The same list of few blocks, by one warp of every CTA into its shared memory, a block a lane: a launch and its
// latency less (three prompts of up to 100 tokens, 32 heads: 17.9 -> 10.8 us; five of 201..777 on prefixes of up to
// 9000, 16 heads: 232 -> 224 us).
__device__ __forceinline__ List plan_few(const Params &p, int2 *table, int64_t *before, int32_t *units)
{
    const LatentPrefillArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    int32_t nb = 0;
    if (lane < a.num_seqs) {
        const int64_t n = clamp64(a.cu_q[lane + 1], a.total_q) - clamp64(a.cu_q[lane], a.total_q);
        nb = n > 0 ? static_cast<int32_t>((n + kBlock - 1) / kBlock) : 0;
    }
    auto scan = [&](int64_t x) {  // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    const int64_t end = scan(nb), sum = __shfl_sync(0xffffffffu, end, 31);
    const int32_t blocks = static_cast<int32_t>(sum <= p.max_blocks ? sum : 0), off = static_cast<int32_t>(end - nb);
    int32_t seq = -1, first = 0;  // the last sequence that begins at or before block `lane`
    for (int b = 0; b < a.num_seqs; ++b) {
        const int32_t at = __shfl_sync(0xffffffffu, off, b);
        if (at <= lane) seq = b, first = at;
    }
    const bool mine = lane < blocks;
    int32_t place = INT32_MAX, n = 0;
    if (mine) {
        Item it;
        it.load(a, seq, lane - first);
        n = it.n;
        place = bucket(n);
    }
    int32_t rank = 0;
    for (int b = 0; b < blocks; ++b) {
        const int32_t other = __shfl_sync(0xffffffffu, place, b);
        rank += other < place || (other == place && b < lane) ? 1 : 0;
    }
    if (mine) {
        table[rank] = make_int2(seq, lane - first);
        units[rank] = n > 0 ? n : 1;
        if (blockIdx.x == 0) p.table[rank] = make_int2(seq, lane - first);  // for the join
    }
    __syncwarp();
    const int64_t through = scan(mine ? units[lane] : 0);
    if (mine) before[lane + 1] = through;
    if (lane == 0) before[0] = 0;
    __syncwarp();
    return List{table, before, blocks, whole_pairs(before, blocks, a.h, p.grid)};
}

// ------------------------------------------------------------------ the kernel --
struct Bars {
    // by parity of the key tile: its key panels and value panels, loaded and handed back
    uint64_t k_full[2][3], k_free[2], v_full[2], v_free[2];  // k_full: by panel
    uint64_t q_full[2], q_free[2], s[2], p[2][2], o[2], drain[2];  // by query tile
    uint64_t seg_full[2], seg_free[2];
};

// A pair, or stretch of one, as the scheduling warp hands it to the others.
struct Segment {
    int32_t q0, k0, nk;         // first query row, first key of the sequence, its keys
    int32_t rows[2], tiles[2];  // by query tile: valid queries, key tiles in the stretch
    int32_t see;                // keys that the block's first query sees
    int32_t j0, j1;             // key tiles of the stretch
    int32_t slot, head, pair;   // slot: as in Walk; pair -1: no more work
    int32_t exact;              // bit s: the first key tile's weights go into query tile s with what their rounding leaves off
};

struct Shared {
    Bars bar;
    Segment seg[2];
    float pair[2][2][T];  // by query tile, half, row: what the two threads of a row tell each other
    uint32_t not_finite[2];  // by parity of the segment: its number + 1 once a value was taken out
    uint32_t tmem_base;
    List few;
    int2 few_table[kFewBlocks];
    int64_t few_before[kFewBlocks + 1];
};
constexpr int kSmem = OFF_SHARED + sizeof(Shared);
static_assert(kSmem <= 232448, "227 KB");

__global__ void __launch_bounds__(kThreads, 1) latent_prefill_kernel(Params p, const __grid_constant__ Maps maps)
{
    extern __shared__ __align__(1024) char smem[];  // all of it: nothing static stands before it
    Shared &sh = *reinterpret_cast<Shared *>(smem + OFF_SHARED);
    Bars &bar = sh.bar;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform

    if (warp == 3) {
        tc::tmem_alloc(&sh.tmem_base, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            sh.not_finite[s] = 0;
            for (int u = 0; u < 3; ++u) mbar_init(&bar.k_full[s][u], 1);
            mbar_init(&bar.v_full[s], 1);
            mbar_init(&bar.k_free[s], 2), mbar_init(&bar.v_free[s], 2);  // handed back by both query tiles
            mbar_init(&bar.drain[s], 1), mbar_init(&bar.seg_full[s], 1), mbar_init(&bar.seg_free[s], kReaders);
            mbar_init(&bar.q_full[s], 1), mbar_init(&bar.q_free[s], 1), mbar_init(&bar.s[s], 1), mbar_init(&bar.o[s], 1);
            mbar_init(&bar.p[s][0], 2 * T), mbar_init(&bar.p[s][1], 2 * T);
        }
        fence_mbar_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    before_next();
    after_previous();
    if (warp == 3 && p.few) {
        if (lane == 0) {
            p.item0[blockIdx.x] = p.item1[blockIdx.x] = -1;
            if (blockIdx.x == 0) *p.status = 0;
        }
        const List list = plan_few(p, sh.few_table, sh.few_before, reinterpret_cast<int32_t *>(sh.pair));  // not in use yet
        if (lane == 0) sh.few = list;
        __syncwarp();
    }
    const uint32_t tmem = uniform(sh.tmem_base);
    uint32_t nseg = 0;  // segments taken

    bool gave_up = false;
    auto wait = [&](uint64_t *b, uint32_t parity) {
        if (!gave_up && !mbar_wait(b, parity, kWaitLimit, p.seconds)) {
            gave_up = true;
            atomicExch(p.status, kStatusExpired);
        }
        return !gave_up;
    };
    // by a whole warp: the test that usually passes first, the bounded wait behind it
    auto all_wait = [&](uint64_t *b, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_test(b, parity))) return true;
        return __all_sync(0xffffffffu, wait(b, parity)) != 0;
    };

    // the next segment, or nullptr behind the last one; `segment_done` (by a whole warp) gives it back
    auto next_segment = [&]() -> const Segment * {
        if (!all_wait(&bar.seg_full[nseg & 1], nseg >> 1 & 1)) return nullptr;
        const Segment *g = &sh.seg[nseg & 1];
        return uniform(g->pair) < 0 ? nullptr : g;
    };
    auto segment_done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.seg_free[nseg & 1]);
        ++nseg;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kServiceRegs) : "memory");
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            uint32_t g = 0, loads0 = 0, loads1 = 0;  // key tiles, query tiles so far
            auto query = [&](const Segment &w, int s, uint32_t &loads) {
                if (w.tiles[s] == 0) return true;
                if (loads > 0 && !all_wait(&bar.q_free[s], (loads - 1) & 1)) return false;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&bar.q_full[s], kQBytes);
#pragma unroll
                    for (int u = 0; u < DQ / 64; ++u)
                        tma_load_3d(smem + s * kQBytes + u * PB, &maps.q, 64 * u, w.head, w.q0 + s * T, &bar.q_full[s]);
                }
                __syncwarp();
                ++loads;
                return true;
            };
            bool ok = true;
            while (const Segment *seg = ok ? next_segment() : nullptr) {
                const Segment &w = *seg;
                if (!(ok = query(w, 0, loads0))) break;
                const int head = w.head, j0 = w.j0, j1 = w.j1, first_key = w.k0;
                for (int32_t j = j0; j < j1; ++j, ++g) {
                    // panel i of tile g lies in slot (5 g + i) % 8: its first key panel where tile g - 2's last one was (waited
                    // for with tile g - 1's values), the others where tile g - 2's values were, its values where tile g - 1's
                    // first keys were
                    const int tok = first_key + j * T;
                    char *const ring = smem + OFF_RING;
                    const int kn_y = p.kn_order == kTokensFirst ? tok : p.kn_order == kOneHead ? 0 : head;
                    const int kn_z = p.kn_order == kTokensFirst ? head : tok;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&bar.k_full[g & 1][0], PB);
                        tma_load_3d(ring + 5 * g % kRing * PB, &maps.kn, 0, kn_y, kn_z, &bar.k_full[g & 1][0]);
                    }
                    __syncwarp();
                    if (g > 1 && !(ok = all_wait(&bar.v_free[g & 1], ((g >> 1) & 1) ^ 1))) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&bar.k_full[g & 1][1], PB);
                        tma_load_3d(ring + (5 * g + 1) % kRing * PB, &maps.kn, 64, kn_y, kn_z, &bar.k_full[g & 1][1]);
                        mbar_arrive_expect_tx(&bar.k_full[g & 1][2], PB);
                        tma_load_3d(ring + (5 * g + 2) % kRing * PB, &maps.kr, 0, 0, tok, &bar.k_full[g & 1][2]);
                    }
                    __syncwarp();
                    if (j == j0 && !(ok = query(w, 1, loads1))) break;
                    if (g > 0 && !(ok = all_wait(&bar.k_free[(g - 1) & 1], (g - 1) >> 1 & 1))) break;
                    if (elect_one()) {
                        const int order = p.v_order, y = order == kTokensFirst ? tok : order == kOneHead ? 0 : head;
                        const int z = order == kTokensFirst ? head : tok;
                        mbar_arrive_expect_tx(&bar.v_full[g & 1], 2 * PB);
                        tma_load_3d(ring + (5 * g + 3) % kRing * PB, &maps.v, 0, y, z, &bar.v_full[g & 1]);
                        tma_load_3d(ring + (5 * g + 4) % kRing * PB, &maps.v, 64, y, z, &bar.v_full[g & 1]);
                    }
                    __syncwarp();
                }
                segment_done();
            }
            if (!ok) {  // gave up: the copies in flight land before the CTA ends
                // what tile g has under way is not told apart: a wait for what was not begun runs out, bounded like the others
                for (uint32_t e = g > 0 ? g - 1 : 0; e <= g; ++e) {
                    for (int u = 0; u < 3; ++u) mbar_wait(&bar.k_full[e & 1][u], e >> 1 & 1, kWaitLimit);
                    mbar_wait(&bar.v_full[e & 1], e >> 1 & 1, kWaitLimit);
                }
                if (loads0 > 0) mbar_wait(&bar.q_full[0], (loads0 - 1) & 1, kWaitLimit);
                if (loads1 > 0) mbar_wait(&bar.q_full[1], (loads1 - 1) & 1, kWaitLimit);
            }
        } else if (warp < 3) {
            // -------------------------------------------- MMAs of query tile s
            // One warp a query tile: while one waits, looks at barriers or forms descriptors, the other's products run (with
            // one warp for both the tensor pipe idled a third of the time behind its serial code).
            const int s = warp - 1;
            constexpr uint32_t kIdS = tc::idesc_bf16(T, T, false), kIdO = tc::idesc_bf16(T, 64, true);
            const uint32_t base = smem_u32(smem), ts = tmem + 128 * s, to = tmem + kColO + 128 * s;
            const uint64_t q_desc = tc::sdesc_sw128(base + s * kQBytes, 16, 1024), ring_desc = tc::sdesc_sw128(base + OFF_RING, 16, 1024);
            uint32_t g = 0, loads = 0, pvs = 0;  // key tiles, query tiles, second products so far
            // panel u of S of key tile g (by one lane)
            auto panel = [&](uint32_t g, int u) {
                const uint64_t a = q_desc + (u * PB >> 4), b = ring_desc + (5 * g + u) % kRing * (PB >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) tc::mma_bf16(ts, a + 2 * ks, b + 2 * ks, kIdS, u > 0 || ks > 0 ? 1u : 0u);
            };
            auto first_done = [&](uint32_t g, bool free_q) {
                tc::commit(&bar.s[s]);
                tc::commit(&bar.k_free[g & 1]);
                if (free_q) tc::commit(&bar.q_free[s]);
            };
            // S of key tile g, panel by panel as they arrive
            auto first = [&](uint32_t g, bool free_q) {
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                    if (!all_wait(&bar.k_full[g & 1][u], g >> 1 & 1)) return false;
                    if (elect_one()) {
                        panel(g, u);
                        if (u == 2) first_done(g, free_q);
                    }
                    __syncwarp();
                }
                return true;
            };
            // O += P V of key tile g and, behind it, S of key tile g + 1 (more).  A look at a barrier costs its time even
            // where the barrier is long open, and behind the product it would leave the tensor pipe idle: so the
            // key panels are looked at before the wait for P, and S follows at once where they are there.
            auto second = [&](uint32_t g, bool fresh, bool exact, bool more, bool free_q) {
                const uint64_t b0 = ring_desc + (5 * g + 3) % kRing * (PB >> 4), b1 = ring_desc + (5 * g + 4) % kRing * (PB >> 4);
                if (!all_wait(&bar.v_full[g & 1], g >> 1 & 1)) return false;
                const uint32_t n = g + 1, par = n >> 1 & 1;
                const bool there = more && __all_sync(0xffffffffu, mbar_test(&bar.k_full[n & 1][0], par) &&
                                                                      mbar_test(&bar.k_full[n & 1][1], par) &&
                                                                      mbar_test(&bar.k_full[n & 1][2], par));
                // P comes in two parts: the first half of each thread's keys, then the second
                if (!all_wait(&bar.p[s][0], pvs & 1)) return false;
                tc::fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ks = 4 * (i >> 1) + (i & 1);
                        tc::mma_bf16_ts(to, ts + 8 * ks, b0 + 128 * ks, kIdO, i > 0 || !fresh ? 1u : 0u);
                        tc::mma_bf16_ts(to + 64, ts + 8 * ks, b1 + 128 * ks, kIdO, i > 0 || !fresh ? 1u : 0u);
                    }
                }
                __syncwarp();
                if (!all_wait(&bar.p[s][1], pvs++ & 1)) return false;
                tc::fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ks = 4 * (i >> 1) + (i & 1) + 2;
                        tc::mma_bf16_ts(to, ts + 8 * ks, b0 + 128 * ks, kIdO, 1u);
                        tc::mma_bf16_ts(to + 64, ts + 8 * ks, b1 + 128 * ks, kIdO, 1u);
                    }
                    if (exact) {  // what the rounding left off, too
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            tc::mma_bf16_ts(to, ts + 64 + 8 * ks, b0 + 128 * ks, kIdO, 1u);
                            tc::mma_bf16_ts(to + 64, ts + 64 + 8 * ks, b1 + 128 * ks, kIdO, 1u);
                        }
                    }
                    tc::commit(&bar.o[s]);
                    tc::commit(&bar.v_free[g & 1]);
                    if (there) {
                        panel(n, 0);
                        panel(n, 1);
                        panel(n, 2);
                        first_done(n, free_q);
                    }
                }
                __syncwarp();
                return !more || there || first(n, free_q);
            };
            bool ok = true;
            while (const Segment *seg = ok ? next_segment() : nullptr) {
                const int nt = uniform(seg->tiles[s]), n = uniform(seg->j1 - seg->j0);
                const bool exact = (uniform(seg->exact) >> s & 1) != 0;
                segment_done();
                if (nt > 0) {
                    if (!(ok = all_wait(&bar.q_full[s], loads++ & 1))) break;
                    tc::fence_after_sync();
                    if (!(ok = first(g, nt == 1))) break;
                }
                for (int j = 0; j < n; ++j, ++g) {
                    if (j < nt) {
                        if (!(ok = second(g, (j & (kSumTiles - 1)) == 0, exact && j == 0, j + 1 < nt, j + 2 == nt))) break;
                    } else {  // the other query tile's alone: handed back once it is there (then the tile two before is)
                        if (!(ok = all_wait(&bar.k_full[g & 1][0], g >> 1 & 1))) break;
                        if (lane == 0) mbar_arrive(&bar.k_free[g & 1]);
                        if (!(ok = all_wait(&bar.v_full[g & 1], g >> 1 & 1))) break;
                        if (lane == 0) mbar_arrive(&bar.v_free[g & 1]);
                        __syncwarp();
                    }
                }
            }
            if (elect_one()) tc::commit(&bar.drain[s]);  // everything issued has completed before tensor memory is given back
            mbar_wait(&bar.drain[s], 0, kWaitLimit);
        } else {
            // -------------------------------------------------------- scheduling
            List list{p.table, p.before, 0, 0};
            if (p.few) list = sh.few;
            else list.blocks = *p.n_blocks, list.whole = *p.whole;
            Walk w;
            w.begin(list);
            for (bool more = true; more; ++nseg) {
                more = w.next(p, list);
                if (nseg > 1 && !all_wait(&bar.seg_free[nseg & 1], ((nseg >> 1) & 1) ^ 1)) break;
                if (lane == 0) {
                    Segment &g = sh.seg[nseg & 1];
                    g.pair = -1;
                    if (more) {
                        g.q0 = w.it.q0, g.k0 = w.it.k0, g.nk = w.it.nk, g.see = w.it.see0;
                        g.rows[0] = w.it.rows0, g.rows[1] = w.it.rows1, g.tiles[0] = w.tiles(0), g.tiles[1] = w.tiles(1);
                        g.j0 = w.j0, g.j1 = w.j1, g.slot = w.slot, g.head = w.head, g.pair = w.pair;
                        g.exact = w.j0 > 0 ? 0 : (w.it.see(0) <= T ? 1 : 0) | (w.it.see(1) <= T ? 2 : 0);
                    }
                    mbar_arrive(&bar.seg_full[nseg & 1]);
                }
                __syncwarp();
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs) : "memory");
        // ------------------------------------------------------- softmax, epilogue
        // Two threads a row: thread `half` has 64 of a tile's 128 keys and 64 of the output's 128 columns.
        const int s = warp >= 12 ? 1 : 0, half = (warp >> 2) - 1 - 2 * s, row = tid & 127;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t ts = tl + 128 * s, to = tl + kColO + 128 * s + kHalf * half;
        const int pair_bar = 1 + 4 * s + (warp & 3);  // the two warps of the same rows
        auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;\n" ::"r"(pair_bar) : "memory"); };
        auto pair_any = [&](bool v) {
            uint32_t r;
            asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                         : "=r"(r)
                         : "r"(v ? 1u : 0u), "r"(pair_bar)
                         : "memory");
            return r != 0;
        };
        uint32_t g0 = 0, steps = 0;  // key tiles of the segments before; key tiles so far (of this query tile)
        // A thread that gave up goes on without waiting, so that the two warps of a row meet at every barrier, and
        // both leave at the next segment.
        while (true) {
            const Segment *seg = next_segment();
            if (pair_any(gave_up) || seg == nullptr) break;
            // a row's 64 scores fill the registers: what is not needed for each tile stays in the segment
            const int32_t nt = seg->tiles[s];
            // keys seen; no query: no mask to pay for
            const int32_t limit = row < seg->rows[s] ? seg->see + s * T + row - seg->j0 * T : INT32_MAX / 2;
            const bool exact = (seg->exact >> s & 1) != 0;
            float m = -INFINITY, l = 0.f, lr = 0.f;  // l, lr: of this thread's keys
            // O, l and lr join what was set aside (`begun`: something was), and come back as the whole (`back`)
            auto set_aside = [&](bool begun, bool back) {
                wait(&bar.o[s], (steps - 1) & 1);
                tc::fence_after_sync();
                float4 *const kept = p.kept + static_cast<int64_t>(blockIdx.x) * (4 * T) + (tid - T);
                float4 k = make_float4(m, 0.f, 0.f, 0.f);
                if (begun) k = *kept;
                const float f = rebase(k.x, m);
                l = fmaf(k.y, f, l), lr = fmaf(k.z, f, lr);
                if (!back) {
                    *kept = make_float4(m, l, lr, 0.f);
                    l = lr = 0.f;
                }
                const int64_t sums_row = (2 * static_cast<int64_t>(blockIdx.x) + (seg->slot != 0 ? 1 : 0)) * kBlock + s * T + row;
                float4 *sums = reinterpret_cast<float4 *>(p.part + sums_row * DV + kHalf * half);  // of this thread's columns
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 16, sums += 4) {
                    uint32_t o[16];
                    tc::ld16(to + c, o);
                    tc::wait_ld();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (begun) x = sums[q];
                        x = make_float4(fmaf(x.x, f, __uint_as_float(o[4 * q])), fmaf(x.y, f, __uint_as_float(o[4 * q + 1])),
                                        fmaf(x.z, f, __uint_as_float(o[4 * q + 2])), fmaf(x.w, f, __uint_as_float(o[4 * q + 3])));
                        if (!back) sums[q] = x;
                        o[4 * q] = __float_as_uint(x.x), o[4 * q + 1] = __float_as_uint(x.y);
                        o[4 * q + 2] = __float_as_uint(x.z), o[4 * q + 3] = __float_as_uint(x.w);
                    }
                    if (back) tc::st16(to + c, o);
                }
                tc::wait_st();
            };
            for (int32_t j = 0; j < nt; ++j, ++steps) {
                if (j > 0 && (j & (kSumTiles - 1)) == 0) set_aside(j > kSumTiles, false);  // the next product does not add to O
                wait(&bar.s[s], steps & 1);
                tc::fence_after_sync();
                float z[kHalf];
                tc::ld32(ts + kHalf * half, *reinterpret_cast<uint32_t (*)[32]>(&z[0]));
                tc::ld32(ts + kHalf * half + 32, *reinterpret_cast<uint32_t (*)[32]>(&z[32]));
                tc::wait_ld();
                const int32_t left = limit - j * T - kHalf * half;  // of this thread's keys, those before `left`
                if (__any_sync(0xffffffffu, left < kHalf)) {
#pragma unroll
                    for (int c = 0; c < kHalf; ++c) z[c] = c < left ? z[c] : -INFINITY;
                }
                float mx = z[0];
#pragma unroll
                for (int c = 1; c + 1 < kHalf; c += 2) mx = fmaxf(mx, fmaxf(z[c], z[c + 1]));
                mx = fmaxf(mx, z[kHalf - 1]);
                sh.pair[s][half][row] = mx;
                tc::fence_before_sync();
                pair_sync();  // both have read their scores, too: P may overwrite them
                tc::fence_after_sync();
                mx = fmaxf(mx, sh.pair[s][half ^ 1][row]) * p.scale_log2;
                const bool grew = mx > m + kLazy && m > -INFINITY;
                if (__any_sync(0xffffffffu, grew)) {
                    const float f = grew ? ex2_approx(m - mx) : 1.f;
                    l *= f;
                    lr *= f;
                    wait(&bar.o[s], (steps - 1) & 1);  // grew only behind the first tile of the item
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < kHalf; c += 16) {
                        uint32_t o[16];
                        tc::ld16(to + c, o);
                        tc::wait_ld();
#pragma unroll
                        for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
                        tc::st16(to + c, o);
                    }
                }
                if (grew || m == -INFINITY) m = mx;
                const float base = m == -INFINITY ? 0.f : m;
                const float2 sc = make_float2(p.scale_log2, p.scale_log2), nb = make_float2(-base, -base);
                // a tile that the block's first query does not see whole: its values are looked at before the product
                const bool look = (seg->j0 + j + 1) * T > seg->see;
                // scores -> probabilities, rounded, into S_s
                float2 sum = make_float2(0.f, 0.f), sum_r = make_float2(0.f, 0.f);
                if (!exact || j > 0) {
#pragma unroll
                    for (int c = 0; c < kHalf / 2; c += 16) {
                        uint32_t pk[16];
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            float2 x = fma2(make_float2(z[2 * (c + q)], z[2 * (c + q) + 1]), sc, nb);
                            x.x = ex2_approx(x.x);
                            x.y = ex2_approx(x.y);
                            sum = add2(sum, x);
                            pk[q] = pack_bf16x2(x.x, x.y);
                            sum_r = add2(sum_r, make_float2(bf16_lo(pk[q]), bf16_hi(pk[q])));
                        }
                        tc::st16(ts + kHalf / 2 * half + c, pk);
                        tc::wait_st();
                        tc::fence_before_sync();
                        if (!look) mbar_arrive(&bar.p[s][c >> 4]);
                    }
                } else {  // what the rounding leaves off goes into the other half of S_s
#pragma unroll
                    for (int c = 0; c < kHalf / 2; c += 16) {
                        uint32_t hi[16], low[16];
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            float2 x = fma2(make_float2(z[2 * (c + q)], z[2 * (c + q) + 1]), sc, nb);
                            x.x = ex2_approx(x.x);
                            x.y = ex2_approx(x.y);
                            sum = add2(sum, x);
                            hi[q] = pack_bf16x2(x.x, x.y);
                            low[q] = pack_bf16x2(x.x - bf16_lo(hi[q]), x.y - bf16_hi(hi[q]));
                        }
                        tc::st16(ts + kHalf / 2 * half + c, hi);
                        tc::st16(ts + 64 + kHalf / 2 * half + c, low);
                    }
                    sum_r = sum;
                    tc::wait_st();
                    tc::fence_before_sync();
                    if (!look) mbar_arrive(&bar.p[s][0]), mbar_arrive(&bar.p[s][1]);
                }
                // Behind the exponentials, which need no values, and with a multiply-add for two of them: 8192 queries, 2 heads
                // took 73 us without a look, 83 with each value compared before the exponentials, and take 76.
                if (look) {
                    const uint32_t g = g0 + j;
                    wait(&bar.v_full[g & 1], g >> 1 & 1);
                    char *v = smem + OFF_RING + (5 * g + 3 + half) % kRing * PB;
                    // rows behind the sequence's last key: whatever they hold must not meet P = 0 (every softmax thread of
                    // the tile writes its share of these zeros for its own product; a second time they change nothing)
                    const int32_t keys = seg->nk - (seg->j0 + j) * T;
                    auto at = [&](int q) { return reinterpret_cast<uint4 *>(v + row * 128 + ((q + row) & 7) * 16); };  // eight rows start in eight banks
                    if (row >= keys) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) *at(q) = make_uint4(0u, 0u, 0u, 0u);
                    } else {
                        uint32_t zero = 0u;  // a sum of 0 x values: no number once one of them is not finite
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint4 u = *at(q);
                            zero = fma_bf16x2(u.x, 0u, fma_bf16x2(u.y, 0u, fma_bf16x2(u.z, 0u, fma_bf16x2(u.w, 0u, zero))));
                        }
                        if (bf16x2_not_finite(zero)) {
                            sh.not_finite[nseg & 1] = nseg + 1;
                            __threadfence_block();  // who finds the zeros finds the mark, too
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
                                const uint4 u = *at(q);
                                *at(q) = make_uint4(u.x & ~bf16x2_not_finite(u.x), u.y & ~bf16x2_not_finite(u.y), u.z & ~bf16x2_not_finite(u.z),
                                                    u.w & ~bf16x2_not_finite(u.w));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&bar.p[s][0]);
                    mbar_arrive(&bar.p[s][1]);
                }
                l += sum.x + sum.y;
                lr += sum_r.x + sum_r.y;
            }
            if (nt > kSumTiles) set_aside(true, true);
            pair_sync();  // the maxima have been read
            sh.pair[s][half][row] = l;
            pair_sync();
            l += sh.pair[s][half ^ 1][row];
            pair_sync();
            sh.pair[s][half][row] = lr;
            pair_sync();
            lr += sh.pair[s][half ^ 1][row];
            const int32_t slot = seg->slot;
            const int64_t out_row = static_cast<int64_t>(seg->q0 + s * T + row) * p.a.h + seg->head;
            const int64_t part_row = (2 * static_cast<int64_t>(blockIdx.x) + slot) * kBlock + s * T + row;
            const bool valid = row < seg->rows[s];
            if (nt > 0) {
                wait(&bar.o[s], (steps - 1) & 1);
                tc::fence_after_sync();
            }
            const float inv = inverse(lr);
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.a.out) + out_row * DV + kHalf * half);
            const bool taken = nt > 0 && *static_cast<volatile uint32_t *>(&sh.not_finite[nseg & 1]) == nseg + 1;
#pragma unroll
            for (int c = 0; c < kHalf; c += 16) {
                uint32_t o[16];
                if (nt > 0) {
                    tc::ld16(to + c, o);
                    tc::wait_ld();
                }
                if (taken && valid) {  // values that were taken out, to the queries that see them
                    int32_t key = seg->see / T * T;
                    if (key < seg->j0 * T) key = seg->j0 * T;
                    const int32_t end = min(limit + seg->j0 * T, (seg->j0 + nt) * T);
                    for (; key < end; ++key) {
                        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.a.v) + (seg->k0 + static_cast<int64_t>(key)) * p.a.v_token +
                                                 seg->head * p.a.v_head + kHalf * half + c;
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float x = __bfloat162float(v[q]);
                            if (!isfinite(x)) o[q] = __float_as_uint(__uint_as_float(o[q]) + x);
                        }
                    }
                }
                if (slot >= 0) {  // a part: as it is
                    if (nt > 0 && valid) {
                        uint4 *part = reinterpret_cast<uint4 *>(p.part + part_row * DV + kHalf * half + c);
#pragma unroll
                        for (int q = 0; q < 4; ++q) part[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                    }
                } else if (valid) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t v[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            v[r] = lr == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[8 * q + 2 * r]) * inv, __uint_as_float(o[8 * q + 2 * r + 1]) * inv);
                        out[c / 8 + q] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            tc::fence_before_sync();
            if (half == 0 && slot >= 0) {
                p.ml[part_row] = make_float4(m, l, lr, 0.f);
                if (row == 0 && s == 0) (slot ? p.item1 : p.item0)[blockIdx.x] = seg->pair;
            } else if (half == 0 && valid && p.a.lse != nullptr) {
                p.a.lse[out_row] = log_sum(m, l);
            }
            pair_sync();  // the sums have been read
            g0 += seg->j1 - seg->j0;
            segment_done();
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 3) tc::tmem_dealloc(tmem, 512);
}

// Joins the parts of the pairs that fell into several stretches: a pair's first part is in slot 1 of some CTA's
// slots, the next ones are in slot 0 of the CTAs behind.  Every warp lists those pairs by a look at one word a CTA
// and takes every n-th (pair, row) of n warps, four columns a lane.
__global__ void __launch_bounds__(256) join_kernel(Params p)
{
    extern __shared__ int32_t heads[];  // [grid]
    __shared__ int32_t listed;
    const int lane = threadIdx.x & 31;
    before_next();
    after_previous();
    if (threadIdx.x < 32) {
        int32_t n = 0;
        for (int32_t j0 = 0; j0 < p.grid; j0 += 32) {
            const bool has = j0 + lane < p.grid && p.item1[j0 + lane] >= 0;
            const uint32_t all = __ballot_sync(0xffffffffu, has);
            if (has) heads[n + __popc(all & ((1u << lane) - 1))] = j0 + lane;
            n += __popc(all);
        }
        if (lane == 0) listed = n;
    }
    __syncthreads();
    for (int32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5); unit < listed * kBlock; unit += gridDim.x * 8) {
        const int c = heads[unit / kBlock], row = unit % kBlock;
        const int32_t pair = p.item1[c];
        const int2 e = p.table[pair / p.a.h];
        Item it;
        it.load(p.a, e.x, e.y);
        if ((row & (T - 1)) >= it.rows(row / T)) continue;
        int32_t last = c;  // CTAs between that took nothing hold other numbers
        for (int32_t j0 = c + 1; j0 < p.grid; j0 += 32) {
            const uint32_t mine = __ballot_sync(0xffffffffu, j0 + lane < p.grid && p.item0[j0 + lane] == pair);
            if (mine != 0) last = j0 + 31 - __clz(mine);
        }
        auto at = [&](int32_t j) { return (2 * static_cast<int64_t>(j) + (j == c ? 1 : 0)) * kBlock + row; };
        float m = -INFINITY, l = 0.f, lr = 0.f;
        for (int32_t j = c + lane; j <= last; j += 32) {
            const float x = p.ml[at(j)].x;
            if (j == c || p.item0[j] == pair) m = fmaxf(m, x);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int32_t j = c; j <= last; ++j) {
            const int32_t of = p.item0[j];
            const float4 ml = p.ml[at(j)];
            const float4 x = *reinterpret_cast<const float4 *>(p.part + at(j) * DV + 4 * lane);
            // not a part of this pair, or one in which the row saw nothing (and whose row may not be written)
            if ((j != c && of != pair) || ml.y == 0.f) continue;
            const float f = ex2_approx(ml.x - (m == -INFINITY ? 0.f : m));
            l += f * ml.y;
            lr += f * ml.z;
            o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
        }
        const float inv = inverse(lr);
        const int64_t out_row = static_cast<int64_t>(it.q0 + row) * p.a.h + pair % p.a.h;
        uint2 v = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.a.out) + out_row * DV)[lane] = v;
        if (lane == 0 && p.a.lse != nullptr) p.a.lse[out_row] = log_sum(m, l);
    }
}

// Boxes of 64 columns x 128 tokens of a bf16 [tokens][heads][cols] tensor (strides in elements), 128-byte
// swizzle, zeros outside.  Of heads and tokens the one with the smaller stride comes first; heads that
// share their rows (stride 0) are one head.
bool encode(CUtensorMap *m, const void *base, int64_t cols, int64_t heads, int64_t tokens, int64_t s_head, int64_t s_token,
            int32_t *order)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = prefill::tensor_map_encoder();
    if (fn == nullptr) return false;
    if (heads == 1 || s_head == 0) heads = 1, s_head = cols;  // a stride of a size-one dimension means nothing
    if (tokens == 1) s_token = heads * s_head;
    const bool tf = s_head > s_token;
    *order = heads == 1 ? kOneHead : tf ? kTokensFirst : kHeadsFirst;
    const bool swap = *order == kTokensFirst;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(swap ? tokens : heads),
                                static_cast<cuuint64_t>(swap ? heads : tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(swap ? s_token : s_head) * 2, static_cast<cuuint64_t>(swap ? s_head : s_token) * 2};
    const cuuint32_t box[3] = {64, swap ? static_cast<cuuint32_t>(T) : 1u, swap ? 1u : static_cast<cuuint32_t>(T)}, elem[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace {
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// [status and counts | blocks | offsets | who holds parts | their statistics | parts | maxima and sums set aside]; returns
// the size.
size_t layout(char *ws, int64_t total_q, int64_t num_seqs, Params *p)
{
    const size_t n = static_cast<size_t>(blocks_bound(total_q, num_seqs)), grid = static_cast<size_t>(sm_count() < kMostCtas ? sm_count() : kMostCtas);
    const size_t before = 256, table = before + (n + 1) * 8, seq = table + n * 8, items = up256(seq + (num_seqs + 1) * 8);
    const size_t ml = up256(items + 8 * grid), part = ml + 2 * grid * kBlock * 16, kept = part + 2 * grid * kBlock * DV * 4;
    const size_t end = kept + grid * 4 * T * 16;
    if (p != nullptr) {
        p->max_blocks = static_cast<int64_t>(n);
        p->grid = static_cast<int32_t>(grid);
        p->status = reinterpret_cast<int32_t *>(ws);
        p->n_blocks = p->status + 1;
        p->whole = p->status + 2;
        p->taken = p->status + 3;
        p->before = reinterpret_cast<int64_t *>(ws + before);
        p->table = reinterpret_cast<int2 *>(ws + table);
        p->seq_off = reinterpret_cast<int32_t *>(ws + seq);
        p->short_off = p->seq_off + num_seqs + 1;
        p->item0 = reinterpret_cast<int32_t *>(ws + items);
        p->item1 = p->item0 + grid;
        p->ml = reinterpret_cast<float4 *>(ws + ml);
        p->part = reinterpret_cast<float *>(ws + part);
        p->kept = reinterpret_cast<float4 *>(ws + kept);
    }
    return end;
}
}  // namespace

size_t latent_prefill_workspace(int64_t total_q, int64_t num_seqs, int32_t) { return layout(nullptr, total_q, num_seqs, nullptr); }

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t st)
{
    Params p{};
    p.a = a;
    p.scale_log2 = a.scale * kLog2e;
    p.seconds = 1 + static_cast<uint32_t>(a.total_k / (static_cast<int64_t>(kTilesPerSecond) * T));
    layout(static_cast<char *>(a.workspace), a.total_q, a.num_seqs, &p);
    Maps maps{};
    int32_t plain;  // q's heads lie within a token (or there is one), k_rope has one
    if (!encode(&maps.q, a.q, DQ, a.h, a.total_q, DQ, static_cast<int64_t>(a.h) * DQ, &plain)) return cudaErrorInvalidValue;
    if (a.total_k > 0 && (!encode(&maps.kn, a.k_nope, DN, a.h, a.total_k, a.kn_head, a.kn_token, &p.kn_order) ||
                          !encode(&maps.v, a.v, DV, a.h, a.total_k, a.v_head, a.v_token, &p.v_order) ||
                          !encode(&maps.kr, a.k_rope, DR, 1, a.total_k, DR, a.kr_token, &plain)))
        return cudaErrorInvalidValue;
    // all three keep one split between shared memory and L1 cache: changing it between kernels costs microseconds
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(join_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
        return e;
    p.few = p.max_blocks <= kFewBlocks && p.max_blocks * a.h < static_cast<int64_t>(kTurnRounds) * p.grid;
    if (!p.few && (e = launch_overlapped(plan_kernel, dim3(1), dim3(1024), 0, st, p)) != cudaSuccess) return e;
    e = cudaFuncSetAttribute(latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    // the register split (setmaxnreg) needs a launch with exactly 96 registers a thread
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, latent_prefill_kernel)) != cudaSuccess) return e;
    if (at.numRegs != 96) return cudaErrorInvalidConfiguration;
    if ((e = launch_overlapped(latent_prefill_kernel, dim3(p.grid), dim3(kThreads), kSmem, st, p, maps)) != cudaSuccess) return e;
    if (a.total_k <= kCutTiles * T) return cudaSuccess;  // no pair is long enough to be cut
    return launch_overlapped(join_kernel, dim3(p.grid * kJoinCtas), dim3(256), static_cast<size_t>(p.grid) * 4, st, p);
}

}  // namespace kda
