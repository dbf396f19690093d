// Expanded latent attention over a varlen batch (kda_latent_prefill).
//
//   S = scale (Q_nope K_nope^T + Q_rope K_rope^T),  P = e^{S - m},  out = P V / l
// per sequence and head, causal with the queries at the end of the keys, the keys visited in tiles
// of 128 with a running maximum m and sum l a row.
//
// plan_kernel (one CTA) lists the query blocks (256 queries of one sequence), longest first by the
// key tiles they see.  One persistent CTA per SM then takes every grid-th (block, head) pair of the
// list.  A block is two query tiles s = 0, 1 of 128 rows that share the key and value tiles:
//   S_s   = Q_s K^T     M = 128, N = 128, K = 192 (two nope panels and the shared rope panel)
//   O_s  += P_s V       M = 128, N = 64 twice, K = 128, P_s in tensor memory
// Tensor memory holds S_0, S_1, O_0, O_1 (128 columns each); P_s (bf16) overlays S_s.  While the
// softmax of one tile runs, the tensor cores do the other tile's two products.  Warps: one issues the
// TMA copies, one the MMAs of each query tile, two warpgroups do the softmax (one row a thread) and the epilogues.
// Key and value panels (128 tokens x 64, 16 KB, 128-byte swizzle) pass through one ring of eight: per
// key tile three key panels (K-major B), then two value panels (MN-major B).  The probabilities are
// handed over in two halves, and the sums are formed behind them, so that they are off the path from
// S_s to O_s.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the last rescale.  The
// probabilities are rounded to bf16, the tensor cores' operand type; the output is normalised by the
// sum of the rounded weights, the log-sum-exp taken from the sum before rounding.  A query tile that
// sees a single key tile has few weights to average the rounding over, so there what the rounding
// left off goes through a second product (the other half of S_s holds it).
// Every wait is bounded; an expired one sets the workspace's status word (7).
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
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kLazy = 8.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kStatusExpired = 7;
constexpr int kBuckets = 1024;

enum Order { kHeadsFirst = 0, kTokensFirst = 1, kOneHead = 2 };  // (x, head, token), (x, token, head), (x, 0, token)

struct Params {
    LatentPrefillArgs a;
    float scale_log2;
    int32_t kn_order, v_order;  // of the map's coordinates: Order
    int32_t *status, *n_blocks;
    int2 *table;         // [max_blocks] (sequence, block of the sequence)
    int32_t *seq_off;    // [num_seqs + 1] blocks before each sequence
    int64_t max_blocks;
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
__global__ void __launch_bounds__(1024) plan_kernel(Params p)
{
    __shared__ int32_t hist[kBuckets], sums[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const LatentPrefillArgs &a = p.a;
    auto scan = [&](int32_t x, int32_t *total) {  // exclusive prefix over the CTA
        int32_t s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        int32_t before = 0, all = 0;
        for (int w = 0; w < 32; ++w) {
            before += w < warp ? sums[w] : 0;
            all += sums[w];
        }
        *total = all;
        return before + s - x;
    };
    if (tid == 0) *p.status = 0;
    hist[tid] = 0;
    int32_t base = 0;
    for (int64_t b0 = 0; b0 < a.num_seqs; b0 += 1024) {
        const int64_t b = b0 + tid;
        int32_t nb = 0;
        if (b < a.num_seqs) {
            const int64_t n = clamp64(a.cu_q[b + 1], a.total_q) - clamp64(a.cu_q[b], a.total_q);
            nb = n > 0 ? static_cast<int32_t>((n + kBlock - 1) / kBlock) : 0;
        }
        int32_t total;
        const int32_t at = base + scan(nb, &total);
        if (b < a.num_seqs) p.seq_off[b] = at;
        base += total;
    }
    // more blocks than the bound only if the offsets are not what the contract says
    const int32_t blocks = base < p.max_blocks ? base : static_cast<int32_t>(p.max_blocks);
    if (tid == 0) *p.n_blocks = blocks;
    __syncthreads();
    auto locate = [&](int32_t i, int2 *e) {
        int64_t lo = 0, hi = a.num_seqs;
        while (lo + 1 < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (p.seq_off[mid] <= i) lo = mid;
            else hi = mid;
        }
        *e = make_int2(static_cast<int>(lo), i - p.seq_off[lo]);
        Item it;
        it.load(a, e->x, e->y);
        return it.n < kBuckets ? kBuckets - 1 - it.n : 0;  // longest first
    };
    int2 e;
    for (int32_t i = tid; i < blocks; i += 1024) atomicAdd(&hist[locate(i, &e)], 1);
    __syncthreads();
    int32_t total;
    const int32_t first = scan(hist[tid], &total);
    __syncthreads();
    hist[tid] = first;
    __syncthreads();
    // the order within a bucket is open: it decides which CTA takes a block, not what it computes
    for (int32_t i = tid; i < blocks; i += 1024) {
        const int bucket = locate(i, &e);
        p.table[atomicAdd(&hist[bucket], 1)] = e;
    }
}

// ------------------------------------------------------------------ the kernel --
struct Bars {
    // by parity of the key tile: its key panels and value panels, loaded and handed back
    uint64_t k_full[2][3], k_free[2], v_full[2], v_free[2];  // k_full: by panel
    uint64_t q_full[2], q_free[2], s[2], p[2], o[2], drain[2];  // by query tile
};

struct Shared {
    Bars bar;
    float pair[2][2][T];  // by query tile, half, row: what the two threads of a row tell each other
    uint32_t tmem_base;
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
            mbar_init(&bar.k_full[s][0], 1), mbar_init(&bar.k_full[s][1], 1), mbar_init(&bar.k_full[s][2], 1), mbar_init(&bar.k_free[s], 2), mbar_init(&bar.v_full[s], 1), mbar_init(&bar.v_free[s], 2);  // handed back by both query tiles
            mbar_init(&bar.drain[s], 1);
            mbar_init(&bar.q_full[s], 1), mbar_init(&bar.q_free[s], 1), mbar_init(&bar.s[s], 1), mbar_init(&bar.o[s], 1);
            mbar_init(&bar.p[s], 2 * T);
        }
        fence_mbar_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = uniform(sh.tmem_base);
    const int32_t H = p.a.h, items = uniform(*p.n_blocks) * H;  // below 2^31: checked on the host

    bool gave_up = false;
    auto wait = [&](uint64_t *b, uint32_t parity) {
        if (!gave_up && !mbar_wait(b, parity, kWaitLimit)) {
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

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kServiceRegs) : "memory");
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            uint32_t g = 0, loads0 = 0, loads1 = 0;  // key tiles, query tiles so far
            auto query = [&](int s, uint32_t &loads, const Item &it, int head) {
                if (it.tiles(s) == 0) return true;
                if (loads > 0 && !all_wait(&bar.q_free[s], (loads - 1) & 1)) return false;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&bar.q_full[s], kQBytes);
#pragma unroll
                    for (int u = 0; u < DQ / 64; ++u)
                        tma_load_3d(smem + s * kQBytes + u * PB, &maps.q, 64 * u, head, it.q0 + s * T, &bar.q_full[s]);
                }
                __syncwarp();
                ++loads;
                return true;
            };
            bool ok = true;
            for (int32_t idx = blockIdx.x; idx < items && ok; idx += gridDim.x) {
                const int2 e = p.table[idx / H];
                const int head = idx % H;
                Item it;
                it.load(p.a, e.x, e.y);
                if (!(ok = query(0, loads0, it, head))) break;
                for (int32_t j = 0; j < it.n; ++j, ++g) {
                    // panel i of tile g lies in slot (5 g + i) % 8: its first key panel where tile g - 2's last one was (waited
                    // for with tile g - 1's values), the others where tile g - 2's values were, its values where tile g - 1's
                    // first keys were
                    const int tok = it.k0 + j * T;
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
                    if (j == 0 && !(ok = query(1, loads1, it, head))) break;
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
            auto second = [&](uint32_t g, bool fresh, bool single, bool more, bool free_q) {
                const uint64_t b0 = ring_desc + (5 * g + 3) % kRing * (PB >> 4), b1 = ring_desc + (5 * g + 4) % kRing * (PB >> 4);
                if (!all_wait(&bar.v_full[g & 1], g >> 1 & 1)) return false;
                const uint32_t n = g + 1, par = n >> 1 & 1;
                const bool there = more && __all_sync(0xffffffffu, mbar_test(&bar.k_full[n & 1][0], par) &&
                                                                      mbar_test(&bar.k_full[n & 1][1], par) &&
                                                                      mbar_test(&bar.k_full[n & 1][2], par));
                if (!all_wait(&bar.p[s], pvs++ & 1)) return false;
                tc::fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        tc::mma_bf16_ts(to, ts + 8 * ks, b0 + 128 * ks, kIdO, ks > 0 || !fresh ? 1u : 0u);
                        tc::mma_bf16_ts(to + 64, ts + 8 * ks, b1 + 128 * ks, kIdO, ks > 0 || !fresh ? 1u : 0u);
                    }
                    if (single) {  // what the rounding left off, too
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
            for (int32_t idx = blockIdx.x; idx < items && ok; idx += gridDim.x) {
                const int2 e = p.table[idx / H];
                Item it;
                it.load(p.a, e.x, e.y);
                const int nt = uniform(it.tiles(s)), n = uniform(it.n);
                if (nt > 0) {
                    if (!(ok = all_wait(&bar.q_full[s], loads++ & 1))) break;
                    tc::fence_after_sync();
                    if (!(ok = first(g, nt == 1))) break;
                }
                for (int j = 0; j < n; ++j, ++g) {
                    if (j < nt) {
                        if (!(ok = second(g, j == 0, nt == 1, j + 1 < nt, j + 2 == nt))) break;
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
        uint32_t g0 = 0, steps = 0;  // key tiles of the items before; key tiles so far (of this query tile)
        for (int32_t idx = blockIdx.x; idx < items; idx += gridDim.x) {
            // through the key tiles only what they need is kept (and the item read again behind them): a row's 64
            // scores fill the registers
            int32_t nt, limit, nk;  // key tiles; keys that this row sees; keys of the sequence
            {
                const int2 e = p.table[idx / H];
                Item it;
                it.load(p.a, e.x, e.y);
                nt = it.tiles(s), limit = row < it.rows(s) ? it.see(s) + row : 0, nk = it.nk;
            }
            float m = -INFINITY, l = 0.f, lr = 0.f;  // l, lr: of this thread's keys
            // a thread that gave up goes on without waiting: all of them meet at every barrier
            for (int32_t j = 0; j < nt; ++j, ++steps) {
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
                // value rows behind the sequence's last key: whatever they hold must not meet P = 0 (every softmax
                // thread of the tile writes its share of these zeros for its own product; a second time they change nothing)
                const int32_t keys = nk - j * T;
                if (keys < T) {
                    const uint32_t g = g0 + j;
                    wait(&bar.v_full[g & 1], g >> 1 & 1);
                    for (int q = row; q < (T - keys) * 8; q += T)
                        *reinterpret_cast<uint4 *>(smem + OFF_RING + (5 * g + 3 + half) % kRing * PB + (keys + (q >> 3)) * 128 + (q & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                // scores -> probabilities, rounded, into S_s
                float2 sum = make_float2(0.f, 0.f), sum_r = make_float2(0.f, 0.f);
                if (nt > 1) {
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
                    }
                    tc::wait_st();
                    tc::fence_before_sync();
                    mbar_arrive(&bar.p[s]);
                } else {  // a single key tile: what the rounding leaves off goes into the other half of S_s
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
                    mbar_arrive(&bar.p[s]);
                }
                l += sum.x + sum.y;
                lr += sum_r.x + sum_r.y;
            }
            pair_sync();  // the maxima have been read
            sh.pair[s][half][row] = l;
            pair_sync();
            l += sh.pair[s][half ^ 1][row];
            pair_sync();
            sh.pair[s][half][row] = lr;
            pair_sync();
            lr += sh.pair[s][half ^ 1][row];
            const int2 e = p.table[idx / H];
            Item it;
            it.load(p.a, e.x, e.y);
            const int64_t out_row = static_cast<int64_t>(it.q0 + s * T + row) * H + idx % H;
            if (nt > 0) {
                wait(&bar.o[s], (steps - 1) & 1);
                tc::fence_after_sync();
            }
            const float inv = lr > 0.f ? 1.f / lr : 0.f;
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.a.out) + out_row * DV + kHalf * half);
#pragma unroll
            for (int c = 0; c < kHalf; c += 16) {
                uint32_t o[16];
                if (nt > 0) {
                    tc::ld16(to + c, o);
                    tc::wait_ld();
                }
                if (row < it.rows(s)) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            w[r] = inv > 0.f ? pack_bf16x2(__uint_as_float(o[8 * q + 2 * r]) * inv, __uint_as_float(o[8 * q + 2 * r + 1]) * inv) : 0u;
                        out[c / 8 + q] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc::fence_before_sync();
            if (half == 0 && row < it.rows(s) && p.a.lse != nullptr) p.a.lse[out_row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            pair_sync();  // the sums have been read
            g0 += it.n;
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 3) tc::tmem_dealloc(tmem, 512);
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

size_t latent_prefill_workspace(int64_t total_q, int64_t num_seqs, int32_t)
{
    const size_t n = static_cast<size_t>(blocks_bound(total_q, num_seqs));
    return 256 + n * sizeof(int2) + static_cast<size_t>(num_seqs + 1) * 4;
}

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t st)
{
    Params p{};
    p.a = a;
    p.scale_log2 = a.scale * kLog2e;
    p.max_blocks = blocks_bound(a.total_q, a.num_seqs);
    p.status = static_cast<int32_t *>(a.workspace);
    p.n_blocks = p.status + 1;
    p.table = reinterpret_cast<int2 *>(static_cast<char *>(a.workspace) + 256);
    p.seq_off = reinterpret_cast<int32_t *>(p.table + p.max_blocks);
    Maps maps{};
    int32_t plain;  // q's heads lie within a token (or there is one), k_rope has one
    if (!encode(&maps.q, a.q, DQ, a.h, a.total_q, DQ, static_cast<int64_t>(a.h) * DQ, &plain)) return cudaErrorInvalidValue;
    if (a.total_k > 0 && (!encode(&maps.kn, a.k_nope, DN, a.h, a.total_k, a.kn_head, a.kn_token, &p.kn_order) ||
                          !encode(&maps.v, a.v, DV, a.h, a.total_k, a.v_head, a.v_token, &p.v_order) ||
                          !encode(&maps.kr, a.k_rope, DR, 1, a.total_k, DR, a.kr_token, &plain)))
        return cudaErrorInvalidValue;
    plan_kernel<<<1, 1024, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    // the register split (setmaxnreg) needs a launch with exactly 96 registers a thread
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, latent_prefill_kernel)) != cudaSuccess) return e;
    if (at.numRegs != 96) return cudaErrorInvalidConfiguration;
    const int64_t items = p.max_blocks * a.h, sms = sm_count();
    latent_prefill_kernel<<<static_cast<unsigned>(items < sms ? items : sms), kThreads, kSmem, st>>>(p, maps);
    return cudaGetLastError();
}

}  // namespace kda
