// Absorbed latent attention of groups of requests that share a prefix (kda_latent_decode_shared).
//
// For a query row, softmax attention over [0, n) is the join of that over [0, b) and over [b, n): with each part's maximum m,
// sum l of e^(z - m) and sum o of e^(z - m) x, everything is brought to the larger m and added.  b is the end of the group's last
// whole shared page.  Four steps on the stream:
//   plan      whether sharing pays; b of each group, a member that holds the pages (the longest), b of each entry
//   prefixes  the rows of all members of a group together, 64 at a time, against [0, b): an item is (group, block of 64 rows);
//             o, m, l to the workspace, in fp32, unnormalised
//   join      of the parts of items that fell into several shares
//   rest      kda_latent_decode's kernels on [b, n), whose epilogue and join add the prefix's part
// One request of 32 heads reads a row of 1,152 bytes for 60 flop a byte; 64 rows of any members make 120 of it, and read it from
// L2 once for two requests and not for each.
//
// The prefixes' kernel has the products, panels and rings of latent_decode.cu at 64 rows (S = Q X^T, O^T = C^T P^T, tiles of 64
// tokens).  Its rows are consecutive rows of q, its mask a limit of each row's own: b, or what the row's query token sees where
// that is less (a request that ends in the prefix).  An item of which a row sees at most a tile of tokens takes what the rounding of
// its first tile's weights leaves off in a second pass, as latent_decode.cu does.  Eight softmax warps, two for the same 16 rows with
// half of a tile's tokens each, since the ring has room for two tiles and a tile keeps its place until its second product is done.
//
// What bounds it: shared memory.  A tile of 64 tokens x 64 rows moves 319 KB through it (operands of S 147, of O^T 98, the copy 74:
// 2,500 cycles at 128 bytes each), and takes about 3,300 cycles: the copies wait for the products' reads, and the ring has room for one
// tile beside the one that is worked on.  64 requests of 32 heads on 32,768 tokens: 181 us of 221..228 us (apart: 344 us); 500 requests
// on seven system prompts of 3,000..6,001 tokens 204 us of 377..380 us (447 us); the rest's kernel then adds the prefix's sums, 64 KB a
// request, which it loads a step ahead.  Tried and not kept: panels copied once for two CTAs of a cluster (multicast, an item of
// 128 rows: 237 and 450 us where it was 233 and 446 then).  Where the plan finds nothing to share, it and two kernels that leave at once
// cost 7..8 us beside kda_latent_decode (8 samples of 4,133 tokens: 28 us and 21 us).
//
// Every wait is bounded; an expired one sets the workspace's status word (6) and ends the CTA.
#include "latent_decode.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int N = 64;          // rows of an item
constexpr int kThreads = 384, kSoft = 256;
constexpr float kLazy = 8.f;   // log2 of the growth that forces a rescale

struct Plan {  // in the workspace
    int32_t *tokens, *slot;  // [groups]: tokens of the prefix, block table row
    int32_t *base;           // [batch]: tokens before the entry's own
    int32_t *any;            // whether a group has a prefix
};

struct SharedParams {
    Params p;
    SharedGroups g;
    Plan plan;
};

struct Maps {
    CUtensorMap q, cache;
};

template <int DL_> struct Cfg {
    static constexpr int DL = DL_, D = DL + 64;
    static constexpr int PANELS = D / 64, PAIRS = DL / 128;  // of a tile: all panels, pairs of value panels
    static constexpr int PB = T * 128;
    static constexpr int ROPE = 2;
    static constexpr int Q_BYTES = PANELS * N * 128, P_BYTES = N * 128;
    // 230,400 bytes: 227 KB less what the kernel declares itself (2 KB at the most)
    static constexpr int RING_FIT = (230400 - Q_BYTES - P_BYTES - ROPE * PB) / (2 * PB);
    static constexpr int RING = RING_FIT < 3 * PAIRS ? RING_FIT : 3 * PAIRS;  // pairs in flight
    static constexpr int OFF_P = Q_BYTES, OFF_ROPE = OFF_P + P_BYTES, OFF_RING = OFF_ROPE + ROPE * PB;
    static constexpr int SMEM = OFF_RING + RING * 2 * PB + 1024;
    static_assert(RING >= PAIRS && SMEM <= 230400, "a tile fits the ring, the ring fits shared memory");
};

template <class C> struct Bars {
    uint64_t full[C::RING], empty[C::RING], rope_full[C::ROPE], rope_empty[C::ROPE];
    uint64_t q_full, q_free, s[2], s_free[2], p, o, drain[2];
};

__device__ __forceinline__ int64_t bound(int64_t x, int64_t most) { return x < 0 ? 0 : x > most ? most : x; }

// Entries of group g, within the batch whatever the offsets hold.
__device__ __forceinline__ void entries_of(const SharedParams &s, int64_t g, int64_t *from, int64_t *to)
{
    *from = bound(s.g.cu[g], s.p.a.batch);
    *to = bound(s.g.cu[g + 1], s.p.a.batch);
    if (*to < *from) *to = *from;
}

// What a tile of 64 tokens takes a CTA, in cycles (the figures that decide best, below): with up to 32 rows of an entry, and with 64 rows (of an entry or of a
// prefix); alike for latents of 256 and of 512, whose tiles wait for the same softmax.  What comes with a block of 64 rows of a prefix
// whatever its length, what joining the prefix's part takes an entry of 32 rows of 512 (in proportion to both), and what launches and
// joins take the GPU, a CTA.
constexpr int64_t kTile32 = 3100, kTile64 = 3430, kItem = 4 * kTile64, kEntry = 4000;
__host__ __device__ constexpr int64_t launches(int32_t dl) { return dl == 512 ? 36000 : 20000; }
// In a share of the prefixes' line an item takes its tiles and this many more (7 prompts of 427..27,485 tokens, 199 entries of 40 heads:
// 186, 167, 171 and 174 us with 3, 6, 9 and 12; one long prefix alike within 2 %).
constexpr int kPrefixUnits = 6;
constexpr int kPlanThreads = 512;
constexpr int kLengths = 8192;  // entries whose lengths the plan loads at once; of those behind them each when it is needed

// By one CTA, a group a warp.  Sharing pays where it saves more tiles' time than the joins and launches take; an entry saves the tiles
// that it would take apart, so one that is shorter than the prefix saves few and an empty one none.  Where it does not pay,
// nothing is shared and each entry takes all of its tokens (measured both ways: 64 entries of 32 heads on 32,768 tokens 221 us
// against 344 us apart; 8 on 4,133 tokens 43 us against 29 us with nothing shared).  752 batches of 1 to 56 rows an entry, latents of 256
// and 512, one to seven prefixes of 200 to 39,000 tokens under 2 to 256 entries, each timed both ways: but for five of them the rule
// takes the faster side or loses less than 5 % (11 % at the most, 0.1 % on average).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(SharedParams s, int32_t ctas)
{
    constexpr int kWarps = kPlanThreads / 32;
    __shared__ int64_t saved[kWarps];
    __shared__ int32_t lengths[kLengths];
    before_next();
    after_previous();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const LatentDecodeArgs &a = s.p.a;
    if (tid == 0) *s.p.status = 0;  // of all the kernels of the call
    for (int64_t r = tid; r < a.batch && r < kLengths; r += blockDim.x) lengths[r] = length_of(a, slot_of(a, r));
    __syncthreads();
    auto length = [&](int64_t r) { return r < kLengths ? lengths[r] : length_of(a, slot_of(a, r)); };
    const int64_t own = s.p.rows <= 32 ? 32 : 64;  // (one group of rows: entries of 64 rows do not come here)
    int64_t mine = 0;
    for (int64_t g = warp; g < s.g.groups; g += kWarps) {
        int64_t from, to;
        entries_of(s, g, &from, &to);
        int64_t best = -1;  // the longest member, of these the first
        for (int64_t r = from + lane; r < to; r += 32) {
            const int64_t key = static_cast<int64_t>(length(r)) << 31 | (0x7fffffff - (r - from));
            best = key > best ? key : best;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const int64_t x = __shfl_xor_sync(0xffffffffu, best, o);
            best = x > best ? x : best;
        }
        // whole pages; alone, a member shares nothing
        const int64_t b = to - from < 2 ? 0 : bound(s.g.shared[g], best >> 31) / a.page * a.page;
        if (lane == 0) {
            s.plan.tokens[g] = static_cast<int32_t>(b);
            s.plan.slot[g] = b > 0 ? static_cast<int32_t>(slot_of(a, from + (0x7fffffff - (best & 0x7fffffff)))) : 0;
        }
        if (b == 0) continue;
        int64_t tiles = 0;  // that the entries do not take themselves
        for (int64_t r = from + lane; r < to; r += 32) {
            const int32_t n = length(r), before = static_cast<int32_t>(b);
            tiles += tiles_of(n) - tiles_of(n > before ? n - before : 0);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        const int64_t rows = (to - from) * s.p.rows;
        mine += tiles * (own == N ? kTile64 : kTile32) - (rows + N - 1) / N * ((b + T - 1) / T * kTile64 + kItem) -
                rows * a.dl * kEntry / (32 * 512);
    }
    if (lane == 0) saved[warp] = mine;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += saved[w];
    const bool pays = all > launches(a.dl) * ctas;
    if (tid == 0) *s.plan.any = pays;
    for (int64_t g = warp; g < s.g.groups; g += kWarps) {
        int64_t from, to;
        entries_of(s, g, &from, &to);
        __syncwarp();
        const int32_t b = pays ? s.plan.tokens[g] : 0;
        __syncwarp();
        if (lane == 0) s.plan.tokens[g] = b;
        for (int64_t r = from + lane; r < to; r += 32) s.plan.base[r] = b;
    }
    const int64_t first = bound(s.g.cu[0], a.batch), last = bound(s.g.cu[s.g.groups], a.batch);  // of all groups' entries
    for (int64_t r = tid; r < a.batch; r += blockDim.x)
        if (r < first || r >= last) s.plan.base[r] = 0;
}

// Position on the line of the prefixes' tiles.
struct PrefixWalk {
    int64_t g, row0, rows;  // group; first row of the item and of the group's rows behind it, of all entries' rows
    int32_t slot, block, tile, n, tiles;

    __device__ int64_t blocks() const { return (rows + N - 1) / N; }
    __device__ void load(const SharedParams &s)
    {
        int64_t from, to;
        entries_of(s, g, &from, &to);
        n = s.plan.tokens[g];
        slot = s.plan.slot[g];
        tiles = tiles_of(n);
        row0 = from * s.p.rows;
        rows = (to - from) * s.p.rows;
    }
    __device__ int64_t first_row() const { return row0 + static_cast<int64_t>(block) * N; }
    __device__ int32_t valid() const { const int64_t v = rows - static_cast<int64_t>(block) * N; return v < N ? static_cast<int32_t>(v) : N; }
    __device__ bool first() const { return tile == 0; }
    __device__ bool last() const { return tile + 1 == tiles; }
    __device__ void next(const SharedParams &s)
    {
        if (++tile < tiles) return;
        tile = 0;
        if (++block < blocks()) return;
        block = 0;
        while (++g < s.g.groups) {
            load(s);
            if (n > 0) return;
        }
    }
};

struct PrefixEdge {
    int64_t g, tiles_before;
    int32_t block, tile;
};

template <int DL>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ SharedParams sp, const __grid_constant__ Maps maps)
{
    using C = Cfg<DL>;
    const Params &p = sp.p;
    extern __shared__ char smem_raw[];
    char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) Bars<C> bar;
    __shared__ uint32_t tmem_base;
    __shared__ uint32_t taken_out[kSumTiles / 32];  // tiles that values were taken out of, since the sums began (a bit a tile)
    __shared__ __align__(8) float kept[3][N];  // what was set aside: maximum that it is relative to, l, lr
    __shared__ float corr[N];              // of the rows that grew; at a segment's end: worth of what was set aside
    float *const worth = corr;
    __shared__ float2 top[N];              // the halves' maxima; at the end the second half's l and lr, then (x) what a row sees
    __shared__ uint32_t grown[2];          // rows that are rescaled
    __shared__ int32_t lowest[2];          // fewest tokens that a row of the segment sees (of those that see any), by parity of the segment
    int64_t *const sums = reinterpret_cast<int64_t *>(kept), *const counts = sums + kThreads / 32;  // at the start
    __shared__ PrefixEdge edge[2];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
    const int cta = blockIdx.x;

    before_next();
    after_previous();
    if (*sp.plan.any == 0) return;
    if (warp == 3) {
        tc::tmem_alloc(&tmem_base, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int j = 0; j < C::RING; ++j) mbar_init(&bar.full[j], 1), mbar_init(&bar.empty[j], 1);
        for (int j = 0; j < C::ROPE; ++j) mbar_init(&bar.rope_full[j], 1), mbar_init(&bar.rope_empty[j], 1);
        mbar_init(&bar.q_full, 1), mbar_init(&bar.q_free, 1), mbar_init(&bar.p, kSoft), mbar_init(&bar.o, 1);
        for (int j = 0; j < 2; ++j) mbar_init(&bar.s[j], 1), mbar_init(&bar.s_free[j], kSoft), mbar_init(&bar.drain[j], 1);
        for (int j = 0; j < kSumTiles / 32; ++j) taken_out[j] = 0;
        lowest[0] = lowest[1] = 0x7fffffff;
        fence_mbar_init();
        p.item0[cta] = p.item1[cta] = -1;
    }
    // This CTA's share of the line, as in find_share(): items are the blocks of groups with a prefix.
    const int64_t per = (sp.g.groups + kThreads - 1) / kThreads, g_lo = per * tid;
    const int64_t g_hi = g_lo + per < sp.g.groups ? g_lo + per : sp.g.groups;
    auto group_of = [&](int64_t g, int64_t *items) {  // its items, and the units of one
        PrefixWalk w{};
        w.g = g;
        w.load(sp);
        *items = w.n > 0 ? w.blocks() : 0;
        return w.tiles + kPrefixUnits;
    };
    int64_t mine = 0, my_items = 0;
    for (int64_t g = g_lo; g < g_hi; ++g) {
        int64_t items;
        const int32_t u = group_of(g, &items);
        mine += items * u, my_items += items;
    }
    int64_t scan = mine, scan_i = my_items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, scan, o), z = __shfl_up_sync(0xffffffffu, scan_i, o);
        if (lane >= o) scan += y, scan_i += z;
    }
    if (lane == 31) sums[warp] = scan, counts[warp] = scan_i;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    int64_t before = scan - mine, before_i = scan_i - my_items, all = 0, all_i = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? sums[w] : 0, before_i += w < warp ? counts[w] : 0;
        all += sums[w], all_i += counts[w];
    }
    const int64_t shares = all < gridDim.x ? all : gridDim.x;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t at = shares > 0 && cta + e <= shares ? all * (cta + e) / shares : all;
        if (tid == 0 && at == all) edge[e] = PrefixEdge{0, all - kPrefixUnits * all_i, 0, 0};
        if (at >= before && at < before + mine) {
            int64_t left = at - before, done = before_i, g = g_lo, items;
            int32_t u;
            for (;; ++g) {
                u = group_of(g, &items);
                if (left < items * u) break;
                left -= items * u, done += items;
            }
            const int32_t block = static_cast<int32_t>(left / u), x = static_cast<int32_t>(left % u);
            const int32_t tile = x > kPrefixUnits ? x - kPrefixUnits : 0;
            // tiles before: units before the item, less kPrefixUnits for each item before it
            edge[e] = PrefixEdge{g, at - x + tile - kPrefixUnits * (done + block), block, tile};
        }
    }
    __syncthreads();
    const uint32_t tmem = tmem_base;
    constexpr uint32_t kColS = 256;

    const int32_t total = static_cast<int32_t>(edge[1].tiles_before - edge[0].tiles_before);
    PrefixWalk w{};
    if (total > 0) {
        w.g = edge[0].g;
        w.load(sp);
        w.block = edge[0].block;
        w.tile = edge[0].tile;
    }
    bool gave_up = false;
    auto wait = [&](uint64_t *b, uint32_t parity) {  // by a whole warp, which goes on or gives up as one
        if (!gave_up && !mbar_wait(b, parity, kWaitLimit)) {
            gave_up = true;
            atomicExch(p.status, kStatusExpired);
        }
        gave_up = __any_sync(0xffffffffu, gave_up) != 0;
        return !gave_up;
    };

    if (warp == 0 || warp == 3) {
        // ---------------------------------------------------------------- copies
        const int part = warp == 0 ? 0 : 1, u0 = part * (C::PAIRS / 2), u1 = u0 + C::PAIRS / 2;
        const int32_t br = p.box_rows, page = static_cast<int32_t>(p.a.page);
        auto lookup = [&](const PrefixWalk &x, int32_t *pg, int32_t *row) {
            const int32_t t = x.tile * T + lane * br;
            *pg = 0, *row = 0;
            if (lane * br < T && t < x.n) {
                const int32_t e = p.a.block_table[x.slot * p.a.table_stride + t / page];
                *pg = e >= 0 && e < p.a.cache.n_rows ? e : static_cast<int32_t>(p.a.cache.n_rows);
                *row = t % page;
            }
        };
        int32_t pg = 0, row = 0, i = 0, segs = 0;
        if (total > 0) lookup(w, &pg, &row);
        bool ok = true;  // the same in every lane
        for (; i < total && ok; ++i) {
            PrefixWalk nx = w;
            nx.next(sp);
            int32_t pg_next = 0, row_next = 0;
            if (i + 1 < total) lookup(nx, &pg_next, &row_next);
            if (part == 0 && (i == 0 || w.first())) {
                if (segs > 0 && !(ok = wait(&bar.q_free, (segs - 1) & 1))) break;
                const int y = static_cast<int>(w.first_row());
                if (elect_one()) {
                    mbar_arrive_expect_tx(&bar.q_full, C::Q_BYTES);
                    for (int e = 0; e < C::PANELS; ++e) tma_load_3d(smem + e * N * 128, &maps.q, 64 * e, y, 0, &bar.q_full);
                }
                __syncwarp();
                ++segs;
            }
            const int32_t valid = w.n - w.tile * T < T ? w.n - w.tile * T : T;
            const int32_t chunks = (valid + br - 1) / br;
            for (int u = u0; u < u1 && ok; ++u) {
                const int k = i * C::PAIRS + u, s = k % C::RING;
                if (!(ok = wait(&bar.empty[s], ((k / C::RING) & 1) ^ 1))) break;
                if (elect_one()) mbar_arrive_expect_tx(&bar.full[s], 2 * chunks * br * 128);
                __syncwarp();
                for (int32_t c = 0; c < chunks; ++c) {
                    const int32_t z = __shfl_sync(0xffffffffu, pg, c), y = __shfl_sync(0xffffffffu, row, c);
                    char *dst = smem + C::OFF_RING + 2 * s * C::PB + c * br * 128;
                    if (elect_one()) {
                        tma_load_3d(dst, &maps.cache, 128 * u, y, z, &bar.full[s]);
                        tma_load_3d(dst + C::PB, &maps.cache, 128 * u + 64, y, z, &bar.full[s]);
                    }
                    __syncwarp();
                }
            }
            if (part == 1 && ok) {
                const int s = i % C::ROPE;
                if (!(ok = wait(&bar.rope_empty[s], ((i / C::ROPE) & 1) ^ 1))) break;
                if (elect_one()) mbar_arrive_expect_tx(&bar.rope_full[s], chunks * br * 128);
                __syncwarp();
                for (int32_t c = 0; c < chunks; ++c) {
                    const int32_t z = __shfl_sync(0xffffffffu, pg, c), y = __shfl_sync(0xffffffffu, row, c);
                    if (elect_one()) tma_load_3d(smem + C::OFF_ROPE + s * C::PB + c * br * 128, &maps.cache, DL, y, z, &bar.rope_full[s]);
                    __syncwarp();
                }
            }
            w = nx, pg = pg_next, row = row_next;
        }
        if (!ok && lane == 0) {
            // gave up: the copies in flight land before the CTA ends (a wait for one that was not begun runs out, bounded)
            const int32_t k = (i + 1) * C::PAIRS;
            for (int32_t e = k > C::RING ? k - C::RING : 0; e < k; ++e)
                if (e % C::PAIRS >= u0 && e % C::PAIRS < u1) mbar_wait(&bar.full[e % C::RING], (e / C::RING) & 1, kWaitLimit);
            for (int32_t e = i > C::ROPE ? i - C::ROPE : 0; part == 1 && e < i; ++e)
                mbar_wait(&bar.rope_full[e % C::ROPE], (e / C::ROPE) & 1, kWaitLimit);
            if (part == 0 && segs > 0) mbar_wait(&bar.q_full, (segs - 1) & 1, kWaitLimit);
        }
    } else if (warp == 1 && total > 0) {
        // ----------------------------------------------------- first product: S
        constexpr uint32_t kId = idesc(64, T, false);
        const uint32_t base = smem_u32(smem);
        const uint64_t q_desc = tc::sdesc_sw128(base, 16, 1024), key_desc = tc::sdesc_sw128(base + C::OFF_RING, 16, 1024),
                       rope_desc = tc::sdesc_sw128(base + C::OFF_ROPE, 16, 1024);
        int slot = 0, rope_slot = 0, segs = 0;
        uint32_t par = 0, rope_par = 0;
        bool ok = true;
        for (int32_t i = 0; i < total && ok; ++i) {
            const uint32_t d = tmem + kColS + T * (i & 1);
            if (i > 1) ok = wait(&bar.s_free[i & 1], ((i >> 1) & 1) ^ 1);
            if (ok && __all_sync(0xffffffffu, i == 0 || w.first())) ok = wait(&bar.q_full, segs++ & 1);
            for (int u = 0; u < C::PAIRS && ok; ++u) {
                if (!(ok = wait(&bar.full[slot], par))) break;
                tc::fence_after_sync();
                if (elect_one()) {
                    const uint64_t q = q_desc + u * (2 * N * 128 >> 4), x = key_desc + slot * (2 * C::PB >> 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        tc::mma_bf16(d, q + (e >> 2) * (N * 128 >> 4) + (e & 3) * 2, x + (e >> 2) * (C::PB >> 4) + (e & 3) * 2, kId,
                                     e > 0 || u > 0 ? 1u : 0u);
                }
                __syncwarp();
                if (++slot == C::RING) slot = 0, par ^= 1u;
            }
            if (!ok || !(ok = wait(&bar.rope_full[rope_slot], rope_par))) break;
            tc::fence_after_sync();
            const bool last = __all_sync(0xffffffffu, w.last()) != 0;
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    tc::mma_bf16(d, q_desc + (2 * C::PAIRS * N * 128 >> 4) + ks * 2, rope_desc + rope_slot * (C::PB >> 4) + ks * 2, kId, 1u);
                tc::commit(&bar.s[i & 1]);
                tc::commit(&bar.rope_empty[rope_slot]);
                if (last) tc::commit(&bar.q_free);
            }
            __syncwarp();
            if (++rope_slot == C::ROPE) rope_slot = 0, rope_par ^= 1u;
            w.next(sp);
        }
        if (elect_one()) tc::commit(&bar.drain[0]);  // everything issued has completed before tensor memory is given back
        mbar_wait(&bar.drain[0], 0, kWaitLimit);
    } else if (warp == 2 && total > 0) {
        // --------------------------------------------------- second product: O^T
        constexpr uint32_t kId = idesc(128, N, true);
        const uint32_t base = smem_u32(smem);
        const uint64_t p_desc = tc::sdesc_sw128(base + C::OFF_P, 16, 1024),
                       val_desc = tc::sdesc_sw128(base + C::OFF_RING, C::PB, 1024);
        int slot = 0, segs = 0;
        uint32_t passes = 0;
        int32_t tile0 = w.tile;  // the segment's first
        bool ok = true;
        for (int32_t i = 0; i < total && ok; ++i) {
            if (i == 0 || w.first()) ++segs;
            if (w.first()) tile0 = 0;
            const uint32_t more = __all_sync(0xffffffffu, ((w.tile - tile0) & (kSumTiles - 1)) == 0) ? 0u : 1u;
            const bool begins = __all_sync(0xffffffffu, w.first()) != 0;
            if (!(ok = wait(&bar.p, passes++ & 1))) break;
            tc::fence_after_sync();
            // (written before the softmax arrived, and again only after this product has arrived there)
            bool again = begins && __all_sync(0xffffffffu, lowest[segs & 1] <= T) != 0;
            for (uint32_t add = more;; add = 1u) {
                if (elect_one()) {
                    int sl = slot;
#pragma unroll
                    for (int mt = 0; mt < C::PAIRS; ++mt) {
                        const uint64_t v = val_desc + sl * (2 * C::PB >> 4);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc::mma_bf16(tmem + mt * N, v + ks * 128, p_desc + ks * 2, kId, ks > 0 ? 1u : add);
                        if (!again) tc::commit(&bar.empty[sl]);
                        sl = sl + 1 == C::RING ? 0 : sl + 1;
                    }
                    tc::commit(&bar.o);
                }
                __syncwarp();
                if (!again || !(ok = wait(&bar.p, passes++ & 1))) break;
                tc::fence_after_sync();
                again = false;
            }
            if (!ok) break;
            slot = (slot + C::PAIRS) % C::RING;
            w.next(sp);
        }
        if (elect_one()) tc::commit(&bar.drain[1]);
        mbar_wait(&bar.drain[1], 0, kWaitLimit);
    } else if (warp >= 4 && total > 0) {
        // --------------------------------------------------- softmax and epilogue
        constexpr int HT = T / 2;  // a half's tokens
        const int quad = warp & 3, half = (warp - 4) >> 2, g = lane >> 2, t = lane & 3, st = tid - 128;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16);
        float m[2], l[2], lr[2];  // of rows 16 quad + g and + 8: the maximum of both halves; sums of this half
        int32_t seen[2];
        int slot_out = 0;
        int32_t segments = 0, tile0 = 0, low = 0;  // tile0: the segment's first; low: fewest tokens that a row sees
        uint32_t passes = 0;  // of the second product, so far
        // The accumulator and l leave tensor memory and registers: they are set aside, or (`end`) the segment ends with them.
        auto finish = [&](bool begun, bool end, bool whole) {
            const int64_t part = 2 * cta + slot_out;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1), lr[e] += __shfl_xor_sync(0xffffffffu, lr[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2), lr[e] += __shfl_xor_sync(0xffffffffu, lr[e], 2);
                if (half == 1 && t == 0) top[16 * quad + 8 * e + g] = make_float2(l[e], lr[e]);
            }
            soft_any<kSoft>(false);
            if (half == 0 && t == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * quad + 8 * e + g;
                    float sum = l[e] + top[row].x, sum_r = lr[e] + top[row].y;
                    const float back = begun ? rebase(kept[0][row], m[e]) : 0.f;
                    if (begun) sum = fmaf(kept[1][row], back, sum), sum_r = fmaf(kept[2][row], back, sum_r);
                    kept[0][row] = m[e], kept[1][row] = sum, kept[2][row] = sum_r;
                    worth[row] = back;
                    top[row].x = __int_as_float(seen[e]);
                    if (end && row < w.valid()) {
                        if (whole) p.pre_ml[w.first_row() + row] = make_float4(m[e], sum, sum_r, 0.f);
                        else p.ml[part * N + row] = make_float4(m[e], sum, sum_r, 0.f);
                    }
                }
            }
            l[0] = l[1] = lr[0] = lr[1] = 0.f;
            wait(&bar.o, (passes - 1) & 1);
            tc::fence_after_sync();
            soft_any<kSoft>(false);  // worth and kept are complete
            const int valid = w.valid(), dim = 32 * quad + lane;
            uint32_t taken = 0;
#pragma unroll
            for (int j = 0; j < kSumTiles / 32; ++j) taken |= taken_out[j];
            const int32_t begin = end ? w.tile - ((w.tile - tile0) & (kSumTiles - 1)) : w.tile - kSumTiles;  // tile that the sums began with
            float *to = end && whole ? p.pre + w.first_row() * DL : p.part + part * N * DL;
            const float *aside = p.part + part * N * DL;
#pragma unroll 1
            for (int c0 = 16 * half; c0 < C::PAIRS * N; c0 += 32) {
                const int mt = c0 / N, row0 = c0 % N;
                uint32_t o[16];
                tc::ld16(tl + c0, o);
                tc::wait_ld();
                if (begun) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = __float_as_uint(fmaf(aside[(row0 + e) * DL + mt * 128 + dim], worth[row0 + e], __uint_as_float(o[e])));
                }
                // Values that were taken out, to the rows that see them: of those tiles alone and eight loads at a time, since every
                // other warp's waits run while this lasts (all of 256 tiles: some 20 ms of their second).
                for (int j = 0; taken != 0 && j < kSumTiles / 32; ++j)
                    for (uint32_t bits = taken_out[j]; bits != 0; bits &= bits - 1) {
                        const int32_t t0 = (begin + 32 * j + __ffs(bits) - 1) * T, last = min(w.n, t0 + T);
                        for (int32_t tok = t0; tok < last; tok += 8) {  // within a page
                            const int32_t e = p.a.block_table[w.slot * p.a.table_stride + tok / p.a.page];
                            if (tok + 8 <= low || e < 0 || e >= p.a.cache.n_rows) continue;
                            const __nv_bfloat16 *from = static_cast<const __nv_bfloat16 *>(p.a.cache.data) + e * p.a.cache.row_stride +
                                                        tok % p.a.page * C::D + mt * 128 + dim;
                            float x[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[k] = __bfloat162float(from[k * C::D]);
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                float bad = x[0];
#pragma unroll
                                for (int u = 1; u < 8; ++u) bad = u == k ? x[u] : bad;
                                if (isfinite(bad) || tok + k < low) continue;
#pragma unroll
                                for (int q = 0; q < 16; ++q)
                                    if (tok + k < __float_as_int(top[row0 + q].x)) o[q] = __float_as_uint(__uint_as_float(o[q]) + bad);
                            }
                        }
                    }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!end || row0 + e < valid) {
                        // a row that sees nothing: 0 times what is not finite
                        if (end && whole && kept[2][row0 + e] == 0.f) o[e] = 0u;
                        to[(row0 + e) * DL + mt * 128 + dim] = __uint_as_float(o[e]);
                    }
            }
            tc::fence_before_sync();
            soft_any<kSoft>(false);  // worth, kept, top and taken_out may be written again
            if (st < kSumTiles / 32) taken_out[st] = 0;
        };
        // a thread that gave up goes on without waiting: all of them meet at every barrier
        for (int32_t i = 0; i < total; ++i) {
            const bool fresh = i == 0 || w.first();
            if (fresh) {
                slot_out = w.first() ? 1 : 0;  // where a part that is not the whole goes
                ++segments;
                tile0 = w.tile;
                int32_t fewest = w.n;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * quad + 8 * e + g;
                    m[e] = -INFINITY;
                    l[e] = lr[e] = 0.f;
                    seen[e] = 0;
                    if (row < w.valid()) {
                        const int64_t f = w.first_row() + row, r = f / p.rows;
                        seen[e] = min(w.n, length_of(p.a, slot_of(p.a, r)) - (p.a.L - 1 - static_cast<int32_t>(f % p.rows) / p.a.h));
                        if (seen[e] > 0) fewest = min(fewest, seen[e]);  // (of a row that sees nothing the sums are put to 0)
                    }
                }
                atomicMin(&lowest[segments & 1], __reduce_min_sync(0xffffffffu, fewest));
                soft_any<kSoft>(false);
                low = lowest[segments & 1];
                if (st == 0) lowest[(segments & 1) ^ 1] = 0x7fffffff;  // read for the last time before this barrier
            } else if (((w.tile - tile0) & (kSumTiles - 1)) == 0) {
                finish(w.tile - tile0 > kSumTiles, false, false);  // this tile's product does not add to it
            }
            wait(&bar.s[i & 1], (i >> 1) & 1);
            tc::fence_after_sync();
            const int32_t t0 = w.tile * T, th = t0 + HT * half;
            uint32_t pk[2][HT / 8];
            float z[2][HT / 4];  // rows g and g + 8; tokens th + 8 j + 2 t, + 1
            float mx[2];
            {
                uint32_t s[16];
                ld_16x256b_x4(tl + kColS + T * (i & 1) + HT * half, s);
                tc::wait_ld();
                tc::fence_before_sync();
                mbar_arrive(&bar.s_free[i & 1]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        z[e][2 * j] = __uint_as_float(s[4 * j + 2 * e]);
                        z[e][2 * j + 1] = __uint_as_float(s[4 * j + 2 * e + 1]);
                    }
            }
            bool grew = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (th + HT > seen[e]) {
#pragma unroll
                    for (int j = 0; j < HT / 4; ++j)
                        if (th + 8 * (j >> 1) + 2 * t + (j & 1) >= seen[e]) z[e][j] = -INFINITY;
                }
                mx[e] = z[e][0];
#pragma unroll
                for (int j = 1; j < HT / 4; ++j) mx[e] = fmaxf(mx[e], z[e][j]);
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2)) * p.scale_log2;
                grew |= m[e] == -INFINITY ? mx[e] != -INFINITY : mx[e] > m[e] + kLazy;
            }
            grew = soft_any<kSoft>(grew);
            if (grew) {  // rarely: both halves take one maximum
                if (st == 0) grown[0] = grown[1] = 0;
                if (t == 0 && half == 1) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) top[16 * quad + 8 * e + g].x = mx[e];
                }
                if (t == 0 && half == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) top[16 * quad + 8 * e + g].y = mx[e];
                }
                soft_any<kSoft>(false);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * quad + 8 * e + g;
                    const float both = fmaxf(top[row].x, top[row].y);
                    if (m[e] == -INFINITY) {
                        m[e] = both;
                    } else if (both > m[e] + kLazy) {
                        const float c = ex2_approx(m[e] - both);
                        l[e] *= c, lr[e] *= c;
                        m[e] = both;
                        if (half == 0 && t == 0) corr[row] = c, atomicOr(&grown[row >> 5], 1u << (row & 31));
                    }
                }
                soft_any<kSoft>(false);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float base = m[e] == -INFINITY ? 0.f : m[e];
                const float2 sc = make_float2(p.scale_log2, p.scale_log2), nb = make_float2(-base, -base);
                float2 sum = make_float2(0.f, 0.f), sum_r = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < HT / 8; ++j) {
                    float2 x = fma2(make_float2(z[e][2 * j], z[e][2 * j + 1]), sc, nb);
                    x.x = ex2_approx(x.x);
                    x.y = ex2_approx(x.y);
                    sum = add2(sum, x);
                    pk[e][j] = pack_bf16x2(x.x, x.y);
                    sum_r = add2(sum_r, make_float2(bf16_lo(pk[e][j]), bf16_hi(pk[e][j])));
                }
                l[e] += sum.x + sum.y;
                lr[e] += sum_r.x + sum_r.y;
            }
            // the second product of the tile before has read P and written O^T
            if (passes > 0) wait(&bar.o, (passes - 1) & 1);
            tc::fence_after_sync();
            auto put = [&]() {  // pk -> the operand P
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * quad + 8 * e + g;
                    char *pr = smem + C::OFF_P + row * 128 + 4 * t;
#pragma unroll
                    for (int j = 0; j < HT / 8; ++j) *reinterpret_cast<uint32_t *>(pr + (((4 * half + j) ^ (row & 7)) << 4)) = pk[e][j];
                }
            };
            put();
            if (w.n - t0 < T || low < min(w.n, t0 + T)) {
                // The copies were complete for S; each one's own barrier, which turns again only behind this tile's second product, is
                // looked at so that this is seen here too.
                const int turn = i * C::PAIRS + lane % C::PAIRS;
                mbar_test(&bar.full[turn % C::RING], (turn / C::RING) & 1);
                __syncwarp();
                // Rows behind the prefix: whatever they hold must not meet P = 0.  Tokens that some row does not see: nor must
                // what is not finite.
                const int from = max(min(low, w.n) - t0, 0);
                for (int e = st; e < (T - from) * 2 * C::PAIRS * 8; e += kSoft) {
                    const int c = e & 7, pan = (e >> 3) % (2 * C::PAIRS), r2 = from + (e >> 3) / (2 * C::PAIRS);
                    const int s = (i * C::PAIRS + (pan >> 1)) % C::RING;
                    uint4 *x = reinterpret_cast<uint4 *>(smem + C::OFF_RING + (2 * s + (pan & 1)) * C::PB + r2 * 128 + c * 16);
                    const uint4 u = *x;
                    const bool behind = t0 + r2 >= w.n;
                    const uint4 bad = make_uint4(bf16x2_not_finite(u.x), bf16x2_not_finite(u.y), bf16x2_not_finite(u.z), bf16x2_not_finite(u.w));
                    if (behind) {
                        *x = make_uint4(0u, 0u, 0u, 0u);
                    } else if (bad.x | bad.y | bad.z | bad.w) {
                        const int32_t k = (w.tile - tile0) & (kSumTiles - 1);
                        atomicOr(&taken_out[k >> 5], 1u << (k & 31));
                        *x = make_uint4(u.x & ~bad.x, u.y & ~bad.y, u.z & ~bad.z, u.w & ~bad.w);
                    }
                }
            }
            if (grew && passes > 0 && ((w.tile - tile0) & (kSumTiles - 1)) != 0) {  // the columns of the rows that grew
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    for (uint32_t rows = grown[q]; rows != 0; rows &= rows - 1) {
                        const int row = 32 * q + __ffs(rows) - 1;
                        uint32_t o[C::PAIRS / 2];
#pragma unroll
                        for (int c = 0; c < C::PAIRS / 2; ++c) ld1(tl + (half * (C::PAIRS / 2) + c) * N + row, o[c]);
                        tc::wait_ld();
#pragma unroll
                        for (int c = 0; c < C::PAIRS / 2; ++c)
                            st1(tl + (half * (C::PAIRS / 2) + c) * N + row, __float_as_uint(__uint_as_float(o[c]) * corr[row]));
                    }
                tc::wait_st();
            }
            fence_proxy_async_smem();
            tc::fence_before_sync();
            mbar_arrive(&bar.p);
            ++passes;
            if (w.first() && low <= T) {  // the second pass: what the rounding left off
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float base = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
                    for (int j = 0; j < HT / 8; ++j)
                        pk[e][j] = pack_bf16x2(ex2_approx(fmaf(z[e][2 * j], p.scale_log2, -base)) - bf16_lo(pk[e][j]),
                                               ex2_approx(fmaf(z[e][2 * j + 1], p.scale_log2, -base)) - bf16_hi(pk[e][j]));
                    lr[e] = l[e];
                }
                wait(&bar.o, (passes - 1) & 1);
                tc::fence_after_sync();
                put();
                fence_proxy_async_smem();
                tc::fence_before_sync();
                mbar_arrive(&bar.p);
                ++passes;
            }
            const bool last = w.last();
            if (last || i + 1 == total) {  // the segment ends here
                const bool whole = last && slot_out == 1;
                if (!whole && st == 0) {
                    (slot_out ? p.item1 : p.item0)[cta] = static_cast<int32_t>(w.first_row());
                    p.item_rows[cta] = w.valid();  // (of the item in slot 1, which the later segment is)
                }
                finish(w.tile - tile0 >= kSumTiles, true, whole);
            }
            w.next(sp);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 3) tc::tmem_dealloc(tmem, 512);
}

// Entries of 64 rows and more fill the plain kernel's groups of rows by themselves: the prefixes' kernel, which takes 64 rows as well, with
// as little room in its ring, has nothing to save there (4 draft tokens x 128 heads of 18 entries on 9,001 tokens: 221 us, with it 309 us).
bool takes_prefixes(int32_t L, int32_t h) { return static_cast<int64_t>(L) * h < N; }

// The workspace: that of the rest's calls (its status word first), the prefixes' lists and parts, the plan, the prefixes' sums.
struct Layout {
    size_t lists, ml, part, plan, pre_ml, pre, total;
};
Layout layout(int64_t batch, int64_t groups, int32_t L, int32_t h, int32_t dl)
{
    const size_t grid = static_cast<size_t>(sm_count()), rows = static_cast<size_t>(batch) * L * h;
    Layout y;
    y.lists = up256(latent_decode_workspace(batch, L, h, dl));
    y.ml = y.lists + up256(12 * grid);
    y.part = y.ml + 2 * grid * N * 16;
    y.plan = y.part + 2 * grid * N * static_cast<size_t>(dl) * 4;
    y.pre_ml = y.plan + up256(static_cast<size_t>(2 * groups + batch + 1) * 4);
    y.pre = y.pre_ml + up256(rows * 16);
    y.total = y.pre + rows * static_cast<size_t>(dl) * 4;
    return y;
}

template <int DL> cudaError_t launch(const LatentDecodeArgs &a, const SharedGroups &g, cudaStream_t st)
{
    using C = Cfg<DL>;
    const int grid = static_cast<int>(sm_count());
    const Layout y = layout(a.batch, g.groups, a.L, a.h, DL);
    char *ws = static_cast<char *>(a.workspace);
    SharedParams s{};
    Params &p = s.p;
    p.a = a;
    p.rows = a.L * a.h;
    p.scale_log2 = a.scale * kLog2e;
    p.box_rows = box_rows(a.page);
    p.status = reinterpret_cast<int32_t *>(ws);
    p.item0 = reinterpret_cast<int32_t *>(ws + y.lists);
    p.item1 = p.item0 + grid;
    p.item_rows = p.item1 + grid;
    p.ml = reinterpret_cast<float4 *>(ws + y.ml);
    p.part = reinterpret_cast<float *>(ws + y.part);
    p.pre_ml = reinterpret_cast<float4 *>(ws + y.pre_ml);
    p.pre = reinterpret_cast<float *>(ws + y.pre);
    s.g = g;
    s.plan.tokens = reinterpret_cast<int32_t *>(ws + y.plan);
    s.plan.slot = s.plan.tokens + g.groups;
    s.plan.base = s.plan.slot + g.groups;
    s.plan.any = s.plan.base + a.batch;
    p.shares_any = s.plan.any;
    Maps maps;
    const int64_t q_rows = a.batch * p.rows;
    if (!encode(&maps.q, a.q, C::D, q_rows, 1, C::D, q_rows * C::D, N) ||
        !encode(&maps.cache, a.cache.data, C::D, a.page, a.cache.n_rows, C::D, a.cache.row_stride, p.box_rows))
        return cudaErrorInvalidValue;
    cudaError_t e = launch_overlapped(plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, s, grid);
    if (e != cudaSuccess) return e;
    auto kern = prefix_kernel<DL>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
    auto join = latent_join_kernel<DL, N, kPrefix>;
    if ((e = cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
        return e;
    if ((e = launch_overlapped(kern, dim3(grid), dim3(kThreads), C::SMEM, st, s, maps)) != cudaSuccess) return e;
    if ((e = launch_overlapped(join, dim3(grid * kJoinCtas), dim3(256), static_cast<size_t>(grid) * 16, st, p, static_cast<int32_t>(grid))) !=
        cudaSuccess)
        return e;
    return launch_latent_decode_own(a, s.plan.base, p.pre_ml, p.pre, st);
}

}  // namespace

size_t latent_shared_workspace(int64_t batch, int64_t groups, int32_t L, int32_t h, int32_t dl)
{
    return takes_prefixes(L, h) ? layout(batch, groups, L, h, dl).total : latent_decode_workspace(batch, L, h, dl);
}

cudaError_t launch_latent_decode_shared(const LatentDecodeArgs &a, const SharedGroups &g, cudaStream_t st)
{
    if (!takes_prefixes(a.L, a.h)) return launch_latent_decode(a, st);
    return a.dl == 512 ? launch<512>(a, g, st) : launch<256>(a, g, st);
}

}  // namespace kda
