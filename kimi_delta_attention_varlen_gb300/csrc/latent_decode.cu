// Absorbed latent attention over paged latents (kda_latent_decode).
//
// For one request the query rows are its L x H (token, head) pairs, all of them against the same
// cache rows x_j = [c_j | r_j].  With S = scale Q X^T and P = e^{S - m}, out = P C / l: the cache
// is read once, as the keys of the first product and (its first dl columns) as the values of the
// second, while the softmax keeps a running maximum m and sum l a row.
//
// One persistent CTA per SM.  The tiles (T tokens of one request, for one group of at most N query
// rows) of the whole batch lie on one line, request by request; CTA c takes the c-th equal share, so
// few long requests fill the GPU as well as many short ones.  A (request, group) that falls into
// several shares leaves unnormalised parts in the workspace, and a second kernel joins them in order
// of their tiles (so the result does not depend on which CTA was first).
//
// Warps of a CTA: two issue the TMA copies, one the MMAs of each product, four do the softmax and
// the epilogue.
//   S   = Q X^T        M = 64 (rows; fewer than 64 leave lanes unused), N = T tokens, K = dl + 64
//   O^T = C^T P^T      M = 128 value dimensions (dl / 128 of them), N rows, K = T tokens
// The second product is transposed so that the accumulator's width is the number of rows, not dl:
// 4 x N tensor-memory columns instead of dl.  A tile arrives as panels of T tokens x 64 dimensions
// (128-byte swizzle), which serve as K-major B of the first product and, two side by side, as
// MN-major A of the second.  Panels travel in pairs through a ring (the rope panel through a ring of
// its own) and are handed back pair by pair as the second product is done with them.
//
// The probabilities enter the second product in bf16, the only operand type the tensor cores take
// beside bf16 values; the output is normalised by the sum of those rounded weights (they then sum
// to one exactly), the log-sum-exp taken from the sum before rounding.  So each weight is off by 2^-8 at most, relative
// to the others, and the output by 2^-7 sum p |x| beside its own rounding; that takes two or three weights that
// outweigh all others and round to opposite sides, else the errors average out.  A query token that sees few tokens
// has no more weights than that, so where one sees no second tile, a second pass adds the product of what the rounding
// left off in the first one (its own rounding is 2^-16 of the weight).
//
// The accumulator is rescaled only when a row's maximum has grown by more than 2^8 since the last
// rescale (the exponents are relative to that older maximum, exact in fp32 and in bf16's range).
// The tensor cores cut every product off at 2^-25 of the sum that it joins (the bits of a 26-bit window), so a sum of N
// may lack N 2^-25 of its size: 1.3 % after a million tokens behind one that holds half of the weight.  After kSumTiles
// tiles of a segment the accumulator, l and lr are therefore added to fp32 sums (the accumulator in the workspace) and
// begin again (16,384 tokens: 2^-11 at the most).
// Rows of a tile behind the request's last token are set to 0 in shared memory before they meet P = 0 (0
// times what they hold need not be 0).  With draft tokens the last L - 1 tokens are not seen by every query
// token: of their values those that are not finite are set to 0 likewise, and where there were any, the
// epilogue adds them to the rows that do see them.
//
// What bounds it: with one token a request the cache's bytes (512 requests of 512..8192 tokens, 32 heads, dl = 512:
// 419..443 us = 5.9..6.2 TB/s), a few short requests the latency of two launches, the first tile and the join (one of
// 1009 tokens: 14 us), with four draft tokens and 128 heads the ring: 64 query rows leave room for two tiles, each of
// which holds its slots for 7,000 cycles from copy to second product, 1,920 of them MMAs (33 requests of 1500..6001
// tokens: 218..233 us = 600..640 TFLOP/s; with P handed over in two parts 10 us more, since the slots then come back
// later).  64-token tiles because of the same ring: 512 requests took 617 us with 96 and 572 with 128 where they took
// 439 with 64.  Four copying warps instead of two: 425 / 420 us, drafts alike.
//
// With a prefix that groups share (latent_shared.cu) the same kernels take the tokens behind it and add its part at the end.
//
// Every wait is bounded; an expired one sets the workspace's status word (6) and ends the CTA.
#include "latent_decode.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 256;
constexpr float kLazy = 8.f;  // log2 of the growth that forces a rescale

template <int DL_, int N_> struct Cfg {
    static constexpr int DL = DL_, N = N_;
    static constexpr int D = DL + 64, PANELS = D / 64, PAIRS = DL / 128;  // of a tile: all panels, pairs of value panels
    static constexpr int PB = T * 128;                                    // bytes of a panel
    static constexpr int ROPE = N == 64 ? 2 : 3;                          // rope panels in flight
    static constexpr int Q_BYTES = PANELS * N * 128, P_BYTES = N * 128;
    // 230,400 bytes: 227 KB less what the kernel declares itself (2 KB at the most)
    static constexpr int RING_FIT = (230400 - Q_BYTES - P_BYTES - ROPE * PB) / (2 * PB);
    static constexpr int RING = RING_FIT < 3 * PAIRS ? RING_FIT : 3 * PAIRS;  // pairs in flight
    static constexpr int OFF_P = Q_BYTES, OFF_ROPE = OFF_P + P_BYTES, OFF_RING = OFF_ROPE + ROPE * PB;
    static constexpr int SMEM = OFF_RING + RING * 2 * PB + 1024;
    static_assert(RING >= PAIRS && SMEM <= 230400, "a tile fits the ring, the ring fits shared memory");
};

struct Maps {
    CUtensorMap q, cache;
};

template <class C> struct Bars {
    uint64_t full[C::RING], empty[C::RING], rope_full[C::ROPE], rope_empty[C::ROPE];
    uint64_t q_full, q_free, s[2], s_free[2], p, o, drain[2];
};

// The accumulator and a thread's l (x, y of `l`: rows g and g + 8) and lr (z, w) join what its segment set aside (`begun`:
// something was) or, at the segment's end, come back with it as the whole (`back`).  By the softmax warps; sums [N][DL]:
// this thread's dimension; kept [3][N]: the maximum that the sums are relative to, l and lr of what was set aside;
// worth [N]: free to be written.  Returns the new l, lr.  Not inlined: it is rarely called, and its code between the
// kernel's own cost a call of one request 0.5 us of 13.8.
template <int DL, int N>
__device__ __noinline__ float4 set_aside(uint32_t tl, float *sums, float (*kept)[N], float *worth, int row, float2 m, float4 l,
                                         bool begun, bool back)
{
    const bool first = (threadIdx.x & 3) == 0;  // of the four threads of a row
    if (row < N) {
        float x[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] += __shfl_xor_sync(0xffffffffu, x[e], 1);
            x[e] += __shfl_xor_sync(0xffffffffu, x[e], 2);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row + 8 * e;
            const float now = e ? m.y : m.x;
            if (first) {
                const float f = begun ? rebase(kept[0][r], now) : 0.f;
                if (begun) x[e] = fmaf(kept[1][r], f, x[e]), x[2 + e] = fmaf(kept[2][r], f, x[2 + e]);
                worth[r] = f;
                kept[0][r] = now, kept[1][r] = x[e], kept[2][r] = x[2 + e];
            }
        }
        l = first && back ? make_float4(x[0], x[1], x[2], x[3]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    soft_any(false);  // worth is complete
#pragma unroll 1
    for (int c0 = 0; c0 < DL / 128 * N; c0 += 16) {
        uint32_t o[16];
        tc::ld16(tl + c0, o);
        tc::wait_ld();
        float *x = sums + static_cast<int64_t>(c0 % N) * DL + c0 / N * 128;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (begun) o[e] = __float_as_uint(fmaf(x[e * DL], worth[c0 % N + e], __uint_as_float(o[e])));
        if (back) {
            tc::st16(tl + c0, o);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e * DL] = __uint_as_float(o[e]);
        }
    }
    tc::wait_st();
    tc::fence_before_sync();
    return l;
}

// Shared: the tokens behind a prefix (whose part, computed before, joins in at the end).
template <int DL, int N, bool Shared>
__global__ void __launch_bounds__(kThreads, 1) latent_decode_kernel(Params p, const __grid_constant__ Maps maps)
{
    using C = Cfg<DL, N>;
    extern __shared__ char smem_raw[];
    char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) Bars<C> bar;
    __shared__ uint32_t tmem_base;
    __shared__ int32_t not_finite;          // segments (from 1) of the last value that was taken out
    __shared__ float corr[2][N], linv[N];  // corr: by parity of the tile, so that a late reader keeps its own
    __shared__ float kept[3][N];           // set aside: maximum that it is relative to, l, lr
    float *const pinv = kept[2];           // of the prefix's part, when nothing is aside any more
    __shared__ int64_t sums[kThreads / 32];
    __shared__ Edge edge[2];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
    const int cta = blockIdx.x;

    if (warp == 3) {
        tc::tmem_alloc(&tmem_base, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int j = 0; j < C::RING; ++j) mbar_init(&bar.full[j], 1), mbar_init(&bar.empty[j], 1);
        for (int j = 0; j < C::ROPE; ++j) mbar_init(&bar.rope_full[j], 1), mbar_init(&bar.rope_empty[j], 1);
        mbar_init(&bar.q_full, 1), mbar_init(&bar.q_free, 1), mbar_init(&bar.s[0], 1), mbar_init(&bar.s[1], 1);
        not_finite = 0;
        mbar_init(&bar.p, kSoftThreads), mbar_init(&bar.o, 1);
        for (int j = 0; j < 2; ++j) mbar_init(&bar.s_free[j], kSoftThreads), mbar_init(&bar.drain[j], 1);
        fence_mbar_init();
    }
    before_next();
    after_previous();
    if (tid == 0) {
        if (!Shared && cta == 0) *p.status = 0;
        p.item0[cta] = p.item1[cta] = -1;
    }
    find_share<kThreads, Shared>(p, sums, edge);
    const uint32_t tmem = tmem_base;
    constexpr uint32_t kColS = 256;

    const int32_t total = static_cast<int32_t>(edge[1].tiles_before - edge[0].tiles_before);
    WalkOf<Shared> w{};
    if (total > 0) {
        w.r = edge[0].r;
        w.load(p);
        w.group = edge[0].group;
        w.tile = edge[0].tile;
    }
    bool gave_up = false;
    auto wait = [&](uint64_t *b, uint32_t parity) {
        if (!gave_up && !mbar_wait(b, parity, kWaitLimit)) {
            gave_up = true;
            atomicExch(p.status, kStatusExpired);
        }
        return !gave_up;
    };

    if (warp == 0 || warp == 3) {
        // ---------------------------------------------------------------- copies
        // Warp 0 copies the queries and the first half of a tile's pairs, warp 3 the other pairs and the rope panel:
        // small pages make many copies (16 tokens: 36 a tile), which one warp issues in about a microsecond.
        const int part = warp == 0 ? 0 : 1, u0 = part * (C::PAIRS / 2), u1 = u0 + C::PAIRS / 2;
        const int32_t br = p.box_rows, page = static_cast<int32_t>(p.a.page);
        // page (an out-of-range coordinate, read as zeros, where the number is invalid) and row of chunk `lane`
        auto lookup = [&](const WalkOf<Shared> &x, int32_t *pg, int32_t *row) {
            const int32_t t = x.token(x.tile) + lane * br;
            *pg = 0, *row = 0;
            if (lane * br < T && lane * br < x.n - x.token(x.tile)) {
                const int32_t e = p.a.block_table[x.slot * p.a.table_stride + t / page];
                *pg = e >= 0 && e < p.a.cache.n_rows ? e : static_cast<int32_t>(p.a.cache.n_rows);
                *row = t % page;
            }
        };
        auto all_wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
        int32_t pg = 0, row = 0, i = 0, segs = 0;
        if (total > 0) lookup(w, &pg, &row);
        bool ok = true;  // the same in every lane
        for (; i < total && ok; ++i) {
            WalkOf<Shared> nx = w;
            nx.next(p);
            int32_t pg_next = 0, row_next = 0;
            if (i + 1 < total) lookup(nx, &pg_next, &row_next);
            if (part == 0 && (i == 0 || w.first())) {
                if (segs > 0 && !(ok = all_wait(&bar.q_free, (segs - 1) & 1))) break;
                const int y = static_cast<int>(w.r * p.rows + w.group * N);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&bar.q_full, C::Q_BYTES);
                    for (int e = 0; e < C::PANELS; ++e) tma_load_3d(smem + e * N * 128, &maps.q, 64 * e, y, 0, &bar.q_full);
                }
                __syncwarp();
                ++segs;
            }
            const int32_t left = w.n - w.token(w.tile), valid = left < T ? left : T;
            const int32_t chunks = (valid + br - 1) / br;
            for (int u = u0; u < u1 && ok; ++u) {
                const int k = i * C::PAIRS + u, s = k % C::RING;
                if (!(ok = all_wait(&bar.empty[s], ((k / C::RING) & 1) ^ 1))) break;
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
                if (!(ok = all_wait(&bar.rope_empty[s], ((i / C::ROPE) & 1) ^ 1))) break;
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
            if (segs > 0) mbar_wait(&bar.q_full, (segs - 1) & 1, kWaitLimit);
        }
    } else if (warp == 1 && total > 0) {
        // ----------------------------------------------------- first product: S
        constexpr uint32_t kId = idesc(64, T, false);
        const uint32_t base = smem_u32(smem);
        const uint64_t q_desc = tc::sdesc_sw128(base, 16, 1024), key_desc = tc::sdesc_sw128(base + C::OFF_RING, 16, 1024),
                       rope_desc = tc::sdesc_sw128(base + C::OFF_ROPE, 16, 1024);
        int slot = 0, rope_slot = 0, segs = 0;
        uint32_t par = 0, rope_par = 0;
        auto ready = [&](uint64_t *b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
        bool ok = true;
        for (int32_t i = 0; i < total && ok; ++i) {
            const uint32_t d = tmem + kColS + T * (i & 1);
            if (i > 1) ok = ready(&bar.s_free[i & 1], ((i >> 1) & 1) ^ 1);
            if (ok && __all_sync(0xffffffffu, i == 0 || w.first())) ok = ready(&bar.q_full, segs++ & 1);
            for (int u = 0; u < C::PAIRS && ok; ++u) {
                if (!(ok = ready(&bar.full[slot], par))) break;
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
            if (!ok || !(ok = ready(&bar.rope_full[rope_slot], rope_par))) break;
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
            w.next(p);
        }
        if (elect_one()) tc::commit(&bar.drain[0]);  // everything issued has completed before tensor memory is given back
        mbar_wait(&bar.drain[0], 0, kWaitLimit);
    } else if (warp == 2 && total > 0) {
        // --------------------------------------------------- second product: O^T
        constexpr uint32_t kId = idesc(128, N, true);
        const uint32_t base = smem_u32(smem);
        const uint64_t p_desc = tc::sdesc_sw128(base + C::OFF_P, 16, 1024),
                       val_desc = tc::sdesc_sw128(base + C::OFF_RING, C::PB, 1024);
        int slot = 0;
        uint32_t passes = 0;
        int32_t tile0 = w.tile;  // the segment's first
        bool ok = true;
        for (int32_t i = 0; i < total && ok; ++i) {
            if (w.first()) tile0 = 0;
            const uint32_t more = __all_sync(0xffffffffu, ((w.tile - tile0) & (kSumTiles - 1)) == 0) ? 0u : 1u;
            const bool two = __all_sync(0xffffffffu, w.twice(p)) != 0;
            for (int pass = two ? 0 : 1; pass < 2; ++pass, ++passes) {
                if (!(ok = __all_sync(0xffffffffu, wait(&bar.p, passes & 1)) != 0)) break;
                tc::fence_after_sync();
                if (elect_one()) {
                    int sl = slot;
#pragma unroll
                    for (int mt = 0; mt < C::PAIRS; ++mt) {
                        const uint64_t v = val_desc + sl * (2 * C::PB >> 4);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc::mma_bf16(tmem + mt * N, v + ks * 128, p_desc + ks * 2, kId,
                                         ks > 0 || (two && pass == 1) ? 1u : more);
                        if (pass == 1) tc::commit(&bar.empty[sl]);
                        sl = sl + 1 == C::RING ? 0 : sl + 1;
                    }
                    tc::commit(&bar.o);
                }
                __syncwarp();
            }
            slot = (slot + C::PAIRS) % C::RING;
            w.next(p);
        }
        if (elect_one()) tc::commit(&bar.drain[1]);
        mbar_wait(&bar.drain[1], 0, kWaitLimit);
    } else if (warp >= 4 && total > 0) {
        // --------------------------------------------------- softmax and epilogue
        const int quad = warp & 3, g = lane >> 2, t = lane & 3;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16);
        const bool active = 16 * quad < N;  // this warp holds rows 16 quad ... + 15 of S
        float m[2], l[2], lr[2];  // l: sum of the probabilities, lr: of their bf16 roundings
        int32_t seen[2];
        int slot_out = 0;
        int32_t segments = 0, tile0 = 0;  // tile0: the segment's first
        uint32_t passes = 0;  // of the second product, so far
        // worth: the half of corr that the tile does not use
        auto aside = [&](float *worth, bool begun, bool back) {
            wait(&bar.o, (passes - 1) & 1);
            tc::fence_after_sync();
            float *sums = p.part + (static_cast<int64_t>(2) * cta + slot_out) * N * DL + 32 * quad + lane;
            const float4 x = set_aside<DL, N>(tl, sums, kept, worth, 16 * quad + g, make_float2(m[0], m[1]),
                                              make_float4(l[0], l[1], lr[0], lr[1]), begun, back);
            l[0] = x.x, l[1] = x.y, lr[0] = x.z, lr[1] = x.w;
        };
        // a thread that gave up goes on without waiting: all of them meet at every barrier
        for (int32_t i = 0; i < total; ++i) {
            const bool fresh = i == 0 || w.first();
            if (fresh) {
                slot_out = w.first() ? 1 : 0;  // where a part that is not the whole goes
                ++segments;
                tile0 = w.tile;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = w.group * N + 16 * quad + 8 * e + g;
                    m[e] = -INFINITY;
                    l[e] = lr[e] = 0.f;
                    seen[e] = row < p.rows ? w.n - (p.a.L - 1 - row / p.a.h) : 0;
                }
            } else if (((w.tile - tile0) & (kSumTiles - 1)) == 0) {
                aside(corr[(i & 1) ^ 1], w.tile - tile0 > kSumTiles, false);  // this tile's product does not add to it
            }
            wait(&bar.s[i & 1], (i >> 1) & 1);
            tc::fence_after_sync();
            const int32_t t0 = w.token(w.tile);
            uint32_t pk[2][T / 8];
            float z[2][T / 4];  // rows g and g + 8 of this warp; columns 8 j + 2 t, + 1
            bool grew = false;
            if (active) {
#pragma unroll
                for (int c0 = 0; c0 < T; c0 += 32) {
                    uint32_t s[16];
                    ld_16x256b_x4(tl + kColS + T * (i & 1) + c0, s);
                    tc::wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            z[e][c0 / 4 + 2 * j] = __uint_as_float(s[4 * j + 2 * e]);
                            z[e][c0 / 4 + 2 * j + 1] = __uint_as_float(s[4 * j + 2 * e + 1]);
                        }
                }
                tc::fence_before_sync();
                mbar_arrive(&bar.s_free[i & 1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (t0 + T > seen[e]) {
#pragma unroll
                        for (int j = 0; j < T / 4; ++j)
                            if (t0 + 8 * (j >> 1) + 2 * t + (j & 1) >= seen[e]) z[e][j] = -INFINITY;
                    }
                    float mx = z[e][0];
#pragma unroll
                    for (int j = 1; j < T / 4; ++j) mx = fmaxf(mx, z[e][j]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * p.scale_log2;
                    float c = 1.f;
                    if (m[e] == -INFINITY) {
                        m[e] = mx;  // nothing summed yet
                    } else if (mx > m[e] + kLazy) {
                        c = ex2_approx(m[e] - mx);
                        l[e] *= c;
                        lr[e] *= c;
                        m[e] = mx;
                        grew = true;
                    }
                    if (t == 0) corr[i & 1][16 * quad + 8 * e + g] = c;
                    const float base = m[e] == -INFINITY ? 0.f : m[e];
                    const float2 sc = make_float2(p.scale_log2, p.scale_log2), nb = make_float2(-base, -base);
                    float2 sum = make_float2(0.f, 0.f), sum_r = make_float2(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < T / 8; ++j) {
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
            } else {
                mbar_arrive(&bar.s_free[i & 1]);
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
                    for (int j = 0; j < T / 8; ++j) *reinterpret_cast<uint32_t *>(pr + ((j ^ (row & 7)) << 4)) = pk[e][j];
                }
            };
            if (active) put();
            // What the copies wrote is read and written below.  They were complete for S; each one's own barrier, which turns again only
            // behind this tile's second product, is looked at so that this is seen here too.
            if (t0 + T > w.n - (p.a.L - 1)) {
                const int k = i * C::PAIRS + lane % C::PAIRS;
                mbar_test(&bar.full[k % C::RING], (k / C::RING) & 1);
                __syncwarp();
            }
            if (w.n - t0 < T) {  // rows behind the last token: whatever they hold must not meet P = 0
                const int from = w.n - t0;
                for (int e = tid - 128; e < (T - from) * 2 * C::PAIRS * 8; e += kSoftThreads) {
                    const int c = e & 7, pan = (e >> 3) % (2 * C::PAIRS), r2 = from + (e >> 3) / (2 * C::PAIRS);
                    const int s = (i * C::PAIRS + (pan >> 1)) % C::RING;
                    *reinterpret_cast<uint4 *>(smem + C::OFF_RING + (2 * s + (pan & 1)) * C::PB + r2 * 128 + c * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
            }
            if (p.a.L > 1 && t0 + T > w.n - (p.a.L - 1)) {  // draft tokens: what is not finite must not meet P = 0 either
                const int from = max(w.n - (p.a.L - 1) - t0, 0), to = min(w.n - t0, T);
                for (int e = tid - 128; e < (to - from) * 2 * C::PAIRS * 8; e += kSoftThreads) {
                    const int c = e & 7, pan = (e >> 3) % (2 * C::PAIRS), r2 = from + (e >> 3) / (2 * C::PAIRS);
                    const int s = (i * C::PAIRS + (pan >> 1)) % C::RING;
                    uint4 *x = reinterpret_cast<uint4 *>(smem + C::OFF_RING + (2 * s + (pan & 1)) * C::PB + r2 * 128 + c * 16);
                    const uint4 u = *x;
                    const uint4 bad = make_uint4(bf16x2_not_finite(u.x), bf16x2_not_finite(u.y), bf16x2_not_finite(u.z), bf16x2_not_finite(u.w));
                    if (bad.x | bad.y | bad.z | bad.w) {
                        not_finite = segments;
                        *x = make_uint4(u.x & ~bad.x, u.y & ~bad.y, u.z & ~bad.z, u.w & ~bad.w);
                    }
                }
            }
            fence_proxy_async_smem();
            if (soft_any(grew) && !fresh) {
#pragma unroll 1
                for (int c0 = 0; c0 < C::PAIRS * N; c0 += 16) {
                    uint32_t o[16];
                    tc::ld16(tl + c0, o);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr[i & 1][(c0 + e) % N]);
                    tc::st16(tl + c0, o);
                }
                tc::wait_st();
            }
            tc::fence_before_sync();
            mbar_arrive(&bar.p);
            ++passes;
            if (w.twice(p)) {  // the second pass: what the rounding left off
                if (active) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float base = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
                        for (int j = 0; j < T / 8; ++j)
                            pk[e][j] = pack_bf16x2(ex2_approx(fmaf(z[e][2 * j], p.scale_log2, -base)) - bf16_lo(pk[e][j]),
                                                   ex2_approx(fmaf(z[e][2 * j + 1], p.scale_log2, -base)) - bf16_hi(pk[e][j]));
                        lr[e] = l[e];
                    }
                }
                wait(&bar.o, (passes - 1) & 1);
                tc::fence_after_sync();
                if (active) put();
                fence_proxy_async_smem();
                tc::fence_before_sync();
                mbar_arrive(&bar.p);
                ++passes;
            }
            const bool last = w.last();
            if (last || i + 1 == total) {  // the segment ends here
                const bool whole = last && slot_out == 1;
                const int64_t part = 2 * cta + slot_out;
                if (w.tile - tile0 >= kSumTiles) aside(corr[(i & 1) ^ 1], true, true);
                if (active) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float sum = l[e], sum_r = lr[e];
                        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                        sum_r += __shfl_xor_sync(0xffffffffu, sum_r, 1);
                        sum_r += __shfl_xor_sync(0xffffffffu, sum_r, 2);
                        const int row = 16 * quad + 8 * e + g, rr = w.group * N + row;
                        if (t == 0) {
                            if (Shared && whole) {
                                float f = 1.f, fy = 0.f, top = m[e];
                                if (w.base > 0 && rr < p.rows) {
                                    const float4 ml = p.pre_ml[w.r * p.rows + rr];
                                    top = fmaxf(m[e], ml.x);
                                    f = rebase(m[e], top), fy = rebase(ml.x, top);
                                    sum = sum * f + ml.y * fy, sum_r = sum_r * f + ml.z * fy, m[e] = top;
                                }
                                linv[row] = f * inverse(sum_r), pinv[row] = fy * inverse(sum_r);
                            } else {
                                linv[row] = inverse(sum_r);
                            }
                            if (!whole) p.ml[part * N + row] = make_float4(m[e], sum, sum_r, 0.f);
                            else if (p.a.lse != nullptr && rr < p.rows)
                                p.a.lse[w.r * p.rows + rr] = log_sum(m[e], sum);
                        }
                    }
                }
                if (!whole && tid == 128) (slot_out ? p.item1 : p.item0)[cta] = static_cast<int32_t>(w.r * p.rows + w.group * N);
                const int valid = p.rows - w.group * N < N ? p.rows - w.group * N : N;
                const int dim = 32 * quad + lane;
                // the prefix's part of 16 columns, loaded while those before them are worked on
                const bool prefixed = Shared && whole && w.base > 0;
                float y[Shared ? 16 : 1];
                auto load_prefix = [&](int c0) {
                    if constexpr (Shared) {
                        if (prefixed) {  // (of the last row in place of those behind it: loads that wait for nothing)
                            const float *pre = p.pre + (w.r * p.rows + w.group * N) * DL + c0 / N * 128 + dim;
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = pre[min(c0 % N + e, valid - 1) * DL];
                        }
                    }
                };
                load_prefix(0);
                wait(&bar.o, (passes - 1) & 1);
                tc::fence_after_sync();
                soft_any(false);  // linv is complete
                const bool taken = not_finite == segments;
#pragma unroll 1
                for (int c0 = 0; c0 < C::PAIRS * N; c0 += 16) {
                    uint32_t o[16];
                    tc::ld16(tl + c0, o);
                    const int mt = c0 / N, row0 = c0 % N;
                    tc::wait_ld();
                    if (taken) {  // draft tokens' values that were taken out, to the rows that see them
                        const int32_t last = min(w.n, w.token(w.tile + 1));
                        for (int32_t tok = max(w.n - (p.a.L - 1), w.token(tile0)); tok < last; ++tok) {
                            const int32_t e = p.a.block_table[w.slot * p.a.table_stride + tok / p.a.page];
                            if (e < 0 || e >= p.a.cache.n_rows) continue;
                            const float x = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.a.cache.data)[
                                e * p.a.cache.row_stride + tok % p.a.page * C::D + mt * 128 + dim]);
                            if (isfinite(x)) continue;
#pragma unroll
                            for (int q = 0; q < 16; ++q) {
                                const int row = w.group * N + row0 + q;
                                if (row < p.rows && tok < w.n - (p.a.L - 1 - row / p.a.h)) o[q] = __float_as_uint(__uint_as_float(o[q]) + x);
                            }
                        }
                    }
                    if (whole) {
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) +
                                             (w.r * p.rows + w.group * N + row0) * DL + mt * 128 + dim;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x = __uint_as_float(o[e]) * linv[row0 + e];
                            if (prefixed) x = fmaf(y[Shared ? e : 0], pinv[row0 + e], x);
                            o[e] = __float_as_uint(x);
                        }
                        if (c0 + 16 < C::PAIRS * N) load_prefix(c0 + 16);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (row0 + e < valid) out[e * DL] = __float2bfloat16_rn(__uint_as_float(o[e]));
                    } else {
                        float *out = p.part + (part * N + row0) * DL + mt * 128 + dim;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (row0 + e < valid) out[e * DL] = __uint_as_float(o[e]);
                    }
                }
                tc::fence_before_sync();
                soft_any(false);  // linv may be written again
            }
            w.next(p);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 3) tc::tmem_dealloc(tmem, 512);
}

int rows_per_group(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int DL, int N, bool Shared> cudaError_t launch(Params p, cudaStream_t st)
{
    using C = Cfg<DL, N>;
    const int grid = static_cast<int>(sm_count());
    char *ws = static_cast<char *>(p.a.workspace);
    p.status = reinterpret_cast<int32_t *>(ws);
    p.item0 = p.status + 64;
    p.item1 = p.item0 + grid;
    p.ml = reinterpret_cast<float4 *>(ws + up256(256 + 8 * static_cast<size_t>(grid)));
    p.part = reinterpret_cast<float *>(p.ml + static_cast<size_t>(2) * grid * N);
    p.groups = (p.rows + N - 1) / N;
    Maps maps;
    const int64_t q_rows = p.a.batch * p.rows, pitch = p.a.cache.row_stride;
    if (!encode(&maps.q, p.a.q, C::D, q_rows, 1, C::D, q_rows * C::D, N) ||
        !encode(&maps.cache, p.a.cache.data, C::D, p.a.page, p.a.cache.n_rows, C::D, pitch, p.box_rows))
        return cudaErrorInvalidValue;
    auto kern = latent_decode_kernel<DL, N, Shared>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    // the join keeps the main kernel's split between shared memory and L1 cache: changing it between kernels that
    // follow each other costs microseconds
    auto join = latent_join_kernel<DL, N, Shared ? kOwn : kPlain>;
    if ((e = cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
        return e;
    if ((e = launch_overlapped(kern, dim3(grid), dim3(kThreads), C::SMEM, st, p, maps)) != cudaSuccess) return e;
    return launch_overlapped(join, dim3(grid * kJoinCtas), dim3(256), static_cast<size_t>(grid) * 16, st, p, static_cast<int32_t>(grid));
}

}  // namespace

size_t latent_decode_workspace(int64_t batch, int32_t L, int32_t h, int32_t dl)
{
    const size_t n = rows_per_group(static_cast<int64_t>(L) * h), grid = static_cast<size_t>(sm_count());
    (void)batch;
    return up256(256 + 8 * grid) + 2 * grid * n * (16 + static_cast<size_t>(dl) * 4);
}

namespace {
template <bool Shared> cudaError_t dispatch(Params p, cudaStream_t st)
{
    p.rows = p.a.L * p.a.h;
    p.scale_log2 = p.a.scale * kLog2e;
    const int n = rows_per_group(p.rows);
    p.box_rows = box_rows(p.a.page);
    if (p.a.dl == 512)
        return n == 16 ? launch<512, 16, Shared>(p, st) : n == 32 ? launch<512, 32, Shared>(p, st) : launch<512, 64, Shared>(p, st);
    return n == 16 ? launch<256, 16, Shared>(p, st) : n == 32 ? launch<256, 32, Shared>(p, st) : launch<256, 64, Shared>(p, st);
}
}  // namespace

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t st)
{
    Params p{};
    p.a = a;
    return dispatch<false>(p, st);
}

cudaError_t launch_latent_decode_own(const LatentDecodeArgs &a, const int32_t *base, void *pre_ml, float *pre, cudaStream_t st)
{
    Params p{};
    p.a = a;
    p.base = base;
    p.pre_ml = static_cast<float4 *>(pre_ml);
    p.pre = pre;
    return dispatch<true>(p, st);
}

}  // namespace kda
