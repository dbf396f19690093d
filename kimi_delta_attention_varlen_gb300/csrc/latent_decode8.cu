// Absorbed latent attention over 8-bit pages (kda_latent_decode8).
//
// A token's row is x = 2^e [code | rope]: e4m3 codes of the latent and a bf16 rope key in one unit 2^e.  So
//   z = scale q . x = scale 2^(a+e) (Q_c code + Q_r rope)   with the query row in units 2^a of its own,
//   out = sum_j p_j 2^(e_j) code_j / l,                     the unit folded into the weight,
// and the codes are operands of the tensor cores as they are: nothing is converted on its way from the page.
//
// The other operand of an e4m3 product is e4m3 too.  Three binary digits follow the leading one there, so
//   a query value (bf16: eight digits)  = q1 + q2 / 16                the parts rows g and g + 8 of one product (exactly down to
//                                                                     2^-15 of the row's largest value; below, e4m3's subnormals
//                                                                     round q2 / 16 to steps of 2^-13, 2^-22 of that value at most),
//   a weight w (to fp16: eleven digits) = (w1 + w2 / 16 + w3 / 256) / 16, the parts side by side in N,
// each part the rounding of what the one before left off; the accumulators of the parts are added up in fp32, those of the
// scores for every tile, those of the outputs once at the end of a segment.
//   S   = [q1; q2] Codes^T  M = 64 (two rows a query row), N = T tokens, K = 64 (bf16) for the rope keys, then K = dl (e4m3)
//   O^T = Codes^T [w1 w2 w3]^T  M = 128 value dimensions (dl / 128 of them), 3 N rows, K = T tokens
// Two running maxima: m over z, for the sum l of p = 2^(z - m), and M over z + e, for the weights w = 2^(z + e - M): tokens of
// large values and tokens of small ones each count to full precision where they matter.  The accumulator is rescaled when a
// row's M has grown by more than kLazy; a weight is then 16 * 2^kLazy at most, which e4m3's 448 takes, and its last part ends
// 2^-21 below 1.  After kSumTiles tiles the accumulator and l are set aside in fp32 and M begins anew, so a token far above
// the rest takes no digits from more than 16,384 others.
//
// Shares, walk and join are those of the bf16 form (latent_decode.cuh); a tile (codes in panels of T tokens x 128 dimensions,
// rope keys, units) is one stage of a ring.  Warps: 0 and 3 copy, 1 and 2 issue one product each, 4 to 11 do the softmax and the
// epilogue, 12 to 15 split the next segment's queries into their parts while this one's tiles run.
//
// What bounds it: the chain of a tile through the softmax warps (scores, maximum, exponentials, parts, hand-over: about 2,200
// cycles, where the bytes of a tile, 41 KB, take 1,800) and the end of a segment (6,800 cycles).  512 requests of 512..8,192 tokens,
// 32 heads: 290..294 us = 4.9 TB/s (bf16 pages: 425 us); two of 131,072: 57 us (66); one of 1,009: 16 us (13).  33 requests x 4 draft
// tokens x 128 heads: 281..286 us (bf16 pages: 225 us): 32 rows to a group where that form has 64, so the pages come twice as
// often, from L2.  Instructions count here as code: the kernel's roles share an instruction cache, and the epilogue in two places
// cost the 512 requests 23 us, unrolled once more 30 us.  dl = 512 at 32 rows spills 220 bytes a thread at its 128 registers.  Tried and not
// kept, when the kernel took 317 us: four softmax warps (341), two groups of four that take the tiles in turn (399); when it took 290:
// weights in two places so that the next are written while these are read (316), the products of a tile's scores a tile ahead (313),
// both (332), queries read twice instead of held (318).
//
// Every wait is bounded; an expired one sets the workspace's status word (6) and ends the CTA.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "latent_decode.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 512, kSoft = 256;  // of the softmax: two warps for the same query rows, half of a tile's tokens each
constexpr float kLazy = 4.f;   // log2 of the growth that forces a rescale
constexpr int kLowest = -100;  // of a query row's exponent

template <int DL_, int N_> struct Cfg {
    static constexpr int DL = DL_, N = N_, D = DL + 64;
    static constexpr int MT = DL / 128;                        // panels of codes, blocks of value dimensions
    static constexpr int PB = T * 128;                         // bytes of a panel
    static constexpr int STAGE = (MT + 1) * PB;                // codes, rope keys
    static constexpr int QB = 2 * N * 128;                     // bytes of a query panel
    static constexpr int Q_BYTES = (MT + 1) * QB, P_BYTES = 3 * N * 128;
    static constexpr int OFF_P = Q_BYTES, OFF_RING = OFF_P + P_BYTES;
    // 229,376 bytes: 227 KB less what the kernel declares itself (3 KB at the most)
    static constexpr int FIT = (229376 - 1024 - OFF_RING) / (STAGE + T * 4);
    static constexpr int RING = FIT < 6 ? FIT : 6;             // tiles in flight
    static constexpr int OFF_UNIT = OFF_RING + RING * STAGE;   // the units (fp32 2^e), T a stage
    static constexpr int SMEM = OFF_UNIT + RING * T * 4 + 1024;
    static constexpr int COL_S = 384;                          // of tensor memory: O^T before it, two tiles of S from there
    static_assert(3 * N * MT <= COL_S && RING >= 2 && SMEM <= 229376, "tensor memory and shared memory");
};

struct Maps {
    CUtensorMap codes, rope;
};

template <class C> struct Bars {
    uint64_t full[C::RING], empty[C::RING], q_full, q_free, s[2], s_free[2], p, o, rope, drain[2];
};

// Two fp32 values -> fp16 pair (low, high); then e4m3 parts of it: code pair of the rounding, `h` left with 16 times the rest.
__device__ __forceinline__ uint32_t half2_of(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t part_of(uint32_t &h)
{
    const __half2 x = *reinterpret_cast<const __half2 *>(&h);
    const __nv_fp8x2_storage_t c = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
    const __half2 r = __hmul2(__hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3))), __float2half2_rn(16.f));
    h = *reinterpret_cast<const uint32_t *>(&r);
    return c;
}

// Smallest k with |x| <= 2^p (1 + f / 2^23) 2^k for the finite magnitude bits `most`.
__device__ __forceinline__ int exponent_for(uint32_t most, int p, uint32_t f)
{
    if (most < 0x00800000u) return kLowest;
    return static_cast<int>(most >> 23) - 127 - p + ((most & 0x007fffffu) > f ? 1 : 0);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
__device__ __forceinline__ uint32_t bf16x2_finite_magnitude(uint32_t u) { return u & 0x7fff7fffu & ~bf16x2_not_finite(u); }

template <int DL, int N>
__global__ void __launch_bounds__(kThreads, 1) latent_decode8_kernel(Params p, const __grid_constant__ Maps maps)
{
    using C = Cfg<DL, N>;
    extern __shared__ char smem_raw[];
    char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) Bars<C> bar;
    __shared__ uint32_t tmem_base;
    __shared__ int32_t not_finite;                    // segments (from 1) of the last value that was taken out
    __shared__ float corr[N], fac[N], worth[N], top[2][N];
    __shared__ float2 lm[2][N];                       // l and m of the halves of a tile's tokens
    __shared__ uint32_t grown;                        // rows that are rescaled
    __shared__ float kept[2][N];                      // set aside: maximum that the sums are relative to, l
    __shared__ float q_unit[4][N];                    // 2^a of a segment's query rows, four segments deep: see the splitting warps
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
        for (int j = 0; j < C::RING; ++j) mbar_init(&bar.full[j], 2), mbar_init(&bar.empty[j], 1);
        mbar_init(&bar.q_full, 128), mbar_init(&bar.q_free, 1);
        mbar_init(&bar.p, kSoft), mbar_init(&bar.o, 1), mbar_init(&bar.rope, 1);
        for (int j = 0; j < 2; ++j) mbar_init(&bar.s[j], 1), mbar_init(&bar.s_free[j], kSoft), mbar_init(&bar.drain[j], 1);
        not_finite = 0;
        fence_mbar_init();
    }
    before_next();
    after_previous();
    if (tid == 0) {
        if (cta == 0) *p.status = 0;
        p.item0[cta] = p.item1[cta] = -1;
    }
    find_share<kThreads>(p, sums, edge);
    const uint32_t tmem = tmem_base;

    const int32_t total = static_cast<int32_t>(edge[1].tiles_before - edge[0].tiles_before);
    Walk w{};
    if (total > 0) {
        w.r = edge[0].r;
        w.load(p);
        w.group = edge[0].group;
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
        // Warp 0 copies the first half of the code panels and the units, warp 3 the other half and the rope keys.
        const int part = warp == 0 ? 0 : 1, u0 = part * (C::MT / 2);
        const int32_t br = p.box_rows, page = static_cast<int32_t>(p.a.page);
        // page (an out-of-range coordinate, read as zeros, where the number is invalid) and row of chunk `lane`
        auto lookup = [&](const Walk &x, int32_t *pg, int32_t *row) {
            const int32_t t = x.tile * T + lane * br;
            *pg = 0, *row = 0;
            if (lane * br < T && t < x.n) {
                const int32_t e = p.a.block_table[x.slot * p.a.table_stride + t / page];
                *pg = e >= 0 && e < p.a.cache.n_rows ? e : static_cast<int32_t>(p.a.cache.n_rows);
                *row = t % page;
            }
        };
        int32_t pg = 0, row = 0, i = 0;
        if (total > 0) lookup(w, &pg, &row);
        bool ok = true;  // the same in every lane
        for (; i < total; ++i) {
            Walk nx = w;
            nx.next(p);
            int32_t pg_next = 0, row_next = 0;
            if (i + 1 < total) lookup(nx, &pg_next, &row_next);
            const int32_t valid = w.n - w.tile * T < T ? w.n - w.tile * T : T;
            const int32_t chunks = (valid + br - 1) / br;
            const int s = i % C::RING;
            if (!(ok = wait(&bar.empty[s], ((i / C::RING) & 1) ^ 1))) break;
            char *stage = smem + C::OFF_RING + s * C::STAGE;
            float *units = reinterpret_cast<float *>(smem + C::OFF_UNIT) + s * T;
            int32_t bytes = chunks * br * (C::MT / 2 * 128 + (part == 0 ? 0 : 128));
            if (part == 0) {  // the units are plain copies: of an invalid page they are zeros from here
                const bool there = lane < chunks && pg < p.a.cache.n_rows;
                bytes += __popc(__ballot_sync(0xffffffffu, there)) * br * 4;
                if (lane < chunks && !there)
                    for (int32_t e = 0; e < br; ++e) units[lane * br + e] = 0.f;
                __syncwarp();
            }
            if (elect_one()) mbar_arrive_expect_tx(&bar.full[s], bytes);
            __syncwarp();
            for (int32_t c = 0; c < chunks; ++c) {
                const int32_t z = __shfl_sync(0xffffffffu, pg, c), y = __shfl_sync(0xffffffffu, row, c);
                if (elect_one()) {
                    char *dst = stage + c * br * 128;
#pragma unroll
                    for (int u = 0; u < C::MT / 2; ++u) tma_load_3d(dst + (u0 + u) * C::PB, &maps.codes, 128 * (u0 + u), y, z, &bar.full[s]);
                    if (part == 1)
                        tma_load_3d(dst + C::MT * C::PB, &maps.rope, 0, y, z, &bar.full[s]);
                    else if (z < p.a.cache.n_rows)
                        bulk_g2s(units + c * br, static_cast<const char *>(p.a.cache.data) + z * p.a.cache.row_stride +
                                     static_cast<int64_t>(page) * (DL + 128) + static_cast<int64_t>(y) * 4,
                                 br * 4, &bar.full[s]);
                }
                __syncwarp();
            }
            w = nx, pg = pg_next, row = row_next;
        }
        if (!ok && lane == 0)  // gave up: the copies in flight land before the CTA ends (bounded)
            for (int32_t e = i > C::RING ? i - C::RING : 0; e < i; ++e) mbar_wait(&bar.full[e % C::RING], (e / C::RING) & 1, kWaitLimit);
    } else if (warp == 1 && total > 0) {
        // ----------------------------------------------------- first product: S
        constexpr uint32_t kId8 = tc::idesc_e4m3(64, T, false), kId16 = tc::idesc_bf16(64, T, false);
        const uint32_t base = smem_u32(smem);
        const uint64_t q_desc = tc::sdesc_sw128(base, 16, 1024), x_desc = tc::sdesc_sw128(base + C::OFF_RING, 16, 1024);
        int slot = 0, segs = 0;
        uint32_t par = 0;
        bool ok = true;
        for (int32_t i = 0; i < total && ok; ++i) {
            const uint32_t d = tmem + C::COL_S + T * (i & 1);
            if (i > 1) ok = wait(&bar.s_free[i & 1], ((i >> 1) & 1) ^ 1);
            if (ok && __all_sync(0xffffffffu, i == 0 || w.first())) ok = wait(&bar.q_full, segs++ & 1);
            if (!ok || !(ok = wait(&bar.full[slot], par))) break;
            tc::fence_after_sync();
            const uint64_t x = x_desc + slot * (C::STAGE >> 4);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    tc::mma_bf16(d, q_desc + (C::MT * C::QB >> 4) + ks * 2, x + (C::MT * C::PB >> 4) + ks * 2, kId16, ks > 0 ? 1u : 0u);
                tc::commit(&bar.rope);
            }
            __syncwarp();
            // products of another operand type join the sum only when these have: their order is promised within a type
            if (!(ok = wait(&bar.rope, i & 1))) break;
            tc::fence_after_sync();
            const bool last = __all_sync(0xffffffffu, w.last()) != 0;
            if (elect_one()) {
#pragma unroll
                for (int u = 0; u < C::MT; ++u)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc::mma_e4m3(d, q_desc + (u * C::QB >> 4) + ks * 2, x + (u * C::PB >> 4) + ks * 2, kId8, 1u);
                tc::commit(&bar.s[i & 1]);
                if (last) tc::commit(&bar.q_free);
            }
            __syncwarp();
            if (++slot == C::RING) slot = 0, par ^= 1u;
            w.next(p);
        }
        if (elect_one()) tc::commit(&bar.drain[0]);  // everything issued has completed before tensor memory is given back
        mbar_wait(&bar.drain[0], 0, kWaitLimit);
    } else if (warp == 2 && total > 0) {
        // --------------------------------------------------- second product: O^T
        constexpr uint32_t kId = tc::idesc_e4m3(128, 3 * N, true);
        const uint32_t base = smem_u32(smem);
        const uint64_t p_desc = tc::sdesc_sw128(base + C::OFF_P, 16, 1024), val_desc = tc::sdesc_sw128(base + C::OFF_RING, C::PB, 1024);
        int slot = 0;
        int32_t tile0 = w.tile;  // the segment's first
        bool ok = true;
        for (int32_t i = 0; i < total && ok; ++i) {
            if (w.first()) tile0 = 0;
            const uint32_t more = __all_sync(0xffffffffu, ((w.tile - tile0) & (kSumTiles - 1)) == 0) ? 0u : 1u;
            if (!(ok = wait(&bar.p, i & 1))) break;
            tc::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)  // 32 tokens a step
                        tc::mma_e4m3(tmem + mt * 3 * N, val_desc + ((slot * C::STAGE + mt * C::PB) >> 4) + ks * 256, p_desc + ks * 2, kId,
                                     ks > 0 ? 1u : more);
                tc::commit(&bar.empty[slot]);
                tc::commit(&bar.o);
            }
            __syncwarp();
            if (++slot == C::RING) slot = 0;
            w.next(p);
        }
        if (elect_one()) tc::commit(&bar.drain[1]);
        mbar_wait(&bar.drain[1], 0, kWaitLimit);
    } else if (warp >= 12 && total > 0) {
        // --------------------------------------------------- queries into their parts
        constexpr int TPR = 128 / N, UNITS = DL / 16 / TPR;  // threads a row; 16 values of the latent part a unit
        const int qt = tid - 384, row = qt / TPR, j = qt % TPR;
        const int rho = 16 * (row >> 3) + (row & 7);  // of the first part; the second is 8 rows behind
        int32_t segs = 0;
        bool ok = true;
        for (int32_t i = 0; i < total && ok; ++segs) {
            const int rr = w.group * N + row;
            uint4 x[UNITS][2], rp[8 / TPR];
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.a.q) + (w.r * p.rows + rr) * C::D;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int u = 0; u < UNITS; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) x[u][e] = rr < p.rows ? ld_v4(q + (u * TPR + j) * 16 + 8 * e) : zero;
#pragma unroll
            for (int e = 0; e < 8 / TPR; ++e) rp[e] = rr < p.rows ? ld_v4(q + DL + (e * TPR + j) * 8) : zero;
            auto magnitude = [](uint4 v) {
                const uint32_t a = __vmaxu2(bf16x2_finite_magnitude(v.x), bf16x2_finite_magnitude(v.y)),
                               b = __vmaxu2(bf16x2_finite_magnitude(v.z), bf16x2_finite_magnitude(v.w));
                return __vmaxu2(a, b);
            };
            uint32_t most = 0, most_r = 0;
#pragma unroll
            for (int u = 0; u < UNITS; ++u) most = __vmaxu2(most, __vmaxu2(magnitude(x[u][0]), magnitude(x[u][1])));
#pragma unroll
            for (int e = 0; e < 8 / TPR; ++e) most_r = __vmaxu2(most_r, magnitude(rp[e]));
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) {
                most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
                most_r = __vmaxu2(most_r, __shfl_xor_sync(0xffffffffu, most_r, o));
            }
            const uint32_t top = max(most << 16, most & 0xffff0000u), top_r = max(most_r << 16, most_r & 0xffff0000u);
            const int a = max(max(exponent_for(top, 8, 0x600000u), exponent_for(top_r, 64, 0u)), kLowest);
            const float down = power_of_two(-a);
            // x: of each 16 values the 16 codes of the first parts and those of the second
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                uint32_t c1[4], c2[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint4 v = x[u][e >> 1];
                    const uint32_t w2[2] = {e & 1 ? v.z : v.x, e & 1 ? v.w : v.y};
                    uint32_t p1[2], p2[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t bad = bf16x2_not_finite(w2[k]);  // infinities as NaN
                        uint32_t h = half2_of(bf16_lo(w2[k]) * down, bf16_hi(w2[k]) * down) | (bad & 0x7fff7fffu);
                        p1[k] = part_of(h);
                        p2[k] = part_of(h);
                    }
                    c1[e] = p1[0] | p1[1] << 16;
                    c2[e] = p2[0] | p2[1] << 16;
                }
                x[u][0] = make_uint4(c1[0], c1[1], c1[2], c1[3]);
                x[u][1] = make_uint4(c2[0], c2[1], c2[2], c2[3]);
            }
#pragma unroll
            for (int e = 0; e < 8 / TPR; ++e) {
                const uint4 v = rp[e];
                rp[e] = make_uint4(pack_bf16x2(bf16_lo(v.x) * down, bf16_hi(v.x) * down), pack_bf16x2(bf16_lo(v.y) * down, bf16_hi(v.y) * down),
                                   pack_bf16x2(bf16_lo(v.z) * down, bf16_hi(v.z) * down), pack_bf16x2(bf16_lo(v.w) * down, bf16_hi(v.w) * down));
            }
            // the products of the segment before have read its parts (q_unit: the softmax has read the unit of the last
            // segment but two, since a tile's scores wait for the softmax of the last tile but one)
            if (segs > 0 && !(ok = wait(&bar.q_free, (segs - 1) & 1))) break;
            if (j == 0) q_unit[segs & 3][row] = power_of_two(a);
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                const int unit = u * TPR + j;
                char *to = smem + (unit >> 3) * C::QB + rho * 128 + (((unit & 7) ^ (rho & 7)) << 4);
                *reinterpret_cast<uint4 *>(to) = x[u][0];
                *reinterpret_cast<uint4 *>(to + 8 * 128) = x[u][1];
            }
#pragma unroll
            for (int e = 0; e < 8 / TPR; ++e) {
                char *to = smem + C::MT * C::QB + rho * 128 + (((e * TPR + j) ^ (rho & 7)) << 4);
                *reinterpret_cast<uint4 *>(to) = rp[e];
                *reinterpret_cast<uint4 *>(to + 8 * 128) = zero;
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar.q_full);
            i += w.tiles - w.tile;  // to the next segment
            w.tile = w.tiles - 1;
            w.next(p);
        }
    } else if (warp >= 4 && total > 0) {
        // --------------------------------------------------- softmax and epilogue
        const int quad = warp & 3, half = (warp - 4) >> 2, g = lane >> 2, t = lane & 3, st = tid - 128;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16);
        const bool active = 8 * quad < N;  // this warp holds the parts of query rows 8 quad ... + 7
        const int row = 8 * quad + g;
        constexpr int HT = T / 2;  // a half's tokens
        float m = -INFINITY, big = -INFINITY, l = 0.f, unit = 0.f;  // m, l: of this half; big: the maximum M of z + e
        int32_t seen = 0;
        int slot_out = 0;
        int32_t segments = 0, tile0 = 0;  // tile0: the segment's first
        // The accumulator and l leave tensor memory and registers: they are set aside, or (`end`) the segment ends with them.
        auto finish = [&](int32_t i, bool begun, bool end, bool whole) {
            const int64_t part = 2 * cta + slot_out;
            if (active) {
                float sum = l;
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (t == 0) lm[half][row] = make_float2(sum, m);
            }
            soft_any<kSoft>(false);
            if (active && half == 0 && t == 0) {
                const float2 a = lm[0][row], b = lm[1][row];
                const float mm = fmaxf(a.y, b.y);
                float sum = a.x * rebase(a.y, mm) + b.x * rebase(b.y, mm);
                float back = begun ? rebase(kept[0][row], mm) : 0.f;
                if (begun) sum = fmaf(kept[1][row], back, sum);
                kept[0][row] = mm, kept[1][row] = sum;
                // a weight's 16 parts, and from M to m: the sums come to be relative to m as l is
                float f = mm == -INFINITY || big == -INFINITY ? 0.0625f : 0.0625f * exp2f(big - mm);
                const int rr = w.group * N + row;
                if (whole) {
                    const float inv = inverse(sum);
                    f *= inv, back *= inv;
                    if (p.a.lse != nullptr && rr < p.rows) p.a.lse[w.r * p.rows + rr] = log_sum(mm, sum);
                } else if (end) {
                    p.ml[part * N + row] = make_float4(mm, sum, sum, 0.f);
                }
                fac[row] = f;
                worth[row] = back;
            }
            l = 0.f, big = -INFINITY;
            wait(&bar.o, i & 1);
            tc::fence_after_sync();
            soft_any<kSoft>(false);  // fac, worth are complete
            const int valid = p.rows - w.group * N < N ? p.rows - w.group * N : N;
            const int dim = 32 * quad + lane;
            const bool taken = end && not_finite == segments;
#pragma unroll 1
            for (int c0 = 16 * half; c0 < C::MT * N; c0 += 32) {
                const int mt = c0 / N, row0 = c0 % N;
                uint32_t o1[16], o2[16], o3[16];
                tc::ld16(tl + mt * 3 * N + row0, o1);
                tc::ld16(tl + mt * 3 * N + N + row0, o2);
                tc::ld16(tl + mt * 3 * N + 2 * N + row0, o3);
                tc::wait_ld();
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[e] = fmaf(fmaf(__uint_as_float(o3[e]), 0.0625f, __uint_as_float(o2[e])), 0.0625f, __uint_as_float(o1[e])) * fac[row0 + e];
                float *part_at = p.part + (part * N + row0) * DL + mt * 128 + dim;
                if (begun) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = fmaf(part_at[e * DL], worth[row0 + e], v[e]);
                }
                if (taken) {  // draft tokens' values that were taken out, to the rows that see them
                    const int32_t last = min(w.n, (w.tile + 1) * T);
                    for (int32_t tok = max(w.n - (p.a.L - 1), tile0 * T); tok < last; ++tok) {
                        const int32_t e = p.a.block_table[w.slot * p.a.table_stride + tok / p.a.page];
                        if (e < 0 || e >= p.a.cache.n_rows) continue;
                        const uint8_t code = static_cast<const uint8_t *>(p.a.cache.data)[e * p.a.cache.row_stride +
                                                                                           tok % p.a.page * DL + mt * 128 + dim];
                        if ((code & 0x7fu) != 0x7fu) continue;
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const int r2 = w.group * N + row0 + q;
                            if (r2 < p.rows && tok < w.n - (p.a.L - 1 - r2 / p.a.h)) v[q] = NAN;
                        }
                    }
                }
                if (whole) {
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.a.out) + (w.r * p.rows + w.group * N + row0) * DL + mt * 128 + dim;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (row0 + e < valid) out[e * DL] = __float2bfloat16_rn(v[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (!end || row0 + e < valid) part_at[e * DL] = v[e];
                }
            }
            tc::fence_before_sync();
            soft_any<kSoft>(false);  // fac and worth may be written again
        };
        // a thread that gave up goes on without waiting: all of them meet at every barrier
        for (int32_t i = 0; i < total; ++i) {
            const bool fresh = i == 0 || w.first();
            if (fresh) {
                slot_out = w.first() ? 1 : 0;  // where a part that is not the whole goes
                ++segments;
                tile0 = w.tile;
                m = big = -INFINITY;
                l = 0.f;
                const int rr = w.group * N + row;
                seen = active && rr < p.rows ? w.n - (p.a.L - 1 - rr / p.a.h) : 0;
            }
            const int stage = i % C::RING;
            wait(&bar.s[i & 1], (i >> 1) & 1);
            tc::fence_after_sync();
            // The copies were complete for S; their own barrier, which turns again only behind this tile's second product, is looked at
            // so that this is seen here too (behind the scores' loads: 512 requests 294 us, drafts 286 us; without the look 291 and 285 us).
            auto seen_here = [&]() {
                if (lane == 0) mbar_test(&bar.full[stage], (i / C::RING) & 1);
                __syncwarp();
            };
            const int32_t t0 = w.tile * T, th = t0 + HT * half;
            float u[HT / 4];  // z + e of tokens th + 8 j + 2 t, + 1
            float mu = -INFINITY;
            if (active) {
                if (fresh) unit = q_unit[(segments - 1) & 3][row] * p.scale_log2;
                float z[HT / 4];
                const float *units = reinterpret_cast<const float *>(smem + C::OFF_UNIT) + stage * T + HT * half + 2 * t;
                uint32_t s[16];
                ld_16x256b_x4(tl + C::COL_S + T * (i & 1) + HT * half, s);
                seen_here();
                tc::wait_ld();
                tc::fence_before_sync();
                mbar_arrive(&bar.s_free[i & 1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 un = *reinterpret_cast<const float2 *>(units + 8 * j);
                    const float2 zz = mul2(mul2(fma2(make_float2(__uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3])),
                                                     make_float2(0.0625f, 0.0625f),
                                                     make_float2(__uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1]))),
                                                un), make_float2(unit, unit));
                    // 2^23 + (e + 127), the exponent's bits behind those of 2^23
                    const float2 e = make_float2(__uint_as_float(__float_as_uint(un.x) >> 23 | 0x4b000000u),
                                                 __uint_as_float(__float_as_uint(un.y) >> 23 | 0x4b000000u));
                    const float2 uu = add2(add2(e, make_float2(-8388735.f, -8388735.f)), zz);
                    z[2 * j] = zz.x, z[2 * j + 1] = zz.y, u[2 * j] = uu.x, u[2 * j + 1] = uu.y;
                }
                if (th + HT > seen) {
#pragma unroll
                    for (int j = 0; j < HT / 4; ++j)
                        if (th + 8 * (j >> 1) + 2 * t + (j & 1) >= seen) z[j] = u[j] = -INFINITY;
                }
                float mx = z[0];
                mu = u[0];
#pragma unroll
                for (int j = 1; j < HT / 4; ++j) mx = fmaxf(mx, z[j]), mu = fmaxf(mu, u[j]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, 2));
                if (mx > m) {
                    if (m != -INFINITY) l *= ex2_approx(m - mx);
                    m = mx;
                }
                const float base = m == -INFINITY ? 0.f : m;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < HT / 4; ++j) sum += ex2_approx(z[j] - base);
                l += sum;
            } else {
                seen_here();
                mbar_arrive(&bar.s_free[i & 1]);
            }
            const bool first = big == -INFINITY;  // nothing summed yet
            const bool grew = soft_any<kSoft>(active && (first ? mu != -INFINITY : mu > big + kLazy));
            if (grew) {  // rarely: both halves take one M, the columns of the rows that grew are rescaled
                if (st == 0) grown = 0;
                if (active && t == 0) top[half][row] = mu;
                soft_any<kSoft>(false);
                if (active) {
                    mu = fmaxf(top[0][row], top[1][row]);
                    if (first) {
                        big = mu;
                    } else if (mu > big + kLazy) {
                        if (half == 0 && t == 0) corr[row] = ex2_approx(big - mu), atomicOr(&grown, 1u << row);
                        big = mu;
                    }
                }
                soft_any<kSoft>(false);
            }
            // the second product of the tile before has read P and written O^T
            if (i > 0 && !__all_sync(0xffffffffu, mbar_test(&bar.o, (i - 1) & 1))) wait(&bar.o, (i - 1) & 1);
            tc::fence_after_sync();
            if (active) {
                const float above = (big == -INFINITY ? 0.f : big) - 4.f;  // weights 16 times, as fp16 pairs
                char *pr = smem + C::OFF_P + row * 128 + 2 * t;
                uint32_t h[HT / 8];
#pragma unroll
                for (int j = 0; j < HT / 8; ++j) h[j] = half2_of(ex2_approx(u[2 * j] - above), ex2_approx(u[2 * j + 1] - above));
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int j = 0; j < HT / 8; ++j)
                        *reinterpret_cast<uint16_t *>(pr + k * N * 128 + (((2 * half + (j >> 1)) ^ (row & 7)) << 4 | (j & 1) << 3)) =
                            static_cast<uint16_t>(part_of(h[j]));
            }
            char *codes = smem + C::OFF_RING + stage * C::STAGE;
            if (w.n - t0 < T) {  // rows behind the last token: whatever they hold must not meet P = 0
                const int from = w.n - t0;
                for (int e = st; e < (T - from) * C::MT * 8; e += kSoft)
                    *reinterpret_cast<uint4 *>(codes + ((e >> 3) % C::MT) * C::PB + (from + (e >> 3) / C::MT) * 128 + (e & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            if (p.a.L > 1 && t0 + T > w.n - (p.a.L - 1)) {  // draft tokens: a NaN must not meet P = 0 either
                const int from = max(w.n - (p.a.L - 1) - t0, 0), to = min(w.n - t0, T);
                for (int e = st; e < (to - from) * C::MT * 8; e += kSoft) {
                    uint4 *x = reinterpret_cast<uint4 *>(codes + ((e >> 3) % C::MT) * C::PB + (from + (e >> 3) / C::MT) * 128 + (e & 7) * 16);
                    const uint4 v = *x;
                    auto nan4 = [](uint32_t c) { return __vcmpeq4(c & 0x7f7f7f7fu, 0x7f7f7f7fu); };
                    const uint4 bad = make_uint4(nan4(v.x), nan4(v.y), nan4(v.z), nan4(v.w));
                    if (bad.x | bad.y | bad.z | bad.w) {
                        not_finite = segments;
                        *x = make_uint4(v.x & ~bad.x, v.y & ~bad.y, v.z & ~bad.z, v.w & ~bad.w);
                    }
                }
            }
            if (grew) {
                for (uint32_t rows = grown; rows != 0; rows &= rows - 1) {
                    const int r2 = __ffs(rows) - 1;
                    constexpr int COLS = 3 * C::MT / 2;  // this half's
                    uint32_t o[COLS];
#pragma unroll
                    for (int c = 0; c < COLS; ++c) ld1(tl + (half * COLS + c) * N + r2, o[c]);
                    tc::wait_ld();
#pragma unroll
                    for (int c = 0; c < COLS; ++c) st1(tl + (half * COLS + c) * N + r2, __float_as_uint(__uint_as_float(o[c]) * corr[r2]));
                }
                tc::wait_st();
            }
            fence_proxy_async_smem();
            tc::fence_before_sync();
            mbar_arrive(&bar.p);
            // the segment ends here, or the next tile's product does not add to what the accumulator holds
            const bool last = w.last(), over = last || i + 1 == total;
            if (over || ((w.tile + 1 - tile0) & (kSumTiles - 1)) == 0) {
                const bool whole = last && slot_out == 1;
                if (over && !whole && st == 0) (slot_out ? p.item1 : p.item0)[cta] = static_cast<int32_t>(w.r * p.rows + w.group * N);
                finish(i, w.tile - tile0 >= kSumTiles, over, whole);
            }
            w.next(p);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 3) tc::tmem_dealloc(tmem, 512);
}

int rows_per_group(int64_t rows) { return rows <= 16 ? 16 : 32; }

// Box of 128 bytes x `rows` rows of [n_pages][page][n0] elements, strides in bytes, 128-byte swizzle.
bool encode8(CUtensorMap *map, CUtensorMapDataType type, int cols, const char *base, int64_t n0, int64_t n1, int64_t n2, int64_t s1,
            int64_t s2, int rows)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = prefill::tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(n0), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1), static_cast<cuuint64_t>(s2)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(rows), 1}, elem[3] = {1, 1, 1};
    return fn(map, type, 3, const_cast<char *>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DL, int N> cudaError_t launch(Params p, cudaStream_t st)
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
    const char *data = static_cast<const char *>(p.a.cache.data);
    const int64_t P = p.a.page, pages = p.a.cache.n_rows, pitch = p.a.cache.row_stride;
    if (!encode8(&maps.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 128, data, DL, P, pages, DL, pitch, p.box_rows) ||
        !encode8(&maps.rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 64, data + P * DL, 64, P, pages, 128, pitch, p.box_rows))
        return cudaErrorInvalidValue;
    auto kern = latent_decode8_kernel<DL, N>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    auto join = latent_join_kernel<DL, N>;  // with the main kernel's split between shared memory and L1 cache, as in the bf16 form
    if ((e = cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
        return e;
    if ((e = launch_overlapped(kern, dim3(grid), dim3(kThreads), C::SMEM, st, p, maps)) != cudaSuccess) return e;
    return launch_overlapped(join, dim3(grid * kJoinCtas), dim3(256), static_cast<size_t>(grid) * 16, st, p, static_cast<int32_t>(grid));
}

}  // namespace

size_t latent_decode8_workspace(int64_t, int32_t L, int32_t h, int32_t dl)
{
    const size_t n = rows_per_group(static_cast<int64_t>(L) * h), grid = static_cast<size_t>(sm_count());
    return up256(256 + 8 * grid) + 2 * grid * n * (16 + static_cast<size_t>(dl) * 4);
}

cudaError_t launch_latent_decode8(const LatentDecodeArgs &a, cudaStream_t st)
{
    Params p{};
    p.a = a;
    p.rows = a.L * a.h;
    p.scale_log2 = a.scale * kLog2e;
    p.box_rows = box_rows(a.page);
    if (rows_per_group(p.rows) == 16) return a.dl == 512 ? launch<512, 16>(p, st) : launch<256, 16>(p, st);
    return a.dl == 512 ? launch<512, 32>(p, st) : launch<256, 32>(p, st);
}

}  // namespace kda
