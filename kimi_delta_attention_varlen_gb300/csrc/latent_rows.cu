// Rows of latents into 8-bit pages (kda_latent_append8) and out of pages (kda_latent_read).
//
// Writing: a token is one warp's, which has the row in registers, takes the largest magnitudes of its latent and of its rope
// key across the warp and from them the token's unit 2^e, scales (exact: a power of two) and rounds once.  One power of two for a
// token and not an fp32 maximum / 448: e4m3's relative step is the same in every binade, so nothing is lost, and code * 2^e and
// rope * 2^-e are exact in bf16, whatever reads them.  Reading back multiplies by 2^e.
//
// What bounds it: bytes (644 + 1,152 a token), and before them the look-ups, five loads that wait for one another (offsets, request,
// length, page, row).  A CTA's rows are looked up together, a row a lane; reading keeps four rows a warp in flight behind them.
// 73,364 tokens: written in 29.9 us = 4.4 TB/s (fp32 rows 36.2 us = 6.0 TB/s), read in 24.1 us = 5.5 TB/s (one
// look-up a warp: 37.5 and 27.6 us); 24 new tokens 3.0 us.
// Loads and stores are whole 16- or 8-byte vectors, consecutive across the warp.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_internal.h"
#include "page_lists.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4, kRope = 64;
constexpr int kLowest = -64;  // of a token's exponent

// Where token `pos` of a page lies, in bytes from the page's start.
struct Place8 {
    int64_t codes, rope, scale;
};
__device__ __forceinline__ Place8 place8(int64_t page_size, int64_t slot, int dl)
{
    return Place8{slot * dl, page_size * dl + slot * 2 * kRope, page_size * (dl + 2 * kRope) + slot * 4};
}

// Smallest k with |x| <= top 2^k for the largest finite |x|, whose bits are `most`; top = 2^p (1 + f), f as fraction bits.
__device__ __forceinline__ int exponent_for(uint32_t most, int p, uint32_t f)
{
    if (most < 0x00800000u) return kLowest;  // 0 or subnormal: below 2^-126
    return static_cast<int>(most >> 23) - 127 - p + ((most & 0x007fffffu) > f ? 1 : 0);
}

__device__ __forceinline__ uint32_t finite_magnitude(float x)
{
    const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

__device__ __forceinline__ uint32_t warp_max(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

__device__ __forceinline__ uint32_t codes2(float a, float b) { return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3); }

// Eight consecutive values of a row of x, as they are (until they are needed they take half of the registers in bf16).
template <typename X> struct Eight8 {
    static constexpr int V = sizeof(X) / 2;
    uint4 u[V];
    __device__ void load(const X *p)
    {
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = ld_v4(p + e * 16 / sizeof(X));
    }
    __device__ void values(float (&v)[8]) const
    {
        if (V == 1) {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
        } else {
            const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[V - 1].x, u[V - 1].y, u[V - 1].z, u[V - 1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
        }
    }
};

// Of a CTA's rows: where each one's token is. By warp 0: the entry of the CTA's first row is looked for by the whole warp, the
// others follow from it (rows of one entry lie together), a row a lane.
struct Spot {
    int32_t page, slot;  // page: -1 where there is no such token, -2 where the row is no entry's
};

template <int Rows, bool Read>
__device__ __forceinline__ void find_spots(const LatentRowsArgs &a, int64_t row0, Spot *spots)
{
    const int lane = threadIdx.x & 31;
    const int64_t begin = a.cu[0], behind = a.cu[a.count];
    const int64_t row = row0 + lane;
    const int64_t from = row0 < begin ? begin : row0;
    Spot x{-2, 0};
    if (from < behind && from < row0 + Rows) {
        int64_t i = entry_of(a.cu, a.count, from);
        if (lane < Rows && row >= begin && row < behind && row < a.total) {
            int64_t end = a.cu[i + 1];
            for (int step = 0; row >= end && i + 1 < a.count; ++step) {
                if (step == 3) {  // many entries without rows between: the last one that begins at or before this row
                    int64_t hi = a.count;
                    while (hi - i > 1) {
                        const int64_t mid = (i + hi) >> 1;
                        if (a.cu[mid] <= row) i = mid;
                        else hi = mid;
                    }
                    end = a.cu[i + 1];
                    break;
                }
                end = a.cu[++i + 1];
            }
            if (row < end) {
                x.page = -1;
                const int64_t req = load_index(a.req, a.idx_type, i);
                if (req >= 0 && req < a.table.requests) {
                    const int64_t n = length_of(a.table, req);
                    const int64_t pos = Read ? row - a.cu[i] + (a.first != nullptr ? a.first[i] : 0) : n - end + row;
                    if (pos >= 0 && pos < n) {
                        const int32_t e = a.table.block_table[req * a.table.table_stride + pos / a.table.page_size];
                        if (e >= 0 && e < a.table.n_pages) x = Spot{e, static_cast<int32_t>(pos % a.table.page_size)};
                    }
                }
            }
        }
    }
    if (lane < Rows) spots[lane] = x;
}

template <typename X, int DL, int Per>
__global__ void __launch_bounds__(32 * kWarps) append8_kernel(const X *x, LatentRowsArgs a)
{
    __shared__ Spot spots[kWarps * Per];
    before_next();
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kWarps * Per;
    Eight8<X> x8[Per][DL / 256];
    float r[Per][2];
    auto load = [&](int k) {
        if (row0 + warp + kWarps * k >= a.total) return;
        const X *from = x + (row0 + warp + kWarps * k) * a.stride;
#pragma unroll
        for (int e = 0; e < DL / 256; ++e) x8[k][e].load(from + 256 * e + 8 * lane);
        r[k][0] = load_as_f32(from + DL + 2 * lane), r[k][1] = load_as_f32(from + DL + 2 * lane + 1);
    };
#pragma unroll
    for (int k = 0; k < Per; ++k) load(k);
    if (warp == 0) find_spots<kWarps * Per, false>(a, row0, spots);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < Per; ++k) {
        const Spot spot = spots[warp + kWarps * k];
        if (spot.page < 0) continue;
        float c[DL / 256][8];
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < DL / 256; ++e) {
            x8[k][e].values(c[e]);
#pragma unroll
            for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(c[e][j]) & 0x7fffffffu);
        }
        most = warp_max(most);
        const bool finite = most < 0x7f800000u;  // of the latent, in every lane alike: then no value needs a look of its own
        if (!finite) {
            most = 0;
#pragma unroll
            for (int e = 0; e < DL / 256; ++e)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    most = max(most, finite_magnitude(c[e][j]));
                    if (!(fabsf(c[e][j]) < INFINITY)) c[e][j] = NAN;  // e4m3 has no infinities
                }
            most = warp_max(most);
        }
        const int kc = exponent_for(most, 8, 0x600000u);  // 448 = 2^8 * 1.75
        const int kr = exponent_for(warp_max(max(finite_magnitude(r[k][0]), finite_magnitude(r[k][1]))), 64, 0u);
        const int exponent = max(max(kc, kr), kLowest);             // at most 120
        const float unit = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);

        const Place8 place = place8(a.table.page_size, spot.slot, DL);
        char *to = static_cast<char *>(a.cache.data) + spot.page * a.cache.row_stride;
#pragma unroll
        for (int e = 0; e < DL / 256; ++e) {
            const float *v = c[e];
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[j] = codes2(v[4 * j] * unit, v[4 * j + 1] * unit) | codes2(v[4 * j + 2] * unit, v[4 * j + 3] * unit) << 16;
            *reinterpret_cast<uint2 *>(to + place.codes + 256 * e + 8 * lane) = make_uint2(w[0], w[1]);
        }
        *reinterpret_cast<uint32_t *>(to + place.rope + 4 * lane) = pack_bf16x2(r[k][0] * unit, r[k][1] * unit);
        if (lane == 0) *reinterpret_cast<float *>(to + place.scale) = __uint_as_float(static_cast<uint32_t>(127 + exponent) << 23);
    }
}

__device__ __forceinline__ uint32_t values2(uint32_t codes, float scale)  // two codes (low halfword) as bf16 values
{
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3));
    const float2 v = __half22float2(h);
    return pack_bf16x2(v.x * scale, v.y * scale);
}

template <int DL, bool Eight, int Per>
__global__ void __launch_bounds__(32 * kWarps) read_kernel(LatentRowsArgs a)
{
    __shared__ Spot spots[kWarps * Per];
    before_next();
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kWarps * Per;
    if (warp == 0) find_spots<kWarps * Per, true>(a, row0, spots);
    __syncthreads();
    uint4 v[Per][DL / 256];  // Eight: the codes in the first half
    uint32_t rope[Per];
    float scale[Per];
#pragma unroll
    for (int k = 0; k < Per; ++k) {  // all loads before the first store
        const Spot spot = spots[warp + kWarps * k];
        rope[k] = 0, scale[k] = 0.f;
#pragma unroll
        for (int e = 0; e < DL / 256; ++e) v[k][e] = make_uint4(0u, 0u, 0u, 0u);
        if (spot.page < 0) continue;
        if (Eight) {
            const char *from = static_cast<const char *>(a.cache.data) + spot.page * a.cache.row_stride;
            const Place8 place = place8(a.table.page_size, spot.slot, DL);
#pragma unroll
            for (int e = 0; e < DL / 256; ++e) {
                const uint2 w = *reinterpret_cast<const uint2 *>(from + place.codes + 256 * e + 8 * lane);
                v[k][e].x = w.x, v[k][e].y = w.y;
            }
            rope[k] = *reinterpret_cast<const uint32_t *>(from + place.rope + 4 * lane);
            scale[k] = *reinterpret_cast<const float *>(from + place.scale);
        } else {
            const __nv_bfloat16 *from = static_cast<const __nv_bfloat16 *>(a.cache.data) + spot.page * a.cache.row_stride +
                                        static_cast<int64_t>(spot.slot) * (DL + kRope);
#pragma unroll
            for (int e = 0; e < DL / 256; ++e) v[k][e] = ld_v4(from + 256 * e + 8 * lane);
            rope[k] = *reinterpret_cast<const uint32_t *>(from + DL + 2 * lane);
        }
    }
#pragma unroll
    for (int k = 0; k < Per; ++k) {
        if (spots[warp + kWarps * k].page == -2) continue;
        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.rows) + (row0 + warp + kWarps * k) * a.stride;
#pragma unroll
        for (int e = 0; e < DL / 256; ++e) {
            const uint4 w = v[k][e];
            *reinterpret_cast<uint4 *>(to + 256 * e + 8 * lane) =
                Eight ? make_uint4(values2(w.x, scale[k]), values2(w.x >> 16, scale[k]), values2(w.y, scale[k]), values2(w.y >> 16, scale[k])) : w;
        }
        *reinterpret_cast<uint32_t *>(to + DL + 2 * lane) = Eight ? pack_bf16x2(bf16_lo(rope[k]) * scale[k], bf16_hi(rope[k]) * scale[k]) : rope[k];
    }
}

// Rows a warp (kWarps times that many are at most 32).  73,364 tokens of 512 + 64 values: written in 29.6 us with 1 or 2, 31.8 with
// 4 (a step's 24 tokens 3.1, 3.8 and 5.2); read in 24.3 us with 4 or 8, 26.6 with 1.
constexpr int kPerAppend = 1, kPerRead = 4;

dim3 grid_of(int64_t total, int per) { return dim3(static_cast<unsigned>((total + kWarps * per - 1) / (kWarps * per))); }

}  // namespace

cudaError_t launch_latent_append8(const LatentRowsArgs &a, cudaStream_t st)
{
    const dim3 grid = grid_of(a.total, kPerAppend), block(32 * kWarps);
    if (a.dtype == KDA_F32) {
        const float *x = static_cast<const float *>(a.rows);
        return launch_overlapped(a.dl == 512 ? append8_kernel<float, 512, kPerAppend> : append8_kernel<float, 256, kPerAppend>, grid, block, 0, st, x, a);
    }
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.rows);
    return launch_overlapped(a.dl == 512 ? append8_kernel<__nv_bfloat16, 512, kPerAppend> : append8_kernel<__nv_bfloat16, 256, kPerAppend>, grid,
                             block, 0, st, x, a);
}

cudaError_t launch_latent_read(const LatentRowsArgs &a, cudaStream_t st)
{
    const dim3 grid = grid_of(a.total, kPerRead), block(32 * kWarps);
    if (a.cache.dtype == KDA_U8)
        return launch_overlapped(a.dl == 512 ? read_kernel<512, true, kPerRead> : read_kernel<256, true, kPerRead>, grid, block, 0, st, a);
    return launch_overlapped(a.dl == 512 ? read_kernel<512, false, kPerRead> : read_kernel<256, false, kPerRead>, grid, block, 0, st, a);
}

}  // namespace kda
