// Rows of latents into 8-bit pages (kda_latent_append8) and out of pages (kda_latent_read).
//
// A token is one warp's: append8 has the row in registers (dl / 32 + 2 values a lane), takes the largest magnitudes of
// its latent and of its rope key by shuffles and from them the token's unit 2^e, scales (exact: a power of two) and
// rounds once.  Reading back multiplies by 2^e, exact in bf16 for every code.  Loads and stores are whole 16- or 8-byte
// vectors, consecutive across the warp.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_internal.h"
#include "page_lists.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8, kRope = 64;
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

__device__ __forceinline__ uint32_t codes2(float a, float b)  // infinities as NaN: e4m3 has none
{
    const float2 v = make_float2(fabsf(a) < INFINITY ? a : NAN, fabsf(b) < INFINITY ? b : NAN);
    return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

// Eight consecutive values of a row of x.
template <typename X> __device__ __forceinline__ void load8(const X *p, float (&v)[8]);
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 u = ld_v4(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
}
template <> __device__ __forceinline__ void load8<float>(const float *p, float (&v)[8])
{
    const uint4 a = ld_v4(p), b = ld_v4(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
}

template <typename X, int DL>
__global__ void __launch_bounds__(32 * kWarps) append8_kernel(const X *x, LatentRowsArgs a)
{
    before_next();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (tok >= a.total || tok < a.cu[0] || tok >= a.cu[a.count]) return;
    const X *from = x + tok * a.stride;
    float c[DL / 256][8], r[2];
#pragma unroll
    for (int e = 0; e < DL / 256; ++e) load8(from + 256 * e + 8 * lane, c[e]);
    r[0] = load_as_f32(from + DL + 2 * lane), r[1] = load_as_f32(from + DL + 2 * lane + 1);
    const int64_t i = entry_of(a.cu, a.count, tok), req = load_index(a.req, a.idx_type, i);
    if (req < 0 || req >= a.table.requests || tok >= a.cu[i + 1]) return;
    const int64_t pos = length_of(a.table, req) - a.cu[i + 1] + tok;
    if (pos < 0) return;
    const int32_t page = a.table.block_table[req * a.table.table_stride + pos / a.table.page_size];
    if (page < 0 || page >= a.table.n_pages) return;

    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < DL / 256; ++e)
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max(most, finite_magnitude(c[e][j]));
    const int k = exponent_for(warp_max(most), 8, 0x600000u);  // 448 = 2^8 * 1.75
    const int kr = exponent_for(warp_max(max(finite_magnitude(r[0]), finite_magnitude(r[1]))), 64, 0u);
    const int exponent = max(max(k, kr), kLowest);             // at most 120
    const float unit = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);

    const Place8 at = place8(a.table.page_size, pos % a.table.page_size, DL);
    char *to = static_cast<char *>(a.cache.data) + page * a.cache.row_stride;
#pragma unroll
    for (int e = 0; e < DL / 256; ++e) {
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[j] = codes2(c[e][4 * j] * unit, c[e][4 * j + 1] * unit) | codes2(c[e][4 * j + 2] * unit, c[e][4 * j + 3] * unit) << 16;
        *reinterpret_cast<uint2 *>(to + at.codes + 256 * e + 8 * lane) = make_uint2(w[0], w[1]);
    }
    *reinterpret_cast<uint32_t *>(to + at.rope + 4 * lane) = pack_bf16x2(r[0] * unit, r[1] * unit);
    if (lane == 0) *reinterpret_cast<float *>(to + at.scale) = __uint_as_float(static_cast<uint32_t>(127 + exponent) << 23);
}

__device__ __forceinline__ uint32_t values2(uint32_t codes, float scale)  // two codes (low halfword) as bf16 values
{
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3));
    const float2 v = __half22float2(h);
    return pack_bf16x2(v.x * scale, v.y * scale);
}

template <int DL, bool Eight>
__global__ void __launch_bounds__(32 * kWarps) read_kernel(LatentRowsArgs a)
{
    before_next();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (row >= a.total || row < a.cu[0] || row >= a.cu[a.count]) return;
    const int64_t i = entry_of(a.cu, a.count, row), req = load_index(a.req, a.idx_type, i);
    if (row >= a.cu[i + 1]) return;
    const int64_t pos = row - a.cu[i] + (a.first != nullptr ? a.first[i] : 0);
    int32_t page = -1;
    if (req >= 0 && req < a.table.requests && pos >= 0 && pos < length_of(a.table, req))
        page = a.table.block_table[req * a.table.table_stride + pos / a.table.page_size];
    const bool valid = page >= 0 && page < a.table.n_pages;
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.rows) + row * a.stride;
    const int64_t slot = pos % a.table.page_size;
    uint4 v[DL / 256];
    uint32_t rope = 0;
#pragma unroll
    for (int e = 0; e < DL / 256; ++e) v[e] = make_uint4(0u, 0u, 0u, 0u);
    if (valid && Eight) {
        const char *from = static_cast<const char *>(a.cache.data) + page * a.cache.row_stride;
        const Place8 at = place8(a.table.page_size, slot, DL);
        uint2 w[DL / 256];
#pragma unroll
        for (int e = 0; e < DL / 256; ++e) w[e] = *reinterpret_cast<const uint2 *>(from + at.codes + 256 * e + 8 * lane);
        const uint32_t r = *reinterpret_cast<const uint32_t *>(from + at.rope + 4 * lane);
        const float scale = *reinterpret_cast<const float *>(from + at.scale);
#pragma unroll
        for (int e = 0; e < DL / 256; ++e)
            v[e] = make_uint4(values2(w[e].x, scale), values2(w[e].x >> 16, scale), values2(w[e].y, scale), values2(w[e].y >> 16, scale));
        rope = pack_bf16x2(bf16_lo(r) * scale, bf16_hi(r) * scale);
    } else if (valid) {
        const __nv_bfloat16 *from = static_cast<const __nv_bfloat16 *>(a.cache.data) + page * a.cache.row_stride + slot * (DL + kRope);
#pragma unroll
        for (int e = 0; e < DL / 256; ++e) v[e] = ld_v4(from + 256 * e + 8 * lane);
        rope = *reinterpret_cast<const uint32_t *>(from + DL + 2 * lane);
    }
#pragma unroll
    for (int e = 0; e < DL / 256; ++e) *reinterpret_cast<uint4 *>(to + 256 * e + 8 * lane) = v[e];
    *reinterpret_cast<uint32_t *>(to + DL + 2 * lane) = rope;
}

dim3 grid_of(int64_t total) { return dim3(static_cast<unsigned>((total + kWarps - 1) / kWarps)); }

}  // namespace

cudaError_t launch_latent_append8(const LatentRowsArgs &a, cudaStream_t st)
{
    const dim3 grid = grid_of(a.total), block(32 * kWarps);
    if (a.dtype == KDA_F32) {
        const float *x = static_cast<const float *>(a.rows);
        return launch_overlapped(a.dl == 512 ? append8_kernel<float, 512> : append8_kernel<float, 256>, grid, block, 0, st, x, a);
    }
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.rows);
    return launch_overlapped(a.dl == 512 ? append8_kernel<__nv_bfloat16, 512> : append8_kernel<__nv_bfloat16, 256>, grid, block, 0, st, x, a);
}

cudaError_t launch_latent_read(const LatentRowsArgs &a, cudaStream_t st)
{
    const dim3 grid = grid_of(a.total), block(32 * kWarps);
    if (a.cache.dtype == KDA_U8)
        return launch_overlapped(a.dl == 512 ? read_kernel<512, true> : read_kernel<256, true>, grid, block, 0, st, a);
    return launch_overlapped(a.dl == 512 ? read_kernel<512, false> : read_kernel<256, false>, grid, block, 0, st, a);
}

}  // namespace kda
