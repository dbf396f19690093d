// Absorbed latent attention over paged latents (kda_latent_decode).
//
// One warp a query row (one head of one query token), eight rows a CTA; tiles
// of 32 tokens pass through shared memory once for the eight rows.  Per tile,
// lane j holds token j's score; the running maximum m, the sum l of
// e^{z - m} and the output are rescaled by e^{m_old - m_new} when m grows, so
// the latents are read once.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kTile = 32;
constexpr int kRows = 8;

template <int DL, int DR>
__global__ void __launch_bounds__(kRows * 32) latent_decode_kernel(LatentDecodeArgs a)
{
    constexpr int D = DL + DR, PER = DL / 32;
    __shared__ __nv_bfloat16 kv[kTile][D + 2];
    __shared__ __nv_bfloat16 qs[kRows][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = blockIdx.y;
    const int row = blockIdx.x * kRows + warp, rows = a.L * a.h;
    int64_t slot = r;
    if (a.req != nullptr)
        slot = a.idx_type == KDA_I32 ? static_cast<const int32_t *>(a.req)[r] : static_cast<const int64_t *>(a.req)[r];
    int64_t n = 0;
    if (slot >= 0 && slot < a.requests) {
        const int64_t most = a.width * a.page;
        n = a.seq_lens[slot];
        n = n < 0 ? 0 : n > most ? most : n;
    }
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + (r * rows + row) * D;
    if (row < rows)
        for (int e = lane; e < D; e += 32) qs[warp][e] = q[e];
    const int64_t seen = row < rows ? n - (a.L - 1 - row / a.h) : 0;
    float m = -INFINITY, l = 0.f, o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    const __nv_bfloat16 *cache = static_cast<const __nv_bfloat16 *>(a.cache.data);
    for (int64_t t0 = 0; t0 < n; t0 += kTile) {
        __syncthreads();
        for (int j = warp; j < kTile; j += kRows) {
            const int64_t t = t0 + j;
            int64_t page = -1;
            if (t < n) page = a.block_table[slot * a.table_stride + t / a.page];
            const bool ok = page >= 0 && page < a.cache.n_rows;
            const __nv_bfloat16 *x = cache + (ok ? page * a.cache.row_stride + (t % a.page) * D : 0);
            for (int e = lane; e < D; e += 32) kv[j][e] = ok ? x[e] : __float2bfloat16_rn(0.f);
        }
        __syncthreads();
        float z = 0.f;
        for (int e = 0; e < D; ++e) z += __bfloat162float(qs[warp][e]) * __bfloat162float(kv[lane][e]);
        z = t0 + lane < seen ? z * a.scale : -INFINITY;
        float mx = z;
        for (int s = 16; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        mx = fmaxf(mx, m);
        const float base = mx == -INFINITY ? 0.f : mx;
        const float p = expf(z - base), c = expf(m - base);
        float sum = p;
        for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        l = l * c + sum;
        m = mx;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] *= c;
        for (int j = 0; j < kTile; ++j) {
            const float w = __shfl_sync(0xffffffffu, p, j);
            if (w != 0.f)  // a token that is not seen adds nothing, whatever its row holds
#pragma unroll
                for (int e = 0; e < PER; ++e) o[e] += w * __bfloat162float(kv[j][lane + 32 * e]);
        }
    }
    if (row >= rows) return;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (r * rows + row) * DL;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) out[lane + 32 * e] = __float2bfloat16_rn(o[e] * inv);
    if (lane == 0 && a.lse != nullptr) a.lse[r * rows + row] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t latent_decode_workspace(int64_t, int32_t, int32_t, int32_t) { return 256; }

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t st)
{
    cudaError_t e = cudaMemsetAsync(a.workspace, 0, 4, st);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((a.L * a.h + kRows - 1) / kRows), static_cast<unsigned>(a.batch));
    if (a.dl == 512) latent_decode_kernel<512, 64><<<grid, kRows * 32, 0, st>>>(a);
    else latent_decode_kernel<256, 64><<<grid, kRows * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
