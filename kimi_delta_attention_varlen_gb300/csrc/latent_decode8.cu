// Absorbed latent attention over 8-bit pages (kda_latent_decode8).
//
// One CTA a query row: blocks of tokens in turn, one token a thread for the scores, then one dimension (or two) a
// thread for the values, with a running maximum and sum.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float value_of(uint8_t code)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}

template <int DL> __global__ void __launch_bounds__(kThreads) decode8_kernel(LatentDecodeArgs a)
{
    constexpr int D = DL + 64, PER = DL / kThreads;
    __shared__ float q[D], p[kThreads], red[kThreads];
    __shared__ int32_t page_of[kThreads];
    const int tid = threadIdx.x;
    before_next();
    after_previous();
    const int64_t rows = static_cast<int64_t>(a.L) * a.h, at = blockIdx.x, r = at / rows;
    const int64_t slot = a.req == nullptr ? r : a.idx_type == KDA_I32 ? static_cast<const int32_t *>(a.req)[r] : static_cast<const int64_t *>(a.req)[r];
    int64_t n = 0;
    if (slot >= 0 && slot < a.requests) {
        n = a.seq_lens[slot];
        n = n < 0 ? 0 : n > a.width * a.page ? a.width * a.page : n;
    }
    n -= a.L - 1 - at % rows / a.h;
    if (at == 0 && tid == 0) *static_cast<int32_t *>(a.workspace) = 0;
    for (int d = tid; d < D; d += kThreads) q[d] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[at * D + d]) * (a.scale * kLog2e);
    float m = -INFINITY, l = 0.f, o[PER] = {};
    for (int64_t t0 = 0; t0 < n; t0 += kThreads) {
        const int64_t t = t0 + tid;
        float z = -INFINITY;
        int32_t page = -1;
        __syncthreads();
        if (t < n) {
            page = a.block_table[slot * a.table_stride + t / a.page];
            z = 0.f;
            if (page >= 0 && page < a.cache.n_rows) {
                const char *base = static_cast<const char *>(a.cache.data) + page * a.cache.row_stride;
                const int64_t s = t % a.page;
                const uint8_t *codes = reinterpret_cast<const uint8_t *>(base + s * DL);
                const __nv_bfloat16 *rope = reinterpret_cast<const __nv_bfloat16 *>(base + a.page * DL + s * 128);
                for (int d = 0; d < DL; ++d) z = fmaf(q[d], value_of(codes[d]), z);
                for (int d = 0; d < 64; ++d) z = fmaf(q[DL + d], __bfloat162float(rope[d]), z);
                z *= *reinterpret_cast<const float *>(base + a.page * (DL + 128) + s * 4);
            } else {
                page = -1;
            }
        }
        page_of[tid] = page;
        red[tid] = z;
        __syncthreads();
        float mx = m;
        for (int j = 0; j < kThreads; ++j) mx = fmaxf(mx, red[j]);
        const float base = mx == -INFINITY ? 0.f : mx, f = m == mx ? 1.f : exp2f(m - base);
        p[tid] = t < n ? exp2f(z - base) : 0.f;
        m = mx;
        float lb = 0.f, ob[PER] = {};  // the block's own sums: small weights are added to each other first
        __syncthreads();
        const int most = n - t0 < kThreads ? static_cast<int>(n - t0) : kThreads;
        for (int j = 0; j < most; ++j) {
            lb += p[j];
            if (page_of[j] < 0) continue;
            const char *base8 = static_cast<const char *>(a.cache.data) + page_of[j] * a.cache.row_stride;
            const int64_t s = (t0 + j) % a.page;
            const float w = p[j] * *reinterpret_cast<const float *>(base8 + a.page * (DL + 128) + s * 4);
            for (int e = 0; e < PER; ++e) ob[e] = fmaf(w, value_of(reinterpret_cast<const uint8_t *>(base8)[s * DL + tid + e * kThreads]), ob[e]);
        }
        l = fmaf(l, f, lb);
        for (int e = 0; e < PER; ++e) o[e] = fmaf(o[e], f, ob[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < PER; ++e) static_cast<__nv_bfloat16 *>(a.out)[at * DL + tid + e * kThreads] = __float2bfloat16_rn(o[e] * inv);
    if (tid == 0 && a.lse != nullptr) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

size_t latent_decode8_workspace(int64_t, int32_t, int32_t, int32_t) { return 256; }

cudaError_t launch_latent_decode8(const LatentDecodeArgs &a, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>(a.batch * a.L * a.h));
    return launch_overlapped(a.dl == 512 ? decode8_kernel<512> : decode8_kernel<256>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace kda
