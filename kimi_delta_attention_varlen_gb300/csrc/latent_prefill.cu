// Expanded latent attention over a varlen batch (kda_latent_prefill).
//
// One warp a query, eight queries of one head a CTA; tiles of 32 keys and
// values pass through shared memory once for the eight queries, with the
// running maximum and sum of the softmax in registers.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kTile = 32;
constexpr int kRows = 8;
constexpr int DN = 128, DR = 64, DV = 128, D = DN + DR;

__global__ void __launch_bounds__(kRows * 32) latent_prefill_kernel(LatentPrefillArgs a)
{
    __shared__ __nv_bfloat16 ks[kTile][D + 2], vs[kTile][DV], qs[kRows][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = blockIdx.y;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows, i = first + warp;
    auto seq_of = [&](int64_t t) {  // the sequence b with cu_q[b] <= t < cu_q[b + 1]
        int64_t lo = 0, hi = a.num_seqs;
        while (lo + 1 < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (a.cu_q[mid] <= t) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    const int64_t last = first + kRows < a.total_q ? first + kRows : a.total_q;
    const int64_t mine = i < a.total_q ? seq_of(i) : -1;
    if (i < a.total_q) {
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + (i * a.h + head) * D;
        for (int e = lane; e < D; e += 32) qs[warp][e] = q[e];
    }
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t b = seq_of(first); b <= seq_of(last - 1); ++b) {  // the CTA's queries may belong to several sequences
        const int64_t k0 = a.cu_k[b], nk = a.cu_k[b + 1] - k0, nq = a.cu_q[b + 1] - a.cu_q[b];
        const int64_t seen = mine == b ? i - a.cu_q[b] + nk - nq + 1 : 0;
        for (int64_t t0 = 0; t0 < nk; t0 += kTile) {
            __syncthreads();
            for (int j = warp; j < kTile; j += kRows) {
                const int64_t t = k0 + t0 + j;
                const bool ok = t0 + j < nk && t < a.total_k;
                const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16 *>(a.k_nope) + t * a.kn_token + head * a.kn_head;
                const __nv_bfloat16 *kr = static_cast<const __nv_bfloat16 *>(a.k_rope) + t * a.kr_token;
                const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + t * a.v_token + head * a.v_head;
                const __nv_bfloat16 zero = __float2bfloat16_rn(0.f);
                for (int e = lane; e < D; e += 32) ks[j][e] = !ok ? zero : e < DN ? kn[e] : kr[e - DN];
                for (int e = lane; e < DV; e += 32) vs[j][e] = ok ? v[e] : zero;
            }
            __syncthreads();
            float z = 0.f;
            for (int e = 0; e < D; ++e) z += __bfloat162float(qs[warp][e]) * __bfloat162float(ks[lane][e]);
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
            for (int e = 0; e < 4; ++e) o[e] *= c;
            for (int j = 0; j < kTile; ++j) {
                const float w = __shfl_sync(0xffffffffu, p, j);
                if (w != 0.f)  // a key that is not seen adds nothing, whatever its value holds
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] += w * __bfloat162float(vs[j][lane + 32 * e]);
            }
        }
    }
    if (i >= a.total_q) return;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (i * a.h + head) * DV;
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[lane + 32 * e] = __float2bfloat16_rn(o[e] * inv);
    if (lane == 0 && a.lse != nullptr) a.lse[i * a.h + head] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t latent_prefill_workspace(int64_t, int64_t, int32_t) { return 256; }

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t st)
{
    cudaError_t e = cudaMemsetAsync(a.workspace, 0, 4, st);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((a.total_q + kRows - 1) / kRows), static_cast<unsigned>(a.h));
    latent_prefill_kernel<<<grid, kRows * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
