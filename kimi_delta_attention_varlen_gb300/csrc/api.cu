// C ABI of the KDA hot path: argument validation on the host (metadata only,
// before any launch) and dispatch to the kernel launchers.
//
// Fail-closed, as the "vllm-ascend KDA state copy" page requires ("Startup
// preparation": bad layouts and metadata are rejected before compile or
// launch; "Numeric contract": an empty selection validates metadata and
// launches nothing).  No call allocates, synchronises or keeps a pointer.
#include <cuda_runtime.h>

#include "kda_internal.h"

namespace {

thread_local cudaError_t t_last_cuda = cudaSuccess;

int cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return KDA_OK;
    t_last_cuda = e;
    return KDA_ERR_CUDA;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t esize(int32_t dtype) { return dtype == KDA_F32 ? 4 : 2; }

bool valid_dtype(int32_t d) { return d == KDA_F32 || d == KDA_BF16; }

bool valid_itype(int32_t t) { return t == KDA_I32 || t == KDA_I64; }

bool built_head_size(int32_t dk, int32_t dv) { return dk == dv && (dk == 32 || dk == 64 || dk == 128); }

// The prefill has a compact form (the fused kernel, no per-chunk records) for bf16 at head size 128.
bool compact_form(int32_t io_dtype, int32_t dk) { return io_dtype == KDA_BF16 && dk == 128; }

// Layout predicate of the state-copy page ("Automatic dispatch"): fp32/bf16,
// n_rows > 0, positive inner sizes, rows that do not overlap.
int check_cache(const kda_cache *c, kda::CacheDesc *out)
{
    if (c == nullptr || c->data == nullptr) return KDA_ERR_NULL;
    if (!valid_dtype(c->dtype)) return KDA_ERR_DTYPE;
    if (c->reserved != 0) return KDA_ERR_LAYOUT;
    if (c->n_rows <= 0 || c->h <= 0 || c->v <= 0 || c->k <= 0) return KDA_ERR_LAYOUT;
    const int64_t lim = INT64_C(1) << 40;
    if (c->h > lim || c->v > lim || c->k > lim) return KDA_ERR_RANGE;
    const __int128 payload = static_cast<__int128>(c->h) * c->v * c->k;
    if (payload > (INT64_C(1) << 40)) return KDA_ERR_RANGE;
    if (c->row_stride < static_cast<int64_t>(payload)) return KDA_ERR_LAYOUT;
    const __int128 bytes = static_cast<__int128>(c->n_rows) * c->row_stride * esize(c->dtype);
    if (bytes > (static_cast<__int128>(1) << 62)) return KDA_ERR_RANGE;
    if (!aligned(c->data, static_cast<uintptr_t>(esize(c->dtype)))) return KDA_ERR_ALIGN;
    *out = kda::CacheDesc{c->data, c->dtype, c->n_rows, c->h, c->v, c->k, c->row_stride};
    return KDA_OK;
}

int check_index_array(const void *idx, int32_t idx_type)
{
    if (idx == nullptr) return KDA_ERR_NULL;
    if (!aligned(idx, idx_type == KDA_I32 ? 4 : 8)) return KDA_ERR_ALIGN;
    return KDA_OK;
}

}  // namespace

int kda::record_cuda_status(cudaError_t e) { return cuda_status(e); }

extern "C" {

int kda_state_gather(const kda_cache *cache, const void *idx, int32_t idx_type, int64_t selected,
                     const uint8_t *flags, void *packed, void *stream)
{
    kda::CacheDesc c{};
    int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if (!valid_itype(idx_type)) return KDA_ERR_DTYPE;
    if (selected < 0) return KDA_ERR_SHAPE;
    if (selected == 0) return KDA_OK;
    if ((rc = check_index_array(idx, idx_type)) != KDA_OK) return rc;
    if (packed == nullptr) return KDA_ERR_NULL;
    if (!aligned(packed, static_cast<uintptr_t>(esize(c.dtype)))) return KDA_ERR_ALIGN;
    if (static_cast<__int128>(selected) * c.h * c.v * c.k * esize(c.dtype) > (static_cast<__int128>(1) << 62))
        return KDA_ERR_RANGE;
    return cuda_status(kda::launch_state_gather(c, idx, idx_type, selected, flags, packed,
                                                static_cast<cudaStream_t>(stream)));
}

int kda_state_scatter(const kda_cache *cache, const void *idx, int32_t idx_type, int64_t selected,
                      const void *packed, int32_t packed_dtype, void *stream)
{
    kda::CacheDesc c{};
    int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if (!valid_itype(idx_type) || !valid_dtype(packed_dtype)) return KDA_ERR_DTYPE;
    if (selected < 0) return KDA_ERR_SHAPE;
    if (selected == 0) return KDA_OK;
    if ((rc = check_index_array(idx, idx_type)) != KDA_OK) return rc;
    if (packed == nullptr) return KDA_ERR_NULL;
    if (!aligned(packed, static_cast<uintptr_t>(esize(packed_dtype)))) return KDA_ERR_ALIGN;
    if (static_cast<__int128>(selected) * c.h * c.v * c.k * 4 > (static_cast<__int128>(1) << 62))
        return KDA_ERR_RANGE;
    return cuda_status(kda::launch_state_scatter(c, idx, idx_type, selected, packed, packed_dtype,
                                                 static_cast<cudaStream_t>(stream)));
}

size_t kda_prefill_workspace_size(int64_t total_tokens, int64_t num_seqs, int32_t h, int32_t dk, int32_t dv)
{
    if (!built_head_size(dk, dv)) return 0;
    kda::PrefillLayout L{};
    if (!kda::prefill_layout(total_tokens, num_seqs, h, dk, &L)) return 0;
    return L.total;
}

size_t kda_prefill_workspace_size_compact(int64_t total_tokens, int64_t num_seqs, int32_t h, int32_t dk, int32_t dv,
                                          int32_t io_dtype)
{
    if (!built_head_size(dk, dv) || !valid_dtype(io_dtype)) return 0;
    kda::PrefillLayout L{};
    if (!kda::prefill_layout(total_tokens, num_seqs, h, dk, &L)) return 0;
    return compact_form(io_dtype, dk) ? L.compact : L.total;
}

namespace {
// Shared by every prefill entry point; `se` says where states come from and go
// (its cache fields are validated by the caller).
int prefill_impl(const void *q, const void *k, const void *v, int32_t io_dtype, const float *g, const float *beta,
                 const int32_t *cu_seqlens, int64_t num_seqs, int64_t total_tokens, int32_t h, int32_t dk,
                 int32_t dv, float scale, int32_t qk_l2norm, const kda::StateEnds &se, void *out, void *workspace,
                 size_t ws_bytes, void *stream, void *const *events)
{
    if (!valid_dtype(io_dtype)) return KDA_ERR_DTYPE;
    if (se.init != nullptr && !valid_dtype(se.init_dtype)) return KDA_ERR_DTYPE;
    if (num_seqs < 1 || total_tokens < 0 || h < 1 || dk < 1 || dv < 1) return KDA_ERR_SHAPE;
    if (!built_head_size(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if (total_tokens >= (INT64_C(1) << 31) || num_seqs >= (INT64_C(1) << 30) || h > 65535)
        return KDA_ERR_RANGE;
    if (static_cast<__int128>(total_tokens) * h * dk >= (static_cast<__int128>(1) << 62)) return KDA_ERR_RANGE;
    if (cu_seqlens == nullptr || workspace == nullptr) return KDA_ERR_NULL;
    if (total_tokens > 0 && (q == nullptr || k == nullptr || v == nullptr || g == nullptr || beta == nullptr ||
                             out == nullptr))
        return KDA_ERR_NULL;
    const void *vec16[] = {q, k, v, g, out, se.init, se.final_state, se.out_cache, se.ckpt};
    for (const void *p : vec16)
        if (p != nullptr && !aligned(p, 16)) return KDA_ERR_ALIGN;
    if (!aligned(beta, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_ALIGN;
    kda::PrefillLayout L{};
    if (!kda::prefill_layout(total_tokens, num_seqs, h, dk, &L)) return KDA_ERR_SHAPE;
    if (L.n_chunk_max >= (INT64_C(1) << 31)) return KDA_ERR_RANGE;
    // one-dimensional launch grids: chunk preparation (chunks x heads) and the state pass
    // ((sequence, head) pairs x at most 8 value slices), checked before anything is launched
    if (L.n_chunk_max * h >= (INT64_C(1) << 31) || num_seqs * h * 8 >= (INT64_C(1) << 31)) return KDA_ERR_RANGE;
    if (!aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
    if (ws_bytes < (compact_form(io_dtype, dk) ? L.compact : L.total)) return KDA_ERR_WORKSPACE;
    kda::PrefillArgs a{q, k, v, io_dtype, g, beta, cu_seqlens, num_seqs, total_tokens, h, dk, scale,
                       qk_l2norm ? 1 : 0, se, out, workspace, ws_bytes, events};
    return cuda_status(kda::launch_prefill(a, L, static_cast<cudaStream_t>(stream)));
}

kda::StateEnds packed_ends(const void *init_state, int32_t init_dtype, float *final_state)
{
    kda::StateEnds se{};
    se.init = init_state;
    se.init_dtype = init_dtype;
    se.final_state = final_state;
    return se;
}
}  // namespace

int kda_prefill_varlen(const void *q, const void *k, const void *v, int32_t io_dtype, const float *g,
                       const float *beta, const int32_t *cu_seqlens, int64_t num_seqs, int64_t total_tokens,
                       int32_t h, int32_t dk, int32_t dv, float scale, int32_t qk_l2norm, const void *init_state,
                       int32_t init_dtype, float *final_state, void *out, void *workspace, size_t ws_bytes,
                       void *stream)
{
    return prefill_impl(q, k, v, io_dtype, g, beta, cu_seqlens, num_seqs, total_tokens, h, dk, dv, scale,
                        qk_l2norm, packed_ends(init_state, init_dtype, final_state), out, workspace, ws_bytes,
                        stream, nullptr);
}

int kda_prefill_varlen_timed(const void *q, const void *k, const void *v, int32_t io_dtype, const float *g,
                             const float *beta, const int32_t *cu_seqlens, int64_t num_seqs,
                             int64_t total_tokens, int32_t h, int32_t dk, int32_t dv, float scale,
                             int32_t qk_l2norm, const void *init_state, int32_t init_dtype, float *final_state,
                             void *out, void *workspace, size_t ws_bytes, void *stream, void *const *events)
{
    if (events == nullptr) return KDA_ERR_NULL;  // NULL entries: boundaries left unrecorded
    return prefill_impl(q, k, v, io_dtype, g, beta, cu_seqlens, num_seqs, total_tokens, h, dk, dv, scale,
                        qk_l2norm, packed_ends(init_state, init_dtype, final_state), out, workspace, ws_bytes,
                        stream, events);
}

int kda_prefill_varlen_cached(const void *q, const void *k, const void *v, int32_t io_dtype, const float *g,
                              const float *beta, const int32_t *cu_seqlens, int64_t num_seqs, int64_t total_tokens,
                              int32_t h, int32_t dk, int32_t dv, float scale, int32_t qk_l2norm,
                              const kda_cache *cache, const void *idx_in, const uint8_t *flags,
                              const void *idx_out, int32_t idx_type, float *final_state, void *checkpoints,
                              int32_t ckpt_dtype, int32_t ckpt_every, int64_t ckpt_slots, void *out,
                              void *workspace, size_t ws_bytes, void *stream)
{
    kda::CacheDesc c{};
    int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if (!valid_itype(idx_type)) return KDA_ERR_DTYPE;
    if (c.h != h || c.k != dk || c.v != dv) return KDA_ERR_SHAPE;
    if (!aligned(c.data, 16) || (c.row_stride * esize(c.dtype)) % 16 != 0) return KDA_ERR_ALIGN;
    if ((rc = check_index_array(idx_in, idx_type)) != KDA_OK) return rc;
    if (idx_out != nullptr && (rc = check_index_array(idx_out, idx_type)) != KDA_OK) return rc;
    if (checkpoints != nullptr) {
        if (!valid_dtype(ckpt_dtype)) return KDA_ERR_DTYPE;
        if (ckpt_every <= 0 || ckpt_every % 64 != 0 || ckpt_slots < 0) return KDA_ERR_SHAPE;
    }
    kda::StateEnds se{};
    se.init = c.data;
    se.init_dtype = c.dtype;
    se.in_idx = idx_in;
    se.in_flags = flags;
    se.idx_type = idx_type;
    se.n_rows = c.n_rows;
    se.row_stride = c.row_stride;
    se.final_state = final_state;
    se.out_cache = idx_out != nullptr ? c.data : nullptr;
    se.out_dtype = c.dtype;
    se.out_idx = idx_out;
    se.ckpt = checkpoints;
    se.ckpt_dtype = ckpt_dtype;
    se.ckpt_every = checkpoints != nullptr ? ckpt_every : 0;
    se.ckpt_slots = ckpt_slots;
    return prefill_impl(q, k, v, io_dtype, g, beta, cu_seqlens, num_seqs, total_tokens, h, dk, dv, scale,
                        qk_l2norm, se, out, workspace, ws_bytes, stream, nullptr);
}

int64_t kda_prefill_checkpoint_count(const int32_t *cu_seqlens_host, int64_t num_seqs, int32_t ckpt_every)
{
    if (cu_seqlens_host == nullptr || num_seqs < 1 || ckpt_every <= 0 || ckpt_every % 64 != 0) return -1;
    int64_t n = 0;
    for (int64_t b = 0; b < num_seqs; ++b) {
        const int64_t len = static_cast<int64_t>(cu_seqlens_host[b + 1]) - cu_seqlens_host[b];
        if (len < 0) return -1;
        n += len / ckpt_every;
    }
    return n;
}

int kda_decode_step(const void *q, const void *k, const void *v, int32_t io_dtype, const float *g,
                    const float *beta, int64_t batch, int32_t h, int32_t dk, int32_t dv, float scale,
                    int32_t qk_l2norm, const kda_cache *cache, const void *idx, int32_t idx_type, void *out,
                    void *stream)
{
    kda::CacheDesc c{};
    int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if (!valid_dtype(io_dtype) || !valid_itype(idx_type)) return KDA_ERR_DTYPE;
    if (batch < 0 || h < 1 || dk < 1 || dv < 1) return KDA_ERR_SHAPE;
    if (!built_head_size(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if (c.h != h || c.k != dk || c.v != dv) return KDA_ERR_SHAPE;
    if (batch == 0) return KDA_OK;
    if (batch * static_cast<int64_t>(h) >= (INT64_C(1) << 31)) return KDA_ERR_RANGE;
    if ((rc = check_index_array(idx, idx_type)) != KDA_OK) return rc;
    if (q == nullptr || k == nullptr || v == nullptr || g == nullptr || beta == nullptr || out == nullptr)
        return KDA_ERR_NULL;
    const void *vec16[] = {q, k, v, g, out, c.data};
    for (const void *p : vec16)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    if (!aligned(beta, 4)) return KDA_ERR_ALIGN;
    if ((c.row_stride * esize(c.dtype)) % 16 != 0) return KDA_ERR_ALIGN;
    kda::DecodeArgs a{q, k, v, io_dtype, g, beta, batch, h, dk, scale, qk_l2norm ? 1 : 0, c, idx, idx_type, out};
    return cuda_status(kda::launch_decode_step(a, static_cast<cudaStream_t>(stream)));
}

namespace {
// Shared checks of the INT8 checkpoint calls: a built head size, 16-byte rows,
// aligned index arrays and checkpoint buffers.
int check_ckpt_args(const kda_cache *active, kda::CacheDesc *c, const void *src, const void *dst,
                    int32_t idx_type, int64_t count, const void *qdata, const void *scale, int64_t n_slots)
{
    int rc = check_cache(active, c);
    if (rc != KDA_OK) return rc;
    if (!valid_itype(idx_type)) return KDA_ERR_DTYPE;
    if (count < 0 || n_slots < 0) return KDA_ERR_SHAPE;
    if (!built_head_size(static_cast<int32_t>(c->k), static_cast<int32_t>(c->v))) return KDA_ERR_UNSUPPORTED;
    if (c->h > 65535) return KDA_ERR_RANGE;
    if (count == 0) return KDA_OK;
    if (count * c->h >= (INT64_C(1) << 31)) return KDA_ERR_RANGE;
    if ((rc = check_index_array(src, idx_type)) != KDA_OK) return rc;
    if ((rc = check_index_array(dst, idx_type)) != KDA_OK) return rc;
    if (qdata == nullptr || scale == nullptr) return KDA_ERR_NULL;
    if (!aligned(qdata, 16) || !aligned(scale, 16) || !aligned(c->data, 16)) return KDA_ERR_ALIGN;
    if ((c->row_stride * esize(c->dtype)) % 16 != 0) return KDA_ERR_ALIGN;
    return KDA_OK;
}
}  // namespace

int kda_ckpt_store_int8(const kda_cache *active, const void *src_rows, const void *dst_slots, int32_t idx_type,
                        int64_t count, int8_t *qdata, float *scale, int64_t n_slots, void *stream)
{
    kda::CacheDesc c{};
    const int rc = check_ckpt_args(active, &c, src_rows, dst_slots, idx_type, count, qdata, scale, n_slots);
    if (rc != KDA_OK || count == 0) return rc;
    return cuda_status(kda::launch_ckpt_store_int8(c, src_rows, dst_slots, idx_type, count, qdata, scale, n_slots,
                                                   static_cast<cudaStream_t>(stream)));
}

int kda_ckpt_load_int8(const int8_t *qdata, const float *scale, int64_t n_slots, const void *src_slots,
                       const void *dst_rows, int32_t idx_type, int64_t count, const kda_cache *active, void *stream)
{
    kda::CacheDesc c{};
    const int rc = check_ckpt_args(active, &c, src_slots, dst_rows, idx_type, count, qdata, scale, n_slots);
    if (rc != KDA_OK || count == 0) return rc;
    return cuda_status(kda::launch_ckpt_load_int8(c, qdata, scale, n_slots, src_slots, dst_rows, idx_type, count,
                                                  static_cast<cudaStream_t>(stream)));
}

int kda_target_verify(const void *q, const void *k, const void *v, int32_t io_dtype, const float *g,
                      const float *beta, int64_t batch, int32_t L, int32_t h, int32_t dk, int32_t dv, float scale,
                      int32_t qk_l2norm, const kda_cache *cache, const void *idx, const kda_cache *pool,
                      const void *inter_idx, int32_t idx_type, void *out, void *stream)
{
    kda::CacheDesc c{}, pl{};
    int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if ((rc = check_cache(pool, &pl)) != KDA_OK) return rc;
    if (!valid_dtype(io_dtype) || !valid_itype(idx_type)) return KDA_ERR_DTYPE;
    if (batch < 0 || L < 1 || h < 1 || dk < 1 || dv < 1) return KDA_ERR_SHAPE;
    if (!built_head_size(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if (c.h != h || c.k != dk || c.v != dv || pl.h != h || pl.k != dk || pl.v != dv) return KDA_ERR_SHAPE;
    if (batch == 0) return KDA_OK;
    if (batch * static_cast<int64_t>(h) >= (INT64_C(1) << 31) || L > (1 << 20)) return KDA_ERR_RANGE;
    if ((rc = check_index_array(idx, idx_type)) != KDA_OK) return rc;
    if ((rc = check_index_array(inter_idx, idx_type)) != KDA_OK) return rc;
    if (q == nullptr || k == nullptr || v == nullptr || g == nullptr || beta == nullptr || out == nullptr)
        return KDA_ERR_NULL;
    const void *vec16[] = {q, k, v, g, c.data, pl.data};
    for (const void *p : vec16)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    if (!aligned(beta, 4) || !aligned(out, 4)) return KDA_ERR_ALIGN;
    if ((c.row_stride * esize(c.dtype)) % 16 != 0 || (pl.row_stride * esize(pl.dtype)) % 16 != 0)
        return KDA_ERR_ALIGN;
    kda::VerifyArgs a{q, k, v, io_dtype, g, beta, batch, L, h, dk, scale, qk_l2norm ? 1 : 0, c, idx, pl, inter_idx,
                      idx_type, out};
    return cuda_status(kda::launch_target_verify(a, static_cast<cudaStream_t>(stream)));
}

namespace {
int check_conv_common(const void *x, int32_t io_dtype, int64_t channels, int32_t width, const float *weight,
                      const float *bias, int32_t activation, const void *y)
{
    if (!valid_dtype(io_dtype)) return KDA_ERR_DTYPE;
    if (width < 2 || width > 4 || channels < 1) return KDA_ERR_UNSUPPORTED;
    if (channels % 8 != 0) return KDA_ERR_SHAPE;
    if (activation != 0 && activation != 1) return KDA_ERR_SHAPE;
    // channel blocks sit in the y dimension of the per-sequence and update grids
    if (channels > INT64_C(65535) * kda::kConvChannelsPerBlock) return KDA_ERR_RANGE;
    if (weight == nullptr) return KDA_ERR_NULL;
    const void *vec16[] = {x, weight, bias, y};
    for (const void *p : vec16)
        if (p != nullptr && !aligned(p, 16)) return KDA_ERR_ALIGN;
    return KDA_OK;
}
}  // namespace

int kda_conv1d_varlen(const void *x, int32_t io_dtype, const int32_t *cu_seqlens, int64_t num_seqs,
                      int64_t total_tokens, int64_t channels, int32_t width, const float *weight, const float *bias,
                      int32_t activation, const void *init_state, void *final_state, int32_t state_dtype, void *y,
                      void *stream)
{
    int rc = check_conv_common(x, io_dtype, channels, width, weight, bias, activation, y);
    if (rc != KDA_OK) return rc;
    if ((init_state != nullptr || final_state != nullptr) && !valid_dtype(state_dtype)) return KDA_ERR_DTYPE;
    if (num_seqs < 1 || total_tokens < 0) return KDA_ERR_SHAPE;
    if (num_seqs >= (INT64_C(1) << 30) || total_tokens >= (INT64_C(1) << 36)) return KDA_ERR_RANGE;
    if ((total_tokens + 15) / 16 >= (INT64_C(1) << 31)) return KDA_ERR_RANGE;
    // one-dimensional grid of (token block, channel block) pairs, token blocks of 8 or more tokens
    const int64_t cblocks = (channels + kda::kConvChannelsPerBlock - 1) / kda::kConvChannelsPerBlock;
    if ((total_tokens + 15) / 8 * cblocks > INT64_C(0x7fffffff)) return KDA_ERR_RANGE;
    if (cu_seqlens == nullptr) return KDA_ERR_NULL;
    if (total_tokens > 0 && (x == nullptr || y == nullptr)) return KDA_ERR_NULL;
    if (!aligned(cu_seqlens, 4)) return KDA_ERR_ALIGN;
    const void *st16[] = {init_state, final_state};
    for (const void *p : st16)
        if (p != nullptr && !aligned(p, 16)) return KDA_ERR_ALIGN;
    kda::Conv1dArgs a{x, io_dtype, cu_seqlens, num_seqs, total_tokens, channels, width, weight, bias, activation,
                      init_state, final_state, state_dtype, y};
    return cuda_status(kda::launch_conv1d_varlen(a, static_cast<cudaStream_t>(stream)));
}

int kda_conv1d_update(const void *x, int32_t io_dtype, int64_t batch, int64_t channels, int32_t width,
                      const float *weight, const float *bias, int32_t activation, const kda_cache *conv_cache,
                      const void *idx, int32_t idx_type, void *y, void *stream)
{
    kda::CacheDesc c{};
    int rc = check_cache(conv_cache, &c);
    if (rc != KDA_OK) return rc;
    if ((rc = check_conv_common(x, io_dtype, channels, width, weight, bias, activation, y)) != KDA_OK) return rc;
    if (!valid_itype(idx_type)) return KDA_ERR_DTYPE;
    if (c.h != 1 || c.v != width - 1 || c.k != channels) return KDA_ERR_SHAPE;
    if (batch < 0) return KDA_ERR_SHAPE;
    if (batch == 0) return KDA_OK;
    if (batch >= (INT64_C(1) << 31)) return KDA_ERR_RANGE;
    if ((rc = check_index_array(idx, idx_type)) != KDA_OK) return rc;
    if (x == nullptr || y == nullptr) return KDA_ERR_NULL;
    if (!aligned(c.data, 16) || (c.row_stride * esize(c.dtype)) % 16 != 0) return KDA_ERR_ALIGN;
    kda::Conv1dUpdateArgs a{x, io_dtype, batch, channels, width, weight, bias, activation, c, idx, idx_type, y};
    return cuda_status(kda::launch_conv1d_update(a, static_cast<cudaStream_t>(stream)));
}

namespace {
// [status word | the kernels' own]: every attention workspace is 256-byte aligned and of the full size.
int check_workspace(const void *ws, size_t have, size_t need)
{
    if (ws == nullptr) return KDA_ERR_NULL;
    return aligned(ws, 256) && have >= need ? KDA_OK : KDA_ERR_WORKSPACE;
}

// A softmax scale: positive (its running maximum is taken before the scale is applied), and finite once the
// kernels have multiplied it by log2(e) for their base-2 exponentials.
bool valid_scale(float s) { return s > 0.f && s <= 2.35e38f; }

int check_page_table(const kda_page_table *t)
{
    if (t == nullptr || t->block_table == nullptr || t->seq_lens == nullptr || t->refcount == nullptr) return KDA_ERR_NULL;
    if (t->reserved != 0 || t->requests < 1 || t->width < 1 || t->n_pages < 1 || t->page_size < 1 ||
        t->table_stride < t->width)
        return KDA_ERR_LAYOUT;
    // page numbers, positions and the requests' page ranks are 32-bit; offsets into the table 64-bit
    const int64_t lim = INT64_C(1) << 31;
    if (t->n_pages >= lim || t->requests >= lim || t->width >= lim || t->width * t->page_size >= lim ||
        t->table_stride > (INT64_C(1) << 40) || static_cast<__int128>(t->requests) * t->table_stride > (INT64_C(1) << 60))
        return KDA_ERR_RANGE;
    if (!aligned(t->block_table, 4) || !aligned(t->seq_lens, 4) || !aligned(t->refcount, 4)) return KDA_ERR_ALIGN;
    return KDA_OK;
}

// Checks shared by the calls that take a list of requests.  KDA_OK with *count == 0: nothing to launch.
int check_page_list(const kda_page_table *t, const void *req, int32_t idx_type, int64_t count)
{
    const int rc = check_page_table(t);
    if (rc != KDA_OK) return rc;
    if (!valid_itype(idx_type)) return KDA_ERR_DTYPE;
    if (count < 0) return KDA_ERR_SHAPE;
    if (count >= (INT64_C(1) << 30)) return KDA_ERR_RANGE;
    return count == 0 ? KDA_OK : check_index_array(req, idx_type);
}
}  // namespace

size_t kda_latent_decode_workspace_size(int64_t batch, int32_t L, int32_t h, int32_t dl, int32_t dr)
{
    if (batch < 0 || L < 1 || h < 1 || (dl != 256 && dl != 512) || dr != 64) return 0;
    if (static_cast<int64_t>(L) * h > 65536 || static_cast<__int128>(batch) * L * h >= (INT64_C(1) << 31)) return 0;
    return kda::latent_decode_workspace(batch, L, h, dl);
}

int kda_latent_decode(const void *q, int32_t io_dtype, int64_t batch, int32_t L, int32_t h, int32_t dl, int32_t dr,
                      float scale, const kda_cache *cache, const int32_t *block_table, int64_t requests, int64_t width,
                      int64_t table_stride, const int32_t *seq_lens, const void *req, int32_t idx_type, void *out,
                      float *lse, void *workspace, size_t ws_bytes, void *stream)
{
    kda::CacheDesc c{};
    int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if (io_dtype != KDA_BF16 || c.dtype != KDA_BF16 || (req != nullptr && !valid_itype(idx_type))) return KDA_ERR_DTYPE;
    if (batch < 0 || L < 1 || h < 1 || dl < 1 || dr < 1 || requests < 1 || width < 1 || table_stride < width ||
        c.h != 1 || c.k != static_cast<int64_t>(dl) + dr || (req == nullptr && requests < batch))
        return KDA_ERR_SHAPE;
    if ((dl != 256 && dl != 512) || dr != 64 || c.v % 8 != 0) return KDA_ERR_UNSUPPORTED;
    if (!valid_scale(scale) || static_cast<int64_t>(L) * h > 65536 || static_cast<__int128>(batch) * L * h >= (INT64_C(1) << 31) ||
        static_cast<__int128>(width) * c.v >= (INT64_C(1) << 31) || c.n_rows >= (INT64_C(1) << 31) ||
        static_cast<__int128>(requests) * table_stride > (INT64_C(1) << 60))
        return KDA_ERR_RANGE;
    if (batch == 0) return KDA_OK;
    if (q == nullptr || block_table == nullptr || seq_lens == nullptr || out == nullptr) return KDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(c.data, 16) || c.row_stride % 8 != 0 || !aligned(lse, 4) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || (req != nullptr && !aligned(req, idx_type == KDA_I32 ? 4 : 8)))
        return KDA_ERR_ALIGN;
    if ((rc = check_workspace(workspace, ws_bytes, kda::latent_decode_workspace(batch, L, h, dl))) != KDA_OK) return rc;
    kda::LatentDecodeArgs a{q, batch, L, h, dl, dr, scale, c, block_table, requests, width, table_stride, c.v, seq_lens, req,
                            idx_type, out, lse, workspace};
    return cuda_status(kda::launch_latent_decode(a, static_cast<cudaStream_t>(stream)));
}

size_t kda_latent_prefill_workspace_size(int64_t total_q, int64_t num_seqs, int32_t h)
{
    if (total_q < 0 || total_q >= (INT64_C(1) << 31) - 256 || num_seqs < 1 || num_seqs >= (1 << 24) || h < 1 || h > 1024) return 0;
    return kda::latent_prefill_workspace(total_q, num_seqs, h);
}

int kda_latent_prefill(const void *q, int32_t io_dtype, const void *k_nope, int64_t kn_token, int64_t kn_head,
                       const void *k_rope, int64_t kr_token, const void *v, int64_t v_token, int64_t v_head,
                       const int32_t *cu_q, const int32_t *cu_k, int64_t num_seqs, int64_t total_q, int64_t total_k,
                       int32_t h, int32_t dn, int32_t dr, int32_t dv, float scale, void *out, float *lse, void *workspace,
                       size_t ws_bytes, void *stream)
{
    if (io_dtype != KDA_BF16) return KDA_ERR_DTYPE;
    if (num_seqs < 1 || total_q < 0 || total_k < 0 || h < 1 || dn < 1 || dr < 1 || dv < 1 || kn_token < 0 || kn_head < 0 ||
        kr_token < 0 || v_token < 0 || v_head < 0)
        return KDA_ERR_SHAPE;
    if (dn != 128 || dv != 128 || dr != 64) return KDA_ERR_UNSUPPORTED;
    const int64_t most = (INT64_C(1) << 31) - 256;
    if (!valid_scale(scale) || total_q >= most || total_k >= most || num_seqs >= (1 << 24) || h > 1024 ||
        (total_q / 256 + num_seqs) * h >= (INT64_C(1) << 31))  // (block of 256 queries, head) pairs
        return KDA_ERR_RANGE;
    const int64_t strides[] = {kn_token, kn_head, kr_token, v_token, v_head};
    for (int64_t s : strides)
        if (s >= (INT64_C(1) << 38)) return KDA_ERR_RANGE;
    if (total_k > 1 && (kn_token == 0 || kr_token == 0 || v_token == 0)) return KDA_ERR_SHAPE;  // tokens that share a row
    if (total_q == 0) return KDA_OK;
    if (q == nullptr || cu_q == nullptr || cu_k == nullptr || out == nullptr) return KDA_ERR_NULL;
    if (total_k > 0 && (k_nope == nullptr || k_rope == nullptr || v == nullptr)) return KDA_ERR_NULL;
    const void *vec16[] = {q, k_nope, k_rope, v, out};
    for (const void *p : vec16)
        if (!aligned(p, 16)) return KDA_ERR_ALIGN;
    for (int64_t s : strides)
        if (s % 8 != 0) return KDA_ERR_ALIGN;
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4)) return KDA_ERR_ALIGN;
    const int rc = check_workspace(workspace, ws_bytes, kda::latent_prefill_workspace(total_q, num_seqs, h));
    if (rc != KDA_OK) return rc;
    kda::LatentPrefillArgs a{q, k_nope, k_rope, v, kn_token, kn_head, kr_token, v_token, v_head, cu_q, cu_k, num_seqs,
                             total_q, total_k, h, scale, out, lse, workspace};
    return cuda_status(kda::launch_latent_prefill(a, static_cast<cudaStream_t>(stream)));
}

int kda_latent_append(const void *x, int64_t x_stride, int64_t total, const int32_t *cu, const void *req, int32_t idx_type,
                      int64_t count, const kda_page_table *table, const kda_cache *cache, void *stream)
{
    kda::CacheDesc c{};
    int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if ((rc = check_page_list(table, req, idx_type, count)) != KDA_OK) return rc;
    if (total < 0 || c.h != 1 || c.v != table->page_size || c.n_rows < table->n_pages || x_stride < c.k) return KDA_ERR_SHAPE;
    if (total >= (INT64_C(1) << 31) || static_cast<__int128>(total) * x_stride > (INT64_C(1) << 60)) return KDA_ERR_RANGE;
    if (total == 0 || count == 0) return KDA_OK;
    if (x == nullptr || cu == nullptr) return KDA_ERR_NULL;
    if (!aligned(x, static_cast<uintptr_t>(esize(c.dtype))) || !aligned(cu, 4)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_latent_append(x, x_stride, total, cu, req, idx_type, count, *table, c,
                                                 static_cast<cudaStream_t>(stream)));
}

size_t kda_pages_workspace_size(int64_t n_pages, int64_t count)
{
    if (n_pages < 1 || n_pages >= (INT64_C(1) << 31) || count < 0 || count >= (INT64_C(1) << 30)) return 0;
    return kda::pages_workspace(n_pages, count);
}

int kda_pages_fork(const kda_page_table *table, const void *src, const void *dst, int32_t idx_type, int64_t count,
                   void *stream)
{
    int rc = check_page_list(table, src, idx_type, count);
    if (rc != KDA_OK || count == 0) return rc;
    if ((rc = check_index_array(dst, idx_type)) != KDA_OK) return rc;
    return cuda_status(kda::launch_pages_fork(*table, src, dst, idx_type, count, static_cast<cudaStream_t>(stream)));
}

int kda_pages_release(const kda_page_table *table, const void *req, int32_t idx_type, const int32_t *keep, int64_t count,
                      void *stream)
{
    const int rc = check_page_list(table, req, idx_type, count);
    if (rc != KDA_OK || count == 0) return rc;
    if (!aligned(keep, 4)) return KDA_ERR_ALIGN;
    return cuda_status(kda::launch_pages_release(*table, req, idx_type, keep, count, static_cast<cudaStream_t>(stream)));
}

int kda_pages_reserve(const kda_page_table *table, const void *req, int32_t idx_type, const int32_t *new_tokens,
                      int64_t count, int32_t *move_src, int32_t *move_dst, int32_t *info, void *workspace, size_t ws_bytes,
                      void *stream)
{
    int rc = check_page_list(table, req, idx_type, count);
    if (rc != KDA_OK || count == 0) return rc;
    if (new_tokens == nullptr || move_src == nullptr || move_dst == nullptr || info == nullptr) return KDA_ERR_NULL;
    const void *vec4[] = {new_tokens, move_src, move_dst, info};
    for (const void *p : vec4)
        if (!aligned(p, 4)) return KDA_ERR_ALIGN;
    if ((rc = check_workspace(workspace, ws_bytes, kda::pages_workspace(table->n_pages, count))) != KDA_OK) return rc;
    return cuda_status(kda::launch_pages_reserve(*table, req, idx_type, new_tokens, count, move_src, move_dst, info,
                                                 workspace, static_cast<cudaStream_t>(stream)));
}

int kda_pages_compact(const kda_page_table *table, int32_t *move_src, int32_t *move_dst, int64_t capacity, int32_t *info,
                      void *workspace, size_t ws_bytes, void *stream)
{
    int rc = check_page_table(table);
    if (rc != KDA_OK) return rc;
    if (capacity < table->n_pages / 2) return KDA_ERR_SHAPE;
    if (capacity >= (INT64_C(1) << 31)) return KDA_ERR_RANGE;
    if (info == nullptr || (capacity > 0 && (move_src == nullptr || move_dst == nullptr))) return KDA_ERR_NULL;
    if (!aligned(move_src, 4) || !aligned(move_dst, 4) || !aligned(info, 4)) return KDA_ERR_ALIGN;
    if ((rc = check_workspace(workspace, ws_bytes, kda::pages_workspace(table->n_pages, 0))) != KDA_OK) return rc;
    return cuda_status(kda::launch_pages_compact(*table, move_src, move_dst, capacity, info, workspace,
                                                 static_cast<cudaStream_t>(stream)));
}

int kda_pages_copy(const kda_cache *cache, const void *move_src, const void *move_dst, int32_t idx_type, int64_t count,
                   void *stream)
{
    kda::CacheDesc c{};
    int rc = check_cache(cache, &c);
    if (rc != KDA_OK) return rc;
    if (!valid_itype(idx_type)) return KDA_ERR_DTYPE;
    if (count < 0) return KDA_ERR_SHAPE;
    // the scalar kernel's one-dimensional grid over a row
    if (c.h * c.v * c.k / 256 >= INT64_C(0x7fffffff)) return KDA_ERR_RANGE;
    if (count == 0) return KDA_OK;
    if ((rc = check_index_array(move_src, idx_type)) != KDA_OK) return rc;
    if ((rc = check_index_array(move_dst, idx_type)) != KDA_OK) return rc;
    return cuda_status(kda::launch_pages_copy(c, move_src, move_dst, idx_type, count, static_cast<cudaStream_t>(stream)));
}

const char *kda_status_string(int32_t status)
{
    switch (status) {
    case KDA_OK: return "KDA_OK";
    case KDA_ERR_NULL: return "KDA_ERR_NULL: a required pointer is NULL";
    case KDA_ERR_DTYPE: return "KDA_ERR_DTYPE: unknown or unsupported element or index type";
    case KDA_ERR_LAYOUT: return "KDA_ERR_LAYOUT: invalid cache layout (n_rows, sizes or row stride)";
    case KDA_ERR_SHAPE: return "KDA_ERR_SHAPE: invalid size or shape";
    case KDA_ERR_RANGE: return "KDA_ERR_RANGE: size beyond the supported range";
    case KDA_ERR_WORKSPACE: return "KDA_ERR_WORKSPACE: workspace missing, too small or misaligned";
    case KDA_ERR_CUDA: return "KDA_ERR_CUDA: CUDA launch failed";
    case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED: head size combination not built";
    case KDA_ERR_ALIGN: return "KDA_ERR_ALIGN: pointer or stride misaligned";
    default: return "unknown kda_status";
    }
}

const char *kda_last_cuda_error_string(void) { return cudaGetErrorString(t_last_cuda); }

int kda_selftest_bounded_wait(int32_t *status_dev, uint32_t polls, int32_t arrive, void *stream)
{
    if (status_dev == nullptr) return KDA_ERR_NULL;
    if (polls == 0) return KDA_ERR_RANGE;
    return cuda_status(kda::launch_bounded_wait_selftest(status_dev, polls, arrive, static_cast<cudaStream_t>(stream)));
}

int kda_prefill_workspace_status(const void *workspace, int32_t *status_out, void *stream)
{
    if (workspace == nullptr || status_out == nullptr) return KDA_ERR_NULL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(status_out, workspace, sizeof(int32_t), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return cuda_status(e);
}

}  // extern "C"
