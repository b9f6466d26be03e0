// kv_api.hip -- the C ABI of the key/value cache (declared in include/q4.h):
// host-side argument validation and dispatch.  As in q4_api.hip, every check
// runs before the first HIP call.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kv_common.hpp"
#include "q4.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
q4_status from_hip(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_EHIP; }
bool dtype_ok(int t) { return t == Q4_F16 || t == Q4_BF16; }

constexpr int kMaxGridYZ = 65535;

// Format, sizes and pointers of a cache.
q4_status check_cache(const q4_kv_cache *c)
{
    if (!c)
        return Q4_EINVAL;
    if (c->format != Q4_NF4 && c->format != Q4_INT4_SYM && c->format != Q4_INT4_ASYM && c->format != Q4_FP4)
        return Q4_EUNSUPPORTED;
    if (c->g != 32 && c->g != 64 && c->g != 128)
        return Q4_EUNSUPPORTED;
    if (c->pages <= 0 || c->heads <= 0 || c->reserved != 0)
        return Q4_EINVAL;
    if (c->dim != 64 && c->dim != 128 && c->dim != 256)
        return Q4_EUNSUPPORTED;
    if (c->dim % c->g != 0)
        return Q4_EINVAL;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256)
        return Q4_EUNSUPPORTED;
    if (c->pages > INT32_MAX || 2 * (int64_t)c->heads > kMaxGridYZ)  // (a grid counts heads of keys and of values)
        return Q4_EUNSUPPORTED;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
        return Q4_EINVAL;
    const bool asym = c->format == Q4_INT4_ASYM;
    if (asym != (c->k_zeros != nullptr) || asym != (c->v_zeros != nullptr))
        return Q4_EINVAL;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) ||
        !aligned(c->v_scales, 16) || !aligned(c->k_zeros, 4) || !aligned(c->v_zeros, 4))
        return Q4_EALIGN;
    return Q4_OK;
}

// A batch over a checked cache.  `rows`: the packed arrays take part too.
q4_status check_batch(const q4_kv_cache *c, const q4_kv_batch *b, bool rows)
{
    if (!b || !b->table || !b->lens)
        return Q4_EINVAL;
    if (b->seqs <= 0 || b->table_width <= 0 || b->max_len < 0)
        return Q4_EINVAL;
    if (b->max_len > (int64_t)b->table_width * c->page)
        return Q4_EINVAL;
    if (b->seqs > kMaxGridYZ || b->max_len > Q4_KV_MAX_LEN)
        return Q4_EUNSUPPORTED;
    if (!aligned(b->table, 4) || !aligned(b->lens, 4) || !aligned(b->starts, 4))
        return Q4_EALIGN;
    if (!rows)
        return Q4_OK;
    if (b->tokens < 0 || b->max_new < 0 || (!b->starts && (b->tokens != b->seqs || b->max_new != 1)))
        return Q4_EINVAL;
    // packed row numbers fit 31 bits, and so do a sequence's work items
    if (b->tokens > INT32_MAX || (int64_t)b->max_new * c->heads * c->dim > (int64_t)1 << 36)
        return Q4_EUNSUPPORTED;
    return Q4_OK;
}

// Strides of a [tokens, heads, dim] array: whole 16-byte steps.
bool strides_ok(int64_t ts, int64_t hs) { return ts >= 0 && hs >= 0 && ts % 8 == 0 && hs % 8 == 0; }

bool empty(const q4_kv_batch *b) { return b->tokens == 0 || b->max_new == 0; }

q4_status check_q(const q4_kv_cache *c, const q4_kv_batch *b, int q_heads)
{
    if (q_heads <= 0 || q_heads % c->heads != 0)
        return Q4_EINVAL;
    if (q_heads / c->heads > Q4_KV_MAX_GROUP || q_heads > kMaxGridYZ ||
        (int64_t)b->max_new * (q_heads / c->heads) > INT32_MAX / 2)
        return Q4_EUNSUPPORTED;
    // the grids count 16-row tiles of all sequences and heads
    if ((((int64_t)b->max_new * (q_heads / c->heads) >> 4) + 1) * b->seqs * c->heads > 1 << 30)
        return Q4_EUNSUPPORTED;
    return Q4_OK;
}

}  // namespace

extern "C" {

q4_status q4_kv_append(const q4_kv_cache *cache, const q4_kv_batch *batch, q4_dtype in_t,
                       const void *k, int64_t k_token_stride, int64_t k_head_stride,
                       const void *v, int64_t v_token_stride, int64_t v_head_stride, void *stream)
{
    q4_status st = check_cache(cache);
    if (st == Q4_OK)
        st = check_batch(cache, batch, true);
    if (st != Q4_OK)
        return st;
    if (!dtype_ok(in_t))
        return Q4_EUNSUPPORTED;
    if (empty(batch))
        return Q4_OK;
    if (!k || !v || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
        return Q4_EINVAL;
    if (!aligned(k, 16) || !aligned(v, 16) || !strides_ok(k_token_stride, k_head_stride) ||
        !strides_ok(v_token_stride, v_head_stride))
        return Q4_EALIGN;
    return from_hip(q4::launch_kv_append(cache->format, q4::kv_cache_args(*cache),
                                         q4::kv_batch_args(*batch), in_t, k, k_token_stride,
                                         k_head_stride, v, v_token_stride, v_head_stride,
                                         (hipStream_t)stream));
}

q4_status q4_kv_read(const q4_kv_cache *cache, const q4_kv_batch *batch, q4_dtype out_t, void *k,
                     void *v, void *stream)
{
    q4_status st = check_cache(cache);
    if (st == Q4_OK)
        st = check_batch(cache, batch, true);
    if (st != Q4_OK)
        return st;
    if (!dtype_ok(out_t))
        return Q4_EUNSUPPORTED;
    if (empty(batch))
        return Q4_OK;
    if (!k || !v)
        return Q4_EINVAL;
    if (!aligned(k, 16) || !aligned(v, 16))
        return Q4_EALIGN;
    return from_hip(q4::launch_kv_read(cache->format, q4::kv_cache_args(*cache),
                                       q4::kv_batch_args(*batch), out_t, k, v, (hipStream_t)stream));
}

size_t q4_kv_workspace_bytes(const q4_kv_cache *cache, const q4_kv_batch *batch, int q_heads, int window,
                             int with_mass)
{
    if (check_cache(cache) != Q4_OK || check_batch(cache, batch, true) != Q4_OK ||
        check_q(cache, batch, q_heads) != Q4_OK || window < 0 || empty(batch))
        return 0;
    return q4::kv_attention_workspace(q4::kv_cache_args(*cache), q4::kv_batch_args(*batch), q_heads, window,
                                      with_mass != 0);
}

q4_status q4_kv_attention(const q4_kv_cache *cache, const q4_kv_batch *batch, q4_dtype act_t,
                          const void *q, int64_t q_token_stride, int64_t q_head_stride,
                          int q_heads, float scale, int window, void *out, float *lse,
                          float *mass, int64_t mass_width, void *workspace,
                          size_t workspace_bytes, void *stream)
{
    q4_status st = check_cache(cache);
    if (st == Q4_OK)
        st = check_batch(cache, batch, true);
    if (st == Q4_OK)
        st = check_q(cache, batch, q_heads);
    if (st != Q4_OK)
        return st;
    if (!dtype_ok(act_t))
        return Q4_EUNSUPPORTED;
    if (!(scale > 0.0f) || !(scale <= 0x1p60f) || window < 0)
        return Q4_EINVAL;
    if (mass && mass_width < batch->max_len)
        return Q4_EINVAL;
    if (empty(batch))
        return Q4_OK;
    if (!q || !out || q_token_stride < 0 || q_head_stride < 0)
        return Q4_EINVAL;
    const q4::KvCache c = q4::kv_cache_args(*cache);
    const q4::KvBatch b = q4::kv_batch_args(*batch);
    const size_t need = q4::kv_attention_workspace(c, b, q_heads, window, mass != nullptr);
    if (need > workspace_bytes || (need && !workspace))
        return Q4_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || !strides_ok(q_token_stride, q_head_stride) ||
        !aligned(lse, 4) || !aligned(mass, 4) || (need && !aligned(workspace, 256)))
        return Q4_EALIGN;
    return from_hip(q4::launch_kv_attention(cache->format, c, b, act_t, q, q_token_stride,
                                            q_head_stride, q_heads, scale, window, out, lse, mass,
                                            mass_width, workspace, (hipStream_t)stream));
}

q4_status q4_kv_evict(const q4_kv_cache *cache, const q4_kv_batch *batch, const float *mass,
                      int64_t mass_width, const int32_t *new_table, int new_table_width,
                      int budget, int recent, int32_t *new_lens, float *new_mass,
                      int64_t new_width, int32_t *kept, void *stream)
{
    q4_status st = check_cache(cache);
    if (st == Q4_OK)
        st = check_batch(cache, batch, false);
    if (st != Q4_OK)
        return st;
    if (!mass || !new_table || !new_lens || !new_mass || !kept)
        return Q4_EINVAL;
    if (budget <= 0 || recent < 0 || recent > budget || new_table_width <= 0 ||
        budget > (int64_t)new_table_width * cache->page || mass_width < batch->max_len ||
        new_width < budget)
        return Q4_EINVAL;
    if (budget > Q4_KV_MAX_LEN)
        return Q4_EUNSUPPORTED;
    if (!aligned(mass, 4) || !aligned(new_table, 4) || !aligned(new_lens, 4) || !aligned(new_mass, 4) ||
        !aligned(kept, 4))
        return Q4_EALIGN;
    return from_hip(q4::launch_kv_evict(cache->format, q4::kv_cache_args(*cache),
                                        q4::kv_batch_args(*batch), mass, mass_width, new_table,
                                        new_table_width, budget, recent, new_lens, new_mass,
                                        new_width, kept, (hipStream_t)stream));
}

}  // extern "C"
