// api_kv.cu -- the C ABI of the 4-bit key/value cache (include/bnb4.h):
// argument checks and the launches on the caller's stream.  Nothing here
// allocates or synchronizes.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bnb4.h"
#include "kernels.h"
#include "kvcache.h"

namespace {

bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? BNB4_OK : BNB4_ERR_CUDA; }

int check_cache(const bnb4_kv_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_absmax || !c->v_absmax || c->reserved != 0)
    return BNB4_ERR_INVALID_ARG;
  if (c->qtype != BNB4_NF4 && c->qtype != BNB4_FP4) return BNB4_ERR_INVALID_ARG;
  if (c->dtype != BNB4_BF16 && c->dtype != BNB4_F16) return BNB4_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return BNB4_ERR_UNSUPPORTED;
  if ((c->blocksize != 32 && c->blocksize != 64 && c->blocksize != 128) ||
      c->blocksize > c->head_dim)
    return BNB4_ERR_UNSUPPORTED;
  if (c->num_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > (1 << 20)) return BNB4_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size % 16 != 0) return BNB4_ERR_SHAPE;
  if (c->num_pages > INT32_MAX / c->page_size) return BNB4_ERR_SHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_absmax, 16) ||
      !aligned(c->v_absmax, 16))
    return BNB4_ERR_ALIGNMENT;
  return BNB4_OK;
}

// Rows of whole 16-byte chunks, `per` elements each, at non-negative strides.
int check_strides(int64_t ts, int64_t hs, int64_t per) {
  if (ts < 0 || hs < 0) return BNB4_ERR_SHAPE;
  return ts % per == 0 && hs % per == 0 ? BNB4_OK : BNB4_ERR_ALIGNMENT;
}

// Whether two of tokens x heads rows of `dim` elements at t * ts + h * hs share an
// element.
bool rows_overlap(int64_t ts, int64_t hs, int64_t tokens, int64_t heads, int64_t dim) {
  if ((tokens > 1 && ts < dim) || (heads > 1 && hs < dim)) return true;
  if (tokens < 2 || heads < 2) return false;
  using Wide = __int128;  // a stride may be anything below 2^63
  // a token's heads end before the next token, or a head's tokens before the next head
  if (ts >= Wide(hs) * (heads - 1) + dim || hs >= Wide(ts) * (tokens - 1) + dim) return false;
  // interleaved: rows (t, h + j) and (t + i, h) for the i that bring them nearest
  const bool by_heads = heads <= tokens;
  const int64_t n = by_heads ? heads : tokens, m = by_heads ? tokens : heads;
  const Wide step = by_heads ? hs : ts, other = by_heads ? ts : hs;
  for (int64_t j = 1; j < n; ++j) {
    const Wide x = step * j, i = x / other;
    if ((i >= 1 && i < m && x - i * other < dim) || (i + 1 < m && (i + 1) * other - x < dim))
      return true;
  }
  return false;
}

// Rows that are written do not lie over one another.
int check_written(int64_t ts, int64_t hs, int64_t tokens, int64_t heads, int64_t dim,
                  int64_t per) {
  const int rc = check_strides(ts, hs, per);
  if (rc != BNB4_OK) return rc;
  return rows_overlap(ts, hs, tokens, heads, dim) ? BNB4_ERR_SHAPE : BNB4_OK;
}

int on_device(const void* p) {
  const void* d;
  return bnb4::resolve_ptr(p, bnb4::Residency::kDevice, &d);
}

int check_cache_memory(const bnb4_kv_cache* c) {
  int rc;
  if ((rc = on_device(c->k_codes)) != BNB4_OK) return rc;
  if ((rc = on_device(c->v_codes)) != BNB4_OK) return rc;
  if ((rc = on_device(c->k_absmax)) != BNB4_OK) return rc;
  return on_device(c->v_absmax);
}

int check_rows(int64_t tokens, const int64_t* slots, const bnb4_kv_cache* c) {
  if (!slots) return BNB4_ERR_INVALID_ARG;
  if (tokens > INT32_MAX / (2 * static_cast<int64_t>(c->n_kv_heads))) return BNB4_ERR_SHAPE;
  return aligned(slots, 8) ? BNB4_OK : BNB4_ERR_ALIGNMENT;
}

}  // namespace

extern "C" {

int bnb_kv_write_4bit(const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v,
                      int64_t v_stride_t, int64_t v_stride_h, int64_t tokens,
                      const int64_t* slots, const bnb4_kv_cache* cache, void* stream) {
  int rc = check_cache(cache);
  if (rc != BNB4_OK) return rc;
  if (tokens < 0) return BNB4_ERR_SHAPE;
  if (tokens == 0) return BNB4_OK;
  if (!k || !v) return BNB4_ERR_INVALID_ARG;
  if ((rc = check_rows(tokens, slots, cache)) != BNB4_OK) return rc;
  if ((rc = check_strides(k_stride_t, k_stride_h, 8)) != BNB4_OK) return rc;
  if ((rc = check_strides(v_stride_t, v_stride_h, 8)) != BNB4_OK) return rc;
  if (!aligned(k, 16) || !aligned(v, 16)) return BNB4_ERR_ALIGNMENT;
  int sms;
  if ((rc = bnb4::device_sms(&sms)) != BNB4_OK) return rc;
  if ((rc = on_device(k)) != BNB4_OK || (rc = on_device(v)) != BNB4_OK) return rc;
  if ((rc = on_device(slots)) != BNB4_OK) return rc;
  if ((rc = check_cache_memory(cache)) != BNB4_OK) return rc;
  const bnb4::KvRows rows{k, v, k_stride_t, k_stride_h, v_stride_t, v_stride_h};
  return from_cuda(bnb4::launch_kv_write(rows, tokens, slots, *cache, sms,
                                         static_cast<cudaStream_t>(stream)));
}

int bnb_kv_read_4bit(const bnb4_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k,
                     int64_t k_stride_t, int64_t k_stride_h, void* v, int64_t v_stride_t,
                     int64_t v_stride_h, int32_t out_dtype, void* stream) {
  int rc = check_cache(cache);
  if (rc != BNB4_OK) return rc;
  if (out_dtype != BNB4_F32 && out_dtype != BNB4_BF16 && out_dtype != BNB4_F16)
    return BNB4_ERR_UNSUPPORTED;
  if (tokens < 0) return BNB4_ERR_SHAPE;
  if (tokens == 0) return BNB4_OK;
  if (!k && !v) return BNB4_ERR_INVALID_ARG;
  if ((rc = check_rows(tokens, slots, cache)) != BNB4_OK) return rc;
  const int64_t per = out_dtype == BNB4_F32 ? 4 : 8;
  const int64_t heads = cache->n_kv_heads, dim = cache->head_dim;
  if (k && (rc = check_written(k_stride_t, k_stride_h, tokens, heads, dim, per)) != BNB4_OK)
    return rc;
  if (v && (rc = check_written(v_stride_t, v_stride_h, tokens, heads, dim, per)) != BNB4_OK)
    return rc;
  if (!aligned(k, 16) || !aligned(v, 16)) return BNB4_ERR_ALIGNMENT;
  if (k == v) return BNB4_ERR_SHAPE;  // (both NULL is refused above)
  int sms;
  if ((rc = bnb4::device_sms(&sms)) != BNB4_OK) return rc;
  if (k && (rc = on_device(k)) != BNB4_OK) return rc;
  if (v && (rc = on_device(v)) != BNB4_OK) return rc;
  if ((rc = on_device(slots)) != BNB4_OK) return rc;
  if ((rc = check_cache_memory(cache)) != BNB4_OK) return rc;
  const bnb4::KvRows rows{k, v, k_stride_t, k_stride_h, v_stride_t, v_stride_h};
  return from_cuda(bnb4::launch_kv_read(*cache, slots, tokens, rows, out_dtype, sms,
                                        static_cast<cudaStream_t>(stream)));
}

// Everything of an attention call but its pointers' memory kinds.
static int check_attn(const bnb4_attn* a) {
  if (!a) return BNB4_ERR_INVALID_ARG;
  int rc = check_cache(a->cache);
  if (rc != BNB4_OK) return rc;
  if (a->reserved != 0 || (a->causal != 0 && a->causal != 1)) return BNB4_ERR_INVALID_ARG;
  if (a->batch < 0 || a->total_q < 0 || a->total_q > INT32_MAX || a->max_q_len < 1 ||
      a->max_seq_len < 0 || a->window < 0)
    return BNB4_ERR_SHAPE;
  if (a->n_heads < 1 || a->n_heads % a->cache->n_kv_heads != 0) return BNB4_ERR_SHAPE;
  if (static_cast<int64_t>(a->max_q_len) * a->n_heads > INT32_MAX) return BNB4_ERR_SHAPE;
  if (!a->cu_seqlens_q && a->total_q != 0 &&
      static_cast<int64_t>(a->batch) * a->max_q_len != a->total_q)
    return BNB4_ERR_SHAPE;
  if (a->block_table_width < 1 || a->block_table_stride < a->block_table_width ||
      a->block_table_width > (1 << 30) / a->cache->page_size)
    return BNB4_ERR_SHAPE;
  // tiles of 16 rows and more, counted in 32 bits
  if (static_cast<int64_t>(a->batch) * a->n_heads > (1 << 24) ||
      static_cast<int64_t>(a->batch) * a->n_heads * (a->max_q_len / 64 + 1) > (1 << 30))
    return BNB4_ERR_SHAPE;
  if (!(a->scale >= 1e-8f && a->scale <= 1e8f)) return BNB4_ERR_INVALID_ARG;
  return BNB4_OK;
}

int bnb4_attn_workspace(const bnb4_attn* a, size_t* bytes) {
  if (!bytes) return BNB4_ERR_INVALID_ARG;
  const int rc = check_attn(a);
  if (rc != BNB4_OK) return rc;
  *bytes = a->batch == 0 || a->total_q == 0 ? 0 : bnb4::attn_workspace_bytes(*a);
  return BNB4_OK;
}

static int run_attn(const bnb4_attn* a, void* stream, uint64_t wait_limit_ns, int withhold) {
  int rc = check_attn(a);
  if (rc != BNB4_OK) return rc;
  if (a->batch == 0 || a->total_q == 0) return BNB4_OK;
  if (!a->q || !a->out || !a->block_table || !a->seq_lens) return BNB4_ERR_INVALID_ARG;
  if ((rc = check_strides(a->q_stride_t, a->q_stride_h, 8)) != BNB4_OK) return rc;
  if ((rc = check_written(a->out_stride_t, a->out_stride_h, a->total_q, a->n_heads,
                          a->cache->head_dim, 8)) != BNB4_OK)
    return rc;
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->block_table, 4) ||
      !aligned(a->seq_lens, 4) || !aligned(a->cu_seqlens_q, 4) || !aligned(a->lse, 4))
    return BNB4_ERR_ALIGNMENT;
  const size_t need = bnb4::attn_workspace_bytes(*a);
  if (need > 0) {
    if (!a->workspace || a->workspace_bytes < need) return BNB4_ERR_WORKSPACE;
    if (!aligned(a->workspace, 16)) return BNB4_ERR_ALIGNMENT;
  }
  int sms;
  if ((rc = bnb4::device_sms(&sms)) != BNB4_OK) return rc;
  if ((rc = on_device(a->q)) != BNB4_OK || (rc = on_device(a->out)) != BNB4_OK) return rc;
  if (a->lse && (rc = on_device(a->lse)) != BNB4_OK) return rc;
  if ((rc = on_device(a->block_table)) != BNB4_OK) return rc;
  if ((rc = on_device(a->seq_lens)) != BNB4_OK) return rc;
  if (a->cu_seqlens_q && (rc = on_device(a->cu_seqlens_q)) != BNB4_OK) return rc;
  if (need > 0 && (rc = on_device(a->workspace)) != BNB4_OK) return rc;
  if ((rc = check_cache_memory(a->cache)) != BNB4_OK) return rc;
  int* err;
  if ((rc = bnb4::device_error_word(&err)) != BNB4_OK) return rc;
  return from_cuda(bnb4::launch_attn(*a, sms, err, static_cast<cudaStream_t>(stream),
                                     wait_limit_ns, withhold));
}

int bnb_attn_4bit(const bnb4_attn* a, void* stream) { return run_attn(a, stream, 0, 0); }

int bnb4_debug_attn_withhold(const bnb4_attn* a, int32_t wait_limit_us, void* stream) {
  if (wait_limit_us < 1 || wait_limit_us > 1000000) return BNB4_ERR_INVALID_ARG;
  return run_attn(a, stream, static_cast<uint64_t>(wait_limit_us) * 1000u, 1);
}

}  // extern "C"
