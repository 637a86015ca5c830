// C ABI entry points of the 8-bit full-rank cache: host-side argument
// checks, then the launchers.
#include <limits.h>

#include "quant.cuh"

using namespace lrkv;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_quant(const lrkv_quant_cache* c) {
  if (!c) return LRKV_ERR_ARG;
  if (c->code != LRKV_CODE_INT8 && c->code != LRKV_CODE_E4M3) return LRKV_ERR_UNSUPPORTED;
  if (c->head_dim != kHeadDim) return LRKV_ERR_UNSUPPORTED;
  if (c->batch < 1 || c->batch > LRKV_MAX_BATCH || c->num_kv_heads < 1 ||
      c->num_kv_heads > 32767)
    return LRKV_ERR_ARG;
  // positions are 32-bit
  if (c->num_pages < 1 || c->max_pages_per_seq < 1 || c->max_pages_per_seq > INT_MAX / kQBlock - 2)
    return LRKV_ERR_ARG;
  if (!c->pages || !c->block_table || !c->tail || !c->seq_len || !c->append_counter || !c->error)
    return LRKV_ERR_ARG;
  if (!aligned16(c->pages) || !aligned16(c->tail)) return LRKV_ERR_ARG;
  return LRKV_OK;
}

int check_quant_heads(const lrkv_quant_cache* c, int H_q, int n) {
  if (H_q < 1 || H_q % c->num_kv_heads != 0 || n < 0) return LRKV_ERR_ARG;
  if (H_q / c->num_kv_heads > 128) return LRKV_ERR_UNSUPPORTED;
  // blocks of the whole batch (the kernels count up to 16 more a unit: what its
  // parts cost) and a unit's rows (queries x grouped heads) are counted in 32 bits
  if ((long long)c->batch * c->num_kv_heads * ((long long)c->max_pages_per_seq + 16) > INT_MAX)
    return LRKV_ERR_UNSUPPORTED;
  const long long rows = (long long)n * (H_q / c->num_kv_heads);
  if (rows > (1 << 30)) return LRKV_ERR_UNSUPPORTED;
  // ... and so are the steps of a unit's row tiles
  if ((rows + 255) / 256 * ((long long)c->max_pages_per_seq + 16) > INT_MAX)
    return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

QuantView view(const lrkv_quant_cache* c) {
  QuantView v;
  v.B = c->batch;
  v.H = c->num_kv_heads;
  v.maxp = c->max_pages_per_seq;
  v.num_pages = c->num_pages;
  v.e4m3 = c->code == LRKV_CODE_E4M3;
  v.pages = static_cast<uint8_t*>(c->pages);
  v.bt = c->block_table;
  v.tail = static_cast<__nv_bfloat16*>(c->tail);
  v.seq_len = c->seq_len;
  v.counter = c->append_counter;
  v.error = c->error;
  return v;
}

bool strides_ok(int64_t a, int64_t b, int64_t c, int m) {
  return a % m == 0 && b % m == 0 && c % m == 0;
}

}  // namespace

extern "C" {

int lrkv_quant_append(const lrkv_quant_cache* cache, const void* k, const void* v,
                      int32_t n_tokens, const int32_t* n_new, int64_t seq_stride,
                      int64_t head_stride, int64_t token_stride, void* stream) {
  const int rc = check_quant(cache);
  if (rc != LRKV_OK) return rc;
  if (n_tokens < 0) return LRKV_ERR_ARG;
  if (n_tokens == 0) return LRKV_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v) ||
      !strides_ok(seq_stride, head_stride, token_stride, 8))
    return LRKV_ERR_ARG;
  if (n_tokens > (long long)cache->max_pages_per_seq * kQBlock) return LRKV_ERR_CAPACITY;
  QuantAppendArgs a;
  a.c = view(cache);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.n = n_tokens;
  a.n_new = n_new;
  a.ss = seq_stride;
  a.hs = head_stride;
  a.ts = token_stride;
  return quant_append_launch(a, static_cast<cudaStream_t>(stream));
}

int lrkv_quant_read(const lrkv_quant_cache* cache, const int32_t* first, int32_t n_tokens,
                    void* k, void* v, int32_t dtype, int64_t seq_stride, int64_t head_stride,
                    int64_t token_stride, void* stream) {
  const int rc = check_quant(cache);
  if (rc != LRKV_OK) return rc;
  if (dtype != LRKV_BF16 && dtype != LRKV_F32) return LRKV_ERR_UNSUPPORTED;
  if (n_tokens < 0) return LRKV_ERR_ARG;
  if (n_tokens == 0) return LRKV_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v) ||
      !strides_ok(seq_stride, head_stride, token_stride, dtype == LRKV_F32 ? 4 : 8))
    return LRKV_ERR_ARG;
  QuantReadArgs a;
  a.c = view(cache);
  a.first = first;
  a.n = n_tokens;
  a.k = k;
  a.v = v;
  a.ss = seq_stride;
  a.hs = head_stride;
  a.ts = token_stride;
  return quant_read_launch(a, dtype, static_cast<cudaStream_t>(stream));
}

size_t lrkv_quant_attn_workspace_bytes(const lrkv_quant_cache* cache, int32_t num_q_heads,
                                       int32_t n_queries) {
  if (check_quant(cache) != LRKV_OK || check_quant_heads(cache, num_q_heads, n_queries) != LRKV_OK)
    return 0;
  return quant_attn_workspace(cache->batch, cache->num_kv_heads, num_q_heads, n_queries);
}

int lrkv_quant_attn(const lrkv_quant_cache* cache, const void* q, int32_t num_q_heads,
                    int32_t n_queries, const int32_t* n_q, int64_t q_seq_stride,
                    int64_t q_head_stride, int64_t q_token_stride, float scale, void* o,
                    int64_t o_seq_stride, int64_t o_head_stride, int64_t o_token_stride,
                    void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_quant(cache);
  if (rc == LRKV_OK) rc = check_quant_heads(cache, num_q_heads, n_queries);
  if (rc != LRKV_OK) return rc;
  if (n_queries == 0) return LRKV_OK;
  if (!q || !o || !workspace || !aligned16(q) || !aligned16(o) || !aligned16(workspace) ||
      !strides_ok(q_seq_stride, q_head_stride, q_token_stride, 8) ||
      !strides_ok(o_seq_stride, o_head_stride, o_token_stride, 8))
    return LRKV_ERR_ARG;
  const size_t need = quant_attn_workspace(cache->batch, cache->num_kv_heads, num_q_heads,
                                           n_queries);
  if (need == 0) return LRKV_ERR_CUDA;  // the device query failed
  if (workspace_bytes < need) return LRKV_ERR_WORKSPACE;
  QuantAttnArgs a;
  a.c = view(cache);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.Hq = num_q_heads;
  a.G = num_q_heads / cache->num_kv_heads;
  a.n = n_queries;
  a.n_q = n_q;
  a.qs = q_seq_stride;
  a.qh = q_head_stride;
  a.qt = q_token_stride;
  a.os = o_seq_stride;
  a.oh = o_head_stride;
  a.ot = o_token_stride;
  a.scale = scale;
  a.ws = workspace;
  int s = 0;
  while ((1 << s) < a.G) ++s;
  a.gmul = a.G == 1 ? 0u : (uint32_t)((1ull << (31 + s)) / a.G + 1);
  a.gshift = a.G == 1 ? 0u : (uint32_t)(s - 1);
  return quant_attn_launch(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
