// C ABI of the rollout-side operators: the 4-bit paged cache and token
// sampling.  Argument checks and dispatch; the contract of every entry point
// is in include/sinkattn.h.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/sinkattn.h"
#include "checks.h"
#include "internal.h"

using sa::aligned16;
using sa::aligned4;
using sa::check_list;
using sa::from_cuda;

namespace {

// Validates `c` and fills `out`.  Touches no CUDA API.
sinkattn_status check_cache(const sinkattn_kv4_cache* c, sa::Kv4Cache& out) {
  if (c == nullptr) return SINKATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_heads_kv < 1 || c->num_slots < 1 || c->max_pages < 1) return SINKATTN_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return SINKATTN_ERR_UNSUPPORTED;
  if (c->num_heads_kv > sa::kMaxHeadsQ) return SINKATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * c->page_size > (1LL << 30)) return SINKATTN_ERR_UNSUPPORTED;
  if (!c->pages || !c->page_table || !c->seqlens || !c->refcount || !c->k_scale || !c->v_scale)
    return SINKATTN_ERR_INVALID_ARG;
  if (!aligned16(c->pages) || !aligned16(c->page_table) || !aligned16(c->seqlens) || !aligned16(c->refcount) ||
      !aligned16(c->k_scale) || !aligned16(c->v_scale))
    return SINKATTN_ERR_ALIGNMENT;
  out.pages = static_cast<uint8_t*>(c->pages);
  out.page_table = c->page_table;
  out.seqlens = c->seqlens;
  out.refcount = c->refcount;
  out.k_scale = c->k_scale;
  out.v_scale = c->v_scale;
  out.num_pages = c->num_pages;
  out.page_size = c->page_size;
  out.num_heads_kv = c->num_heads_kv;
  out.num_slots = c->num_slots;
  out.max_pages = c->max_pages;
  out.page_log2 = 0;
  while ((1 << out.page_log2) < c->page_size) ++out.page_log2;
  out.blocks_log2 = out.page_log2 - 4;
  return SINKATTN_OK;
}

// Whether two lists of n int32 share memory.
bool lists_overlap(const int32_t* a, const int32_t* b, int32_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return (x < y ? y - x : x - y) < static_cast<uintptr_t>(n) * 4;
}

sinkattn_status tokens_common(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t n, const int32_t* cu,
                              int32_t total, const void* k, const void* v, sa::Kv4Cache& c) {
  sinkattn_status st = check_cache(cache, c);
  if (st != SINKATTN_OK) return st;
  if (total < 0) return SINKATTN_ERR_INVALID_ARG;
  if ((st = check_list(n, slots)) != SINKATTN_OK) return st;
  if (n == 0 && total > 0 && cu == nullptr) return SINKATTN_ERR_INVALID_ARG;
  if (cu == nullptr && n > 0 && total % n != 0) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned4(cu)) return SINKATTN_ERR_ALIGNMENT;
  if (n == 0 || total == 0) return SINKATTN_OK;
  if (!k || !v) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return SINKATTN_ERR_ALIGNMENT;
  if ((total / 16 + 2LL * n) * c.num_heads_kv / 8 >= 0x7fffffffLL) return SINKATTN_ERR_UNSUPPORTED;
  return SINKATTN_OK;
}

}  // namespace

extern "C" {

sinkattn_status sinkattn_kv4_reserve(const sinkattn_kv4_cache* cache, const int32_t* slots, const int32_t* new_tokens,
                                     int32_t n, int32_t* done, void* stream) {
  sa::Kv4Cache c;
  sinkattn_status st = check_cache(cache, c);
  if (st != SINKATTN_OK) return st;
  if ((st = check_list(n, slots)) != SINKATTN_OK || (st = check_list(n, new_tokens)) != SINKATTN_OK ||
      (st = check_list(n, done)) != SINKATTN_OK)
    return st;
  if (n == 0) return SINKATTN_OK;
  return from_cuda(sa::launch_kv4_reserve(c, slots, new_tokens, n, done, static_cast<cudaStream_t>(stream)));
}

sinkattn_status sinkattn_kv4_fork(const sinkattn_kv4_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                                  int32_t* done, void* stream) {
  sa::Kv4Cache c;
  sinkattn_status st = check_cache(cache, c);
  if (st != SINKATTN_OK) return st;
  if ((st = check_list(n, src)) != SINKATTN_OK || (st = check_list(n, dst)) != SINKATTN_OK ||
      (st = check_list(n, done)) != SINKATTN_OK)
    return st;
  if (n == 0) return SINKATTN_OK;
  // the second of fork's launches reads src and dst again
  if (lists_overlap(done, src, n) || lists_overlap(done, dst, n)) return SINKATTN_ERR_INVALID_ARG;
  return from_cuda(sa::launch_kv4_fork(c, src, dst, n, done, static_cast<cudaStream_t>(stream)));
}

sinkattn_status sinkattn_kv4_free(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t n, void* stream) {
  sa::Kv4Cache c;
  sinkattn_status st = check_cache(cache, c);
  if (st != SINKATTN_OK) return st;
  if ((st = check_list(n, slots)) != SINKATTN_OK) return st;
  if (n == 0) return SINKATTN_OK;
  return from_cuda(sa::launch_kv4_free(c, slots, n, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_kv4_compact_workspace_size(const sinkattn_kv4_cache* from) {
  sa::Kv4Cache c;
  if (check_cache(from, c) != SINKATTN_OK) return 0;
  return sa::kv4_compact_workspace_bytes(c.num_pages);
}

sinkattn_status sinkattn_kv4_compact(const sinkattn_kv4_cache* from, const sinkattn_kv4_cache* to, int32_t* count,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  sa::Kv4Cache a, b;
  sinkattn_status st = check_cache(from, a);
  if (st != SINKATTN_OK || (st = check_cache(to, b)) != SINKATTN_OK) return st;
  if (a.page_size != b.page_size || a.num_heads_kv != b.num_heads_kv || a.num_slots != b.num_slots ||
      a.max_pages != b.max_pages)
    return SINKATTN_ERR_INVALID_ARG;
  if (a.pages == b.pages || a.page_table == b.page_table || a.seqlens == b.seqlens || a.refcount == b.refcount)
    return SINKATTN_ERR_INVALID_ARG;
  if (!count) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned4(count)) return SINKATTN_ERR_ALIGNMENT;
  if (workspace_bytes < sa::kv4_compact_workspace_bytes(a.num_pages)) return SINKATTN_ERR_WORKSPACE;
  if (workspace == nullptr || !aligned16(workspace)) return workspace ? SINKATTN_ERR_ALIGNMENT : SINKATTN_ERR_INVALID_ARG;
  return from_cuda(sa::launch_kv4_compact(a, b, count, workspace, static_cast<cudaStream_t>(stream)));
}

sinkattn_status sinkattn_kv4_append(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t num_seqs,
                                    const int32_t* cu_new, int32_t total, const void* k, const void* v, void* stream) {
  sa::Kv4Cache c;
  const sinkattn_status st = tokens_common(cache, slots, num_seqs, cu_new, total, k, v, c);
  if (st != SINKATTN_OK || num_seqs == 0 || total == 0) return st;
  return from_cuda(sa::launch_kv4_append(c, slots, num_seqs, cu_new, total, k, v, static_cast<cudaStream_t>(stream)));
}

sinkattn_status sinkattn_kv4_read(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t num_seqs,
                                  const int32_t* cu, int32_t total, void* k, void* v, void* stream) {
  sa::Kv4Cache c;
  const sinkattn_status st = tokens_common(cache, slots, num_seqs, cu, total, k, v, c);
  if (st != SINKATTN_OK || num_seqs == 0 || total == 0) return st;
  return from_cuda(sa::launch_kv4_read(c, slots, num_seqs, cu, total, k, v, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_kv4_decode_workspace_size(int64_t num_rows, int32_t num_heads_q) {
  if (num_rows < 0 || num_rows > sa::kKv4MaxRequests * 128LL || num_heads_q < 1 || num_heads_q > sa::kMaxHeadsQ)
    return 0;
  return sa::kv4_decode_workspace_bytes(num_rows, num_heads_q);
}

sinkattn_status sinkattn_kv4_decode_fwd(const sinkattn_kv4_cache* cache, const int32_t* slots, int32_t num_seqs,
                                        int32_t q_per_seq, int32_t num_heads_q, int64_t window, int64_t prefix,
                                        float scale, const void* q, const float* sink, void* o, float* lse,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  sa::Kv4Cache c;
  sinkattn_status st = check_cache(cache, c);
  if (st != SINKATTN_OK) return st;
  if (q_per_seq < 1 || num_heads_q < 1 || num_heads_q % c.num_heads_kv != 0) return SINKATTN_ERR_INVALID_ARG;
  if (num_heads_q > sa::kMaxHeadsQ) return SINKATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_heads_q / c.num_heads_kv) * q_per_seq > 128) return SINKATTN_ERR_UNSUPPORTED;
  if (window < -1 || prefix < 0) return SINKATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SINKATTN_ERR_INVALID_ARG;
  if ((st = check_list(num_seqs, slots)) != SINKATTN_OK) return st;
  if (num_seqs == 0) return SINKATTN_OK;
  if (!q || !sink || !o || !lse) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(sink) || !aligned16(o) || !aligned16(lse)) return SINKATTN_ERR_ALIGNMENT;
  const long long rows = static_cast<long long>(num_seqs) * q_per_seq;
  if (workspace_bytes < sa::kv4_decode_workspace_bytes(rows, num_heads_q)) return SINKATTN_ERR_WORKSPACE;
  if (workspace == nullptr || !aligned16(workspace)) return workspace ? SINKATTN_ERR_ALIGNMENT : SINKATTN_ERR_INVALID_ARG;
  // positions stay below 2^30: a longer window or prefix covers everything
  const int w = window < 0 || window >= (1LL << 30) ? -1 : static_cast<int>(window);
  const int p = static_cast<int>(std::min<int64_t>(prefix, 1LL << 30));
  const sa::Kv4DecodeArgs a{slots, q, sink, o, lse, workspace, num_seqs, q_per_seq, num_heads_q, w, p, scale};
  int* status = sa::device_status_word();
  if (status == nullptr) return SINKATTN_ERR_CUDA;
  return from_cuda(sa::launch_kv4_decode(c, a, status, static_cast<cudaStream_t>(stream)));
}

sinkattn_status sinkattn_sample_tokens(const void* logits, int32_t dtype, int32_t rows, int32_t vocab,
                                       int64_t row_stride, const float* u, const float* temperature,
                                       const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                                       float* logp, float* logq, void* stream) {
  if (dtype < 0 || dtype > 2 || rows < 0 || vocab < 1 || row_stride < vocab) return SINKATTN_ERR_INVALID_ARG;
  if (vocab > (1 << 18) || rows > (1 << 24)) return SINKATTN_ERR_UNSUPPORTED;
  if (rows == 0) return SINKATTN_OK;
  if (!logits || !u || !temperature || !top_k || !top_p || !min_p || !tokens || !logp || !logq)
    return SINKATTN_ERR_INVALID_ARG;
  const uintptr_t size = dtype == 0 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size != 0 || !aligned4(u) || !aligned4(temperature) || !aligned4(top_k) ||
      !aligned4(top_p) || !aligned4(min_p) || !aligned4(tokens) || !aligned4(logp) || !aligned4(logq))
    return SINKATTN_ERR_ALIGNMENT;
  const sa::SampleArgs a{logits, dtype, rows, vocab, row_stride, u, temperature, top_k, top_p, min_p, tokens, logp, logq};
  return from_cuda(sa::launch_sample(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
