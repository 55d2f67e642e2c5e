// C ABI of the pages of bf16 keys and values and of the verification of
// drafted tokens.  Argument checks and dispatch; the contract of every entry
// point is in include/sinkattn.h.
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
sinkattn_status check_pages(const sinkattn_kv_pages* c, sa::KvPages& out) {
  if (c == nullptr) return SINKATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_heads_kv < 1 || c->num_slots < 1 || c->max_pages < 1) return SINKATTN_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return SINKATTN_ERR_UNSUPPORTED;
  if (c->num_heads_kv > sa::kMaxHeadsQ) return SINKATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * c->page_size > (1LL << 30)) return SINKATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->num_pages) * c->page_size >= (1LL << 31)) return SINKATTN_ERR_UNSUPPORTED;
  if (!c->k_pages || !c->v_pages || !c->block_table || !c->seqlens || !c->owner) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned16(c->block_table) || !aligned16(c->seqlens) ||
      !aligned16(c->owner))
    return SINKATTN_ERR_ALIGNMENT;
  out.k = static_cast<__nv_bfloat16*>(c->k_pages);
  out.v = static_cast<__nv_bfloat16*>(c->v_pages);
  out.block_table = c->block_table;
  out.seqlens = c->seqlens;
  out.owner = c->owner;
  out.num_pages = c->num_pages;
  out.page_size = c->page_size;
  out.num_heads_kv = c->num_heads_kv;
  out.num_slots = c->num_slots;
  out.max_pages = c->max_pages;
  out.page_log2 = 0;
  while ((1 << out.page_log2) < c->page_size) ++out.page_log2;
  return SINKATTN_OK;
}

}  // namespace

extern "C" {

sinkattn_status sinkattn_kv_plan(const sinkattn_kv_pages* pages, const int32_t* slots, const int32_t* drop,
                                 const int32_t* new_tokens, int32_t n, int32_t* live, int32_t* cu, int32_t* slot_map,
                                 int32_t* positions, int32_t total, void* stream) {
  sa::KvPages c;
  sinkattn_status st = check_pages(pages, c);
  if (st != SINKATTN_OK) return st;
  if ((st = check_list(n, slots)) != SINKATTN_OK || (st = check_list(n, new_tokens)) != SINKATTN_OK ||
      (st = check_list(n, live)) != SINKATTN_OK)
    return st;
  if (total < 0 || !cu || (total > 0 && (!slot_map || !positions))) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned4(drop) || !aligned4(cu) || !aligned4(slot_map) || !aligned4(positions)) return SINKATTN_ERR_ALIGNMENT;
  const sa::KvPlanArgs a{slots, drop, new_tokens, n, total, live, cu, slot_map, positions};
  return from_cuda(sa::launch_kv_plan(c, a, static_cast<cudaStream_t>(stream)));
}

sinkattn_status sinkattn_kv_write(const sinkattn_kv_pages* pages, const int32_t* slot_map, int32_t rows, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride, void* stream) {
  sa::KvPages c;
  sinkattn_status st = check_pages(pages, c);
  if (st != SINKATTN_OK) return st;
  if (rows < 0) return SINKATTN_ERR_INVALID_ARG;
  if (rows == 0) return SINKATTN_OK;
  const int64_t row = static_cast<int64_t>(c.num_heads_kv) * sa::kHeadDim;
  if (!slot_map || !k || !v || k_stride < row || v_stride < row) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned4(slot_map) || !aligned16(k) || !aligned16(v) || k_stride % 8 != 0 || v_stride % 8 != 0)
    return SINKATTN_ERR_ALIGNMENT;
  const sa::KvWriteArgs a{slot_map, static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
                          k_stride, v_stride, rows};
  return from_cuda(sa::launch_kv_write(c, a, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_kv_decode_workspace_size(int32_t num_heads_kv) {
  if (num_heads_kv < 1 || num_heads_kv > sa::kMaxHeadsQ) return 0;
  return sa::kv_decode_workspace_bytes(num_heads_kv);
}

sinkattn_status sinkattn_kv_decode_fwd(const sinkattn_kv_pages* pages, const int32_t* slots, const int32_t* cu_rows,
                                       int32_t num_seqs, int32_t q_per_seq, int32_t rows, int32_t num_heads_q,
                                       int64_t window, int64_t prefix, float scale, const void* q, const float* sink,
                                       void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  sa::KvPages c;
  sinkattn_status st = check_pages(pages, c);
  if (st != SINKATTN_OK) return st;
  if (q_per_seq < 1 || rows < 0 || num_heads_q < 1 || num_heads_q % c.num_heads_kv != 0) return SINKATTN_ERR_INVALID_ARG;
  if (num_heads_q > sa::kMaxHeadsQ) return SINKATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_heads_q / c.num_heads_kv) * q_per_seq > 128) return SINKATTN_ERR_UNSUPPORTED;
  if (window < -1 || prefix < 0) return SINKATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SINKATTN_ERR_INVALID_ARG;
  if ((st = check_list(num_seqs, slots)) != SINKATTN_OK) return st;
  if (!aligned4(cu_rows)) return SINKATTN_ERR_ALIGNMENT;
  if (cu_rows == nullptr && rows != static_cast<long long>(num_seqs) * q_per_seq) return SINKATTN_ERR_INVALID_ARG;
  if (num_seqs == 0 || rows == 0) return SINKATTN_OK;
  if (!q || !sink || !o || !lse) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(sink) || !aligned16(o) || !aligned16(lse)) return SINKATTN_ERR_ALIGNMENT;
  if (workspace_bytes < sa::kv_decode_workspace_bytes(c.num_heads_kv)) return SINKATTN_ERR_WORKSPACE;
  if (workspace == nullptr || !aligned16(workspace)) return workspace ? SINKATTN_ERR_ALIGNMENT : SINKATTN_ERR_INVALID_ARG;
  // positions stay below 2^30: a longer window or prefix covers everything
  const int w = window < 0 || window >= (1LL << 30) ? -1 : static_cast<int>(window);
  const int p = static_cast<int>(std::min<int64_t>(prefix, 1LL << 30));
  const sa::KvDecodeArgs a{slots, cu_rows, q, sink, o, lse, workspace, num_seqs, rows, q_per_seq, num_heads_q, w, p, scale};
  int* status = sa::device_status_word();
  if (status == nullptr) return SINKATTN_ERR_CUDA;
  return from_cuda(sa::launch_kv_decode(c, a, status, static_cast<cudaStream_t>(stream)));
}

size_t sinkattn_verify_workspace_size(int32_t dtype, int32_t rows, int32_t vocab) {
  if (dtype < 0 || dtype > 2 || rows < 0 || rows > (1 << 20) || vocab < 1 || vocab > (1 << 18)) return 0;
  return sa::verify_workspace_bytes(dtype, rows, vocab);
}

sinkattn_status sinkattn_verify_tokens(const void* logits, int64_t row_stride, const void* draft_logits,
                                       int64_t draft_stride, int32_t dtype, int32_t rows, int32_t num_drafts,
                                       int32_t vocab, const int32_t* drafts, const int32_t* cu_rows, int32_t num_seqs,
                                       const float* u, const float* temperature, int32_t* tokens, float* logp,
                                       int32_t* accepted, int32_t* rejected, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  return sinkattn_verify_live_tokens(logits, row_stride, draft_logits, draft_stride, dtype, rows, num_drafts, vocab,
                                     drafts, cu_rows, nullptr, num_seqs, u, temperature, tokens, logp, accepted, rejected,
                                     workspace, workspace_bytes, stream);
}

sinkattn_status sinkattn_verify_live_tokens(const void* logits, int64_t row_stride, const void* draft_logits,
                                            int64_t draft_stride, int32_t dtype, int32_t rows, int32_t num_drafts,
                                            int32_t vocab, const int32_t* drafts, const int32_t* cu_rows,
                                            const int32_t* live, int32_t num_seqs, const float* u,
                                            const float* temperature, int32_t* tokens, float* logp, int32_t* accepted,
                                            int32_t* rejected, void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype < 0 || dtype > 2 || rows < 0 || num_drafts < 0 || num_drafts > rows || vocab < 1 || row_stride < vocab ||
      (draft_logits != nullptr && draft_stride < vocab))
    return SINKATTN_ERR_INVALID_ARG;
  if (vocab > (1 << 18) || rows > (1 << 20)) return SINKATTN_ERR_UNSUPPORTED;
  sinkattn_status st = check_list(num_seqs, temperature);
  if (st != SINKATTN_OK || (st = check_list(num_seqs, accepted)) != SINKATTN_OK ||
      (st = check_list(num_seqs, rejected)) != SINKATTN_OK)
    return st;
  if (num_seqs == 0) return SINKATTN_OK;
  if (!cu_rows) return SINKATTN_ERR_INVALID_ARG;
  if (!aligned4(cu_rows) || !aligned4(live)) return SINKATTN_ERR_ALIGNMENT;
  if ((rows > 0 && (!logits || !u || !tokens || !logp)) || (num_drafts > 0 && !drafts)) return SINKATTN_ERR_INVALID_ARG;
  const uintptr_t size = dtype == 0 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size != 0 || reinterpret_cast<uintptr_t>(draft_logits) % size != 0 ||
      !aligned4(drafts) || !aligned4(u) || !aligned4(tokens) || !aligned4(logp))
    return SINKATTN_ERR_ALIGNMENT;
  if (workspace_bytes < sa::verify_workspace_bytes(dtype, rows, vocab)) return SINKATTN_ERR_WORKSPACE;
  if (rows > 0 && (workspace == nullptr || !aligned16(workspace)))
    return workspace ? SINKATTN_ERR_ALIGNMENT : SINKATTN_ERR_INVALID_ARG;
  const sa::VerifyArgs a{logits, draft_logits, dtype, rows, num_drafts, vocab, num_seqs, row_stride, draft_stride,
                         drafts, cu_rows, live, u, temperature, tokens, logp, accepted, rejected,
                         static_cast<float4*>(workspace)};
  return from_cuda(sa::launch_verify(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
