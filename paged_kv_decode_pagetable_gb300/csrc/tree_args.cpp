// The speculative calls with their arguments in a record: each unpacks it and makes the call.
#include <cstring>

#include "pkv_internal.h"

namespace {

// The record may stand at any address (a byte string's).
template <typename T>
T taken(const void *args) {
  T a;
  std::memcpy(&a, args, sizeof a);
  return a;
}

}  // namespace

extern "C" int tree_qkv_norm_rope_append_args(const void *args) {
  if (!args) return pkv::fail(PKV_E_BAD_ARG, "tree_qkv_norm_rope_append: NULL record");
  const auto a = taken<pkv_tree_append_args>(args);
  return tree_qkv_norm_rope_append(
      a.q, a.k, a.v, a.q_stride, a.k_stride, a.v_stride, a.gamma_q, a.gamma_k, a.batch_idx,
      a.ctx_lens, a.row_start, a.parents, a.theta, a.eps, a.rotary_dims, a.v_norm, a.B, a.N, a.Hq,
      a.Hkv, a.D, a.dev_table, a.n_slots, a.max_pages_per_seq, a.page_size, a.n_pages, a.k_cache,
      a.v_cache, a.q_out, a.err_word, a.stream);
}

extern "C" int paged_tree_attn_args(const void *args) {
  if (!args) return pkv::fail(PKV_E_BAD_ARG, "paged_tree_attn: NULL record");
  const auto a = taken<pkv_tree_attn_args>(args);
  return paged_tree_attn(a.q, a.k_cache, a.v_cache, a.dev_table, a.n_slots, a.max_pages_per_seq,
                         a.page_size, a.n_pages, a.batch_idx, a.ctx_lens, a.row_start, a.parents,
                         a.window, a.scale, a.B, a.N, a.Hq, a.Hkv, a.D, a.workspace,
                         a.workspace_bytes, a.out, a.err_word, a.stream);
}

extern "C" int tree_verify_args(const void *args) {
  if (!args) return pkv::fail(PKV_E_BAD_ARG, "tree_verify: NULL record");
  const auto a = taken<pkv_tree_verify_args>(args);
  return tree_verify(a.target_probs, a.target_stride, a.draft_probs, a.draft_stride, a.tokens,
                     a.row_start, a.parents, a.u_accept, a.u_pick, a.B, a.N, a.V, a.path_cols,
                     a.accepted, a.path, a.next_token, a.err_word, a.stream);
}

extern "C" int kv_keep_path_args(const void *args) {
  if (!args) return pkv::fail(PKV_E_BAD_ARG, "kv_keep_path: NULL record");
  const auto a = taken<pkv_keep_path_args>(args);
  return kv_keep_path(a.caches, a.heads, a.token_bytes, a.n_caches, a.dev_table, a.n_slots,
                      a.max_pages_per_seq, a.page_size, a.n_pages, a.batch_idx, a.ctx_lens,
                      a.accepted, a.path, a.path_cols, a.B, a.err_word, a.stream);
}
