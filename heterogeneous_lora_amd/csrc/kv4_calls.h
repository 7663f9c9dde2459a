// Entry points of the cache in 4 bits (defined where this is included: kv4_read.hip).
#pragma once

#include "kv_calls.h"

namespace slora {

inline int kv4_token_bytes(int32_t n_kv_heads, int32_t head_dim, int64_t* bytes) {
  const char* what = "kv4_token_bytes";
  clear_error();
  if (!bytes) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  const int rc = check_shape(what, n_kv_heads, head_dim);
  if (rc) return rc;
  *bytes = kv4_layout(n_kv_heads, head_dim).token_bytes;
  return SLORA_OK;
}

inline int kv4_read(const slora_kv* kv, const slora_kv_rows* r, void* stream) {
  const char* what = "kv4_read";
  clear_error();
  if (!kv || !r) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  int rc = check_slots(what, kv);
  if (!rc) rc = check_pages(what, kv, 4);
  if (rc) return rc;
  if (r->n_tokens < 0) return fail(SLORA_E_INVALID, "%s: n_tokens %d < 0", what, r->n_tokens);
  if (r->n_tokens == 0 || (!r->k && !r->v)) return SLORA_OK;
  if (r->k && (rc = check_rows(what, "k", r->k, r->k_token_stride, r->k_head_stride))) return rc;
  if (r->v && (rc = check_rows(what, "v", r->v, r->v_token_stride, r->v_head_stride))) return rc;
  if ((r->k && !r->k_slots) || (r->v && !r->v_slots))
    return fail(SLORA_E_INVALID, "%s: k_slots or v_slots is NULL", what);
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      timed_call(SLORA_K_KV4_READ, s, [&](const LaunchEvents& ev) { return launch_kv4_read(*kv, *r, s, ev); });
  return e == hipSuccess ? SLORA_OK : launch_failed(e, what);
}

}  // namespace slora

extern "C" {

int slora_kv4_token_bytes(int32_t n_kv_heads, int32_t head_dim, int64_t* bytes) {
  return slora::guarded(__func__, [&] { return slora::kv4_token_bytes(n_kv_heads, head_dim, bytes); });
}

int slora_kv4_write(const slora_kv* kv, const slora_qkv* qkv, void* stream) {
  return slora::guarded(__func__, [&] {
    return slora::kv_write("kv4_write", 4, SLORA_K_KV4_WRITE, slora::launch_kv4_write, kv, qkv, stream);
  });
}

int slora_kv4_read(const slora_kv* kv, const slora_kv_rows* rows, void* stream) {
  return slora::guarded(__func__, [&] { return slora::kv4_read(kv, rows, stream); });
}

int slora_attn4_workspace_size(const slora_kv* kv, const slora_attn* attn, int32_t n_tokens, int64_t* bytes) {
  return slora::guarded(__func__,
                        [&] { return slora::workspace_size("attn4_workspace_size", 4, kv, attn, n_tokens, bytes); });
}

int slora_attn4_decode(const slora_kv* kv, const slora_attn* attn, void* ws, int64_t ws_bytes, void* stream) {
  return slora::guarded(__func__, [&] {
    return slora::attn_decode("attn4_decode", 4, SLORA_K_ATTN4_DECODE, slora::launch_attn4_decode, kv, attn, ws, ws_bytes,
                              stream);
  });
}

int slora_attn4_prefill(const slora_kv* kv, const slora_attn* attn, const int32_t* q_offsets, int32_t n_tokens, void* ws,
                        int64_t ws_bytes, void* stream) {
  return slora::guarded(__func__, [&] {
    return slora::attn_prefill("attn4_prefill", 4, SLORA_K_ATTN4_PREFILL, slora::launch_attn4_prefill, kv, attn, q_offsets,
                               n_tokens, ws, ws_bytes, stream);
  });
}

}  // extern "C"
