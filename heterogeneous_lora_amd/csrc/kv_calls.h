// KV cache and attention calls: argument checks and kernel arguments, for caches of 16 and of 4
// bits a value (kv.cpp, kv4_calls.h). Everything that depends on device data (lengths, tables,
// slots) is checked by the kernels.
#pragma once

#include <float.h>
#include <math.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "guard.h"
#include "internal.h"

namespace slora {

using LaunchWrite = hipError_t (*)(const slora_kv&, const slora_qkv&, hipStream_t, const LaunchEvents&);
using LaunchAttn = hipError_t (*)(const AttnArgs&, int32_t, hipStream_t, const LaunchEvents&);

inline int launch_failed(hipError_t e, const char* what) {
  char text[64];
  snprintf(text, sizeof text, "%s launch", what);
  return hip_fail(e, text);
}

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// What a call that takes slots uses of them.
inline int check_slots(const char* what, const slora_kv* kv) {
  if (kv->n_pages < 0 || kv->n_pages > INT32_MAX)
    return fail(SLORA_E_INVALID, "%s: n_pages %lld outside 0..2^31-1", what, (long long)kv->n_pages);
  if (kv->tokens_per_page < 1) return fail(SLORA_E_INVALID, "%s: tokens_per_page %d < 1", what, kv->tokens_per_page);
  return SLORA_OK;
}

// The cache's lengths: what slora_kv_tables uses of it.
inline int check_lengths(const char* what, const slora_kv* kv) {
  const int rc = check_slots(what, kv);
  if (rc) return rc;
  if (kv->n_requests < 0 || kv->n_requests > SLORA_KV_MAX_REQUESTS)
    return fail(SLORA_E_INVALID, "%s: n_requests %d outside 0..%d", what, kv->n_requests, SLORA_KV_MAX_REQUESTS);
  if (kv->max_blocks < 0 || (int64_t)kv->max_blocks * kv->tokens_per_page > (int64_t(1) << 30))
    return fail(SLORA_E_INVALID, "%s: max_blocks %d x tokens_per_page %d outside 0..2^30", what, kv->max_blocks,
                kv->tokens_per_page);
  return SLORA_OK;
}

inline int check_shape(const char* what, int32_t n_kv_heads, int32_t head_dim) {
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(SLORA_E_INVALID, "%s: head_dim %d is not a multiple of 8 in 8..256", what, head_dim);
  if (n_kv_heads < 1 || n_kv_heads > 1024)
    return fail(SLORA_E_INVALID, "%s: n_kv_heads %d outside 1..1024", what, n_kv_heads);
  return SLORA_OK;
}

// The cache's pages. bits: of a value in it, 16 or 4.
inline int check_pages(const char* what, const slora_kv* kv, int bits) {
  if (!kv->pool || misaligned(kv->pool, 16))
    return fail(SLORA_E_INVALID, "%s: pool must be a 16-byte aligned device pointer", what);
  if (kv->dtype != SLORA_F16 && kv->dtype != SLORA_BF16)
    return fail(SLORA_E_INVALID, "%s: unknown dtype %d", what, kv->dtype);
  if (kv->page_elems < 8 || kv->page_elems % 8)
    return fail(SLORA_E_INVALID, "%s: page_elems %d is not a positive multiple of 8", what, kv->page_elems);
  const int rc = check_shape(what, kv->n_kv_heads, kv->head_dim);
  if (rc) return rc;
  if (bits == 4) {
    const int64_t token = kv4_layout(kv->n_kv_heads, kv->head_dim).token_bytes;
    if (kv->tokens_per_page * token > 2 * (int64_t)kv->page_elems)
      return fail(SLORA_E_INVALID, "%s: %d tokens of %lld bytes (%d heads x %d in 4 bits) do not fit a page of %lld bytes",
                  what, kv->tokens_per_page, (long long)token, kv->n_kv_heads, kv->head_dim,
                  2 * (long long)kv->page_elems);
  } else if ((int64_t)kv->tokens_per_page * kv->n_kv_heads * kv->head_dim > kv->page_elems)
    return fail(SLORA_E_INVALID, "%s: %d tokens of %d heads x %d do not fit a page of %d elements", what,
                kv->tokens_per_page, kv->n_kv_heads, kv->head_dim, kv->page_elems);
  return SLORA_OK;
}

inline int check_rows(const char* what, const char* name, const void* p, int64_t token_stride, int64_t head_stride) {
  if (!p || misaligned(p, 16)) return fail(SLORA_E_INVALID, "%s: %s must be a 16-byte aligned device pointer", what, name);
  if (token_stride % 8 || head_stride % 8)
    return fail(SLORA_E_INVALID, "%s: %s strides %lld, %lld are not multiples of 8 elements", what, name,
                (long long)token_stride, (long long)head_stride);
  return SLORA_OK;
}

// `launch` and kernel id `id` of a call on a cache of `bits` bits a value, below too.
inline int kv_write(const char* what, int bits, int id, LaunchWrite launch, const slora_kv* kv, const slora_qkv* w,
                    void* stream) {
  clear_error();
  if (!kv || !w) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  int rc = check_slots(what, kv);
  if (!rc) rc = check_pages(what, kv, bits);
  if (rc) return rc;
  if (w->n_tokens < 0) return fail(SLORA_E_INVALID, "%s: n_tokens %d < 0", what, w->n_tokens);
  if (w->n_q_heads < 1 || w->n_q_heads > 16384)
    return fail(SLORA_E_INVALID, "%s: n_q_heads %d outside 1..16384", what, w->n_q_heads);
  if (w->rotary_dim < 0 || w->rotary_dim > kv->head_dim || w->rotary_dim % 8)
    return fail(SLORA_E_INVALID, "%s: rotary_dim %d is not a multiple of 8 in 0..head_dim %d", what, w->rotary_dim,
                kv->head_dim);
  if (w->norm && !(w->eps >= 0.f)) return fail(SLORA_E_INVALID, "%s: eps %g < 0", what, (double)w->eps);
  if (w->n_tokens == 0) return SLORA_OK;
  if ((rc = check_rows(what, "q", w->q, w->q_token_stride, w->q_head_stride))) return rc;
  if ((rc = check_rows(what, "q_out", w->q_out, w->out_token_stride, w->out_head_stride))) return rc;
  if (!w->k != !w->v) return fail(SLORA_E_INVALID, "%s: k and v are given together or not at all", what);
  if (w->k) {
    if ((rc = check_rows(what, "k", w->k, w->k_token_stride, w->k_head_stride))) return rc;
    if ((rc = check_rows(what, "v", w->v, w->v_token_stride, w->v_head_stride))) return rc;
    if (!w->k_slots || !w->v_slots) return fail(SLORA_E_INVALID, "%s: k_slots or v_slots is NULL", what);
  }
  if (w->q_out == w->q && (w->out_token_stride != w->q_token_stride || w->out_head_stride != w->q_head_stride))
    return fail(SLORA_E_INVALID, "%s: q_out is q with other strides", what);
  if (!w->position || (w->rotary_dim && !w->turns)) return fail(SLORA_E_INVALID, "%s: position or turns is NULL", what);
  if (w->norm && ((w->q_weight && misaligned(w->q_weight, 16)) || (w->k_weight && misaligned(w->k_weight, 16))))
    return fail(SLORA_E_INVALID, "%s: norm weights must be 16-byte aligned", what);
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = timed_call(id, s, [&](const LaunchEvents& ev) { return launch(*kv, *w, s, ev); });
  return e == hipSuccess ? SLORA_OK : launch_failed(e, what);
}

inline int check_heads(const char* what, int bits, const slora_kv* kv, const slora_attn* at) {
  int rc = check_lengths(what, kv);
  if (!rc) rc = check_pages(what, kv, bits);
  if (rc) return rc;
  if (at->n_q_heads < 1 || at->n_q_heads > 16384 || at->n_q_heads % kv->n_kv_heads)
    return fail(SLORA_E_INVALID, "%s: n_q_heads %d is not a multiple of n_kv_heads %d in 1..16384", what,
                at->n_q_heads, kv->n_kv_heads);
  return SLORA_OK;
}

inline int64_t decode4_cut_bytes(int32_t n_req) { return ((int64_t)n_req * 8 + 255) / 256 * 256; }

inline int64_t decode_workspace(int bits, const slora_kv* kv, const slora_attn* at) {
  const int group = at->n_q_heads / kv->n_kv_heads, n = kv->n_requests;
  const int64_t row = at->n_q_heads * attn_part_floats(kv->head_dim) * (int64_t)sizeof(float);
  int64_t rest = ((int64_t)n + decode_chunks(decode_units(n, kv->n_kv_heads, group))) * row;
  if (bits == 4) {  // (enough for any window)
    const Decode4 d = decode4_plan(n, kv->n_kv_heads, group, kv->head_dim, kv->max_blocks * kv->tokens_per_page, 0);
    rest = std::max(rest, decode4_cut_bytes(n) + 2 * row * d.spans);
  }
  return kAttnCounterBytes + rest;
}

inline int64_t prefill_workspace(const slora_kv* kv, const slora_attn* at, int32_t n_tokens) {
  const int group = at->n_q_heads / kv->n_kv_heads;
  const int64_t chunks = prefill_chunks(n_tokens, group, kv->n_kv_heads, kv->max_blocks * kv->tokens_per_page);
  return kAttnCounterBytes + 2 * chunks * kv->n_kv_heads * prefill_waves(n_tokens, group) *
                                 part_floats(attn_instance(kv->head_dim)) * (int64_t)sizeof(float);
}
inline Prefill4 prefill4_of(const slora_kv* kv, const slora_attn* at, int32_t n_tokens) {
  return prefill4_plan(kv->n_requests, n_tokens, at->n_q_heads / kv->n_kv_heads, kv->n_kv_heads, kv->head_dim,
                       kv->max_blocks * kv->tokens_per_page);
}
inline int64_t prefill_workspace(int bits, const slora_kv* kv, const slora_attn* at, int32_t n_tokens) {
  const int64_t rest = prefill_workspace(kv, at, n_tokens);
  if (bits != 4) return rest;
  const Prefill4 p = prefill4_of(kv, at, n_tokens);
  return p.back ? (rest + 255) / 256 * 256 + p.table_bytes + p.bytes : rest;
}

inline int workspace_size(const char* what, int bits, const slora_kv* kv, const slora_attn* at, int32_t n_tokens,
                   int64_t* bytes) {
  clear_error();
  if (!kv || !at || !bytes) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  if (n_tokens < 0) return fail(SLORA_E_INVALID, "%s: n_tokens %d < 0", what, n_tokens);
  const int rc = check_heads(what, bits, kv, at);
  if (rc) return rc;
  *bytes = n_tokens ? prefill_workspace(bits, kv, at, n_tokens) : decode_workspace(bits, kv, at);
  return SLORA_OK;
}

// Checks an attention call and fills the kernels' arguments.
inline int attn_args(const char* what, int bits, const slora_kv* kv, const slora_attn* at, void* ws, int64_t ws_bytes, int64_t need,
              AttnArgs* a) {
  if (!(at->softcap >= 0.f) || !std::isfinite(at->softcap) || !std::isfinite(at->scale))
    return fail(SLORA_E_INVALID, "%s: scale %g must be finite and softcap %g finite and >= 0", what, (double)at->scale,
                (double)at->softcap);
  if (at->window < 0) return fail(SLORA_E_INVALID, "%s: window %d < 0", what, at->window);
  if (!at->seq_len) return fail(SLORA_E_INVALID, "%s: seq_len is NULL", what);
  if (kv->max_blocks && (!at->k_table || !at->v_table)) return fail(SLORA_E_INVALID, "%s: k_table or v_table is NULL", what);
  int rc = check_rows(what, "q", at->q, at->q_token_stride, at->q_head_stride);
  if (!rc) rc = check_rows(what, "out", at->out, at->out_token_stride, at->out_head_stride);
  if (rc) return rc;
  if (!ws || misaligned(ws, 256)) return fail(SLORA_E_INVALID, "%s: ws must be 256-byte aligned", what);
  if (ws_bytes < need)
    return fail(SLORA_E_INVALID, "%s: workspace of %lld bytes is smaller than the %lld needed", what, (long long)ws_bytes,
                (long long)need);
  *a = AttnArgs();
  a->pool = (const uint16_t*)kv->pool;
  a->n_pages_u = (uint32_t)kv->n_pages;
  a->P = kv->page_elems;
  a->tpp = kv->tokens_per_page;
  divisor(a->tpp, &a->tpp_magic, &a->tpp_shift);
  a->hk = kv->n_kv_heads;
  divisor(a->hk, &a->hk_magic, &a->hk_shift);
  a->D = kv->head_dim;
  a->row = a->hk * a->D;
  a->n_req = kv->n_requests;
  a->max_blocks = kv->max_blocks;
  a->max_len = kv->max_blocks * kv->tokens_per_page;
  a->group = at->n_q_heads / kv->n_kv_heads;
  divisor(a->group, &a->group_magic, &a->group_shift);
  a->kt = at->k_table;
  a->vt = at->v_table;
  a->seq = at->seq_len;
  a->prefix = at->prefix_len;
  a->q = (const uint16_t*)at->q;
  a->q_ts = at->q_token_stride;
  a->q_hs = at->q_head_stride;
  a->out = (uint16_t*)at->out;
  a->o_ts = at->out_token_stride;
  a->o_hs = at->out_head_stride;
  a->lse = at->lse;
  const double log2e = 1.4426950408889634;
  a->scale2 = (float)(at->scale * log2e);
  if (at->softcap > 0.f) {
    // (finite: times a score of 0 it is 0; cap_out may be infinite, its form is then not used)
    a->cap_in = (float)std::clamp(2.0 * log2e * at->scale / at->softcap, -(double)FLT_MAX, (double)FLT_MAX);
    a->cap_out = (float)(at->softcap * log2e);
  }
  // (a window that covers any request is none: positions minus it stay in range)
  a->window = at->window < a->max_len ? at->window : 0;
  a->slopes = at->slopes;
  a->counters = (int32_t*)ws;
  a->part = (float*)((uint8_t*)ws + kAttnCounterBytes);
  a->wg_heads = decode_wg_heads(a->n_req, a->hk, a->group);
  a->chunks = decode_chunks(decode_units(a->n_req, a->hk, a->group));
  if (bits == 4) {
    const Decode4 d = decode4_plan(a->n_req, a->hk, a->group, a->D, a->max_len, a->window);
    a->kv4 = kv4_layout(a->hk, a->D);
    a->wave_heads = d.heads;
    a->wave_runs = d.runs;
    a->wg_units = d.wg_units;
    a->spans = d.spans;
  }
  return SLORA_OK;
}

inline int attn_decode(const char* what, int bits, int id, LaunchAttn launch, const slora_kv* kv, const slora_attn* at,
                       void* ws, int64_t ws_bytes, void* stream) {
  clear_error();
  if (!kv || !at) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  int rc = check_heads(what, bits, kv, at);
  if (rc) return rc;
  if (kv->n_requests == 0) return SLORA_OK;
  AttnArgs a;
  if ((rc = attn_args(what, bits, kv, at, ws, ws_bytes, decode_workspace(bits, kv, at), &a))) return rc;
  if (a.spans) {
    a.cut = (int2*)a.part;
    a.part += decode4_cut_bytes(a.n_req) / (int64_t)sizeof(float);
  }
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = timed_call(id, s, [&](const LaunchEvents& ev) { return launch(a, kv->dtype, s, ev); });
  return e == hipSuccess ? SLORA_OK : launch_failed(e, what);
}

inline int attn_prefill(const char* what, int bits, int id, LaunchAttn launch, const slora_kv* kv, const slora_attn* at,
                        const int32_t* q_offsets, int32_t n_tokens, void* ws, int64_t ws_bytes, void* stream) {
  clear_error();
  if (!kv || !at) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  if (n_tokens < 0) return fail(SLORA_E_INVALID, "%s: n_tokens %d < 0", what, n_tokens);
  int rc = check_heads(what, bits, kv, at);
  if (rc) return rc;
  if (kv->n_requests == 0 || n_tokens == 0) return SLORA_OK;
  if (!q_offsets) return fail(SLORA_E_INVALID, "%s: q_offsets is NULL", what);
  AttnArgs a;
  if ((rc = attn_args(what, bits, kv, at, ws, ws_bytes, prefill_workspace(bits, kv, at, n_tokens), &a))) return rc;
  a.q_offsets = q_offsets;
  a.n_tok = n_tokens;
  a.chunks = prefill_chunks(n_tokens, a.group, a.hk, a.max_len);
  a.part_waves = prefill_waves(n_tokens, a.group);
  if (bits == 4 && prefill4_of(kv, at, n_tokens).back)
    a.back = (int32_t*)((uint8_t*)ws + (prefill_workspace(kv, at, n_tokens) + 255) / 256 * 256);
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = timed_call(id, s, [&](const LaunchEvents& ev) { return launch(a, kv->dtype, s, ev); });
  return e == hipSuccess ? SLORA_OK : launch_failed(e, what);
}

}  // namespace slora
