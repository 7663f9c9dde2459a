// KV cache and attention entry points: argument checks and kernel arguments. Everything
// that depends on device data (lengths, tables, slots) is checked by the kernels.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "guard.h"
#include "internal.h"

using namespace slora;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// The cache's lengths: what slora_kv_tables uses of it.
int check_lengths(const char* what, const slora_kv* kv) {
  if (kv->n_pages < 0 || kv->n_pages > INT32_MAX)
    return fail(SLORA_E_INVALID, "%s: n_pages %lld outside 0..2^31-1", what, (long long)kv->n_pages);
  if (kv->tokens_per_page < 1) return fail(SLORA_E_INVALID, "%s: tokens_per_page %d < 1", what, kv->tokens_per_page);
  if (kv->n_requests < 0 || kv->n_requests > SLORA_KV_MAX_REQUESTS)
    return fail(SLORA_E_INVALID, "%s: n_requests %d outside 0..%d", what, kv->n_requests, SLORA_KV_MAX_REQUESTS);
  if (kv->max_blocks < 0 || (int64_t)kv->max_blocks * kv->tokens_per_page > (int64_t(1) << 30))
    return fail(SLORA_E_INVALID, "%s: max_blocks %d x tokens_per_page %d outside 0..2^30", what, kv->max_blocks,
                kv->tokens_per_page);
  return SLORA_OK;
}

// The cache's pages.
int check_pages(const char* what, const slora_kv* kv) {
  if (!kv->pool || misaligned(kv->pool, 16))
    return fail(SLORA_E_INVALID, "%s: pool must be a 16-byte aligned device pointer", what);
  if (kv->dtype != SLORA_F16 && kv->dtype != SLORA_BF16)
    return fail(SLORA_E_INVALID, "%s: unknown dtype %d", what, kv->dtype);
  if (kv->page_elems < 8 || kv->page_elems % 8)
    return fail(SLORA_E_INVALID, "%s: page_elems %d is not a positive multiple of 8", what, kv->page_elems);
  if (kv->head_dim < 8 || kv->head_dim > 256 || kv->head_dim % 8)
    return fail(SLORA_E_INVALID, "%s: head_dim %d is not a multiple of 8 in 8..256", what, kv->head_dim);
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024)
    return fail(SLORA_E_INVALID, "%s: n_kv_heads %d outside 1..1024", what, kv->n_kv_heads);
  if ((int64_t)kv->tokens_per_page * kv->n_kv_heads * kv->head_dim > kv->page_elems)
    return fail(SLORA_E_INVALID, "%s: %d tokens of %d heads x %d do not fit a page of %d elements", what,
                kv->tokens_per_page, kv->n_kv_heads, kv->head_dim, kv->page_elems);
  return SLORA_OK;
}

int check_rows(const char* what, const char* name, const void* p, int64_t token_stride, int64_t head_stride) {
  if (!p || misaligned(p, 16)) return fail(SLORA_E_INVALID, "%s: %s must be a 16-byte aligned device pointer", what, name);
  if (token_stride % 8 || head_stride % 8)
    return fail(SLORA_E_INVALID, "%s: %s strides %lld, %lld are not multiples of 8 elements", what, name,
                (long long)token_stride, (long long)head_stride);
  return SLORA_OK;
}

int kv_tables(const slora_kv* kv, const slora_kv_step* st, void* stream) {
  const char* what = "kv_tables";
  clear_error();
  if (!kv || !st) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  int rc = check_lengths(what, kv);
  if (rc) return rc;
  if (st->n_planes < 1 || st->n_planes > SLORA_KV_MAX_PLANES)
    return fail(SLORA_E_INVALID, "%s: n_planes %d outside 1..%d", what, st->n_planes, SLORA_KV_MAX_PLANES);
  if (st->n_tokens < 0 || st->n_page_ids < 0)
    return fail(SLORA_E_INVALID, "%s: n_tokens %d or n_page_ids %lld < 0", what, st->n_tokens, (long long)st->n_page_ids);
  if (!st->q_offsets || (kv->n_requests && (!st->past_len || !st->new_len || !st->seq_len)))
    return fail(SLORA_E_INVALID, "%s: a length array is NULL", what);
  if ((st->n_page_ids && !st->pages) || (kv->n_requests && kv->max_blocks && !st->tables))
    return fail(SLORA_E_INVALID, "%s: pages or tables is NULL", what);
  if (st->n_tokens && (!st->token_request || !st->position || !st->slots))
    return fail(SLORA_E_INVALID, "%s: a token array is NULL", what);
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      timed_call(SLORA_K_KV_TABLES, s, [&](const LaunchEvents& ev) { return launch_kv_tables(*kv, *st, s, ev); });
  return e == hipSuccess ? SLORA_OK : hip_fail(e, "kv_tables launch");
}

int rope_turns(const slora_rope* rope, double* turns) {
  const char* what = "rope_turns";
  clear_error();
  if (!rope || !turns) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  const int d = rope->rotary_dim;
  if (d < 8 || d > 256 || d % 8) return fail(SLORA_E_INVALID, "%s: rotary_dim %d is not a multiple of 8 in 8..256", what, d);
  if (!(rope->theta > 0) || !(rope->factor > 0) || !std::isfinite(rope->theta) || !std::isfinite(rope->factor))
    return fail(SLORA_E_INVALID, "%s: theta and factor must be positive", what);
  if (rope->scaling < SLORA_ROPE_NONE || rope->scaling > SLORA_ROPE_BANDS)
    return fail(SLORA_E_INVALID, "%s: unknown scaling %d", what, rope->scaling);
  const double lo = rope->low_turns, hi = rope->high_turns;
  if (rope->scaling == SLORA_ROPE_BANDS && !(lo > 0 && hi > lo && std::isfinite(hi) && rope->original_len > 0 &&
                                             std::isfinite(rope->original_len)))
    return fail(SLORA_E_INVALID, "%s: bands need original_len > 0 and 0 < low_turns < high_turns", what);
  const double theta =
      rope->scaling == SLORA_ROPE_BASE ? rope->theta * pow(rope->factor, (double)d / (d - 2)) : rope->theta;
  for (int i = 0; i < d / 2; ++i) {
    double t = pow(theta, -2.0 * i / d) / kTwoPi;
    if (rope->scaling == SLORA_ROPE_LINEAR) t /= rope->factor;
    if (rope->scaling == SLORA_ROPE_BANDS) {
      double keep = (t * rope->original_len - lo) / (hi - lo);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      t = t * keep + t / rope->factor * (1 - keep);
    }
    turns[i] = t;
  }
  return SLORA_OK;
}

int kv_write(const slora_kv* kv, const slora_qkv* w, void* stream) {
  const char* what = "kv_write";
  clear_error();
  if (!kv || !w) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  if (kv->n_pages < 0 || kv->n_pages > INT32_MAX)
    return fail(SLORA_E_INVALID, "%s: n_pages %lld outside 0..2^31-1", what, (long long)kv->n_pages);
  if (kv->tokens_per_page < 1) return fail(SLORA_E_INVALID, "%s: tokens_per_page %d < 1", what, kv->tokens_per_page);
  int rc = check_pages(what, kv);
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
  const hipError_t e =
      timed_call(SLORA_K_KV_WRITE, s, [&](const LaunchEvents& ev) { return launch_kv_write(*kv, *w, s, ev); });
  return e == hipSuccess ? SLORA_OK : hip_fail(e, "kv_write launch");
}

int check_heads(const char* what, const slora_kv* kv, const slora_attn* at) {
  int rc = check_lengths(what, kv);
  if (!rc) rc = check_pages(what, kv);
  if (rc) return rc;
  if (at->n_q_heads < 1 || at->n_q_heads > 16384 || at->n_q_heads % kv->n_kv_heads)
    return fail(SLORA_E_INVALID, "%s: n_q_heads %d is not a multiple of n_kv_heads %d in 1..16384", what,
                at->n_q_heads, kv->n_kv_heads);
  return SLORA_OK;
}

int64_t decode_workspace(const slora_kv* kv, const slora_attn* at) {
  const int units = decode_units(kv->n_requests, kv->n_kv_heads, at->n_q_heads / kv->n_kv_heads);
  return kAttnCounterBytes + ((int64_t)kv->n_requests + decode_chunks(units)) * at->n_q_heads *
                                 attn_part_floats(kv->head_dim) * (int64_t)sizeof(float);
}

int64_t prefill_workspace(const slora_kv* kv, const slora_attn* at, int32_t n_tokens) {
  const int group = at->n_q_heads / kv->n_kv_heads;
  const int64_t chunks = prefill_chunks(n_tokens, group, kv->n_kv_heads, kv->max_blocks * kv->tokens_per_page);
  return kAttnCounterBytes + 2 * chunks * kv->n_kv_heads * prefill_waves(n_tokens, group) *
                                 part_floats(attn_instance(kv->head_dim)) * (int64_t)sizeof(float);
}

int workspace_size(const slora_kv* kv, const slora_attn* at, int32_t n_tokens, int64_t* bytes) {
  const char* what = "attn_workspace_size";
  clear_error();
  if (!kv || !at || !bytes) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  if (n_tokens < 0) return fail(SLORA_E_INVALID, "%s: n_tokens %d < 0", what, n_tokens);
  const int rc = check_heads(what, kv, at);
  if (rc) return rc;
  *bytes = n_tokens ? prefill_workspace(kv, at, n_tokens) : decode_workspace(kv, at);
  return SLORA_OK;
}

// Checks an attention call and fills the kernels' arguments.
int attn_args(const char* what, const slora_kv* kv, const slora_attn* at, void* ws, int64_t ws_bytes, int64_t need,
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
  return SLORA_OK;
}

int attn_decode(const slora_kv* kv, const slora_attn* at, void* ws, int64_t ws_bytes, void* stream) {
  const char* what = "attn_decode";
  clear_error();
  if (!kv || !at) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  int rc = check_heads(what, kv, at);
  if (rc) return rc;
  if (kv->n_requests == 0) return SLORA_OK;
  AttnArgs a;
  if ((rc = attn_args(what, kv, at, ws, ws_bytes, decode_workspace(kv, at), &a))) return rc;
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = timed_call(SLORA_K_ATTN_DECODE, s,
                                  [&](const LaunchEvents& ev) { return launch_attn_decode(a, kv->dtype, s, ev); });
  return e == hipSuccess ? SLORA_OK : hip_fail(e, "attn_decode launch");
}

int attn_prefill(const slora_kv* kv, const slora_attn* at, const int32_t* q_offsets, int32_t n_tokens, void* ws,
                 int64_t ws_bytes, void* stream) {
  const char* what = "attn_prefill";
  clear_error();
  if (!kv || !at) return fail(SLORA_E_INVALID, "%s: NULL argument", what);
  if (n_tokens < 0) return fail(SLORA_E_INVALID, "%s: n_tokens %d < 0", what, n_tokens);
  int rc = check_heads(what, kv, at);
  if (rc) return rc;
  if (kv->n_requests == 0 || n_tokens == 0) return SLORA_OK;
  if (!q_offsets) return fail(SLORA_E_INVALID, "%s: q_offsets is NULL", what);
  AttnArgs a;
  if ((rc = attn_args(what, kv, at, ws, ws_bytes, prefill_workspace(kv, at, n_tokens), &a))) return rc;
  a.q_offsets = q_offsets;
  a.n_tok = n_tokens;
  a.chunks = prefill_chunks(n_tokens, a.group, a.hk, a.max_len);
  a.part_waves = prefill_waves(n_tokens, a.group);
  const hipStream_t s = (hipStream_t)stream;
  const hipError_t e = timed_call(SLORA_K_ATTN_PREFILL, s,
                                  [&](const LaunchEvents& ev) { return launch_attn_prefill(a, kv->dtype, s, ev); });
  return e == hipSuccess ? SLORA_OK : hip_fail(e, "attn_prefill launch");
}

}  // namespace

extern "C" {

int slora_kv_tables(const slora_kv* kv, const slora_kv_step* step, void* stream) {
  return slora::guarded(__func__, [&] { return kv_tables(kv, step, stream); });
}

int slora_rope_turns(const slora_rope* rope, double* turns) {
  return slora::guarded(__func__, [&] { return rope_turns(rope, turns); });
}

int slora_kv_write(const slora_kv* kv, const slora_qkv* qkv, void* stream) {
  return slora::guarded(__func__, [&] { return kv_write(kv, qkv, stream); });
}

int slora_attn_workspace_size(const slora_kv* kv, const slora_attn* attn, int32_t n_tokens, int64_t* bytes) {
  return slora::guarded(__func__, [&] { return workspace_size(kv, attn, n_tokens, bytes); });
}

int slora_attn_decode(const slora_kv* kv, const slora_attn* attn, void* ws, int64_t ws_bytes, void* stream) {
  return slora::guarded(__func__, [&] { return attn_decode(kv, attn, ws, ws_bytes, stream); });
}

int slora_attn_prefill(const slora_kv* kv, const slora_attn* attn, const int32_t* q_offsets, int32_t n_tokens, void* ws,
                       int64_t ws_bytes, void* stream) {
  return slora::guarded(__func__, [&] { return attn_prefill(kv, attn, q_offsets, n_tokens, ws, ws_bytes, stream); });
}

}  // extern "C"
