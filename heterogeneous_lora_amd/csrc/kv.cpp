// KV cache and attention entry points. Everything that depends on device data (lengths, tables,
// slots) is checked by the kernels.
#include "kv_calls.h"

using namespace slora;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

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

}  // namespace

extern "C" {

int slora_kv_tables(const slora_kv* kv, const slora_kv_step* step, void* stream) {
  return slora::guarded(__func__, [&] { return kv_tables(kv, step, stream); });
}

int slora_rope_turns(const slora_rope* rope, double* turns) {
  return slora::guarded(__func__, [&] { return rope_turns(rope, turns); });
}

int slora_kv_write(const slora_kv* kv, const slora_qkv* qkv, void* stream) {
  return slora::guarded(__func__, [&] { return kv_write("kv_write", 16, SLORA_K_KV_WRITE, launch_kv_write, kv, qkv, stream); });
}

int slora_attn_workspace_size(const slora_kv* kv, const slora_attn* attn, int32_t n_tokens, int64_t* bytes) {
  return slora::guarded(__func__, [&] { return workspace_size("attn_workspace_size", 16, kv, attn, n_tokens, bytes); });
}

int slora_attn_decode(const slora_kv* kv, const slora_attn* attn, void* ws, int64_t ws_bytes, void* stream) {
  return slora::guarded(__func__, [&] {
    return attn_decode("attn_decode", 16, SLORA_K_ATTN_DECODE, launch_attn_decode, kv, attn, ws, ws_bytes, stream);
  });
}

int slora_attn_prefill(const slora_kv* kv, const slora_attn* attn, const int32_t* q_offsets, int32_t n_tokens, void* ws,
                       int64_t ws_bytes, void* stream) {
  return slora::guarded(__func__, [&] {
    return attn_prefill("attn_prefill", 16, SLORA_K_ATTN_PREFILL, launch_attn_prefill, kv, attn, q_offsets, n_tokens, ws,
                        ws_bytes, stream);
  });
}

}  // extern "C"
