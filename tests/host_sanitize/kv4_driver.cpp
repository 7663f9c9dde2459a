// The host code of the cache in 4 bits (kv4_calls.h) under AddressSanitizer and
// UndefinedBehaviorSanitizer, built by tests/test_host_sanitize_kv4.py. The launches are stand-ins
// that look at the arguments the kernels would get: for random shapes and lengths they cut the keys
// as the kernels do and check that every partial result, every request's cut and every block that
// keys are read back to lies in its own place inside the workspace whose size the library asked for.
// No GPU is touched.
#include <stdarg.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <random>
#include <vector>

#include "kv4_calls.h"

static int64_t g_fail = 0, g_few = 0, g_spans = 0, g_cut = 0, g_back = 0, g_straight = 0, g_refused = 0, g_allocations = 0;
void* operator new(size_t n) {
  ++g_allocations;
  if (void* p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }
#define CHECK(c)                                                                            \
  do {                                                                                      \
    if (!(c) && ++g_fail <= 20) std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
  } while (0)

static void* const kFakeDev = reinterpret_cast<void*>(0x7F0000000000ull);
static std::mt19937_64 g_rng(1);
static int64_t g_ws_bytes = 0;              // of the call being made
static std::vector<int32_t> g_seq, g_new;   // its requests
static int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(g_rng() % (uint64_t)(hi - lo + 1)); }
static int64_t pick_log(int64_t lo, int64_t hi) {
  return std::min(hi, std::max(lo, (int64_t)std::exp(std::uniform_real_distribution<>(std::log((double)lo), std::log((double)hi + 1))(g_rng))));
}

namespace slora {

int fail(int code, const char* fmt, ...) {
  char text[512];
  va_list va;
  va_start(va, fmt);
  vsnprintf(text, sizeof text, fmt, va);
  va_end(va);
  ++g_refused;
  return code;
}
int hip_fail(hipError_t, const char*) { return SLORA_E_HIP; }
void clear_error() {}
hipError_t timed_call(int, hipStream_t, hipError_t (*launch)(const void*, const LaunchEvents&), const void* arg) {
  return launch(arg, LaunchEvents());
}

static int64_t offset(const void* p) { return (const uint8_t*)p - (const uint8_t*)kFakeDev; }
static int32_t seen(const AttnArgs& a, int32_t n) { return a.window ? std::min(n, a.window) : n; }

static void few_keys(const AttnArgs& a) {
  ++g_few;
  CHECK(offset(a.part) == kAttnCounterBytes);
  const int units = decode_units(a.n_req, a.hk, a.group), round = 32 * (4 / a.wg_heads);
  float total = 0.f;
  for (int32_t n : g_seq) total += (float)seen(a, n);
  const float per_chunk = 1.0f / std::fmax(total / (float)a.chunks + (float)round, 1.f);
  int64_t first = 0;
  for (int r = 0; r < a.n_req; ++r) {
    const int64_t c = std::max((int)((float)seen(a, g_seq[(size_t)r]) * per_chunk + 0.5f), 1);
    if (c > 1) {
      ++g_cut;
      CHECK((first - r) * units + units - 1 < kAttnCounters);
      CHECK((first + c) * a.hk * a.group * (a.D + 2) * 4 + kAttnCounterBytes <= g_ws_bytes);
    }
    first += c;
  }
}

hipError_t launch_attn4_decode(const AttnArgs& a, int32_t, hipStream_t, const LaunchEvents&) {
  if (!a.spans) {
    few_keys(a);
    return hipSuccess;
  }
  ++g_spans;
  const int row_groups = (a.group + 15) / 16, nc = (a.D + 31) / 32;
  CHECK(a.wave_heads >= 1 && a.wave_heads * std::min(a.group, 16) <= 16 && (a.wave_heads == 1 || row_groups == 1));
  CHECK(a.wg_units == 1 || a.wg_units == 2 || a.wg_units == 4);
  CHECK(a.wave_runs == 1 || a.wave_runs == 2 || (a.wave_runs == 4 && nc <= 4));
  // steps of a wave's heads, from the 16 bytes that the first one's are in, fit a key's place in LDS
  const int step_bytes = a.kv4.step_bytes;
  for (int kv0 = 0; kv0 < a.hk; kv0 += a.wave_heads) {
    const int skip = kv0 * step_bytes % 16, heads = std::min(a.wave_heads, a.hk - kv0);
    CHECK((skip + heads * step_bytes + 15) / 16 * 16 <= 64 / a.wave_runs);
    CHECK(((int64_t)kv0 * step_bytes - skip) + (skip + heads * step_bytes + 15) / 16 * 16 + a.kv4.steps_at <= a.kv4.token_bytes);
  }
  CHECK(a.spans % 8 == 0 && offset(a.cut) == kAttnCounterBytes);
  CHECK(offset(a.part) >= kAttnCounterBytes + 8 * (int64_t)a.n_req && offset(a.part) % 8 == 0);
  const int64_t round = 128 / a.wg_units * a.wave_runs, row = (int64_t)a.hk * a.group * (a.D + 2) * 4;
  auto rounds = [&](int r) { return std::max<int64_t>((seen(a, g_seq[(size_t)r]) + round - 1) / round, 1); };
  int64_t total = 0;
  for (int r = 0; r < a.n_req; ++r) total += rounds(r);
  const int64_t length = (total + a.spans - 1) / a.spans;
  CHECK(length * a.spans >= total);
  int64_t at = 0, last_place = -1;
  for (int r = 0; r < a.n_req; at += rounds(r), ++r) {
    const int64_t first = at / length, off = at % length, here = std::min(length - off, rounds(r));
    const int64_t n = here == rounds(r) ? 1 : (rounds(r) - here + length - 1) / length + 1;
    CHECK(first + n <= a.spans);
    if (n == 1) continue;
    ++g_cut;
    for (int64_t c = 0; c < n; ++c) {
      const int64_t place = 2 * (first + c) + (c == 0);
      CHECK(place > last_place);  // no two parts in one place
      last_place = place;
      CHECK(offset(a.part) + (place + 1) * row <= g_ws_bytes);
    }
  }
  return hipSuccess;
}

hipError_t launch_attn4_prefill(const AttnArgs& a, int32_t, hipStream_t, const LaunchEvents&) {
  int64_t extra = 0, parts = kAttnCounterBytes;
  float work = 0.f;
  auto tiles_of = [&](int r) { return ((int64_t)g_new[(size_t)r] * a.group + 127) / 128; };
  for (int r = 0; r < a.n_req; ++r) work += (float)tiles_of(r) * (float)seen(a, g_seq[(size_t)r]);
  const float length = std::fmax(work / (float)std::max(a.chunks, 1), 512.f);
  for (int r = 0; r < a.n_req; ++r) {
    const int64_t c = a.chunks ? (int64_t)std::fmax((float)seen(a, g_seq[(size_t)r]) / length + 0.5f, 1.f) : 1;
    for (int64_t t = 0; t < tiles_of(r); ++t, extra += c - 1)
      if (c > 1) {
        ++g_cut;
        CHECK(extra * a.hk + a.hk - 1 < kAttnCounters);
        const int64_t part = ((2 * extra + c - 1) * a.hk + a.hk - 1) * a.part_waves + a.part_waves;
        parts = std::max(parts, part * part_floats(attn_instance(a.D)) * 4 + kAttnCounterBytes);
      }
  }
  CHECK(extra <= a.chunks && parts <= g_ws_bytes);
  if (!a.back) {
    ++g_straight;
    return hipSuccess;
  }
  ++g_back;
  const Prefill4 p = prefill4_plan(a.n_req, a.n_tok, a.group, a.hk, a.D, a.max_len);
  CHECK(p.back && offset(a.back) >= parts && offset(a.back) % 256 == 0 && p.table_bytes % 256 == 0);
  CHECK((int64_t)p.blocks * kBackTokens >= a.max_len && 2 * (int64_t)a.n_req * p.blocks * 4 <= p.table_bytes);
  CHECK((int64_t)p.blocks * kBackTokens <= (int64_t)1 << 30 && p.blocks <= INT32_MAX / (2 * a.n_req));
  const int64_t block = (int64_t)kBackTokens * a.row * 2;
  CHECK(offset(a.back) + p.table_bytes + 2 * (int64_t)a.n_req * p.blocks * block <= g_ws_bytes);
  return hipSuccess;
}
hipError_t launch_kv4_write(const slora_kv&, const slora_qkv&, hipStream_t, const LaunchEvents&) { return hipSuccess; }
hipError_t launch_kv4_read(const slora_kv&, const slora_kv_rows&, hipStream_t, const LaunchEvents&) { return hipSuccess; }

}  // namespace slora

using namespace slora;

static slora_kv make_kv(int32_t hk, int32_t D, int32_t tpp, int32_t n_req, int32_t max_blocks) {
  slora_kv kv;
  memset(&kv, 0, sizeof kv);
  kv.pool = kFakeDev;
  kv.n_pages = pick_log(1, INT32_MAX);
  int64_t bytes = 0;
  if (slora_kv4_token_bytes(hk, D, &bytes) == SLORA_OK) kv.page_elems = (int32_t)(bytes / 2 * tpp);
  CHECK(bytes % 16 == 0 && bytes > 0);
  kv.dtype = g_rng() & 1 ? SLORA_F16 : SLORA_BF16;
  kv.n_kv_heads = hk;
  kv.head_dim = D;
  kv.tokens_per_page = tpp;
  kv.n_requests = n_req;
  kv.max_blocks = max_blocks;
  return kv;
}

static slora_attn make_attn(int32_t hq, int32_t D) {
  slora_attn at;
  memset(&at, 0, sizeof at);
  at.n_q_heads = hq;
  at.scale = 0.1f;
  at.k_table = at.v_table = at.seq_len = (const int32_t*)kFakeDev;
  at.q = at.out = kFakeDev;
  at.q_head_stride = at.out_head_stride = D;
  at.q_token_stride = at.out_token_stride = (int64_t)hq * D;
  return at;
}

static void attention_round() {
  const int32_t hk = (int32_t)pick_log(1, g_rng() % 4 ? 80 : 1024), D = 8 * (int32_t)pick(1, 32);
  const int32_t group = (int32_t)pick_log(1, std::min(g_rng() % 4 ? 40 : 16384, 16384 / hk));
  const int32_t n_req = (int32_t)pick_log(1, g_rng() % 8 ? 300 : SLORA_KV_MAX_REQUESTS);
  const int32_t max_len = (int32_t)pick_log(1, g_rng() % 4 ? 1 << 17 : 1 << 30);
  const int64_t n_tok = pick_log(1, g_rng() % 2 ? 4096 : 200000);
  slora_kv kv = make_kv(hk, D, 1, n_req, max_len);
  slora_attn at = make_attn(hk * group, D);
  const int32_t windows[] = {0, 0, 1, 700, max_len, INT32_MAX};
  at.window = windows[g_rng() % 6];
  g_seq.resize((size_t)n_req);
  for (auto& n : g_seq) n = g_rng() % 4 ? (int32_t)pick_log(1, max_len) : (int32_t)pick(0, max_len);
  if (g_rng() % 3 == 0) std::fill(g_seq.begin(), g_seq.end(), max_len);
  if (g_rng() % 5 == 0) std::fill(g_seq.begin(), g_seq.end(), 0);
  int64_t bytes = 0;
  CHECK(slora_attn4_workspace_size(&kv, &at, 0, &bytes) == SLORA_OK);
  g_ws_bytes = bytes;
  CHECK(slora_attn4_decode(&kv, &at, kFakeDev, bytes, nullptr) == SLORA_OK);
  CHECK(slora_attn4_decode(&kv, &at, kFakeDev, bytes - 1, nullptr) == SLORA_E_INVALID);
  g_new.assign((size_t)n_req, 0);
  int64_t left = n_tok;
  for (int r = 0; r < n_req && left; ++r) {
    const int64_t n = r == n_req - 1 ? left : pick(0, std::min<int64_t>(left, 2 * n_tok / n_req + 1));
    g_new[(size_t)r] = (int32_t)n;
    left -= n;
  }
  CHECK(slora_attn4_workspace_size(&kv, &at, (int32_t)n_tok, &bytes) == SLORA_OK);
  g_ws_bytes = bytes;
  CHECK(slora_attn4_prefill(&kv, &at, (const int32_t*)kFakeDev, (int32_t)n_tok, kFakeDev, bytes, nullptr) == SLORA_OK);
  CHECK(slora_attn4_prefill(&kv, &at, (const int32_t*)kFakeDev, (int32_t)n_tok, kFakeDev, bytes - 1, nullptr) == SLORA_E_INVALID);
}

// Fields at the edges of what is accepted: a refusal or a call, never a fault.
static void any_round() {
  const int32_t some[] = {INT32_MIN, -1, 0, 1, 7, 8, 64, 256, 264, 1024, 16384, 1 << 30, INT32_MAX};
  auto any = [&] { return some[g_rng() % 13]; };
  slora_kv kv = make_kv(2, 64, 2, 3, 8);
  slora_attn at = make_attn(4, 64);
  slora_qkv w;
  memset(&w, 0, sizeof w);
  w.n_tokens = w.n_q_heads = 4;
  w.q = w.k = w.v = w.q_out = kFakeDev;
  w.q_token_stride = w.out_token_stride = 256;
  w.k_token_stride = w.v_token_stride = 128;
  w.q_head_stride = w.k_head_stride = w.v_head_stride = w.out_head_stride = 64;
  w.position = (const int32_t*)kFakeDev;
  w.k_slots = w.v_slots = (const int64_t*)kFakeDev;
  slora_kv_rows rows;
  memset(&rows, 0, sizeof rows);
  rows.n_tokens = 4;
  rows.k = rows.v = kFakeDev;
  rows.k_slots = rows.v_slots = (const int64_t*)kFakeDev;
  for (int i = (int)pick(0, 3); i > 0; --i) switch (g_rng() % 14) {
    case 0: kv.n_pages = any(); break;
    case 1: kv.page_elems = any(); break;
    case 2: kv.dtype = any(); break;
    case 3: kv.n_kv_heads = any(); break;
    case 4: kv.head_dim = any(); break;
    case 5: kv.tokens_per_page = any(); break;
    case 6: kv.n_requests = any(); break;
    case 7: kv.max_blocks = any(); break;
    case 8: at.n_q_heads = w.n_q_heads = any(); break;
    case 9: at.window = any(); break;
    case 10: rows.k_token_stride = w.k_head_stride = any(); break;
    case 11: w.n_tokens = rows.n_tokens = any(); break;
    case 12: w.rotary_dim = any(); break;
    default: at.k_table = nullptr; w.k = nullptr; rows.v_slots = nullptr;
  }
  g_seq.assign((size_t)std::max(kv.n_requests, 0) % 20000, 1);
  g_new.assign(g_seq.size(), 0);
  const int32_t n_tok = any();
  int64_t bytes = 0;
  auto ok = [](int rc) { CHECK(rc == SLORA_OK || rc == SLORA_E_INVALID); return rc == SLORA_OK; };
  if (ok(slora_attn4_workspace_size(&kv, &at, 0, &bytes))) {
    CHECK(bytes >= kAttnCounterBytes);
    g_ws_bytes = bytes;
    for (auto& n : g_seq) n = std::min(n, kv.max_blocks * kv.tokens_per_page);
    ok(slora_attn4_decode(&kv, &at, kFakeDev, bytes, nullptr));
  }
  if (ok(slora_attn4_workspace_size(&kv, &at, n_tok, &bytes))) {
    g_ws_bytes = bytes;
    ok(slora_attn4_prefill(&kv, &at, (const int32_t*)kFakeDev, n_tok, kFakeDev, bytes, nullptr));
  }
  ok(slora_kv4_write(&kv, &w, nullptr));
  ok(slora_kv4_read(&kv, &rows, nullptr));
  ok(slora_kv4_token_bytes(any(), any(), &bytes));
  const int64_t before = g_allocations;  // the calls allocate nothing
  ok(slora_kv4_read(&kv, &rows, nullptr));
  CHECK(g_allocations == before);
}

int main(int argc, char** argv) {
  const int rounds = argc > 1 ? std::atoi(argv[1]) : 20;
  for (int i = 0; i < 20 * rounds; ++i) attention_round();
  for (int i = 0; i < 200 * rounds; ++i) any_round();
  std::printf("%lld few, %lld spans, %lld straight, %lld back, %lld cut, %lld refusals; %lld failed checks\n", (long long)g_few,
              (long long)g_spans, (long long)g_straight, (long long)g_back, (long long)g_cut, (long long)g_refused,
              (long long)g_fail);
  return g_fail ? 1 : 0;
}
