// The KV cache and attention entry points' host code (kv.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer, built by tests/test_host_sanitize_kv.py. The launches are
// stand-ins that look at the arguments the kernels would get: for random shapes and lengths
// they cut the keys as the kernels do and check that every counter and every partial result
// lies inside the workspace whose size the library asked for. No GPU is touched.
#include <stdarg.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <random>
#include <vector>

#include "internal.h"

static int64_t g_fail = 0, g_calls = 0, g_cut = 0, g_most_counters = 0, g_refused = 0;
static int64_t g_allocations = 0;
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
static int64_t g_ws_bytes = 0;                       // of the call being made
static std::vector<int32_t> g_seq, g_new;            // its requests
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

// Keys that a request's last row sees.
static int32_t seen(const AttnArgs& a, int32_t n) { return a.window ? std::min(n, a.window) : n; }

hipError_t launch_attn_decode(const AttnArgs& a, int32_t, hipStream_t, const LaunchEvents&) {
  ++g_calls;
  const int units = decode_units(a.n_req, a.hk, a.group);
  CHECK(a.wg_heads == decode_wg_heads(a.n_req, a.hk, a.group) && a.hk % a.wg_heads == 0);
  CHECK(units == a.hk / a.wg_heads * ((a.group + 15) / 16));
  const int round = 32 * (4 / a.wg_heads);
  float total = 0.f;
  for (int32_t n : g_seq) total += (float)seen(a, n);
  const float per_chunk = 1.0f / std::fmax(total / (float)a.chunks + (float)round, 1.f);
  int64_t first = 0;
  const int64_t row = a.D + 2;
  for (int r = 0; r < a.n_req; ++r) {
    const int32_t n = seen(a, g_seq[(size_t)r]);
    const int64_t c = std::max((int)((float)n * per_chunk + 0.5f), 1);
    CHECK(c <= std::max<int64_t>((n + round - 1) / round, 1));  // the grid's other bound
    if (c > 1) {
      ++g_cut;
      const int64_t counter = (first - r) * units + units - 1;
      g_most_counters = std::max(g_most_counters, counter + 1);
      CHECK(first - r >= 0 && counter < kAttnCounters);
      const int64_t end = ((first + c) * a.hk * a.group) * row * 4 + kAttnCounterBytes;
      CHECK(end <= g_ws_bytes);
    }
    first += c;
  }
  CHECK(first <= (int64_t)a.n_req + a.chunks);
  return hipSuccess;
}

hipError_t launch_attn_prefill(const AttnArgs& a, int32_t, hipStream_t, const LaunchEvents&) {
  ++g_calls;
  int64_t tiles_all = 0, extra = 0;
  float work = 0.f;
  auto tiles_of = [&](int r) { return ((int64_t)g_new[(size_t)r] * a.group + 127) / 128; };
  for (int r = 0; r < a.n_req; ++r) work += (float)tiles_of(r) * (float)seen(a, g_seq[(size_t)r]);
  const float length = std::fmax(work / (float)std::max(a.chunks, 1), 512.f);
  for (int r = 0; r < a.n_req; ++r) {
    const int64_t c = a.chunks ? (int64_t)std::fmax((float)seen(a, g_seq[(size_t)r]) / length + 0.5f, 1.f) : 1;
    for (int64_t t = 0; t < tiles_of(r); ++t) {
      if (c > 1) {
        ++g_cut;
        const int64_t counter = extra * a.hk + a.hk - 1;
        g_most_counters = std::max(g_most_counters, counter + 1);
        CHECK(counter < kAttnCounters);
        const int64_t part = ((2 * extra + c - 1) * a.hk + a.hk - 1) * a.part_waves + a.part_waves;
        CHECK(part * part_floats(attn_instance(a.D)) * 4 + kAttnCounterBytes <= g_ws_bytes);
      }
      extra += c - 1;
      ++tiles_all;
    }
  }
  CHECK(extra <= a.chunks);
  // workgroups: as many as the launch makes
  CHECK(tiles_all + extra <= ((int64_t)a.n_tok * a.group + 127) / 128 + a.n_req + a.chunks);
  return hipSuccess;
}

hipError_t launch_kv_tables(const slora_kv&, const slora_kv_step&, hipStream_t, const LaunchEvents&) { ++g_calls; return hipSuccess; }
hipError_t launch_kv_write(const slora_kv&, const slora_qkv&, hipStream_t, const LaunchEvents&) { ++g_calls; return hipSuccess; }

}  // namespace slora

using namespace slora;

static slora_kv make_kv(int32_t hk, int32_t D, int32_t tpp, int32_t n_req, int32_t max_blocks) {
  slora_kv kv;
  memset(&kv, 0, sizeof kv);
  kv.pool = kFakeDev;
  kv.n_pages = pick_log(1, INT32_MAX);
  kv.page_elems = tpp * hk * D;
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

static void attention(int32_t hk, int32_t group, int32_t D, int32_t n_req, int32_t max_len, int64_t n_tok) {
  slora_kv kv = make_kv(hk, D, 1, n_req, max_len);
  slora_attn at = make_attn(hk * group, D);
  const float caps[] = {0.f, 1e-45f, 30.f, 3.4e38f};
  const int32_t windows[] = {0, 1, max_len, INT32_MAX};
  at.softcap = caps[g_rng() % 4];
  at.window = windows[g_rng() % 4];
  g_seq.resize((size_t)n_req);
  for (auto& n : g_seq) n = g_rng() % 4 ? (int32_t)pick_log(1, std::max(max_len, 1)) : (int32_t)pick(0, max_len);
  for (auto& n : g_seq) n = std::min(n, max_len);
  if (g_rng() % 3 == 0) std::fill(g_seq.begin(), g_seq.end(), max_len);
  int64_t bytes = 0;
  CHECK(slora_attn_workspace_size(&kv, &at, 0, &bytes) == SLORA_OK);
  g_ws_bytes = bytes;
  CHECK(slora_attn_decode(&kv, &at, kFakeDev, bytes, nullptr) == SLORA_OK);
  if (n_req) CHECK(slora_attn_decode(&kv, &at, kFakeDev, bytes - 1, nullptr) == SLORA_E_INVALID);
  // a prompt call: n_tok rows spread over the requests
  g_new.assign((size_t)n_req, 0);
  int64_t left = n_tok;
  for (int r = 0; r < n_req && left; ++r) {
    const int64_t n = r == n_req - 1 ? left : pick(0, std::min<int64_t>(left, 2 * n_tok / n_req + 1));
    g_new[(size_t)r] = (int32_t)n;
    left -= n;
  }
  if (!n_tok || !n_req) return;
  CHECK(slora_attn_workspace_size(&kv, &at, (int32_t)n_tok, &bytes) == SLORA_OK);
  g_ws_bytes = bytes;
  CHECK(slora_attn_prefill(&kv, &at, (const int32_t*)kFakeDev, (int32_t)n_tok, kFakeDev, bytes, nullptr) == SLORA_OK);
  CHECK(slora_attn_prefill(&kv, &at, (const int32_t*)kFakeDev, (int32_t)n_tok, kFakeDev, bytes - 1, nullptr) == SLORA_E_INVALID);
}

static void attention_round() {
  const int32_t hk = (int32_t)pick_log(1, 1024);
  const int32_t group = (int32_t)pick_log(1, 16384 / hk);
  const int32_t D = 8 * (int32_t)pick(1, 32);
  attention(hk, group, D, (int32_t)pick_log(1, g_rng() % 8 ? 300 : SLORA_KV_MAX_REQUESTS),
            (int32_t)pick_log(1, 1 << 20), pick_log(1, 4096));
}

// Counters of every number of heads, whatever the requests (the kernels' largest index).
static void counters_of_all_heads() {
  for (int32_t hk = 1; hk <= 1024; ++hk)
    for (int32_t group = 1; group * hk <= 16384; group += group < 40 ? 1 : 13)
      for (int32_t n_req : {1, 2, 63, 1000, 16384}) {
        const int32_t units = decode_units(n_req, hk, group);
        CHECK((int64_t)decode_chunks(units) * units <= kAttnCounters);
        for (int64_t n_tok : {1, 5, 300}) CHECK((int64_t)prefill_chunks(n_tok, group, hk, 1 << 30) * hk <= kAttnCounters);
      }
}

static void divisors() {
  for (int64_t d = 1; d < INT32_MAX; d = d < 5000 ? d + 1 : d + d / 7 + 1) {
    uint32_t magic, shift;
    divisor((int32_t)d, &magic, &shift);
    for (int i = 0; i < 40; ++i) {
      const int64_t k = pick(0, INT32_MAX / d);
      for (int64_t n : {k * d, k * d - 1, k * d + d - 1, pick(0, INT32_MAX), (int64_t)INT32_MAX})
        if (d > 1 && n >= 0 && n <= INT32_MAX) CHECK((int64_t)(((uint64_t)n * magic >> 32) >> shift) == n / d);
    }
  }
}

static void rope_round() {
  slora_rope r;
  r.rotary_dim = 8 * (int32_t)pick(-1, 34);
  r.scaling = (int32_t)pick(-1, 4);
  const double values[] = {0, -1, 1, 4, 1e4, 1e-300, 1e300, INFINITY, NAN};
  auto value = [&] { return values[g_rng() % 9]; };
  r.theta = value();
  r.factor = value();
  r.original_len = value();
  r.low_turns = value();
  r.high_turns = value();
  std::vector<double> turns((size_t)std::max(r.rotary_dim / 2, 0));
  const int rc = slora_rope_turns(&r, turns.empty() ? nullptr : turns.data());
  CHECK(rc == SLORA_OK || rc == SLORA_E_INVALID);
  if (rc == SLORA_OK) ++g_calls;
}

// Fields at the edges of what is accepted: a refusal or a call, never a fault.
static void any_round() {
  const int32_t some[] = {INT32_MIN, -1, 0, 1, 7, 8, 64, 256, 264, 1024, 16384, 1 << 30, INT32_MAX};
  auto any = [&] { return some[g_rng() % 13]; };
  slora_kv kv = make_kv(2, 64, 2, 3, 8);
  slora_attn at = make_attn(4, 64);
  slora_kv_step st;
  memset(&st, 0, sizeof st);
  st.n_planes = 2;
  st.pages = st.past_len = st.new_len = (const int32_t*)kFakeDev;
  st.n_page_ids = 5;
  st.n_tokens = 4;
  st.tables = st.seq_len = st.q_offsets = st.token_request = st.position = (int32_t*)kFakeDev;
  st.slots = (int64_t*)kFakeDev;
  slora_qkv w;
  memset(&w, 0, sizeof w);
  w.n_tokens = 4;
  w.n_q_heads = 4;
  w.q = w.k = w.v = w.q_out = kFakeDev;
  w.q_token_stride = w.out_token_stride = 256;
  w.k_token_stride = w.v_token_stride = 128;
  w.q_head_stride = w.k_head_stride = w.v_head_stride = w.out_head_stride = 64;
  w.position = (const int32_t*)kFakeDev;
  w.k_slots = w.v_slots = (const int64_t*)kFakeDev;
  w.turns = (const double*)kFakeDev;
  w.rotary_dim = 64;
  for (int i = (int)pick(0, 3); i > 0; --i) switch (g_rng() % 18) {
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
    case 10: at.softcap = (float)any() * 1e30f; break;
    case 11: at.q_token_stride = w.k_head_stride = any(); break;
    case 12: at.scale = INFINITY; break;
    case 13: st.n_planes = any(); break;
    case 14: st.n_tokens = w.n_tokens = any(); break;
    case 15: st.n_page_ids = any(); break;
    case 16: w.rotary_dim = any(); break;
    default: at.k_table = nullptr; w.k = nullptr; st.tables = nullptr;
  }
  g_seq.assign((size_t)std::max(kv.n_requests, 0) % 20000, 1);
  g_new.assign(g_seq.size(), 0);
  const int32_t n_tok = any();
  int64_t bytes = 0;
  auto ok = [](int rc) { CHECK(rc == SLORA_OK || rc == SLORA_E_INVALID); return rc == SLORA_OK; };
  if (ok(slora_attn_workspace_size(&kv, &at, 0, &bytes))) {
    CHECK(bytes >= kAttnCounterBytes);
    g_ws_bytes = bytes;
    for (auto& n : g_seq) n = std::min(n, kv.max_blocks * kv.tokens_per_page);
    ok(slora_attn_decode(&kv, &at, kFakeDev, bytes, nullptr));
  }
  if (ok(slora_attn_workspace_size(&kv, &at, n_tok, &bytes))) {
    g_ws_bytes = bytes;
    ok(slora_attn_prefill(&kv, &at, (const int32_t*)kFakeDev, n_tok, kFakeDev, bytes, nullptr));
  }
  ok(slora_kv_tables(&kv, &st, nullptr));
  ok(slora_kv_write(&kv, &w, nullptr));
}

// The calls allocate nothing on the way to their launches.
static void no_allocations() {
  slora_kv kv = make_kv(2, 64, 2, 3, 8);
  slora_attn at = make_attn(4, 64);
  slora_kv_step st;
  memset(&st, 0, sizeof st);
  st.n_planes = 2;
  st.past_len = st.new_len = (const int32_t*)kFakeDev;
  st.tables = st.seq_len = st.q_offsets = (int32_t*)kFakeDev;
  slora_qkv w;
  memset(&w, 0, sizeof w);
  w.n_tokens = w.n_q_heads = 4;
  w.q = w.q_out = kFakeDev;
  w.position = (const int32_t*)kFakeDev;
  g_seq.assign(3, 8);
  g_new.assign(3, 1);
  const int64_t calls = g_calls, before = g_allocations;
  g_ws_bytes = 1 << 20;
  CHECK(slora_kv_tables(&kv, &st, nullptr) == SLORA_OK);
  CHECK(slora_kv_write(&kv, &w, nullptr) == SLORA_OK);
  CHECK(slora_attn_decode(&kv, &at, kFakeDev, g_ws_bytes, nullptr) == SLORA_OK);
  CHECK(slora_attn_prefill(&kv, &at, (const int32_t*)kFakeDev, 3, kFakeDev, g_ws_bytes, nullptr) == SLORA_OK);
  CHECK(g_calls == calls + 4 && g_allocations == before);
}

int main(int argc, char** argv) {
  const int rounds = argc > 1 ? std::atoi(argv[1]) : 20;
  no_allocations();
  divisors();
  counters_of_all_heads();
  for (int32_t hk : {1, 2, 3, 5, 8, 512, 513, 1021, 1024})  // few rows over long caches
    for (int32_t group : {1, 16, 17})
      if (hk * group <= 16384)
        for (int32_t n_req : {1, 3, 40})
          attention(hk, group, 64, n_req, 1 << 20, 2 * n_req);
  for (int i = 0; i < rounds; ++i) {
    for (int j = 0; j < 10; ++j) attention_round();
    for (int j = 0; j < 20; ++j) rope_round();
    for (int j = 0; j < 50; ++j) any_round();
  }
  std::printf("%lld calls, %lld refusals, %lld cut rows, %lld counters of %lld at most; %lld failed checks\n",
              (long long)g_calls, (long long)g_refused, (long long)g_cut, (long long)g_most_counters,
              (long long)kAttnCounters, (long long)g_fail);
  return g_fail != 0;
}
