// Workspace sizes at the largest numbers that the calls accept, of a cache of 16 and of 4 bits, under
// AddressSanitizer and UndefinedBehaviorSanitizer, built by tests/test_host_sanitize_kv4_limits.py.
// No GPU is touched and no memory of these sizes is asked for.
#include <cstdio>
#include <cstring>

#include "kv4_calls.h"

static int64_t g_fail = 0, g_calls = 0;
#define CHECK(c)                                                                            \
  do {                                                                                      \
    if (!(c) && ++g_fail <= 20) std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
  } while (0)

namespace slora {
int fail(int code, const char*, ...) { return code; }
int hip_fail(hipError_t, const char*) { return SLORA_E_HIP; }
void clear_error() {}
hipError_t timed_call(int, hipStream_t, hipError_t (*)(const void*, const LaunchEvents&), const void*) { return hipSuccess; }
hipError_t launch_attn4_decode(const AttnArgs&, int32_t, hipStream_t, const LaunchEvents&) { return hipSuccess; }
hipError_t launch_attn4_prefill(const AttnArgs&, int32_t, hipStream_t, const LaunchEvents&) { return hipSuccess; }
hipError_t launch_kv4_write(const slora_kv&, const slora_qkv&, hipStream_t, const LaunchEvents&) { return hipSuccess; }
hipError_t launch_kv4_read(const slora_kv&, const slora_kv_rows&, hipStream_t, const LaunchEvents&) { return hipSuccess; }
}  // namespace slora

using namespace slora;

int main() {
  const int32_t requests[] = {1, 3, SLORA_KV_MAX_REQUESTS / 2, SLORA_KV_MAX_REQUESTS}, heads[] = {1, 5, 512, 1024},
                dims[] = {8, 136, 256}, blocks[] = {1, 1 << 24, (1 << 30) - 1, 1 << 30}, tokens[] = {0, 1, 1 << 24, INT32_MAX};
  for (int32_t r : requests)
    for (int32_t hk : heads)
      for (int32_t d : dims)
        for (int32_t b : blocks)
          for (int32_t n : tokens)
            for (int32_t hq : {hk, 16384 / hk * hk}) {
              slora_kv kv;
              memset(&kv, 0, sizeof kv);
              kv.pool = (void*)0x1000;
              kv.n_pages = INT32_MAX;
              kv.page_elems = hk * d;
              kv.dtype = SLORA_BF16;
              kv.n_kv_heads = hk;
              kv.head_dim = d;
              kv.tokens_per_page = 1;
              kv.n_requests = r;
              kv.max_blocks = b;
              slora_attn at;
              memset(&at, 0, sizeof at);
              at.n_q_heads = hq;
              int64_t wide = 0, bytes = 0;
              CHECK(workspace_size("16 bits", 16, &kv, &at, n, &wide) == SLORA_OK && wide > 0);
              kv.page_elems = kv4_layout(hk, d).token_bytes / 2;
              CHECK(slora_attn4_workspace_size(&kv, &at, n, &bytes) == SLORA_OK);
              // (tables of 8 bytes a block beside the blocks of 64 tokens)
              CHECK(bytes >= wide && (n == 0 || bytes <= wide + kBackBytes + kBackBytes / 256 + 512));
              // (and K and V read back in no more than 4 times the bytes of q and out)
              CHECK(n == 0 || bytes - wide <= 4 * (4 * (int64_t)n * hq * d) + kBackBytes / 256 + 512);
              ++g_calls;
            }
  const int32_t keys[] = {0, 1, 100, 1 << 25, 1 << 30}, news[] = {0, 1, 99, 100, 1 << 25, INT32_MAX - 1, INT32_MAX},
                windows[] = {0, 1, 70, (1 << 25) - 1, (1 << 30) - 1};
  for (int32_t n : keys)
    for (int32_t m : news)
      for (int32_t w : windows) {
        const int32_t lo = first_key_seen(n, m, w);
        CHECK(lo >= 0 && lo <= n);
        // the first new row is at n - m; a window holds its own position and w - 1 before it
        const int64_t position = (int64_t)n - m;
        CHECK(w == 0 ? lo == 0 : position - w + 1 <= 0 ? lo == 0 : lo == position - w + 1);
      }
  std::printf("%lld sizes; %lld failed checks\n", (long long)g_calls, (long long)g_fail);
  return g_fail ? 1 : 0;
}
