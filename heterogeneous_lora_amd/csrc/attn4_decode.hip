// Attention of one new token per request over a cache in 4 bits (slora_attn4_decode).
//
//   s_j = q . k_j (scaled, capped, biased),  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// attn_decode.hip's kernel with another way from the cache to the products.
#include "attn_decode_dev.h"

namespace slora {
namespace {

template <int DT, int NC>
hipError_t launch_nc(const AttnArgs& a, dim3 grid, hipStream_t s, const LaunchEvents& ev) {
  const int rows = a.group < kRows ? a.group : kRows;
  const size_t lds = sizeof(float) * kWaves * rows * (a.D + 4);
  if (lds > 48 * 1024) {  // with the static part past the 64 KiB a launch has by default
    const hipError_t e = hipFuncSetAttribute((const void*)attn_decode_kernel<DT, NC, 4>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipExtLaunchKernelGGL((attn_decode_kernel<DT, NC, 4>), grid, dim3(kWaves * 64), lds, s, ev.start, ev.stop, 0, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(AttnArgs a, hipStream_t s, const LaunchEvents& ev) {
  const int units = a.hk / a.wg_heads * ((a.group + kRows - 1) / kRows);
  // No request has more chunks than rounds of keys.
  const int64_t round = kTile * (kWaves / a.wg_heads);
  const int64_t most = (a.max_len + round - 1) / round, all = (int64_t)a.n_req * (most > 1 ? most : 1);
  const int64_t chunks = all < (int64_t)a.n_req + a.chunks ? all : (int64_t)a.n_req + a.chunks;
  a.xcd_log2 = chunks >= 32 ? 3 : 0;
  const int64_t rounds = (chunks + (1 << a.xcd_log2) - 1) >> a.xcd_log2;
  if ((rounds << a.xcd_log2) * units * kWaves * 64 >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)units << a.xcd_log2, (unsigned)rounds);
  switch (a.kv4.groups) {
    case 1: return launch_nc<DT, 1>(a, grid, s, ev);
    case 2: return launch_nc<DT, 2>(a, grid, s, ev);
    case 3: return launch_nc<DT, 3>(a, grid, s, ev);
    case 4: return launch_nc<DT, 4>(a, grid, s, ev);
    case 5: return launch_nc<DT, 5>(a, grid, s, ev);
    case 6: return launch_nc<DT, 6>(a, grid, s, ev);
    case 7: return launch_nc<DT, 7>(a, grid, s, ev);
    default: return launch_nc<DT, 8>(a, grid, s, ev);
  }
}

}  // namespace

hipError_t launch_attn4_decode(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
