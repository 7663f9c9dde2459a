// Attention of the new tokens of each request over a cache in 4 bits (slora_attn4_prefill).
//
//   s_ij = q_i . k_j (scaled, capped, biased, masked),  out_i = sum_j softmax(s_i)_j v_j
//
// attn_prefill.hip's kernel with another way from the cache to LDS.
#include "attn_prefill_dev.h"

namespace slora {
namespace {

template <int DT, int MODE>
hipError_t launch_mode(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  const int64_t tiles = ((int64_t)a.n_tok * a.group + kTileM - 1) / kTileM + a.n_req + a.chunks;
  if (tiles * a.hk * kThreads >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(tiles * a.hk));
  const int nc = (a.D + 31) / 32;
  auto go = [&](auto kernel) {
    hipExtLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
    return hipGetLastError();
  };
  return nc <= 2   ? go(attn_prefill_kernel<DT, 2, MODE, 4>)
         : nc == 3 ? go(attn_prefill_kernel<DT, 3, MODE, 4>)
         : nc == 4 ? go(attn_prefill_kernel<DT, 4, MODE, 4>)
         : nc <= 6 ? go(attn_prefill_kernel<DT, 6, MODE, 4>)
                   : go(attn_prefill_kernel<DT, 8, MODE, 4>);
}

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  const bool cap = a.cap_out != 0.f, bias = a.slopes || !(a.scale2 > 0.f);
  if (a.cap_out > kNearCap * kLog2e) return launch_mode<DT, kWideCap>(a, s, ev);
  return bias && cap ? launch_mode<DT, kBiasCap>(a, s, ev)
         : bias      ? launch_mode<DT, kBias>(a, s, ev)
         : cap       ? launch_mode<DT, kCap>(a, s, ev)
                     : launch_mode<DT, kPlain>(a, s, ev);
}

}  // namespace

hipError_t launch_attn4_prefill(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
