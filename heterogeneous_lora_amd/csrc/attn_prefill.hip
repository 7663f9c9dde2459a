// Attention of the new tokens of each request over its paged keys (slora_attn_prefill):
// causal, optionally within a window, with a prefix all rows see, capped or biased scores.
//
//   s_ij = q_i . k_j (scaled, capped, biased, masked),  out_i = sum_j softmax(s_i)_j v_j
//
// Bound by matrix work once prompts are long: a workgroup takes 128 rows (tokens x the
// query heads that share a KV head, flattened) of one request and KV head, 32 to each of
// its 4 waves, and walks the keys those rows see in tiles of 64 (32 for heads above 128).
// Both products are v_mfma_f32_32x32x16 with the keys (or dimensions) as rows and the
// queries as columns, so a lane keeps one query's statistics, and its scores are, after
// rounding, the B operand of the second product without an exchange: the first product
// takes K's rows with bits 2 and 3 of the key's number swapped, which makes the 8 scores a
// lane holds for 16 keys those of 8 consecutive keys.
//
// The next tile's products run beside this tile's weights, and this tile's values beside the
// next one's scores, so that the matrix and the vector units of a wave both have work.
//
// Pages are gathered straight into LDS (global_load_lds, 16 bytes a lane), one tile ahead
// of the products, a load between two of them; the addresses of a tile's keys are made a tile
// earlier, its page ids read another earlier. A tile's rows lie as in the page, in 16-byte units whose places
// within a row are xored with bits of the row's number: K is read a row to a lane
// (ds_read_b128), V four keys x 16 dimensions to 16 lanes, turned on the way
// (ds_read_b64_tr_b16), both without bank conflicts (counted: none). Two workgroups share a
// CU, so that one has work while the other waits.
//
// Two prompts of 8000 tokens after 7000-8192 cached, 32 query heads on 8 KV heads of 128,
// bf16: 3.2 ms (970 TFLOP/s), with softcap 3.6 ms (860; it triples the transcendentals). A
// library product of 8192^3 reaches 1262 on the same card. 64 prompts of 8 to 512 tokens, 32
// heads of 128: 187 us.
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
  return nc <= 2   ? go(attn_prefill_kernel<DT, 2, MODE, 16>)
         : nc == 3 ? go(attn_prefill_kernel<DT, 3, MODE, 16>)
         : nc == 4 ? go(attn_prefill_kernel<DT, 4, MODE, 16>)
         : nc <= 6 ? go(attn_prefill_kernel<DT, 6, MODE, 16>)
                   : go(attn_prefill_kernel<DT, 8, MODE, 16>);
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

hipError_t launch_attn_prefill(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
