// Attention of one new token per request over its paged keys (slora_attn_decode).
//
//   s_j = q . k_j (scaled, capped, biased),  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Bound by the bytes of K and V, each read once. A wave owns one KV head of one request's
// run of keys, with the query heads that share it as up to 16 rows, and takes tiles of 32
// keys. Where there are enough requests to fill the device with one chunk each, the 4 waves
// of a workgroup take up to 4 neighbouring heads, whose vectors lie together in the pages
// (5.88 TB/s against 5.45 for 512 requests of 40 heads). Otherwise they share one head's
// keys, each with its own maximum m, sum and output, joined in LDS at the end, and long
// requests are cut into chunks (a wave to a head would leave four times the partial
// results). Their partial results are joined by the workgroup that
// finishes last (a counter in the workspace), in the chunks' order, so the result does not
// depend on which one that is.
//
// 512 requests of 64 to 2048 keys, 40 heads of 128: 1.89 ms (5.9 TB/s); three of 100000 to
// 131072 keys, 64 query heads on 8: 270 us (5.3 TB/s); 64 with a window of 1024: 44 us.
//
// A tile never goes through LDS. v_mfma_f32_16x16x32 with A = K (16 keys x 32 dimensions)
// and B = q leaves lane l with scores of keys 4 (l / 16) + i of query row l % 16. The two
// 16-key products of a tile take their keys in such an order (row r of product t is key 8
// (r / 4) + 4 t + r % 4) that the 8 scores of a lane are those of keys 8 (l / 16) .. + 7:
// just what the next product, A = V^T (16 dimensions x 32 keys) and B = weights, wants as
// its B operand. For A a lane loads 8 dimensions of those 8 keys and turns the 8 x 8 block
// in registers (v_perm); product e of the tile then makes dimensions 8 m + e. Each row's
// keys, page ids and addresses are looked up once per tile, 64 lanes wide, and handed out
// through LDS. Loads run one tile ahead of the products, page ids two.
#include "attn_decode_dev.h"

namespace slora {
namespace {

template <int DT, int NC>
hipError_t launch_nc(const AttnArgs& a, dim3 grid, hipStream_t s, const LaunchEvents& ev) {
  const int rows = a.group < kRows ? a.group : kRows;
  const size_t lds = sizeof(float) * kWaves * rows * (a.D + 4);
  if (lds > 48 * 1024) {  // with the static part past the 64 KiB a launch has by default
    const hipError_t e = hipFuncSetAttribute((const void*)attn_decode_kernel<DT, NC, 16>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipExtLaunchKernelGGL((attn_decode_kernel<DT, NC, 16>), grid, dim3(kWaves * 64), lds, s, ev.start, ev.stop, 0, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  const int units = a.hk / a.wg_heads * ((a.group + kRows - 1) / kRows);
  // No request has more chunks than rounds of keys.
  const int64_t round = kTile * (kWaves / a.wg_heads);
  const int64_t most = (a.max_len + round - 1) / round, all = (int64_t)a.n_req * (most > 1 ? most : 1);
  const int64_t chunks = all < (int64_t)a.n_req + a.chunks ? all : (int64_t)a.n_req + a.chunks;
  if (chunks * units * kWaves * 64 >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)units, (unsigned)chunks);  // neighbouring heads in neighbouring workgroups
  const int nc = (a.D + 31) / 32;
  return nc <= 2   ? launch_nc<DT, 2>(a, grid, s, ev)
         : nc == 3 ? launch_nc<DT, 3>(a, grid, s, ev)
         : nc == 4 ? launch_nc<DT, 4>(a, grid, s, ev)
         : nc <= 6 ? launch_nc<DT, 6>(a, grid, s, ev)
                   : launch_nc<DT, 8>(a, grid, s, ev);
}

}  // namespace

hipError_t launch_attn_decode(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
