// Attention of the new tokens of each request over a cache in 4 bits (slora_attn4_prefill).
//
//   s_ij = q_i . k_j (scaled, capped, biased, masked),  out_i = sum_j softmax(s_i)_j v_j
//
// Bound by matrix work once prompts are long. attn_prefill.hip's kernel, with products in f16 (step
// times level is exact there) and another way from the cache to LDS: a thread takes a quarter of a
// key's codes, of K and of V, holds them from one tile to the next and makes values of them between
// the products, 2 instructions for 2 values and 16 bytes of LDS a store. That is done by every row
// tile again and costs as many vector instructions as the weights do: long prompts 3785 us against
// 3200 with a cache of 16 bits. Where a key is seen by many row tiles (Prefill4) it is read back to
// 16 bits once, into the workspace, and the 16-bit kernel runs over that.
//
// Two prompts of 8000 tokens after 7000-8192 cached, 32 query heads on 8 KV heads of 128, bf16: 3.05
// to 3.13 ms (1000 TFLOP/s; f16 3.18), 41 us of it the reading back; 64 prompts of 8 to 512 tokens, 32 heads of
// 128, straight from the codes: 238 us (with every tile's page ids and codes waited for before the
// next one's are asked for, at a prompt's beginning: 248).
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

// K and V of the keys that some row sees, in 16 bits, as a cache of blocks of kBackTokens tokens: a
// workgroup a quarter of a block of K or V, a wave a token, a thread 8 dimensions at a time. (A token
// waits for its page id, then for its codes, and a wave's tokens for each other: one prompt of 1024
// tokens takes 42 us in all, 54 with a whole block to a workgroup; long prompts 3128 and 3142.)
constexpr int kBackSplit = 4, kBackPart = kBackTokens / kBackSplit;
template <int DT>
__global__ __launch_bounds__(kThreads) void attn4_back_kernel(AttnArgs a, Prefill4 p) {
  const int r = (int)blockIdx.y, v = (int)blockIdx.z, b = (int)blockIdx.x / kBackSplit, part = (int)blockIdx.x % kBackSplit;
  const int32_t id = (v * a.n_req + r) * p.blocks + b;
  if (threadIdx.x == 0) a.back[id] = id;
  const int32_t n = a.seq[r];
  if (n < 0 || n > a.max_len) return;
  const int32_t q0 = min(max(a.q_offsets[r], 0), a.n_tok), n_new = max(min(max(a.q_offsets[r + 1], 0), a.n_tok) - q0, 0);
  const int32_t lo = first_key_seen(n, n_new, a.window);
  const int32_t prefix = a.prefix ? a.prefix[r] : 0;
  const int32_t j0 = b * kBackTokens, j1 = min(j0 + kBackTokens, n);
  if (n_new == 0 || (j1 <= lo && j0 >= prefix)) return;
  const int per_head = a.D / 8, per_token = a.hk * per_head;
  uint16_t* const to = (uint16_t*)((uint8_t*)a.back + p.table_bytes) + (int64_t)id * (kBackTokens * a.row);
  const int32_t* const table = (v ? a.vt : a.kt) + (int64_t)r * a.max_blocks;
  const int end = min(j0 + (part + 1) * kBackPart, j1);
  for (int j = j0 + part * kBackPart + (int)threadIdx.x / 64; j < end; j += kThreads / 64) {
    const int32_t page = table[div_tpp(a, (uint32_t)j)];
    for (int u = (int)threadIdx.x % 64; u < per_token; u += 64) {
      const int head = u / per_head, x = u - head * per_head;
      const Key4 k = key4_addr(a, page, j, head);
      const uint32_t w = load_codes<8>(k.good ? k.codes + ((x & 3) * a.kv4.groups + (x >> 2)) * 4 : fill_addr<DT>(true));
      const uint32_t st = k.good ? *(const SLORA_GLOBAL uint8_t*)(k.steps + (x >> 2)) : 255u;
      const float step = (float)__builtin_bit_cast(_Float16, (uint16_t)(st << 7));
      uint32_t o[4];
      auto two = [&](auto y, int i) { o[i] = pack2<DT>((float)y[0] * step, (float)y[1] * step); };
      two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), 0);
      two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1), 1);
      two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), 2);
      two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3), 3);
      st16(to + (int64_t)(j - j0) * a.row + u * 8, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

hipError_t launch_back(AttnArgs a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  const Prefill4 p = prefill4_plan(a.n_req, a.n_tok, a.group, a.hk, a.D, a.max_len);
  const dim3 grid((unsigned)p.blocks * kBackSplit, (unsigned)a.n_req, 2);
  if (dtype == SLORA_F16)
    hipExtLaunchKernelGGL(attn4_back_kernel<SLORA_F16>, grid, dim3(kThreads), 0, s, ev.start, nullptr, 0, a, p);
  else
    hipExtLaunchKernelGGL(attn4_back_kernel<SLORA_BF16>, grid, dim3(kThreads), 0, s, ev.start, nullptr, 0, a, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.pool = (const uint16_t*)((const uint8_t*)a.back + p.table_bytes);
  a.n_pages_u = (uint32_t)(2 * a.n_req * p.blocks);
  a.P = kBackTokens * a.row;
  a.tpp = kBackTokens;
  divisor(a.tpp, &a.tpp_magic, &a.tpp_shift);
  a.max_blocks = p.blocks;
  a.kt = a.back;
  a.vt = a.back + a.n_req * p.blocks;
  LaunchEvents rest;
  rest.stop = ev.stop;
  return launch_attn_prefill(a, dtype, s, rest);
}

}  // namespace

hipError_t launch_attn4_prefill(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  if (a.back) return launch_back(a, dtype, s, ev);
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
