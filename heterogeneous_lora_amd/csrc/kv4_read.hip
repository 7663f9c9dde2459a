// K and V of tokens out of a cache in 4 bits (slora_kv4_read): value = step * level, which both
// storage types hold exactly.
//
// Bound by the bytes written: 16 for each 4 of codes read. A thread takes 4 pieces of 8 dimensions,
// each wave's pieces neighbours, so that its stores are whole lines. K and V of 65000 tokens of 8
// heads of 128: 70 us (4.8 TB/s, as a copy; 94 us where each piece waited for its own slot).
#include "device_common.h"
#include "kv4_calls.h"

namespace slora {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;  // of 8 dimensions, a thread's

struct ReadArgs {
  const uint8_t* pool;
  int64_t n_pages, page_bytes;
  int32_t tpp, n_tok, hk, per_head, per_token;  // units of 8 dimensions
  uint32_t head_magic, head_shift, token_magic, token_shift, tpp_magic, tpp_shift;
  Kv4Layout lay;
  uint16_t* out[2];  // K, V
  int64_t ts[2], hs[2];
  const int64_t* slots[2];
};

__device__ __forceinline__ uint32_t divided(uint32_t n, int32_t d, uint32_t magic, uint32_t shift) {
  return d == 1 ? n : __umulhi(n, magic) >> shift;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(ReadArgs a) {
  const int which = (int)blockIdx.y;
  if (!a.out[which]) return;
  const int64_t first = (int64_t)blockIdx.x * (kUnits * kThreads), tok0 = first / a.per_token;
  const uint32_t in0 = (uint32_t)(first - tok0 * a.per_token) + threadIdx.x;
  // (the units' slots together, then their codes: no wait for memory stands between two of them)
  uint32_t t[kUnits], in[kUnits];
  int64_t slot[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    t[k] = divided(in0 + k * kThreads, a.per_token, a.token_magic, a.token_shift);
    in[k] = in0 + k * kThreads - t[k] * a.per_token;
    slot[k] = a.slots[which][min(tok0 + t[k], (int64_t)a.n_tok - 1)];
  }
  uint32_t w[kUnits], byte[kUnits], head[kUnits], piece[kUnits];
  bool is[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    head[k] = divided(in[k], a.per_head, a.head_magic, a.head_shift);
    piece[k] = in[k] - head[k] * a.per_head;
    const int64_t at = slot[k],
                  page = (at >> 31) ? at / a.tpp : (int64_t)divided((uint32_t)at, a.tpp, a.tpp_magic, a.tpp_shift);
    is[k] = tok0 + t[k] < a.n_tok && at >= 0 && page < a.n_pages;
    const uint8_t* token = a.pool + page * a.page_bytes + (at - page * a.tpp) * a.lay.token_bytes;
    const uint32_t group = piece[k] >> 2, word = head[k] * 4 * a.lay.groups + (piece[k] & 3) * a.lay.groups + group;
    const uint8_t* const zero = reinterpret_cast<const uint8_t*>(dev::fill_zero());
    const uint8_t* const codes = is[k] ? token + word * 4 : zero;
    const uint8_t* const step = is[k] ? token + a.lay.steps_at + head[k] * a.lay.step_bytes + group : zero;
    w[k] = *(const __attribute__((address_space(1))) uint32_t*)codes;
    byte[k] = *(const __attribute__((address_space(1))) uint8_t*)step;
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (!is[k]) continue;
    const float step = (float)__builtin_bit_cast(_Float16, (uint16_t)(byte[k] << 7));
    uint32_t o[4];
    auto two = [&](auto x, int i) { o[i] = dev::pack2<DT>((float)x[0] * step, (float)x[1] * step); };
    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 0), 0);
    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 1), 1);
    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 2), 2);
    two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[k], 1.0f, 3), 3);
    dev::st16(a.out[which] + (tok0 + t[k]) * a.ts[which] + (int64_t)head[k] * a.hs[which] + piece[k] * 8,
              make_uint4(o[0], o[1], o[2], o[3]));
  }
}

}  // namespace

hipError_t launch_kv4_read(const slora_kv& kv, const slora_kv_rows& r, hipStream_t s, const LaunchEvents& ev) {
  ReadArgs a;
  a.pool = (const uint8_t*)kv.pool;
  a.n_pages = kv.n_pages;
  a.page_bytes = 2 * (int64_t)kv.page_elems;
  a.tpp = kv.tokens_per_page;
  a.n_tok = r.n_tokens;
  a.hk = kv.n_kv_heads;
  a.per_head = kv.head_dim / 8;
  a.per_token = a.hk * a.per_head;
  divisor(a.per_head, &a.head_magic, &a.head_shift);
  divisor(a.per_token, &a.token_magic, &a.token_shift);
  divisor(a.tpp, &a.tpp_magic, &a.tpp_shift);
  a.lay = kv4_layout(kv.n_kv_heads, kv.head_dim);
  a.out[0] = (uint16_t*)r.k;
  a.out[1] = (uint16_t*)r.v;
  a.ts[0] = r.k_token_stride;
  a.ts[1] = r.v_token_stride;
  a.hs[0] = r.k_head_stride;
  a.hs[1] = r.v_head_stride;
  a.slots[0] = r.k_slots;
  a.slots[1] = r.v_slots;
  const int64_t each = (int64_t)kThreads * kUnits, blocks = ((int64_t)a.n_tok * a.per_token + each - 1) / each;
  if (blocks * kThreads >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, 2);
  if (kv.dtype == SLORA_F16)
    hipExtLaunchKernelGGL((kv4_read_kernel<SLORA_F16>), grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
  else
    hipExtLaunchKernelGGL((kv4_read_kernel<SLORA_BF16>), grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
  return hipGetLastError();
}

}  // namespace slora
