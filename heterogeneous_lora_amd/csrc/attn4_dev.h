// A cache in 4 bits (slora.h) as the attention kernels read it: values in f16, step times level,
// which f16 holds exactly.
#pragma once

#include "attn_dev.h"

namespace slora {
namespace dev {

constexpr int kMaxStep = 226;  // the largest step byte of numbers

// Where the codes of keys whose page is outside the pool are read (their steps are NaN): as
// long as 16 of the largest heads' codes.
__device__ uint4 kNoCodes[128];

// (A factor that has overflowed would make NaN of a score of 0.)
__device__ __forceinline__ float finite(float x) { return fminf(fmaxf(x, -3.402823466e38f), 3.402823466e38f); }

// Loads from an address. (Said to be of global memory: the compiler cannot tell, and a load that
// may be of LDS is waited for with everything else that is on its way.)
#define SLORA_GLOBAL __attribute__((address_space(1)))
typedef uint32_t words2 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t words4 __attribute__((ext_vector_type(4), aligned(4)));
// Words, 4-byte aligned.
template <int N>
__device__ __forceinline__ void load_words(uint64_t from, uint32_t (&w)[N]) {
  const SLORA_GLOBAL uint32_t* p = (const SLORA_GLOBAL uint32_t*)from;
#pragma unroll
  for (int i = 0; i + 4 <= N; i += 4) {
    const words4 x = *(const SLORA_GLOBAL words4*)(p + i);
    w[i] = x[0]; w[i + 1] = x[1]; w[i + 2] = x[2]; w[i + 3] = x[3];
  }
  if constexpr (N % 4 >= 2) {
    const words2 x = *(const SLORA_GLOBAL words2*)(p + N / 4 * 4);
    w[N / 4 * 4] = x[0]; w[N / 4 * 4 + 1] = x[1];
  }
  if constexpr (N % 2) w[N - 1] = p[N - 1];
}
// A head's steps, a byte each.
template <int G, int N>
__device__ __forceinline__ void load_steps(uint64_t from, uint32_t (&w)[N]) {
  if constexpr (G == 1) w[0] = *(const SLORA_GLOBAL uint8_t*)from;
  else if constexpr (G == 2) w[0] = *(const SLORA_GLOBAL uint16_t*)from;
  else load_words<N>(from, w);
}
// The codes of 8 (or 4, in the low half) dimensions.
template <int D>
__device__ __forceinline__ uint32_t load_codes(uint64_t from) {
  if constexpr (D == 8) return *(const SLORA_GLOBAL uint32_t*)from;
  else return *(const SLORA_GLOBAL uint16_t*)from;
}

// A key's codes and steps (of KV head `head`); good: its page is in the pool.
struct Key4 {
  uint64_t codes, steps;
  bool good;
};
__device__ __forceinline__ Key4 key4_addr(const AttnArgs& a, int32_t page, int32_t j, int head) {
  const uint32_t in = a.tpp == 1 ? 0u : (uint32_t)j - div_tpp(a, (uint32_t)j) * (uint32_t)a.tpp;
  const uint64_t at = (uint64_t)(a.pool + (int64_t)page * a.P) + in * (uint32_t)a.kv4.token_bytes;
  return {at + (uint32_t)(head * 16 * a.kv4.groups), at + (uint32_t)(a.kv4.steps_at + head * a.kv4.step_bytes),
          (uint32_t)page < a.n_pages_u};
}

// Byte i of w as a step in f16, twice (its bits are the byte's, moved up by 7).
__device__ __forceinline__ half2_t step_twice(uint32_t w, int i) {
  return __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(w, w, 0x0c000c00u + (uint32_t)i * 0x10001u) << 7);
}
// The 2 values whose codes are in byte i of `codes` (i is a constant where this is used).
__device__ __forceinline__ uint32_t values2(uint32_t codes, int i, half2_t step) {
  half2_t x;
  switch (i) {
    case 0: x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0); break;
    case 1: x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1); break;
    case 2: x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2); break;
    default: x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3);
  }
  return __builtin_bit_cast(uint32_t, x * step);
}
__device__ __forceinline__ uint4 values8(uint32_t codes, half2_t step) {
  return make_uint4(values2(codes, 0, step), values2(codes, 1, step), values2(codes, 2, step), values2(codes, 3, step));
}

// q in bf16 goes to f16 by a power of two that brings its row's largest element to 2^14 .. 2^15:
// exactly, down to 2^-32 of that element. (An infinity stays one; what is finite beside it goes.)
__device__ __forceinline__ float largest_bf16(const uint4& x) {
  float m = 0.f;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = fmaxf(m, fmaxf(fabsf(lo_f32<SLORA_BF16>(w[i])), fabsf(hi_f32<SLORA_BF16>(w[i]))));
  return m;
}
__device__ __forceinline__ int f16_shift(float largest) {
  const int e = (int)(__float_as_uint(largest) >> 23);
  return 14 + 127 - min(max(e, 1), 254);
}
__device__ __forceinline__ uint4 bf16_to_f16(const uint4& x, int up) {
  auto two = [&](uint32_t w) {
    return round2<SLORA_F16>(ldexpf(lo_f32<SLORA_BF16>(w), up), ldexpf(hi_f32<SLORA_BF16>(w), up));
  };
  return make_uint4(two(x.x), two(x.y), two(x.z), two(x.w));
}

}  // namespace dev
}  // namespace slora
