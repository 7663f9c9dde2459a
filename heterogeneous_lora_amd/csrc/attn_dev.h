// Device code shared by the attention kernels: which keys a row sees, where a key's
// vector lies in the pool, the score, matrix instructions, lane exchanges.
#pragma once

#include "device_common.h"

namespace slora {
namespace dev {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A vector of zeros and one of quiet NaN (as long as the largest head), where loads of
// keys past the end, and through a page id outside the pool, are pointed: every load
// issues unconditionally, and no place of the pool that holds no key of the row is read.
struct alignas(16) AttnFill {
  uint16_t zero[256];
  uint16_t nan_f16[256];
  uint16_t nan_bf16[256];
};
constexpr AttnFill make_attn_fill() {
  AttnFill f{};
  for (int i = 0; i < 256; ++i) {
    f.zero[i] = 0;
    f.nan_f16[i] = 0x7E00;
    f.nan_bf16[i] = 0x7FC0;
  }
  return f;
}
__device__ AttnFill kAttnFill = make_attn_fill();

template <int DT>
__device__ __forceinline__ uint64_t fill_addr(bool zero) {
  return (uint64_t)(zero ? kAttnFill.zero : DT == SLORA_F16 ? kAttnFill.nan_f16 : kAttnFill.nan_bf16);
}

// n / tpp for n < 2^31 (magic and shift from the host).
__device__ __forceinline__ uint32_t div_tpp(const AttnArgs& a, uint32_t n) {
  return a.tpp == 1 ? n : __umulhi(n, a.tpp_magic) >> a.tpp_shift;
}

// n / group for n < 2^31.
__device__ __forceinline__ uint32_t div_group(const AttnArgs& a, uint32_t n) {
  return a.group == 1 ? n : __umulhi(n, a.group_magic) >> a.group_shift;
}

// The keys the rows of one workgroup see, as one run of indices [0, count): below `pre`
// the key of that number, from there on that number + gap (a window leaves a hole behind
// the prefix).
struct Keys {
  int32_t count, pre, gap;
  __device__ __forceinline__ int32_t key(int32_t i) const { return i < pre ? i : i + gap; }
};

// For rows at positions p_min .. p_max of a request with n cached keys (p_max < n) and a
// prefix of 0 .. n. The hole behind the prefix begins at a multiple of `unit` (above 1: the
// run then has keys that no row sees).
__device__ __forceinline__ Keys keys_of(const AttnArgs& a, int32_t prefix, int32_t n, int32_t p_min, int32_t p_max,
                                        int32_t unit) {
  const int32_t lo = a.window ? max(p_min - a.window + 1, 0) : 0;
  const int32_t end = max(p_max + 1, prefix);
  Keys k;
  k.pre = min((prefix + unit - 1) / unit * unit, lo);
  k.gap = lo - k.pre;
  if (lo >= end) {  // nothing past the prefix
    k.gap = 0;
    k.count = prefix;
  } else {
    k.count = end - k.gap;
  }
  return k;
}

// Address of the first element of key j's vector (head h), given its page id; `nans` where
// the page is outside the pool.
__device__ __forceinline__ uint64_t key_addr(const AttnArgs& a, int32_t page, int32_t j, int32_t h_off,
                                             uint64_t nans) {
  const uint32_t in = a.tpp == 1 ? 0u : (uint32_t)j - div_tpp(a, (uint32_t)j) * (uint32_t)a.tpp;
  const uint64_t at = (uint64_t)(a.pool + (int64_t)page * a.P + (uint32_t)(in * (uint32_t)a.row) + h_off);
  return (uint32_t)page < a.n_pages_u ? at : nans;
}

// Softcap of a product, in units of log 2 (weights are exp2 of differences), as
//   cap tanh(x / cap) = cap - 2 cap / (exp(2 x / cap) + 1),
// whose error is 2^-22 cap whatever the score: for caps up to kNearCap, where that is 2^-14
// beside 2^-11 (f16) and 2^-8 of a weight's rounding to the storage type.
constexpr float kNearCap = 256.0f;
__device__ __forceinline__ float capped_near(const AttnArgs& a, float s) {
  const float e = __builtin_amdgcn_exp2f(s * a.cap_in);
  return a.cap_out - 2.0f * a.cap_out * __builtin_amdgcn_rcpf(e + 1.0f);
}
// For any cap: where |y| = |x / cap| < 1/8 the odd series of tanh, x (1 - y^2 / 3 + 2 y^4 / 15)
// (the next term is below 2^-22), else the form above; off by 2^-19 of the score at most. (z
// is the square of 2 log2(e) y.)
__device__ __forceinline__ float capped(const AttnArgs& a, float s) {
  constexpr float k = kLn2 * kLn2 / 4;
  const float y = s * a.cap_in, z = y * y;
  const float p = __builtin_fmaf(z, __builtin_fmaf(z, 2.0f / 15 * k * k, -1.0f / 3 * k), 1.0f);
  return z < 0x1p-6f / k ? s * a.scale2 * p : capped_near(a, s);
}

template <int DT>
__device__ __forceinline__ f32x4 mfma16x16(const uint4& x, const uint4& y, f32x4 c) {
  if constexpr (DT == SLORA_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}
template <int DT>
__device__ __forceinline__ f32x16 mfma32x32(const uint4& x, const uint4& y, f32x16 c) {
  if constexpr (DT == SLORA_F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
}

// Lane l with lane l ^ 32 (and l ^ 16).
__device__ __forceinline__ float max32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sums over lanes 0 .. l of a wave, in registers (a row is 16 lanes; the last two steps
// carry a row's sum into the next, then the lower half's into the upper).
template <int CTRL, int ROWS>
__device__ __forceinline__ int lanes_shifted(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int running_sum(int x) {
  x += lanes_shifted<0x111, 0xf>(x);
  x += lanes_shifted<0x112, 0xf>(x);
  x += lanes_shifted<0x114, 0xf>(x);
  x += lanes_shifted<0x118, 0xf>(x);
  x += lanes_shifted<0x142, 0xa>(x);
  x += lanes_shifted<0x143, 0xc>(x);
  return x;
}
// The sum over all lanes, the same on every lane.
__device__ __forceinline__ float wave_sum(float x) {
  auto step = [&](int moved) { x += __int_as_float(moved); };
  step(lanes_shifted<0x111, 0xf>(__float_as_int(x)));
  step(lanes_shifted<0x112, 0xf>(__float_as_int(x)));
  step(lanes_shifted<0x114, 0xf>(__float_as_int(x)));
  step(lanes_shifted<0x118, 0xf>(__float_as_int(x)));
  step(lanes_shifted<0x142, 0xa>(__float_as_int(x)));
  step(lanes_shifted<0x143, 0xc>(__float_as_int(x)));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// Halves of dwords a and b at the same place: (a.lo, b.lo) or (a.hi, b.hi).
__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Two values rounded to nearest even, in one instruction.
template <int DT>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 x = {lo, hi};
  if constexpr (DT == SLORA_F16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, half2_t));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf162_t));
}

// Weights are exp2(score - maximum + this). The maximum may lag by 8 (kRescale), so f16's
// weights, which reach 2^15, keep all bits down to 2^-21 of the largest and some down to 2^-31
// (at 0 it would be 2^-14 and 2^-24: 131072 keys of a long cache could vanish together).
template <int DT>
constexpr float kWeightLog2 = DT == SLORA_F16 ? 7.0f : 0.0f;
// log(sum exp(s)) of a row from its maximum and its sum of weights.
template <int DT>
__device__ __forceinline__ float log_sum(float m, float l) {
  return (m - kWeightLog2<DT>) * kLn2 + logf(l);
}

// Two weights (>= 0) as a sum of two storage values each: one cut off towards zero and the
// rounded rest, which leaves 2^-15 (bf16) or 2^-21 (f16, down to 2^-24 in all) of the weight.
// Where the first is above zero so is the rest, as times an infinity in V a zero makes a NaN.
template <int DT>
__device__ __forceinline__ void split2(float x, float y, uint32_t* top, uint32_t* rest) {
  if constexpr (DT == SLORA_F16) {
    const float least = 0x1p-24f;  // of the type
    *top = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(x, y));
    *rest = round2<DT>(fmaxf(x - lo_f32<DT>(*top), fminf(x, least)), fmaxf(y - hi_f32<DT>(*top), fminf(y, least)));
  } else {
    const float below = 1.0f - 0x1p-10f;
    *top = pair_hi(__float_as_uint(x * below), __float_as_uint(y * below));
    *rest = round2<DT>(x - lo_f32<DT>(*top), y - hi_f32<DT>(*top));
  }
}

// Partial results travel between workgroups, on other XCDs as well: stored and loaded at
// the device's coherence point.
__device__ __forceinline__ void put_pair(float* p, float x, float y) {
  __hip_atomic_store((uint64_t*)p, (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

// exp2(m_part - m) as a weight of a partial result: 0 for a part that saw nothing.
__device__ __forceinline__ float part_weight(float m_part, float m) {
  return m_part == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m_part - m);
}

}  // namespace dev
}  // namespace slora
