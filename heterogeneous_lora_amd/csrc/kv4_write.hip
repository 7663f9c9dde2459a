// Per-head norm of q and k, rotary positions, and K and V to their cache slots in 4 bits, in one
// pass over the new tokens' projections (slora_kv4_write).
//
//   step = RN(max |x| / 6) over 32 dimensions,   code = the level nearest to x / step
//
// Heads are held as in kv_write_dev.h; q is what slora_kv_write makes of it. A group's largest
// magnitude is that of its pieces, which travel between the lanes of a head through LDS.
//
// A code is a decision: two ways of rounding K that differ in the last of 32 bits would now and
// then pick another level, a sixth of the group's range away. So K's norm and rotation are in 64
// bits. What comes after needs only to know on which side of few-bit numbers a value lies (levels'
// borders times the step, ties of the step times 6), which its 24 leading bits say if the last one
// is set where something is cut off: step and level are those of the exactly computed value, unless
// 2^-50 of it decides. (V has no arithmetic before its step, and is exact.)
//
// Bound by the vector unit, which K keeps busy longest (73% of its cycles when it took 108 us). 16411
// tokens of 32 query and 8 + 8 KV heads of 128 with norms: 96 us (108 with a token's position and
// slots asked for by each head; 131 with steps and quotients in 64 bits too; one more wave a SIMD
// spills, 118; 4 or 8 tokens to a workgroup instead of 2, or K's heads dealt evenly to its waves,
// change nothing). slora_kv_write, which stores four times as much of K and V, takes 91.
#include "kv_write_dev.h"

namespace slora {
namespace {

struct Write4 {
  WriteArgs a;
  Kv4Layout lay;
};

// x cut off to 24 bits, the last of them set if anything was lost (a multiple of 2^-149; what is
// finite past the largest float becomes that).
__device__ __forceinline__ float cut(double x) {
  const float f = (float)x;
  if (fabs(x) < (double)INFINITY && !(fabsf(f) < INFINITY)) return copysignf(0x1.fffffep127f, f);
  const double lost = fabs(x) - fabs((double)f);
  const int bits = __float_as_int(f);
  return __int_as_float(lost == 0.0 || !(fabsf(f) < INFINITY) ? bits : (lost < 0.0 ? bits - 1 : bits) | 1);
}

// Upper bits of the f16 value nearest to `most` / 6 among those with 3 bits behind the leading
// one: a group's step byte. 226 is the largest whose 6-fold is finite in f16.
constexpr int kMaxStep = 226, kNanStep = 255;
__device__ __forceinline__ int step_byte(float most) {
  if (!(most < INFINITY)) return kNanStep;
  const float x = most / 6.0f;
  // multiples of 2^(e - 3), e = the exponent, -14 at least
  const int e = max((__float_as_int(x) >> 23) - 127, -14);
  if (e > 14) return kMaxStep;
  const int n = (int)rintf(ldexpf(x, 3 - e));  // 0 .. 16
  return min((e + 14) * 8 + n, kMaxStep);      // n = 16 carries into the exponent
}

// Codes of a piece, 4 bits each. The quotient is the nearest float to x / step: corrected, as the
// product with a rounded reciprocal may pass a border.
template <int V>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[V], int byte) {
  const float step = byte < kNanStep ? (float)__builtin_bit_cast(_Float16, (uint16_t)(byte << 7)) : 0.f;
  const float inv = step == 0.f ? 0.f : 1.0f / step;
  float t[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    t[e] = x[e] * inv;
    t[e] = fmaf(fmaf(-t[e], step, x[e]), inv, t[e]);
    t[e] = copysignf(fminf(fabsf(t[e]), 6.f), x[e]);  // (also of zeros)
  }
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[0], t[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[2], t[3], 1.0f, 1);
  if constexpr (V == 8) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[4], t[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[6], t[7], 1.0f, 3);
  }
  return byte == kNanStep ? 0 : w;
}

// V, G, INTER as for slora_kv_write.
template <int DT, int V, int G, bool INTER>
__global__ __launch_bounds__(kThreads) void kv4_write_kernel(Write4 b) {
  const WriteArgs& a = b.a;
  const Kv4Layout& lay = b.lay;
  __shared__ double2 angle[kAngles];
  __shared__ uint32_t sm_most[kThreads * 2];  // largest magnitudes of the pieces, by group of lanes
  __shared__ uint8_t* places[kMaxTok][2];     // of a token's K and V, NULL: none
  __shared__ int32_t position[kMaxTok];
  const int tid = (int)threadIdx.x;
  const int tok0 = (int)blockIdx.x * a.tpw, n_tok = min(a.tpw, a.n_tok - tok0);
  const int pairs = a.pairs;
  for (int i = tid; i < n_tok * pairs; i += kThreads) {
    const int t = i / pairs, c = i - t * pairs;
    double f = (double)a.pos[tok0 + t] * a.turns[c];
    f -= rint(f);
    double sn, cs;
    sincospi(2.0 * f, &sn, &cs);
    angle[i] = make_double2(cs * a.cs, sn * a.cs);
  }
  // (looked up once a token: in the loop below a head would wait for it first)
  for (int i = tid; i < 2 * n_tok; i += kThreads) {
    const int64_t tok = tok0 + (i >> 1), slot = a.hk ? (i & 1 ? a.vs : a.ks)[tok] : -1;
    const int64_t page = (slot >> 32) ? slot / a.tpp : (int64_t)((uint32_t)slot / (uint32_t)a.tpp);
    places[i >> 1][i & 1] =
        slot < 0 || page >= a.n_pages ? nullptr : (uint8_t*)(a.pool + page * a.P) + (slot - page * a.tpp) * lay.token_bytes;
    position[i >> 1] = a.pos[tok];
  }
  __syncthreads();

  const Place at = place_of<V, INTER>(a, tid % G);
  uint32_t* const most = sm_most + tid / G * 2 * G;

  // What the cache holds of the lane's pieces x and y, to head hh of a token. (Magnitudes are
  // compared as whole numbers, in which an infinity is above all others and NaN above that.)
  auto put = [&](uint8_t* token, int hh, const float (&x)[V], const float (&y)[V]) {
    uint32_t mx = 0, my = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      mx = max(mx, __float_as_uint(x[e]) & 0x7fffffffu);
      my = max(my, __float_as_uint(y[e]) & 0x7fffffffu);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    most[at.c0] = mx;
    most[at.c1] = my;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int kIn = 32 / V;  // pieces of a group of 32
    auto store = [&](int c, const float (&z)[V]) {
      const int group = c / kIn;
      if (group >= lay.groups) {  // a head's steps are filled up with zeros
        if (c % kIn == 0 && group < lay.step_bytes) token[lay.steps_at + hh * lay.step_bytes + group] = 0;
        return;
      }
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kIn; ++i) m = max(m, most[group * kIn + i]);
      const int byte = step_byte(__uint_as_float(m));
      const uint32_t w = codes_of<V>(z, byte);
      const int p = c * V / 8, word = (p & 3) * lay.groups + (p >> 2);  // its 8 dimensions' place
      uint8_t* to = token + hh * 16 * lay.groups + word * 4;
      if constexpr (V == 8) *reinterpret_cast<uint32_t*>(to) = w;
      else *reinterpret_cast<uint16_t*>(to + (c & 1) * 2) = (uint16_t)w;
      if (c % kIn == 0) token[lay.steps_at + hh * lay.step_bytes + group] = (uint8_t)byte;
    };
    store(at.c0, x);
    store(at.c1, y);
  };

  const int heads = a.hq + 2 * a.hk;
  const int h_begin = (int)blockIdx.y * a.heads_y, h_end = min(h_begin + a.heads_y, heads);
  const int n_heads = h_end - h_begin;
  for (int i = tid / G; i < n_tok * n_heads; i += kThreads / G) {
    const int t = i / n_heads, h = h_begin + i - t * n_heads;
    const int64_t tok = tok0 + t;
    if (position[t] < 0) continue;
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hk;
    const int hh = is_q ? h : is_v ? h - a.hq - a.hk : h - a.hq;
    const uint16_t* src = is_q ? a.q.p + tok * a.q.ts + hh * a.q.hs
                          : is_v ? a.v.p + tok * a.v.ts + hh * a.v.hs
                                 : a.k.p + tok * a.k.ts + hh * a.k.hs;
    uint8_t* const token = places[t][is_v];
    if (!is_q && !token) continue;
    Piece<V> r0{}, r1{};
    if (at.has0) r0 = load<V>(src + at.c0 * V);
    if (at.has1) r1 = load<V>(src + at.c1 * V);
    float x[V], y[V];
    unpack<DT, V>(r0, x);
    unpack<DT, V>(r1, y);
    const double2* ang = angle + t * pairs;
    if (is_q) {
      norm_and_turn<DT, V, G, INTER>(a, ang, a.qw, at, x, y);
      uint16_t* dst = a.qo + tok * a.ots + hh * a.ohs;
      if (at.has0) store<V>(dst + at.c0 * V, pack<DT, V>(x));
      if (at.has1) store<V>(dst + at.c1 * V, pack<DT, V>(y));
    } else if (is_v) {
      put(token, hh, x, y);
    } else {
      double kx[V], ky[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        kx[e] = x[e];
        ky[e] = y[e];
      }
      norm_and_turn<DT, V, G, INTER>(a, ang, a.kw, at, kx, ky);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[e] = cut(kx[e]);
        y[e] = cut(ky[e]);
      }
      put(token, hh, x, y);
    }
  }
}

template <int DT, int V, int G>
void launch_one(bool inter, const Write4& a, dim3 grid, hipStream_t s, const LaunchEvents& ev) {
  if (inter)
    hipExtLaunchKernelGGL((kv4_write_kernel<DT, V, G, true>), grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
  else
    hipExtLaunchKernelGGL((kv4_write_kernel<DT, V, G, false>), grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
}

template <int DT>
void launch_dt(const Plan& p, const Write4& a, hipStream_t s, const LaunchEvents& ev) {
  if (p.v == 8) {
    if (p.g <= 4) launch_one<DT, 8, 4>(p.inter, a, p.grid, s, ev);
    else if (p.g <= 8) launch_one<DT, 8, 8>(p.inter, a, p.grid, s, ev);
    else launch_one<DT, 8, 16>(p.inter, a, p.grid, s, ev);
  } else {
    if (p.g <= 8) launch_one<DT, 4, 8>(p.inter, a, p.grid, s, ev);
    else if (p.g <= 16) launch_one<DT, 4, 16>(p.inter, a, p.grid, s, ev);
    else launch_one<DT, 4, 32>(p.inter, a, p.grid, s, ev);
  }
}

}  // namespace

hipError_t launch_kv4_write(const slora_kv& kv, const slora_qkv& w, hipStream_t s, const LaunchEvents& ev) {
  const Plan p = plan_write(kv, w);
  if ((int64_t)p.grid.x * kThreads >= kMaxThreads) return hipErrorInvalidConfiguration;
  const Write4 a = {p.a, kv4_layout(kv.n_kv_heads, kv.head_dim)};
  if (kv.dtype == SLORA_F16) launch_dt<SLORA_F16>(p, a, s, ev);
  else launch_dt<SLORA_BF16>(p, a, s, ev);
  return hipGetLastError();
}

}  // namespace slora
