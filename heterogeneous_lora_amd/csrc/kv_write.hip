// Per-head norm of q and k, rotary positions, and the store of K and V to their cache
// slots, in one pass over the new tokens' projections (slora_kv_write).
//
//   x = x / sqrt(mean(x^2) + eps) * weight                    (optional)
//   (x1, x2) -> (x1 cos a - x2 sin a, x2 cos a + x1 sin a)    a = 2 pi position turns[i]
//
// Bound by bytes: each of q, k, v is read once and written once. A head's vector is held
// by a group of lanes, two 16-byte pieces each, chosen so that both halves of every
// rotated pair are in one lane: pieces i and i + rotary_dim / 16 in the half layout (the
// interleaved layout has its pairs inside a piece). So the rotation needs no exchange,
// and the norm one sum over the group. The angle is reduced to a fraction of a turn in 64
// bits; the cosines and sines of a token are computed once per workgroup, into LDS, and
// serve all of its heads there. Sums, products and the rotation are in fp32, with one
// rounding to the storage type at the end. 16411 tokens of 32 query and 8 + 8 KV heads of 128
// with norms: 91 us (4.4 TB/s; a copy of 2 GiB reaches 4.9 on the same card).
#include "device_common.h"

namespace slora {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 2;        // tokens of one workgroup at most
constexpr int kAngles = kMaxTok * 128;  // cos / sin pairs in LDS

struct Rows {
  const uint16_t* p;
  int64_t ts, hs;
};

struct WriteArgs {
  Rows q, k, v;
  uint16_t* qo;
  int64_t ots, ohs;
  uint16_t* pool;
  int64_t n_pages;
  int32_t P, tpp, row;  // row: n_kv_heads * head_dim
  int32_t n_tok, hq, hk, D;
  const int32_t* pos;
  const int64_t *ks, *vs;
  const double* turns;
  int32_t pairs;        // rotary_dim / 2
  float cs, eps;
  const uint16_t *qw, *kw;
  int32_t norm;
  int32_t tpw;          // tokens of a workgroup
  int32_t heads_y;      // heads (q, then k, then v) of a workgroup
};

template <int V>
struct Piece {
  uint32_t w[V / 2];
};
template <int V>
__device__ __forceinline__ Piece<V> load(const uint16_t* p) {
  Piece<V> r;
  if constexpr (V == 8) {
    const uint4 x = dev::ld16(p);
    r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    r.w[0] = x.x; r.w[1] = x.y;
  }
  return r;
}
template <int V>
__device__ __forceinline__ void store(uint16_t* p, const Piece<V>& r) {
  if constexpr (V == 8) dev::st16(p, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
  else *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
}
template <int DT, int V>
__device__ __forceinline__ void unpack(const Piece<V>& r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    x[2 * i] = dev::lo_f32<DT>(r.w[i]);
    x[2 * i + 1] = dev::hi_f32<DT>(r.w[i]);
  }
}
template <int DT, int V>
__device__ __forceinline__ Piece<V> pack(const float (&x)[V]) {
  Piece<V> r;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) r.w[i] = dev::pack2<DT>(x[2 * i], x[2 * i + 1]);
  return r;
}

// V: elements of a piece (8; 4 when a half of the rotated part is not whole pieces of 8).
// G: lanes of a head's group, a power of two, 2 V G >= head_dim.
template <int DT, int V, int G, bool INTER>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(WriteArgs a) {
  __shared__ float2 angle[kAngles];
  const int tid = (int)threadIdx.x;
  const int tok0 = (int)blockIdx.x * a.tpw, n_tok = min(a.tpw, a.n_tok - tok0);
  const int pairs = a.pairs;
  for (int i = tid; i < n_tok * pairs; i += kThreads) {
    const int t = i / pairs, c = i - t * pairs;
    double f = (double)a.pos[tok0 + t] * a.turns[c];
    f -= rint(f);
    float sn, cs;
    sincospif(2.0f * (float)f, &sn, &cs);
    angle[i] = make_float2(cs * a.cs, sn * a.cs);
  }
  __syncthreads();

  // the lane's two pieces of a head, in units of V dimensions: the rotated pairs first,
  // the rest of the head two by two
  const int g = tid % G;
  const int n_pieces = a.D / V, half = INTER ? 0 : pairs / V;
  int c0, c1;
  if (INTER) {
    c0 = 2 * g;
    c1 = 2 * g + 1;
  } else {
    c0 = g < half ? g : 2 * half + 2 * (g - half);
    c1 = g < half ? g + half : c0 + 1;
  }
  const bool has0 = c0 < n_pieces, has1 = c1 < n_pieces;

  const int heads = a.hq + 2 * a.hk;
  const int h_begin = (int)blockIdx.y * a.heads_y, h_end = min(h_begin + a.heads_y, heads);
  const int n_heads = h_end - h_begin;
  for (int i = tid / G; i < n_tok * n_heads; i += kThreads / G) {
    const int t = i / n_heads, h = h_begin + i - t * n_heads;
    const int64_t tok = tok0 + t;
    if (a.pos[tok] < 0) continue;
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hk;
    const int hh = is_q ? h : is_v ? h - a.hq - a.hk : h - a.hq;
    const uint16_t* src = is_q ? a.q.p + tok * a.q.ts + hh * a.q.hs
                          : is_v ? a.v.p + tok * a.v.ts + hh * a.v.hs
                                 : a.k.p + tok * a.k.ts + hh * a.k.hs;
    uint16_t* dst;
    if (is_q) {
      dst = a.qo + tok * a.ots + hh * a.ohs;
    } else {
      const int64_t slot = (is_v ? a.vs : a.ks)[tok];
      const int64_t page = (slot >> 32) ? slot / a.tpp : (int64_t)((uint32_t)slot / (uint32_t)a.tpp);
      if (slot < 0 || page >= a.n_pages) continue;
      dst = a.pool + page * a.P + (slot - page * a.tpp) * a.row + (int64_t)hh * a.D;
    }
    Piece<V> r0{}, r1{};
    if (has0) r0 = load<V>(src + c0 * V);
    if (has1) r1 = load<V>(src + c1 * V);
    if (!is_v) {
      float x[V], y[V];
      unpack<DT, V>(r0, x);
      unpack<DT, V>(r1, y);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) ss += x[e] * x[e] + y[e] * y[e];
#pragma unroll
        for (int d = 1; d < G; d <<= 1) ss += __shfl_xor(ss, d);
        const float inv = 1.0f / sqrtf(ss / (float)a.D + a.eps);
        const uint16_t* w = is_q ? a.qw : a.kw;
        float wx[V], wy[V];
#pragma unroll
        for (int e = 0; e < V; ++e) wx[e] = wy[e] = 1.f;
        if (w) {
          if (has0) unpack<DT, V>(load<V>(w + c0 * V), wx);
          if (has1) unpack<DT, V>(load<V>(w + c1 * V), wy);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[e] = x[e] * inv * wx[e];
          y[e] = y[e] * inv * wy[e];
        }
      }
      const float2* ang = angle + t * pairs;
      if (INTER) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const int i0 = (c0 * V + e) / 2, i1 = (c1 * V + e) / 2;
          if (i0 < pairs) {
            const float2 s = ang[i0];
            const float p = x[e], q = x[e + 1];
            x[e] = p * s.x - q * s.y;
            x[e + 1] = q * s.x + p * s.y;
          }
          if (i1 < pairs) {
            const float2 s = ang[i1];
            const float p = y[e], q = y[e + 1];
            y[e] = p * s.x - q * s.y;
            y[e + 1] = q * s.x + p * s.y;
          }
        }
      } else if (g < half) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 s = ang[c0 * V + e];
          const float p = x[e], q = y[e];
          x[e] = p * s.x - q * s.y;
          y[e] = q * s.x + p * s.y;
        }
      }
      r0 = pack<DT, V>(x);
      r1 = pack<DT, V>(y);
    }
    if (has0) store<V>(dst + c0 * V, r0);
    if (has1) store<V>(dst + c1 * V, r1);
  }
}

template <int DT, int V, int G>
void launch_one(bool inter, const WriteArgs& a, dim3 grid, hipStream_t s, const LaunchEvents& ev) {
  if (inter)
    hipExtLaunchKernelGGL((kv_write_kernel<DT, V, G, true>), grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
  else
    hipExtLaunchKernelGGL((kv_write_kernel<DT, V, G, false>), grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
}

template <int DT>
void launch_dt(bool inter, int v, int g, const WriteArgs& a, dim3 grid, hipStream_t s, const LaunchEvents& ev) {
  if (v == 8) {
    if (g <= 4) launch_one<DT, 8, 4>(inter, a, grid, s, ev);
    else if (g <= 8) launch_one<DT, 8, 8>(inter, a, grid, s, ev);
    else launch_one<DT, 8, 16>(inter, a, grid, s, ev);
  } else {
    if (g <= 8) launch_one<DT, 4, 8>(inter, a, grid, s, ev);
    else if (g <= 16) launch_one<DT, 4, 16>(inter, a, grid, s, ev);
    else launch_one<DT, 4, 32>(inter, a, grid, s, ev);
  }
}

}  // namespace

hipError_t launch_kv_write(const slora_kv& kv, const slora_qkv& w, hipStream_t s, const LaunchEvents& ev) {
  WriteArgs a;
  const bool store = w.k != nullptr;
  a.q = {(const uint16_t*)w.q, w.q_token_stride, w.q_head_stride};
  a.k = {(const uint16_t*)w.k, w.k_token_stride, w.k_head_stride};
  a.v = {(const uint16_t*)w.v, w.v_token_stride, w.v_head_stride};
  a.qo = (uint16_t*)w.q_out;
  a.ots = w.out_token_stride;
  a.ohs = w.out_head_stride;
  a.pool = (uint16_t*)kv.pool;
  a.n_pages = kv.n_pages;
  a.P = kv.page_elems;
  a.tpp = kv.tokens_per_page;
  a.row = kv.n_kv_heads * kv.head_dim;
  a.n_tok = w.n_tokens;
  a.hq = w.n_q_heads;
  a.hk = store ? kv.n_kv_heads : 0;
  a.D = kv.head_dim;
  a.pos = w.position;
  a.ks = w.k_slots;
  a.vs = w.v_slots;
  a.turns = w.turns;
  a.pairs = w.rotary_dim / 2;
  a.cs = w.cos_sin_scale;
  a.eps = w.eps;
  a.qw = (const uint16_t*)w.q_weight;
  a.kw = (const uint16_t*)w.k_weight;
  a.norm = w.norm;
  // pieces of 8, or of 4 where the half layout's halves are not whole pieces of 8
  const bool inter = w.interleaved != 0;
  const int v = !inter && a.pairs % 8 ? 4 : 8;
  const int g = (a.D / v + 1) / 2;
  // Tokens and heads of a workgroup (two tokens at most: 91 us for the case above, 94 with 4,
  // 109 with 8): few of both while the step is small (a decode step
  // of one token spreads its heads over workgroups), more tokens when there are enough
  // workgroups anyway, so that a token's angles are computed once for all its heads.
  const int heads = a.hq + 2 * a.hk;
  const int groups = kThreads / (v == 8 ? (g <= 4 ? 4 : g <= 8 ? 8 : 16) : (g <= 8 ? 8 : g <= 16 ? 16 : 32));
  int tpw = 1;
  while (tpw < kMaxTok && a.n_tok / (2 * tpw) >= 2048) tpw *= 2;
  int split = 1;
  while (split * 2 * groups <= heads + groups && (int64_t)a.n_tok * split < 1024) split *= 2;
  a.tpw = tpw;
  a.heads_y = (heads + split - 1) / split;
  const dim3 grid((unsigned)((a.n_tok + tpw - 1) / tpw), (unsigned)((heads + a.heads_y - 1) / a.heads_y));
  if ((int64_t)grid.x * kThreads >= kMaxThreads) return hipErrorInvalidConfiguration;
  if (kv.dtype == SLORA_F16) launch_dt<SLORA_F16>(inter, v, g, a, grid, s, ev);
  else launch_dt<SLORA_BF16>(inter, v, g, a, grid, s, ev);
  return hipGetLastError();
}

}  // namespace slora
