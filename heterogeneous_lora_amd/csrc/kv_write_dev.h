// What the kernels that store new keys and values share (kv_write.hip, kv4_write.hip): their
// arguments, the pieces of a head a lane holds, tokens and heads of a workgroup.
#pragma once

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

// The lane's two pieces of a head, in units of V dimensions: the rotated pairs first, the rest
// of the head two by two. g: the lane's number in its group.
struct Place {
  int g, half, c0, c1;
  bool has0, has1;  // inside the head
};
template <int V, bool INTER>
__device__ __forceinline__ Place place_of(const WriteArgs& a, int g) {
  const int n_pieces = a.D / V, half = INTER ? 0 : a.pairs / V;
  int c0, c1;
  if (INTER) {
    c0 = 2 * g;
    c1 = 2 * g + 1;
  } else {
    c0 = g < half ? g : 2 * half + 2 * (g - half);
    c1 = g < half ? g + half : c0 + 1;
  }
  return {g, half, c0, c1, c0 < n_pieces, c1 < n_pieces};
}

// Norm and rotation of a head of q or k, in F's arithmetic: the lane's two pieces, the weight of
// the norm (NULL: none), cosines and sines of the token.
template <int DT, int V, int G, bool INTER, typename F, typename Angle>
__device__ __forceinline__ void norm_and_turn(const WriteArgs& a, const Angle* ang, const uint16_t* w, const Place& at,
                                              F (&x)[V], F (&y)[V]) {
  if (a.norm) {
    F ss = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) ss += x[e] * x[e] + y[e] * y[e];
#pragma unroll
    for (int d = 1; d < G; d <<= 1) ss += __shfl_xor(ss, d);
    const F inv = (F)1 / sqrt(ss / (F)a.D + (F)a.eps);
    float wx[V], wy[V];
#pragma unroll
    for (int e = 0; e < V; ++e) wx[e] = wy[e] = 1.f;
    if (w) {
      if (at.has0) unpack<DT, V>(load<V>(w + at.c0 * V), wx);
      if (at.has1) unpack<DT, V>(load<V>(w + at.c1 * V), wy);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[e] = x[e] * inv * (F)wx[e];
      y[e] = y[e] * inv * (F)wy[e];
    }
  }
  if (INTER) {
    // (the rotated part ends with a piece)
    auto turn = [&](int c, F (&z)[V]) {
      if (c * V / 2 >= a.pairs) return;
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const F co = (F)ang[(c * V + e) / 2].x, s = (F)ang[(c * V + e) / 2].y;
        const F p = z[e], q = z[e + 1];
        z[e] = p * co - q * s;
        z[e + 1] = q * co + p * s;
      }
    };
    turn(at.c0, x);
    turn(at.c1, y);
  } else if (at.g < at.half) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const F c = (F)ang[at.c0 * V + e].x, s = (F)ang[at.c0 * V + e].y;
      const F p = x[e], q = y[e];
      x[e] = p * c - q * s;
      y[e] = q * c + p * s;
    }
  }
}

// A launch: pieces of v elements, the lanes g that a head needs, the grid.
struct Plan {
  WriteArgs a;
  bool inter;
  int v, g;
  dim3 grid;
};
inline Plan plan_write(const slora_kv& kv, const slora_qkv& w) {
  Plan p;
  WriteArgs& a = p.a;
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
  p.inter = w.interleaved != 0;
  const int v = !p.inter && a.pairs % 8 ? 4 : 8;
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
  p.v = v;
  p.g = g;
  p.grid = dim3((unsigned)((a.n_tok + tpw - 1) / tpw), (unsigned)((heads + a.heads_y - 1) / a.heads_y));
  return p;
}

}  // namespace
}  // namespace slora
