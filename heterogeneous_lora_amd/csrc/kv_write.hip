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
#include "kv_write_dev.h"

namespace slora {
namespace {

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

  const Place at = place_of<V, INTER>(a, tid % G);
  const int c0 = at.c0, c1 = at.c1;
  const bool has0 = at.has0, has1 = at.has1;

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
      norm_and_turn<DT, V, G, INTER>(a, angle + t * pairs, is_q ? a.qw : a.kw, at, x, y);
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
  const Plan p = plan_write(kv, w);
  if ((int64_t)p.grid.x * kThreads >= kMaxThreads) return hipErrorInvalidConfiguration;
  if (kv.dtype == SLORA_F16) launch_dt<SLORA_F16>(p.inter, p.v, p.g, p.a, p.grid, s, ev);
  else launch_dt<SLORA_BF16>(p.inter, p.v, p.g, p.a, p.grid, s, ev);
  return hipGetLastError();
}

}  // namespace slora
