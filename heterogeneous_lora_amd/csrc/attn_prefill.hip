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
// rounding, the B operand of the second product without an exchange: K's rows lie in LDS
// with bits 2 and 3 of the key's number swapped, which makes the 8 scores a lane holds
// for 16 keys those of 8 consecutive keys. V is turned (8 keys x 4 dimensions per thread,
// in registers) on its way to LDS. Both tiles are laid out in 16-byte units whose index is
// xored with a few higher bits, so neither side has bank conflicts. Pages are gathered:
// addresses of a tile's keys are made two tiles ahead, its loads issued one tile ahead
// into registers and stored to the other LDS buffer after the products.
#include "attn_dev.h"

namespace slora {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWaveRows = 32;
constexpr int kTileM = 128;           // rows of a workgroup
constexpr float kRescale = 8.0f;      // growth of a maximum (log 2) that moves the sums

// NC: head_dim in pieces of 32, rounded up to an instance.
template <int NC>
struct Shape {
  static constexpr int BN = NC <= 4 ? 64 : 32;  // keys of a tile
  static constexpr int KT = BN / 32;
  static constexpr int kUnits = BN * NC * 4;    // 16-byte units of the K tile, and of the V tile
  static constexpr int kLoadK = kUnits / kThreads;
  static constexpr int kBlocksV = BN / 8 * NC * 8;  // 8 keys x 4 dimensions
  static_assert(kUnits % kThreads == 0 && kBlocksV <= kThreads, "tile loads");
};

struct RowTile {
  int r;       // request, -1: none
  int tile;    // row tile of the request
};

// The x-th row tile over all requests.
__device__ __forceinline__ int new_tokens(const AttnArgs& a, int r) {
  const int q0 = min(max(a.q_offsets[r], 0), a.n_tok), q1 = min(max(a.q_offsets[r + 1], 0), a.n_tok);
  return max(q1 - q0, 0);
}
__device__ __forceinline__ RowTile find_tile(const AttnArgs& a, int lane, int x) {
  int before = 0;
  for (int r0 = 0; r0 < a.n_req; r0 += 64) {
    const int r = r0 + lane;
    const int c = r < a.n_req ? (int)(((int64_t)new_tokens(a, r) * a.group + kTileM - 1) / kTileM) : 0;
    int sum = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const uint64_t hit = __ballot(x < before + sum);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      // later tiles of a request see more keys: they go first
      return {r0 + l, before + __shfl(sum, l) - 1 - x};
    }
    before += __shfl(sum, 63);
  }
  return {-1, 0};
}

// A dword of two storage values holds an infinity or NaN.
template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  constexpr uint32_t e = DT == SLORA_F16 ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}

__device__ __forceinline__ int k_unit(int bn, int chunk, int row) { return chunk * bn + (row ^ (chunk & 15)); }
__device__ __forceinline__ int v_unit(int dims, int kg, int d) { return kg * dims + (d ^ ((d >> 4) & 3)); }

template <int DT, int NC>
__global__ __launch_bounds__(kThreads, NC <= 4 ? 2 : 1) void attn_prefill_kernel(AttnArgs a) {
  using S = Shape<NC>;
  constexpr int BN = S::BN, KT = S::KT, kDims = NC * 32;
  __shared__ uint4 sm_k[2][S::kUnits];
  __shared__ uint4 sm_v[2][S::kUnits];
  __shared__ uint64_t sm_addr[2][2 * BN];
  __shared__ uint32_t sm_flag[4];  // tile t (mod 4) has infinities or NaN in V that some row must not see

  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m32 = lane & 31, h = lane >> 5;
  const int kv_head = (int)(blockIdx.x % (uint32_t)a.hk);
  const RowTile rt = find_tile(a, lane, (int)(blockIdx.x / (uint32_t)a.hk));
  if (rt.r < 0) return;
  const int r = __builtin_amdgcn_readfirstlane(rt.r);
  const int row_tile = __builtin_amdgcn_readfirstlane(rt.tile);
  const int q0 = min(max(a.q_offsets[r], 0), a.n_tok), n_new = new_tokens(a, r);
  const int64_t n_rows = (int64_t)n_new * a.group;
  const int64_t wg_row = (int64_t)row_tile * kTileM;
  const int64_t wg_last = min(wg_row + kTileM, n_rows) - 1;
  int32_t n = a.seq[r];
  const bool bad = n < 0 || n > a.max_len;
  if (bad) n = 0;
  const int first_pos = n - n_new;
  const int prefix = a.prefix ? min(max(a.prefix[r], 0), n) : 0;

  // this lane's row
  const int64_t my_row = wg_row + wave * kWaveRows + m32;
  const int64_t row_c = min(my_row, wg_last);
  const int tok = (int)(row_c / a.group), head = kv_head * a.group + (int)(row_c - (int64_t)tok * a.group);
  const int pos = first_pos + tok;
  const int wave_p0 = first_pos + (int)(min(wg_row + wave * kWaveRows, wg_last) / a.group);
  const int wave_p1 = first_pos + (int)(min(wg_row + wave * kWaveRows + kWaveRows - 1, wg_last) / a.group);
  const int wg_p0 = first_pos + (int)(wg_row / a.group), wg_p1 = first_pos + (int)(wg_last / a.group);
  const Keys keys = n > 0 ? keys_of(a, r, n, wg_p0, wg_p1) : Keys{0, 0, 0};
  const int n_tiles = (keys.count + BN - 1) / BN;
  const int h_off = kv_head * a.D;

  // q, as the B operand: lane holds dimensions 16 c + 8 h .. + 7 of its row
  uint4 q[NC * 2];
  {
    const uint16_t* qp = a.q + (int64_t)(q0 + tok) * a.q_ts + (int64_t)head * a.q_hs;
#pragma unroll
    for (int c = 0; c < NC * 2; ++c) {
      const int d = c * 16 + h * 8;
      q[c] = ld16(d < a.D ? qp + d : kAttnFill.zero);
    }
  }
  const float slope = a.slopes ? a.slopes[head] * kLog2e : 0.f;

  f32x16 acc[NC];
#pragma unroll
  for (int d = 0; d < NC; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  // addresses of a tile's keys: threads [0, BN) K, [BN, 2 BN) V
  const int32_t* table = (tid < BN ? a.kt : a.vt) + (int64_t)r * a.max_blocks;
  auto page_of = [&](int t) -> int32_t {
    if (tid >= 2 * BN) return 0;
    return table[div_tpp(a, (uint32_t)keys.key(min(t * BN + tid % BN, keys.count - 1)))];
  };
  auto put_addr = [&](int t, int32_t page) {
    if (tid >= 2 * BN) return;
    const int i = t * BN + tid % BN;
    const uint64_t p = key_addr<DT>(a, page, keys.key(min(i, keys.count - 1)), h_off);
    sm_addr[t & 1][tid] = i < keys.count ? p : fill_addr<DT>(true);
  };
  uint4 rk[S::kLoadK];
  uint2 rv[8];
  const int v_kg = tid / (NC * 8), v_d = tid % (NC * 8) * 4;
  const bool has_v = tid < S::kBlocksV;
  auto fetch = [&](int t) {
    const uint64_t* ad = sm_addr[t & 1];
#pragma unroll
    for (int u = 0; u < S::kLoadK; ++u) {
      const int i = tid + u * kThreads, key = i / (NC * 4), d = i % (NC * 4) * 8;
      rk[u] = ld16(d < a.D ? (const uint16_t*)ad[key] + d : kAttnFill.zero);
    }
    if (has_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t* p = (const uint16_t*)ad[BN + v_kg * 8 + i];
        rv[i] = *reinterpret_cast<const uint2*>(v_d < a.D ? p + v_d : kAttnFill.zero);
      }
    }
  };
  // Every row of the workgroup sees every key of tile t.
  auto all_seen = [&](int t, int p0, int p1) {
    const int i1 = t * BN + BN - 1;
    if (i1 >= keys.count) return false;
    const int j0 = keys.key(t * BN), j1 = keys.key(i1);
    return j1 < prefix || (j1 <= p0 && (a.window == 0 || p1 - j0 < a.window));
  };
  auto put_tile = [&](int t) {
    const int b = t & 1;
#pragma unroll
    for (int u = 0; u < S::kLoadK; ++u) {
      const int i = tid + u * kThreads, key = i / (NC * 4), chunk = i % (NC * 4);
      const int row = (key & ~12) | (key & 4) << 1 | (key & 8) >> 1;
      sm_k[b][k_unit(BN, chunk, row)] = rk[u];
    }
    if (has_v) {
      bool odd = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = e < 2 ? rv[2 * i].x : rv[2 * i].y, y = e < 2 ? rv[2 * i + 1].x : rv[2 * i + 1].y;
          w[i] = e & 1 ? pair_hi(x, y) : pair_lo(x, y);
          odd |= not_finite<DT>(w[i]);
        }
        sm_v[b][v_unit(kDims, v_kg, v_d + e)] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (odd && !all_seen(t, wg_p0, wg_p1)) sm_flag[t & 3] = 1;
    }
  };

  if (tid < 4) sm_flag[tid] = 0;
  if (n_tiles > 0) {
    put_addr(0, page_of(0));
    __syncthreads();
    fetch(0);
    put_addr(1, page_of(1));
    put_tile(0);
  }
  __syncthreads();

  for (int t = 0; t < n_tiles; ++t) {
    const int b = t & 1;
    int32_t next = 0;
    if (t + 1 < n_tiles) {
      fetch(t + 1);
      next = page_of(t + 2);
    }
    if (tid == 0) sm_flag[(t + 2) & 3] = 0;

    const int j0 = keys.key(t * BN), j1 = keys.key(min(t * BN + BN, keys.count) - 1);
    const bool none = j0 >= prefix && (j0 > wave_p1 || (a.window != 0 && wave_p0 - j1 >= a.window));
    uint4 p[KT][2];
    if (!none) {
      f32x16 s[KT];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kt][i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC * 2; ++c)
          s[kt] = mfma32x32<DT>(sm_k[b][k_unit(BN, 2 * c + h, kt * 32 + m32)], q[c], s[kt]);
      }
      if (a.cap_out != 0.f) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[kt][i] = capped(a, s[kt][i]);
      } else {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[kt][i] *= a.scale2;
      }
      // register i of product kt: key kt * 32 + 16 (i / 8) + 8 h + i % 8 of the tile
      if (a.slopes || !all_seen(t, wave_p0, wave_p1)) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = t * BN + kt * 32 + 16 * (i / 8) + 8 * h + i % 8, j = keys.key(at);
            const float x = s[kt][i] + slope * (float)(j - pos);
            s[kt][i] = at < keys.count && sees(a, prefix, pos, j) ? x : -INFINITY;
          }
      }
      float mx = s[0][0];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kt][i]);
      mx = max32(mx);
      // The maximum is moved only when it has grown by kRescale: until then the weights
      // reach 2^kRescale, which costs neither range nor precision in 32 bits.
      if (__any(mx > m + kRescale)) {
        const float mn = fmaxf(m, mx);
        const float f = part_weight(m, mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < NC; ++d) acc[d] *= f;
      }
      const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[kt][i] = __builtin_amdgcn_exp2f(s[kt][i] - ms);
          l += s[kt][i];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
          p[kt][u] = make_uint4(pack2<DT>(s[kt][8 * u], s[kt][8 * u + 1]), pack2<DT>(s[kt][8 * u + 2], s[kt][8 * u + 3]),
                                pack2<DT>(s[kt][8 * u + 4], s[kt][8 * u + 5]),
                                pack2<DT>(s[kt][8 * u + 6], s[kt][8 * u + 7]));
      }
    }
    // A weight of zero does not keep an infinity or NaN in V out of a product. Where a key
    // that some rows must not see holds one, such values are added to the rows that do see
    // them here (they decide these rows' results, whatever their weight) and cleared from
    // the tile. No ordinary tile comes here.
    if (sm_flag[t & 3]) {
      const uint16_t* vt = (const uint16_t*)sm_v[b];
      if (!none) {
        for (int k = 0; k < BN; ++k) {
          const int at = t * BN + k;
          const bool on = at < keys.count && sees(a, prefix, pos, keys.key(at));
#pragma unroll
          for (int d = 0; d < NC; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int dim = d * 32 + 8 * (i / 4) + 4 * h + i % 4;
              const uint32_t w = vt[v_unit(kDims, k >> 3, dim) * 8 + (k & 7)];
              if (on && not_finite<DT>(w)) acc[d][i] += lo_f32<DT>(w);
            }
        }
      }
      __syncthreads();
      for (int i = tid; i < S::kUnits * 8; i += kThreads) {
        uint16_t* w = (uint16_t*)sm_v[b] + i;
        if (not_finite<DT>(*w)) *w = 0;
      }
      __syncthreads();
    }
    if (!none) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int d = 0; d < NC; ++d)
            acc[d] = mfma32x32<DT>(sm_v[b][v_unit(kDims, kt * 4 + u * 2 + h, d * 32 + m32)], p[kt][u], acc[d]);
    }
    if (t + 1 < n_tiles) {
      put_tile(t + 1);
      put_addr(t + 2, next);
    }
    __syncthreads();
  }

  l = sum32(l);
  if (my_row > wg_last) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  uint16_t* o = a.out + (int64_t)(q0 + tok) * a.o_ts + (int64_t)head * a.o_hs;
#pragma unroll
  for (int d = 0; d < NC; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int dim = d * 32 + 8 * (i / 4) + 4 * h;
      if (dim < a.D) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = bad ? NAN : l == 0.f ? 0.f : acc[d][i + e] * inv;
        *reinterpret_cast<uint2*>(o + dim) = make_uint2(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]));
      }
    }
  if (a.lse && h == 0)
    a.lse[(int64_t)(q0 + tok) * (a.hk * a.group) + head] = bad ? NAN : m * kLn2 + logf(l);
}

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  const int64_t tiles = ((int64_t)a.n_tok * a.group + kTileM - 1) / kTileM + a.n_req;
  if (tiles * a.hk * kThreads >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(tiles * a.hk));
  const int nc = (a.D + 31) / 32;
  auto go = [&](auto kernel) {
    hipExtLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
    return hipGetLastError();
  };
  return nc <= 2   ? go(attn_prefill_kernel<DT, 2>)
         : nc == 3 ? go(attn_prefill_kernel<DT, 3>)
         : nc == 4 ? go(attn_prefill_kernel<DT, 4>)
         : nc <= 6 ? go(attn_prefill_kernel<DT, 6>)
                   : go(attn_prefill_kernel<DT, 8>);
}

}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
