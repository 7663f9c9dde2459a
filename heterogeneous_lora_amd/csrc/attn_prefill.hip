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
// rounding, the B operand of the second product without an exchange: the first product
// takes K's rows with bits 2 and 3 of the key's number swapped, which makes the 8 scores a
// lane holds for 16 keys those of 8 consecutive keys.
//
// Pages are gathered straight into LDS (global_load_lds, 16 bytes a lane), one tile ahead
// of the products; the addresses of a tile's keys are made two tiles ahead, its page ids
// are read three ahead. A tile's rows lie as in the page, in 16-byte units whose places
// within a row are xored with bits of the row's number: K is read a row to a lane
// (ds_read_b128), V four keys x 16 dimensions to 16 lanes, turned on the way
// (ds_read_b64_tr_b16), both without bank conflicts. Two workgroups share a CU, so that one
// has products to run while the other is at its weights.
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
  static constexpr int CH = NC * 4;             // 16-byte units of a row
  static constexpr int kUnits = BN * CH;        // of a tile (K or V)
  static constexpr int kLoads = kUnits / kThreads;
  static_assert(kUnits % kThreads == 0, "tile loads");
  // The place of unit c of row `key`: LDS has 16 units a bank row. K is read one unit of
  // 16 rows at a time, V four units of 4 rows.
  __device__ static __forceinline__ int k_at(int key, int c) {
    if constexpr (CH == 12) return c ^ (key >> 2 & 3);
    else if constexpr (CH % 16) return c ^ (key >> 1 & 7);
    else return c ^ (key & 15);
  }
  __device__ static __forceinline__ int v_at(int key, int c) {
    if constexpr (CH == 12) return c;
    else if constexpr (CH % 16) return c ^ (key >> 1 & 1) * 4;
    else return c ^ (key & 3) * 4;
  }
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

// The halves of a dword of two storage values that hold an infinity or NaN; the rest 0.
template <int DT>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t e = DT == SLORA_F16 ? 0x7C00u : 0x7F80u;
  const uint32_t lo = (w & e) == e ? 0xffffu : 0u, hi = (w & e << 16) == e << 16 ? 0xffff0000u : 0u;
  return w & (lo | hi);
}
// Keeps the compiler from moving what made x into one arm of a later choice, as a branch.
template <typename T>
__device__ __forceinline__ T settled(T x) {
  asm volatile("" : "+v"(x));
  return x;
}

// 16 bytes of every lane from its address to LDS: lane l's land at lds + 16 l. Written out
// because the compiler, which cannot tell the tile being filled from the one being read,
// would wait for these loads before every read of LDS; landed() is the wait.
__device__ __forceinline__ void load_to_lds(uint64_t from, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :: "{m0}"(lds), "v"(from) : "memory");
}
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

typedef __attribute__((address_space(3))) void lds_void;
__device__ __forceinline__ uint32_t lds_offset(const void* p) { return (uint32_t)(uintptr_t)(lds_void*)p; }

// Four 16-bit values of this lane's column (16 lanes: 4 rows of 16 values, 4 to a lane).
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 read_turned(const uint16_t* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// What a score passes through between the two products. kPlain: the scale alone, taken in
// the subtraction of the maximum. kCap: softcap. kAny: a bias that depends on distance, with
// or without softcap, and scales of zero or below (which would turn a masked -infinity).
enum Mode { kPlain, kCap, kAny };

template <int DT, int NC, int MODE>
__global__ __launch_bounds__(kThreads, 2) void attn_prefill_kernel(AttnArgs a) {
  using S = Shape<NC>;
  constexpr int BN = S::BN, KT = S::KT, CH = S::CH;
  __shared__ uint4 sm_k[2][S::kUnits];
  __shared__ uint4 sm_v[2][S::kUnits];
  __shared__ uint64_t sm_addr[2][2 * BN];
  __shared__ uint32_t sm_flag[4];  // tile t (mod 4) has infinities or NaN in V that some row must not see

  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m32 = lane & 31, h = lane >> 5;
  const int kv_head = (int)(blockIdx.x % (uint32_t)a.hk);
  const RowTile rt = find_tile(a, lane, (int)(blockIdx.x / (uint32_t)a.hk));
  const int r = __builtin_amdgcn_readfirstlane(rt.r);
  if (r < 0) return;
  const int row_tile = __builtin_amdgcn_readfirstlane(rt.tile);
  const int q0 = min(max(a.q_offsets[r], 0), a.n_tok), n_new = new_tokens(a, r);
  int32_t n = a.seq[r];
  const bool bad = n < 0 || n > a.max_len;
  if (bad) n = 0;
  const int first_pos = n - n_new;
  const int prefix = a.prefix ? min(max(a.prefix[r], 0), n) : 0;

  // Row i of the tile: token tok0 + (head0 + i) / group, query head (head0 + i) % group.
  const int rows = (int)min((int64_t)n_new * a.group - (int64_t)row_tile * kTileM, (int64_t)kTileM);
  const int tile_q = row_tile / a.group, tile_r = row_tile - tile_q * a.group;
  const int tok0 = tile_q * kTileM + (int)div_group(a, (uint32_t)(tile_r * kTileM));
  const int head0 = tile_r * kTileM - (tok0 - tile_q * kTileM) * a.group;
  auto pos_of = [&](int i) { return first_pos + tok0 + (int)div_group(a, (uint32_t)(head0 + min(i, rows - 1))); };
  // this lane's row
  const int my_row = wave * kWaveRows + m32;
  const int pos = pos_of(my_row), tok = pos - first_pos;
  const int head = kv_head * a.group + head0 + min(my_row, rows - 1) - (tok - tok0) * a.group;
  const int wave_p0 = pos_of(wave * kWaveRows), wave_p1 = pos_of(wave * kWaveRows + kWaveRows - 1);
  const int wg_p0 = first_pos + tok0, wg_p1 = pos_of(kTileM - 1);
  const Keys keys = n > 0 ? keys_of(a, r, n, wg_p0, wg_p1) : Keys{0, 0, 0};
  const int n_tiles = (keys.count + BN - 1) / BN;
  const int h_off = kv_head * a.D;
  // In terms of the run's indices the row sees [0, prefix) and [see_lo, see_hi].
  const int see_hi = pos - keys.gap, see_lo = a.window ? see_hi - a.window + 1 : -1;

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
  const float slope = MODE == kAny && a.slopes ? a.slopes[head] * kLog2e : 0.f;
  const float mul = MODE == kPlain ? a.scale2 : 1.f;

  f32x16 acc[NC];
#pragma unroll
  for (int d = 0; d < NC; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  // Addresses of a tile's keys: threads [0, BN) K, [BN, 2 BN) V, the others the same again.
  // (The loop has no branch that lanes could disagree on, one body, and no other place that
  // changes the accumulators: otherwise the compiler keeps a second set of them, and every
  // tile pays for copies between the two.)
  const int my_key = tid % BN;
  const uint64_t zeros = settled(fill_addr<DT>(true)), nans = settled(fill_addr<DT>(false));
  const int32_t* table = (tid / BN % 2 ? a.vt : a.kt) + (int64_t)r * a.max_blocks;
  auto page_of = [&](int t) -> int32_t {
    return table[div_tpp(a, (uint32_t)keys.key(min(t * BN + my_key, keys.count - 1)))];
  };
  auto put_addr = [&](int t, int32_t page) {
    const int i = t * BN + my_key;
    const uint64_t p = settled(key_addr(a, page, keys.key(min(i, keys.count - 1)), h_off, nans));
    sm_addr[t & 1][tid % (2 * BN)] = i < keys.count ? p : zeros;
  };
  const uint32_t lds_k = lds_offset(sm_k) + wave * 1024, lds_v = lds_offset(sm_v) + wave * 1024;
  auto fetch = [&](int t) {
    const uint64_t* ad = sm_addr[t & 1];
    const uint32_t b = (uint32_t)(t & 1) * S::kUnits * 16;
#pragma unroll
    for (int u = 0; u < S::kLoads; ++u) {
      const int i = tid + u * kThreads, key = i / CH, d = S::k_at(key, i % CH) * 8;
      const uint64_t row = settled(ad[key]);
      load_to_lds(settled(d < a.D ? row + d * 2 : zeros), lds_k + b + u * kThreads * 16);
    }
#pragma unroll
    for (int u = 0; u < S::kLoads; ++u) {
      const int i = tid + u * kThreads, key = i / CH, d = S::v_at(key, i % CH) * 8;
      const uint64_t row = settled(ad[BN + key]);
      load_to_lds(settled(d < a.D ? row + d * 2 : zeros), lds_v + b + u * kThreads * 16);
    }
  };
  // Every row from position p0 to p1 sees every key of tile t.
  auto all_seen = [&](int t, int p0, int p1) {
    const int i1 = t * BN + BN - 1;
    if (i1 >= keys.count) return false;
    const int j0 = keys.key(t * BN), j1 = keys.key(i1);
    return j1 < prefix || (j1 <= p0 && (a.window == 0 || p1 - j0 < a.window));
  };

  sm_flag[tid & 3] = 0;
  int32_t next = 0;
  if (n_tiles > 0) {
    put_addr(0, page_of(0));
    put_addr(1, page_of(1));
    next = page_of(2);
    __syncthreads();
    fetch(0);
  }

  const int k_row = (m32 & ~12) | (m32 & 4) << 1 | (m32 & 8) >> 1;
  const int v_key = h * 8 + (lane >> 2 & 3), v_c = (lane >> 4 & 1) * 2 + (lane >> 1 & 1), v_in = (lane & 1) * 4;
  // Scores of tile t. Register i of product kt: index t * BN + kt * 32 + 16 (i / 8) + 8 h +
  // i % 8 of the run.
  auto scores = [&](int t, f32x16 (&s)[KT]) {
    const uint4* kb = sm_k[t & 1];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[kt][i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC * 2; ++c)
        s[kt] = mfma32x32<DT>(kb[(kt * 32 + k_row) * CH + S::k_at(k_row, 2 * c + h)], q[c], s[kt]);
    }
    if (MODE == kCap || (MODE == kAny && a.cap_out != 0.f)) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kt][i] = capped(a, s[kt][i]);
    } else if (MODE == kAny) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kt][i] *= a.scale2;
    }
    if (MODE == kAny) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[kt][i] += slope * (float)(keys.key(t * BN + kt * 32 + 16 * (i / 8) + 8 * h + i % 8) - pos);
    }
  };
  // The running maximum and sum take the scores in; the weights, as the B operand.
  auto weights = [&](f32x16 (&s)[KT], uint4 (&p)[KT][2]) {
    float mx = s[0][0];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kt][i]);
    mx = max32(mx) * mul;
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
        s[kt][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][i], mul, -ms));
        l += s[kt][i];
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        p[kt][u] = make_uint4(round2<DT>(s[kt][8 * u], s[kt][8 * u + 1]), round2<DT>(s[kt][8 * u + 2], s[kt][8 * u + 3]),
                              round2<DT>(s[kt][8 * u + 4], s[kt][8 * u + 5]),
                              round2<DT>(s[kt][8 * u + 6], s[kt][8 * u + 7]));
    }
  };
  auto add_values = [&](int t, const uint4 (&p)[KT][2]) {
    const uint16_t* vt = (const uint16_t*)sm_v[t & 1];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int d = 0; d < NC; ++d) {
          const int key = kt * 32 + u * 16 + v_key;
          const uint16_t* at = vt + (key * CH + S::v_at(v_key, d * 4 + v_c)) * 8 + v_in;
          const uint2 x = read_turned(at), y = read_turned(at + 4 * CH * 8);
          acc[d] = mfma32x32<DT>(make_uint4(x.x, x.y, y.x, y.y), p[kt][u], acc[d]);
        }
  };

  bool cleared = false;  // some tile held an infinity or NaN
  for (int t = 0; t < n_tiles; ++t) {
    landed();         // this wave's share of tile t
    __syncthreads();  // everyone's; and everyone is done with tile t - 1
    if (t + 1 < n_tiles) {
      fetch(t + 1);
      put_addr(t + 2, next);
      next = page_of(t + 3);
    }
    // A tile on some row's border. A weight of zero does not keep an infinity or NaN in V
    // out of a product, so these are taken out of such a tile and dealt with at the end. No
    // ordinary tile gets past the look.
    const bool edge = !all_seen(t, wg_p0, wg_p1);
    if (edge) {
      sm_flag[(t + 2) & 3] = 0;
      uint4* vt = sm_v[t & 1];
      uint32_t odd = 0;
#pragma unroll
      for (int u = 0; u < S::kLoads; ++u) {
        const uint4 w = vt[tid + u * kThreads];
        odd |= not_finite<DT>(w.x) | not_finite<DT>(w.y) | not_finite<DT>(w.z) | not_finite<DT>(w.w);
      }
      if (__any(odd != 0)) sm_flag[t & 3] = 1;
      __syncthreads();
      if (__builtin_amdgcn_readfirstlane(sm_flag[t & 3])) {
        cleared = true;
#pragma unroll 1
        for (int u = 0; u < S::kLoads; ++u) {
          uint4 w = vt[tid + u * kThreads];
          w.x ^= not_finite<DT>(w.x);
          w.y ^= not_finite<DT>(w.y);
          w.z ^= not_finite<DT>(w.z);
          w.w ^= not_finite<DT>(w.w);
          vt[tid + u * kThreads] = w;
        }
        __syncthreads();
      }
    }
    const int j0 = keys.key(t * BN), j1 = keys.key(min(t * BN + BN, keys.count) - 1);
    if (j0 >= prefix && (j0 > wave_p1 || (a.window != 0 && wave_p0 - j1 >= a.window))) continue;  // nothing for this wave
    f32x16 s[KT];
    uint4 p[KT][2];
    scores(t, s);
    if (edge) {
      const int at = t * BN + 8 * h, hi = see_hi - at, lo = see_lo - at, pre = prefix - at;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = kt * 32 + 16 * (i / 8) + i % 8;
          s[kt][i] = (((k <= hi) & (k >= lo)) | (k < pre)) ? s[kt][i] : -INFINITY;
        }
    }
    weights(s, p);
    add_values(t, p);
  }
  // The infinities and NaN taken out, to the rows that see them: they decide these rows'
  // results, whatever their weight.
  if (cleared) {
    const int32_t* vt = a.vt + (int64_t)r * a.max_blocks;
#pragma unroll 1
    for (int i = 0; i < n_tiles * BN; ++i) {
      if (i % BN == 0 && all_seen(i / BN, wg_p0, wg_p1)) {
        i += BN - 1;
        continue;
      }
      if (i >= keys.count) break;
      const int j = keys.key(i);
      const uint64_t row = key_addr(a, vt[div_tpp(a, (uint32_t)j)], j, h_off, nans);
      const uint32_t on = (((i <= see_hi) & (i >= see_lo)) | (i < prefix)) ? ~0u : 0u;
#pragma unroll
      for (int d = 0; d < NC; ++d)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int dim = d * 32 + 8 * u + 4 * h;
          const uint64_t w = *(const __attribute__((address_space(1))) uint64_t*)(dim < a.D ? row + dim * 2 : zeros);
          const uint32_t x0 = not_finite<DT>((uint32_t)w) & on, x1 = not_finite<DT>((uint32_t)(w >> 32)) & on;
          acc[d][4 * u] += lo_f32<DT>(x0);
          acc[d][4 * u + 1] += hi_f32<DT>(x0);
          acc[d][4 * u + 2] += lo_f32<DT>(x1);
          acc[d][4 * u + 3] += hi_f32<DT>(x1);
        }
    }
  }

  l = sum32(l);
  if (my_row >= rows) return;
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
        *reinterpret_cast<uint2*>(o + dim) = make_uint2(round2<DT>(x[0], x[1]), round2<DT>(x[2], x[3]));
      }
    }
  if (a.lse && h == 0)
    a.lse[(int64_t)(q0 + tok) * (a.hk * a.group) + head] = bad ? NAN : m * kLn2 + logf(l);
}

template <int DT, int MODE>
hipError_t launch_mode(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  const int64_t tiles = ((int64_t)a.n_tok * a.group + kTileM - 1) / kTileM + a.n_req;
  if (tiles * a.hk * kThreads >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(tiles * a.hk));
  const int nc = (a.D + 31) / 32;
  auto go = [&](auto kernel) {
    hipExtLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, ev.start, ev.stop, 0, a);
    return hipGetLastError();
  };
  return nc <= 2   ? go(attn_prefill_kernel<DT, 2, MODE>)
         : nc == 3 ? go(attn_prefill_kernel<DT, 3, MODE>)
         : nc == 4 ? go(attn_prefill_kernel<DT, 4, MODE>)
         : nc <= 6 ? go(attn_prefill_kernel<DT, 6, MODE>)
                   : go(attn_prefill_kernel<DT, 8, MODE>);
}

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  return a.slopes || !(a.scale2 > 0.f) ? launch_mode<DT, kAny>(a, s, ev)
         : a.cap_out != 0.f           ? launch_mode<DT, kCap>(a, s, ev)
                                      : launch_mode<DT, kPlain>(a, s, ev);
}

}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
