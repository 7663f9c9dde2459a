// Attention of one new token per request over its paged keys (slora_attn_decode).
//
//   s_j = q . k_j (scaled, capped, biased),  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Bound by the bytes of K and V, each read once. A workgroup owns one KV head of one
// request's run of keys, with the query heads that share it as up to 16 rows; its 4 waves
// take tiles of 32 keys in turn and keep their own maximum m, sum and output, joined in
// LDS at the end. When there are few requests, long ones are cut into runs that are joined
// by a second kernel.
//
// A tile never goes through LDS. v_mfma_f32_16x16x32 with A = K (16 keys x 32 dimensions)
// and B = q leaves lane l with scores of keys 4 (l / 16) + i of query row l % 16. The two
// 16-key products of a tile take their keys in such an order (row r of product t is key 8
// (r / 4) + 4 t + r % 4) that the 8 scores of a lane are those of keys 8 (l / 16) .. + 7:
// just what the next product, A = V^T (16 dimensions x 32 keys) and B = weights, wants as
// its B operand. For A a lane loads 8 dimensions of those 8 keys and turns the 8 x 8 block
// in registers (v_perm); product e of the tile then makes dimensions 8 m + e. Each row's
// keys, page ids and addresses are looked up once per tile, 64 lanes wide, and handed out
// through LDS. Loads run one tile ahead of the products, page ids two.
#include "attn_dev.h"

namespace slora {
namespace {

using namespace dev;

constexpr int kWaves = 4;
constexpr int kTile = 32;              // keys of a wave's tile
constexpr int kRound = kWaves * kTile; // keys a workgroup takes in one round
constexpr int kRows = 16;
constexpr float kRescale = 8.0f;       // growth of a maximum (log 2) that moves the sums

struct Seen {
  Keys keys;
  int32_t n;     // seq_len
  bool bad;      // seq_len outside the table
};

__device__ __forceinline__ Seen seen_by(const AttnArgs& a, int r) {
  Seen s;
  s.n = a.seq[r];
  s.bad = s.n < 0 || s.n > a.max_len;
  if (s.bad) s.n = 0;
  const int32_t prefix = a.prefix ? min(max(a.prefix[r], 0), s.n) : 0;
  s.keys = s.n > 0 ? keys_of(a, prefix, s.n, s.n - 1, s.n - 1) : Keys{0, 0, 0};
  return s;
}

// Keys of a chunk: all requests' keys spread over the workgroups aimed for, in whole
// rounds. The same on every wave of the call.
__device__ __forceinline__ int64_t chunk_keys(const AttnArgs& a, int lane, int units) {
  int64_t total = 0;
  for (int r = lane; r < a.n_req; r += 64) total += seen_by(a, r).keys.count;
  for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
  const int64_t chunks = (a.target + units - 1) / units;
  const int64_t c = (total + chunks - 1) / chunks;
  return max((c + kRound - 1) / kRound * kRound, (int64_t)kRound);
}

__device__ __forceinline__ int chunks_of(int32_t count, int64_t chunk) {
  return count <= chunk ? 1 : (int)((count + chunk - 1) / chunk);
}

struct Place {
  int r, first, n;  // request, its first chunk's number, its chunks
};

// The request whose chunks hold number x (r = -1: past the last).
__device__ __forceinline__ Place find_chunk(const AttnArgs& a, int lane, int64_t chunk, int x) {
  int before = 0;
  for (int r0 = 0; r0 < a.n_req; r0 += 64) {
    const int r = r0 + lane;
    const int c = r < a.n_req ? chunks_of(seen_by(a, r).keys.count, chunk) : 0;
    int sum = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const uint64_t hit = __ballot(x < before + sum);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int at = __shfl(sum, l), n = __shfl(c, l);
      return {r0 + l, before + at - n, n};
    }
    before += __shfl(sum, 63);
  }
  return {-1, 0, 0};
}

// The chunks of request r, all requests before it counted.
__device__ __forceinline__ Place chunks_before(const AttnArgs& a, int lane, int64_t chunk, int r) {
  int before = 0;
  for (int i = lane; i < r; i += 64) before += chunks_of(seen_by(a, i).keys.count, chunk);
  for (int d = 32; d; d >>= 1) before += __shfl_xor(before, d);
  return {r, before, chunks_of(seen_by(a, r).keys.count, chunk)};
}

// NC: head_dim in pieces of 32, rounded up to an instance; VD: dimensions a lane loads of a
// V vector at once (16 lanes cover it in VH turns).
template <int NC>
struct Shape {
  static constexpr int VD = NC <= 2 ? 4 : 8;
  static constexpr int VH = NC <= 4 ? 1 : 2;
  // pieces below this are inside any head_dim that uses the instance
  static constexpr int kFull = NC == 2 ? 0 : NC == 3 ? 2 : NC == 4 ? 3 : NC == 6 ? 4 : 6;
};

template <int NC>
struct Tile {
  uint4 k[2][NC];
  uint32_t v[8][Shape<NC>::VH][Shape<NC>::VD / 2];
};

template <int DT, int NC>
__global__ __launch_bounds__(kWaves * 64, NC <= 4 ? 2 : 1) void attn_decode_kernel(AttnArgs a) {
  using S = Shape<NC>;
  constexpr int VD = S::VD, VH = S::VH;
  extern __shared__ float sm_out[];                       // [wave][row][D]
  __shared__ uint64_t sm_addr[kWaves][2][64];
  __shared__ float sm_m[kWaves][kRows], sm_l[kWaves][kRows];

  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m16 = lane & 15, g = lane >> 4;
  const int row_groups = (a.group + kRows - 1) / kRows;
  const int units = a.hk * row_groups;
  const int unit = (int)(blockIdx.x % (uint32_t)units), x = (int)(blockIdx.x / (uint32_t)units);
  const int64_t chunk = chunk_keys(a, lane, units);
  const Place at = find_chunk(a, lane, chunk, x);
  if (at.r < 0) return;
  const int r = __builtin_amdgcn_readfirstlane(at.r);
  const Seen seen = seen_by(a, r);
  const int kv_head = unit / row_groups, row0 = (unit % row_groups) * kRows;
  const int rows = min(a.group - row0, kRows);
  const int head0 = kv_head * a.group + row0;
  const int h_off = kv_head * a.D;
  const int begin = (int)((x - at.first) * chunk);
  const int end = (int)min((int64_t)seen.keys.count, begin + chunk);

  // q, as the B operand: lane l holds dimensions 32 c + 8 (l / 16) .. + 7 of row l % 16
  uint4 q[NC];
  {
    const uint16_t* qp = a.q + (int64_t)r * a.q_ts + (int64_t)(head0 + min(m16, rows - 1)) * a.q_hs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = c * 32 + g * 8;
      q[c] = ld16(c < S::kFull || d < a.D ? qp + d : kAttnFill.zero);
    }
  }
  const float slope = a.slopes ? a.slopes[head0 + min(m16, rows - 1)] * kLog2e : 0.f;

  f32x4 acc[VH][VD];
#pragma unroll
  for (int h = 0; h < VH; ++h)
#pragma unroll
    for (int e = 0; e < VD; ++e) acc[h][e] = {0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  const int n_tiles = end > begin + wave * kTile ? (end - begin - wave * kTile + kRound - 1) / kRound : 0;
  // lane l looks up key l % 32 of the tile: its K page (l < 32) or V page
  const int32_t* table = (lane < 32 ? a.kt : a.vt) + (int64_t)r * a.max_blocks;
  auto tile_begin = [&](int t) { return begin + wave * kTile + t * kRound; };
  auto page_of = [&](int t) -> int32_t {
    const int i = min(tile_begin(t) + (lane & 31), end - 1);
    return table[div_tpp(a, (uint32_t)seen.keys.key(i))];
  };
  auto put_addr = [&](int t, int32_t page) {
    const int i = tile_begin(t) + (lane & 31);
    const uint64_t p = key_addr(a, page, seen.keys.key(min(i, end - 1)), h_off, fill_addr<DT>(false));
    sm_addr[wave][t & 1][lane] = i < end ? p : fill_addr<DT>(true);
  };
  auto fetch = [&](int t, Tile<NC>& x) {
    const uint64_t* ad = sm_addr[wave][t & 1];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint16_t* p = (const uint16_t*)ad[(m16 >> 2) * 8 + u * 4 + (m16 & 3)];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d = c * 32 + g * 8;
        x.k[u][c] = ld16(c < S::kFull || d < a.D ? p + d : kAttnFill.zero);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t* p = (const uint16_t*)ad[32 + g * 8 + i];
#pragma unroll
      for (int h = 0; h < VH; ++h) {
        int d = h * 128 + m16 * VD;
        if (d >= a.D) d = 0;  // these lanes' products are dimensions past the head: dropped
        if constexpr (VD == 8) {
          const uint4 w = ld16(p + d);
          x.v[i][h][0] = w.x; x.v[i][h][1] = w.y; x.v[i][h][2] = w.z; x.v[i][h][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(p + d);
          x.v[i][h][0] = w.x; x.v[i][h][1] = w.y;
        }
      }
    }
  };
  auto compute = [&](int t, const Tile<NC>& x) {
    const int i0 = tile_begin(t) + g * 8;
    float s[8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 c4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) c4 = mfma16x16<DT>(x.k[u][c], q[c], c4);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[u * 4 + i] = c4[i];
    }
    if (a.cap_out != 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = capped(a, s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] *= a.scale2;
    }
    if (a.slopes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += slope * (float)(seen.keys.key(i0 + i) - (seen.n - 1));
    }
    if (tile_begin(t) + kTile > end) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = i0 + i < end ? s[i] : -INFINITY;
    }
    float mx = s[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
    mx = max32(max16(mx));
    // The maximum is moved only when it has grown by kRescale: until then the weights
    // reach 2^kRescale, which costs neither range nor precision in 32 bits.
    if (__any(mx > m + kRescale)) {
      const float mn = fmaxf(m, mx);
      const float f = part_weight(m, mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int h = 0; h < VH; ++h)
#pragma unroll
        for (int e = 0; e < VD; ++e) acc[h][e] *= f;
    }
    const float ms = m == -INFINITY ? 0.f : m;
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = __builtin_amdgcn_exp2f(s[i] - ms);
      l += s[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pack2<DT>(s[2 * i], s[2 * i + 1]);
    const uint4 pb = make_uint4(p[0], p[1], p[2], p[3]);
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
      for (int e = 0; e < VD; ++e) {
        const int w = e >> 1;
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          b[i] = e & 1 ? pair_hi(x.v[2 * i][h][w], x.v[2 * i + 1][h][w])
                       : pair_lo(x.v[2 * i][h][w], x.v[2 * i + 1][h][w]);
        acc[h][e] = mfma16x16<DT>(make_uint4(b[0], b[1], b[2], b[3]), pb, acc[h][e]);
      }
  };
  // addresses are written and read by the lanes of one wave, in order
  auto fence = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); __builtin_amdgcn_wave_barrier(); };

  if (n_tiles > 0) {
    Tile<NC> x0, x1;
    put_addr(0, page_of(0));
    int32_t next = page_of(1);
    fence();
    fetch(0, x0);
    auto step = [&](int t, Tile<NC>& cur, Tile<NC>& nxt) {
      if (t + 1 < n_tiles) {
        fence();
        put_addr(t + 1, next);
        next = page_of(t + 2);
        fence();
        fetch(t + 1, nxt);
      }
      compute(t, cur);
    };
    for (int t = 0; t < n_tiles; t += 2) {
      step(t, x0, x1);
      if (t + 1 < n_tiles) step(t + 1, x1, x0);
    }
  }

  // join the waves
  l = sum32(sum16(l));
  if (g == 0) {
    sm_m[wave][m16] = m;
    sm_l[wave][m16] = l;
  }
  if (m16 < rows) {
    float* o = sm_out + ((int64_t)wave * rows + m16) * a.D;
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = h * 128 + (g * 4 + i) * VD;
        if (d < a.D) {
#pragma unroll
          for (int e = 0; e < VD; ++e) o[d + e] = acc[h][e][i];
        }
      }
  }
  __syncthreads();
  for (int i = tid; i < rows * a.D; i += kWaves * 64) {
    const int row = i / a.D, d = i - row * a.D;
    float mt = sm_m[0][row];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mt = fmaxf(mt, sm_m[w][row]);
    float o = 0.f, lt = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = part_weight(sm_m[w][row], mt);
      o += f * sm_out[((int64_t)w * rows + row) * a.D + d];
      lt += f * sm_l[w][row];
    }
    const int head = head0 + row;
    if (at.n == 1) {
      const float v = seen.bad ? NAN : lt == 0.f ? 0.f : o / lt;
      a.out[(int64_t)r * a.o_ts + (int64_t)head * a.o_hs + d] = (uint16_t)to_bits<DT>(v);
      if (a.lse && d == 0)
        a.lse[(int64_t)r * (a.hk * a.group) + head] = seen.bad ? NAN : mt * kLn2 + logf(lt);
    } else {
      float* part = a.part + ((int64_t)x * (a.hk * a.group) + head) * (a.D + 2);
      part[2 + d] = o;
      if (d == 0) {
        part[0] = mt;
        part[1] = lt;
      }
    }
  }
}

// Joins the chunks of requests that were cut: workgroup (request, query head).
template <int DT>
__global__ __launch_bounds__(64) void attn_decode_join(AttnArgs a) {
  const int lane = (int)threadIdx.x;
  const int heads = a.hk * a.group;
  const int r = (int)(blockIdx.x / (uint32_t)heads), head = (int)(blockIdx.x % (uint32_t)heads);
  const int units = a.hk * ((a.group + kRows - 1) / kRows);
  const int64_t chunk = chunk_keys(a, lane, units);
  if (chunks_of(seen_by(a, r).keys.count, chunk) == 1) return;
  const Place at = chunks_before(a, lane, chunk, r);
  const float* part = a.part + ((int64_t)at.first * heads + head) * (a.D + 2);
  const int64_t stride = (int64_t)heads * (a.D + 2);
  float mt = -INFINITY;
  for (int c = lane; c < at.n; c += 64) mt = fmaxf(mt, part[c * stride]);
  for (int d = 32; d; d >>= 1) mt = fmaxf(mt, __shfl_xor(mt, d));
  float lt = 0.f;
  for (int c = lane; c < at.n; c += 64) lt += part_weight(part[c * stride], mt) * part[c * stride + 1];
  for (int d = 32; d; d >>= 1) lt += __shfl_xor(lt, d);
  for (int d = lane; d < a.D; d += 64) {
    float o = 0.f;
    for (int c = 0; c < at.n; ++c) o += part_weight(part[c * stride], mt) * part[c * stride + 2 + d];
    a.out[(int64_t)r * a.o_ts + (int64_t)head * a.o_hs + d] = (uint16_t)to_bits<DT>(lt == 0.f ? 0.f : o / lt);
  }
  if (a.lse && lane == 0) a.lse[(int64_t)r * heads + head] = mt * kLn2 + logf(lt);
}

template <int DT, int NC>
hipError_t launch_nc(const AttnArgs& a, unsigned grid, hipStream_t s, const LaunchEvents& ev) {
  const int rows = a.group < kRows ? a.group : kRows;
  const size_t lds = sizeof(float) * kWaves * rows * a.D;
  if (lds > 48 * 1024) {  // with the static part past the 64 KiB a launch has by default
    const hipError_t e = hipFuncSetAttribute((const void*)attn_decode_kernel<DT, NC>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipExtLaunchKernelGGL((attn_decode_kernel<DT, NC>), dim3(grid), dim3(kWaves * 64), lds, s, ev.start, ev.stop, 0, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  const int units = a.hk * ((a.group + kRows - 1) / kRows);
  const int64_t wgs = decode_max_chunks(a.n_req, units) * units;
  if (wgs * kWaves * 64 >= kMaxThreads || (int64_t)a.n_req * a.hk * a.group * 64 >= kMaxThreads)
    return hipErrorInvalidConfiguration;
  const unsigned grid = (unsigned)wgs;
  LaunchEvents first = ev, second = ev;
  first.stop = nullptr;
  second.start = nullptr;
  const int nc = (a.D + 31) / 32;
  hipError_t e = nc <= 2   ? launch_nc<DT, 2>(a, grid, s, first)
                 : nc == 3 ? launch_nc<DT, 3>(a, grid, s, first)
                 : nc == 4 ? launch_nc<DT, 4>(a, grid, s, first)
                 : nc <= 6 ? launch_nc<DT, 6>(a, grid, s, first)
                           : launch_nc<DT, 8>(a, grid, s, first);
  if (e != hipSuccess) return e;
  hipExtLaunchKernelGGL((attn_decode_join<DT>), dim3((unsigned)(a.n_req * a.hk * a.group)), dim3(64), 0, s,
                        second.start, second.stop, 0, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_decode(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
