// Attention of one new token per request over its paged keys (slora_attn_decode).
//
//   s_j = q . k_j (scaled, capped, biased),  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Bound by the bytes of K and V, each read once. A wave owns one KV head of one request's
// run of keys, with the query heads that share it as up to 16 rows, and takes tiles of 32
// keys. Where there are enough requests to fill the device with one chunk each, the 4 waves
// of a workgroup take up to 4 neighbouring heads, whose vectors lie together in the pages
// (5.88 TB/s against 5.45 for 512 requests of 40 heads). Otherwise they share one head's
// keys, each with its own maximum m, sum and output, joined in LDS at the end, and long
// requests are cut into chunks (a wave to a head would leave four times the partial
// results). Their partial results are joined by the workgroup that
// finishes last (a counter in the workspace), in the chunks' order, so the result does not
// depend on which one that is.
//
// 512 requests of 64 to 2048 keys, 40 heads of 128: 1.89 ms (5.9 TB/s); three of 100000 to
// 131072 keys, 64 query heads on 8: 270 us (5.3 TB/s); 64 with a window of 1024: 44 us.
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
constexpr int kRows = 16;
constexpr float kRescale = 8.0f;       // growth of a maximum (log 2) that moves the sums

struct Seen {
  Keys keys;
  int32_t n;     // seq_len
  bool bad;      // seq_len outside the table
};

__device__ __forceinline__ Seen seen_by(const AttnArgs& a, int32_t seq, int32_t prefix) {
  Seen s;
  s.n = seq;
  s.bad = s.n < 0 || s.n > a.max_len;
  if (s.bad) s.n = 0;
  s.keys = s.n > 0 ? keys_of(a, min(max(prefix, 0), s.n), s.n, s.n - 1, s.n - 1, 1) : Keys{0, 0, 0};
  return s;
}

struct Place {
  int r;           // request, -1: none
  int first, n;    // its first chunk's number, its chunks
  int32_t seq, prefix;
};

// The number nearest to count / chunk: one key more does not make a chunk of its own.
__device__ __forceinline__ int chunks_of(int32_t count, float per_chunk) {
  return max((int)((float)count * per_chunk + 0.5f), 1);
}

// The request whose chunks hold number x. A chunk is all requests' keys spread over the
// workgroups aimed for, in whole rounds of keys; every wave of the call finds the same. A
// lane takes HOLD requests at a time, all their loads in flight at once, and keeps them where
// one turn covers the call: each turn is one memory latency that nothing hides.
template <int HOLD>
__device__ __forceinline__ Place find_chunk(const AttnArgs& a, int lane, int x, int round) {
  constexpr int kTurn = 64 * HOLD;
  int32_t seq[HOLD], prefix[HOLD], count[HOLD];
  auto load = [&](int r0) {
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
      const int r = min(r0 + lane * HOLD + k, a.n_req - 1);
      seq[k] = a.seq[r];
      prefix[k] = a.prefix ? a.prefix[r] : 0;
    }
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      count[k] = r0 + lane * HOLD + k < a.n_req ? seen_by(a, seq[k], prefix[k]).keys.count : -1;
  };
  float total = 0.f;
  for (int r0 = 0; r0 < a.n_req; r0 += kTurn) {
    load(r0);
#pragma unroll
    for (int k = 0; k < HOLD; ++k) total += (float)max(count[k], 0);
  }
  // (In 32 bits the keys may be off by a part in 10^6: the chunks past one a request stay a
  // whole number not above a.chunks, which is what the workspace is sized for.)
  const float per_chunk = 1.0f / fmaxf(wave_sum(total) / (float)a.chunks + (float)round, 1.f);

  int before = 0;
  for (int r0 = 0; r0 < a.n_req; r0 += kTurn) {
    if (a.n_req > kTurn) load(r0);
    int mine = 0;
#pragma unroll
    for (int k = 0; k < HOLD; ++k) mine += count[k] < 0 ? 0 : chunks_of(count[k], per_chunk);
    const int sum = running_sum(mine);
    const uint64_t hit = __ballot(x < before + sum);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      Place p{-1, before + sum - mine, 0, 0, 0};
      bool found = false;
#pragma unroll
      for (int k = 0; k < HOLD; ++k) {  // lane l's requests; the other lanes' result is not read
        const int c = count[k] < 0 ? 0 : chunks_of(count[k], per_chunk);
        if (!found && x < p.first + c) {
          p.r = r0 + lane * HOLD + k;
          p.n = c;
          p.seq = seq[k];
          p.prefix = prefix[k];
          found = true;
        }
        if (!found) p.first += c;
      }
      return {__builtin_amdgcn_readlane(p.r, l), __builtin_amdgcn_readlane(p.first, l), __builtin_amdgcn_readlane(p.n, l),
              __builtin_amdgcn_readlane(p.seq, l), __builtin_amdgcn_readlane(p.prefix, l)};
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return {-1, 0, 0, 0, 0};
}

__device__ __forceinline__ float get_part(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_pair(const float* p) {
  return __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

// Two workgroups a CU leave a wave 256 registers: the two tiles that a wave holds fit for heads
// up to 128; above, they would spill (256: 5.2 ms against 1.96 for 512 requests).
template <int DT, int NC>
__global__ __launch_bounds__(kWaves * 64, NC <= 4 ? 2 : 1) void attn_decode_kernel(AttnArgs a) {
  using S = Shape<NC>;
  constexpr int VD = S::VD, VH = S::VH;
  extern __shared__ float sm_out[];                       // [wave][row][D + 4]
  __shared__ uint64_t sm_addr[kWaves][2][64];
  __shared__ float sm_m[kWaves][kRows], sm_l[kWaves][kRows];
  __shared__ int32_t sm_last;

  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m16 = lane & 15, g = lane >> 4;
  // a workgroup: `heads` neighbouring KV heads, `phases` waves on each
  const int heads_log2 = a.wg_heads >> 1, heads = a.wg_heads;  // 1, 2, 4: 0, 1, 2
  const int phases = kWaves >> heads_log2, phase = wave >> heads_log2, my_head = wave & (heads - 1);
  const int round_log2 = 7 - heads_log2, round = 1 << round_log2;  // phases * kTile
  const int row_groups = (a.group + kRows - 1) / kRows;
  const int units = (int)gridDim.x, unit = (int)blockIdx.x, x_chunk = (int)blockIdx.y;
  const Place at = a.n_req <= 64 ? find_chunk<1>(a, lane, x_chunk, round) : find_chunk<8>(a, lane, x_chunk, round);
  if (at.r < 0) return;
  const int r = at.r;
  const Seen seen = seen_by(a, at.seq, at.prefix);
  const int head_unit = row_groups == 1 ? unit : unit / row_groups;
  const int kv_head = (head_unit << heads_log2) + my_head, row0 = (unit - head_unit * row_groups) * kRows;
  const int rows = min(a.group - row0, kRows);
  const int head0 = kv_head * a.group + row0;
  const int h_off = kv_head * a.D;
  // its chunks are of one length, in whole rounds (the last ones may be empty)
  const int32_t count = seen.keys.count;
  const int32_t each = at.n == 1 ? count : (int32_t)((uint32_t)(count + at.n - 1) / (uint32_t)at.n);
  const int32_t length = (each + round - 1) >> round_log2 << round_log2;
  const int begin = min((x_chunk - at.first) * length, count), end = min(begin + length, count);

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

  const int n_tiles = end > begin + phase * kTile ? (end - begin - phase * kTile + round - 1) >> round_log2 : 0;
  // lane l looks up key l % 32 of the tile: its K page (l < 32) or V page
  const int32_t* table = (lane < 32 ? a.kt : a.vt) + (int64_t)r * a.max_blocks;
  auto tile_begin = [&](int t) { return begin + phase * kTile + t * round; };
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
    if (a.cap_out > kNearCap * kLog2e) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = capped(a, s[i]);
    } else if (a.cap_out != 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = capped_near(a, s[i]);
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
    // reach 2^kRescale (times 2^kWeightLog2, which f16 holds).
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
    const float ms = (m == -INFINITY ? 0.f : m) - kWeightLog2<DT>;
    // The matrix unit takes weights of the storage type. Rounded to it once they would bring as
    // much error as the result's own rounding, so each goes in as two values and two products:
    // loads are what this kernel waits for (512 requests 1889 us, with one product each 1893).
    uint32_t p[4], rest[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = __builtin_amdgcn_exp2f(s[i] - ms);
      l += s[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<DT>(s[2 * i], s[2 * i + 1], &p[i], &rest[i]);
    const uint4 pb = make_uint4(p[0], p[1], p[2], p[3]), rb = make_uint4(rest[0], rest[1], rest[2], rest[3]);
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
        const uint4 v8 = make_uint4(b[0], b[1], b[2], b[3]);
        acc[h][e] = mfma16x16<DT>(v8, pb, mfma16x16<DT>(v8, rb, acc[h][e]));
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

  l = sum32(sum16(l));
  const int heads_q = a.hk * a.group;
  if (phases == 1 && at.n == 1) {  // a head of this wave's alone: straight from the registers
    if (m16 >= rows) return;
    const int head = head0 + m16;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint16_t* o = a.out + (int64_t)r * a.o_ts + (int64_t)head * a.o_hs;
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = h * 128 + (g * 4 + i) * VD;
        if (d >= a.D) continue;
        uint32_t w[VD / 2];
#pragma unroll
        for (int e = 0; e < VD; e += 2)
          w[e / 2] = round2<DT>(seen.bad ? NAN : l == 0.f ? 0.f : acc[h][e][i] * inv,
                                seen.bad ? NAN : l == 0.f ? 0.f : acc[h][e + 1][i] * inv);
        if constexpr (VD == 8) st16(o + d, make_uint4(w[0], w[1], w[2], w[3]));
        else *reinterpret_cast<uint2*>(o + d) = make_uint2(w[0], w[1]);
      }
    if (a.lse && g == 0) a.lse[(int64_t)r * heads_q + head] = seen.bad ? NAN : log_sum<DT>(m, l);
    return;
  }

  // Join the waves of each head. Rows are 4 floats apart from a multiple of 8, so the 16
  // rows' stores meet no bank twice.
  const int stride = a.D + 4;
  if (g == 0) {
    sm_m[wave][m16] = m;
    sm_l[wave][m16] = l;
  }
  if (m16 < rows) {
    float* o = sm_out + (wave * rows + m16) * stride;
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = h * 128 + (g * 4 + i) * VD;
        if (d < a.D) {
#pragma unroll
          for (int e = 0; e < VD; e += 4)
            *reinterpret_cast<float4*>(o + d + e) = make_float4(acc[h][e][i], acc[h][e + 1][i], acc[h][e + 2][i], acc[h][e + 3][i]);
        }
      }
  }
  __syncthreads();
  // A chunk's result: [chunk][query head][m, l, out].
  const int64_t part_row = a.D + 2, part_chunk = heads_q * part_row;
  const int pairs = a.D / 2;
  for (int i = tid; i < heads * rows * pairs; i += kWaves * 64) {
    const int hr = i / pairs, d = (i - hr * pairs) * 2, hw = hr / rows, row = hr - hw * rows;
    float mt = -INFINITY, lt = 0.f, x = 0.f, y = 0.f;
    for (int w = hw; w < kWaves; w += heads) mt = fmaxf(mt, sm_m[w][row]);
    for (int w = hw; w < kWaves; w += heads) {
      const float f = part_weight(sm_m[w][row], mt);
      const float2 o = *reinterpret_cast<const float2*>(sm_out + (w * rows + row) * stride + d);
      lt += f * sm_l[w][row];
      x += f * o.x;
      y += f * o.y;
    }
    const int hq = ((head_unit << heads_log2) + hw) * a.group + row0 + row;
    if (at.n == 1) {
      const float inv = lt == 0.f ? 0.f : 1.0f / lt;
      *reinterpret_cast<uint32_t*>(a.out + (int64_t)r * a.o_ts + (int64_t)hq * a.o_hs + d) =
          round2<DT>(seen.bad ? NAN : lt == 0.f ? 0.f : x * inv, seen.bad ? NAN : lt == 0.f ? 0.f : y * inv);
      if (a.lse && d == 0) a.lse[(int64_t)r * heads_q + hq] = seen.bad ? NAN : log_sum<DT>(mt, lt);
    } else {
      float* part = a.part + (int64_t)x_chunk * part_chunk + hq * part_row;
      put_pair(part + 2 + d, x, y);
      if (d == 0) put_pair(part, mt, lt);
    }
  }
  if (at.n == 1) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // stored, before this workgroup counts
  __syncthreads();
  // Requests before this one hold at.first - r chunks more than they are: the cut requests'
  // counters are apart and there are no more than chunks aimed for.
  if (tid == 0) {
    int32_t* counter = a.counters + (at.first - r) * units + unit;
    const int32_t n = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sm_last = n == at.n - 1;
    if (n == at.n - 1) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
  }
  __syncthreads();
  if (!__builtin_amdgcn_readfirstlane(sm_last)) return;
  // rows of all the workgroup's heads, a wave to each in turn
  for (int i = wave; i < heads * rows; i += kWaves) {
    const int hq = ((head_unit << heads_log2) + i / rows) * a.group + row0 + i % rows;
    const float* part = a.part + (int64_t)at.first * part_chunk + hq * part_row;
    float mt = -INFINITY;
    for (int c = lane; c < at.n; c += 64) mt = fmaxf(mt, get_part(part + c * part_chunk));
    mt = max32(max16(mt));
    for (int d = 8; d; d >>= 1) mt = fmaxf(mt, __shfl_xor(mt, d));
    constexpr int kPairs = NC <= 4 ? 1 : 2;  // pairs of dimensions of a lane
    float o[kPairs][2] = {}, lt = 0.f;
    for (int c0 = 0; c0 < at.n; c0 += 64) {
      const float* mine = part + min(c0 + lane, at.n - 1) * part_chunk;
      const float f = part_weight(get_part(mine), mt), lf = f * get_part(mine + 1);
      lt += c0 + lane < at.n ? lf : 0.f;
      const int many = min(64, at.n - c0);
      for (int c = 0; c < many; c += 8) {  // 8 chunks' loads in flight
        uint64_t v[8][kPairs];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int e = 0; e < kPairs; ++e)
            v[j][e] = get_pair(part + (c0 + min(c + j, many - 1)) * part_chunk + 2 + min(lane * 2 + e * 128, a.D - 2));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (c + j >= many) break;
          const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), c + j));
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            o[e][0] += w * __uint_as_float((uint32_t)v[j][e]);
            o[e][1] += w * __uint_as_float((uint32_t)(v[j][e] >> 32));
          }
        }
      }
    }
    for (int d = 32; d; d >>= 1) lt += __shfl_xor(lt, d);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      const int d = lane * 2 + e * 128;
      if (d < a.D)
        *reinterpret_cast<uint32_t*>(a.out + (int64_t)r * a.o_ts + (int64_t)hq * a.o_hs + d) =
            lt == 0.f ? 0u : round2<DT>(o[e][0] / lt, o[e][1] / lt);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)r * heads_q + hq] = log_sum<DT>(mt, lt);
  }
}

template <int DT, int NC>
hipError_t launch_nc(const AttnArgs& a, dim3 grid, hipStream_t s, const LaunchEvents& ev) {
  const int rows = a.group < kRows ? a.group : kRows;
  const size_t lds = sizeof(float) * kWaves * rows * (a.D + 4);
  if (lds > 48 * 1024) {  // with the static part past the 64 KiB a launch has by default
    const hipError_t e = hipFuncSetAttribute((const void*)attn_decode_kernel<DT, NC>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipExtLaunchKernelGGL((attn_decode_kernel<DT, NC>), grid, dim3(kWaves * 64), lds, s, ev.start, ev.stop, 0, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  const int units = a.hk / a.wg_heads * ((a.group + kRows - 1) / kRows);
  // No request has more chunks than rounds of keys.
  const int64_t round = kTile * (kWaves / a.wg_heads);
  const int64_t most = (a.max_len + round - 1) / round, all = (int64_t)a.n_req * (most > 1 ? most : 1);
  const int64_t chunks = all < (int64_t)a.n_req + a.chunks ? all : (int64_t)a.n_req + a.chunks;
  if (chunks * units * kWaves * 64 >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)units, (unsigned)chunks);  // neighbouring heads in neighbouring workgroups
  const int nc = (a.D + 31) / 32;
  return nc <= 2   ? launch_nc<DT, 2>(a, grid, s, ev)
         : nc == 3 ? launch_nc<DT, 3>(a, grid, s, ev)
         : nc == 4 ? launch_nc<DT, 4>(a, grid, s, ev)
         : nc <= 6 ? launch_nc<DT, 6>(a, grid, s, ev)
                   : launch_nc<DT, 8>(a, grid, s, ev);
}

}  // namespace

hipError_t launch_attn_decode(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
