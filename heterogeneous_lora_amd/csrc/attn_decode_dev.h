// The kernel of attention of one new token per request (attn_decode.hip: a cache of 16 bits a
// value; attn4_decode.hip: of 4).
#pragma once

#include "attn_dev.h"
#include "attn4_dev.h"

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

// What a lane holds of a tile: K's rows and V's dimensions of it in the cache's form. In 4 bits
// (NC: the head's groups) 8 values are a word; `steps`: those of the lane's key, K's or V's.
template <int NC, int BITS>
struct Tile {
  uint4 k[2][NC];
  uint32_t v[8][Shape<NC>::VH][Shape<NC>::VD / 2];
};
template <int NC>
struct Tile<NC, 4> {
  uint32_t k[2][NC];
  uint32_t v[8][Shape<NC>::VH];
  uint32_t steps[NC <= 4 ? 1 : 2];
};


// Two workgroups a CU leave a wave 256 registers: the two tiles that a wave holds fit for heads
// up to 128; above, they would spill (256: 5.2 ms against 1.96 for 512 requests).
template <int DT, int NC, int BITS>
__global__ __launch_bounds__(kWaves * 64, BITS == 4 ? (NC <= 3 ? 4 : NC == 4 ? 3 : 2) : NC <= 4 ? 2 : 1) void attn_decode_kernel(AttnArgs a) {
  using S = Shape<NC>;
  constexpr int VD = S::VD, VH = S::VH;
  constexpr bool k4 = BITS == 4;
  constexpr int MT = k4 ? SLORA_F16 : DT;  // the products' type
  constexpr bool kTwo = !k4 || DT == SLORA_F16;  // weights as two values each
  constexpr int kStepWords = NC <= 4 ? 1 : 2;
  extern __shared__ float sm_out[];                       // [wave][row][D + 4]
  __shared__ uint64_t sm_addr[kWaves][2][64];
  __shared__ float sm_m[kWaves][kRows], sm_l[kWaves][kRows];
  __shared__ int32_t sm_last;
  __shared__ __attribute__((aligned(16))) uint32_t sm_steps[k4 ? kWaves : 1][k4 ? 64 : 1][kStepWords];

  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m16 = lane & 15, g = lane >> 4;
  // a workgroup: `heads` neighbouring KV heads, `phases` waves on each
  const int heads_log2 = a.wg_heads >> 1, heads = a.wg_heads;  // 1, 2, 4: 0, 1, 2
  const int phases = kWaves >> heads_log2, phase = wave >> heads_log2, my_head = wave & (heads - 1);
  const int round_log2 = 7 - heads_log2, round = 1 << round_log2;  // phases * kTile
  const int row_groups = (a.group + kRows - 1) / kRows;
  // (of 4 bits a chunk's workgroups go to one XCD: neighbouring heads share lines)
  const int xcd_log2 = k4 ? a.xcd_log2 : 0, xcd = k4 ? (int)blockIdx.x & ((1 << xcd_log2) - 1) : 0;
  const int units = (int)gridDim.x >> xcd_log2, unit = (int)blockIdx.x >> xcd_log2;
  const int x_chunk = ((int)blockIdx.y << xcd_log2) + xcd;
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
  float q_row = 1.f;  // of 4 bits, bf16: what the row is divided by to be in f16
  {
    const uint16_t* qp = a.q + (int64_t)r * a.q_ts + (int64_t)(head0 + min(m16, rows - 1)) * a.q_hs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = c * 32 + g * 8;
      q[c] = ld16((k4 ? c + 1 < NC : c < S::kFull) || d < a.D ? qp + d : kAttnFill.zero);
    }
    if constexpr (k4 && DT == SLORA_BF16) {
      float most = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) most = fmaxf(most, largest_bf16(q[c]));
      const int up = f16_shift(max32(max16(most)));
      q_row = ldexpf(1.f, -up);
#pragma unroll
      for (int c = 0; c < NC; ++c) q[c] = bf16_to_f16(q[c], up);
    }
  }
  const float slope = a.slopes ? a.slopes[head0 + min(m16, rows - 1)] * kLog2e : 0.f;

  f32x4 acc[VH][VD];
#pragma unroll
  for (int h = 0; h < VH; ++h)
#pragma unroll
    for (int e = 0; e < VD; ++e) acc[h][e] = {0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  // Of 4 bits: where the lane's dimensions of V begin in a key's codes (those past the head's
  // groups make dimensions that are dropped: any will do), which byte of its steps is theirs.
  int v_at[VH];
#pragma unroll
  for (int h = 0; h < VH; ++h) {
    const int p = min(VD == 8 ? h * 16 + m16 : m16 >> 1, NC * 4 - 1);
    v_at[h] = ((p & 3) * NC + (p >> 2)) * 4 + (VD == 8 ? 0 : (m16 & 1) * 2);
  }
  const uint32_t v_group = VD == 8 ? m16 >> 2 : m16 >> 3, v_step = 0x0c040c00u + v_group * 0x10001u;

  const int n_tiles = end > begin + phase * kTile ? (end - begin - phase * kTile + round - 1) >> round_log2 : 0;
  // lane l looks up key l % 32 of the tile: its K page (l < 32) or V page
  const int32_t* table = (lane < 32 ? a.kt : a.vt) + (int64_t)r * a.max_blocks;
  auto tile_begin = [&](int t) { return begin + phase * kTile + t * round; };
  auto page_of = [&](int t) -> int32_t {
    const int i = min(tile_begin(t) + (lane & 31), end - 1);
    return table[div_tpp(a, (uint32_t)seen.keys.key(i))];
  };
  auto put_addr = [&](int t, int32_t page, Tile<NC, BITS>& x) {
    const int i = tile_begin(t) + (lane & 31);
    if constexpr (k4) {
      const Key4 k = key4_addr(a, page, seen.keys.key(min(i, end - 1)), kv_head);
      sm_addr[wave][t & 1][lane] = i < end && k.good ? k.codes : fill_addr<DT>(true);
      load_steps<NC>(i >= end ? fill_addr<DT>(true) : k.good ? k.steps : (uint64_t)kAttnFill.nan_steps, x.steps);
    } else {
      const uint64_t p = key_addr(a, page, seen.keys.key(min(i, end - 1)), h_off, fill_addr<DT>(false));
      sm_addr[wave][t & 1][lane] = i < end ? p : fill_addr<DT>(true);
    }
  };
  auto fetch = [&](int t, Tile<NC, BITS>& x) {
    const uint64_t* ad = sm_addr[wave][t & 1];
    if constexpr (k4) {
#pragma unroll
      for (int u = 0; u < 2; ++u) load_words<NC>(ad[(m16 >> 2) * 8 + u * 4 + (m16 & 3)] + g * NC * 4, x.k[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < VH; ++h) x.v[i][h] = load_codes<VD>(ad[32 + g * 8 + i] + v_at[h]);
    } else {
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
    }
  };
  // addresses are written and read by the lanes of one wave, in order
  auto fence = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); __builtin_amdgcn_wave_barrier(); };
  auto compute = [&](int t, const Tile<NC, BITS>& x) {
    const int i0 = tile_begin(t) + g * 8;
    float s[8];
    if constexpr (k4) {
      fence();
#pragma unroll
      for (int w = 0; w < kStepWords; ++w) sm_steps[wave][lane][w] = x.steps[w];
      fence();
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x4 c4 = {0.f, 0.f, 0.f, 0.f};
      if constexpr (k4) {
        uint32_t st[kStepWords];
#pragma unroll
        for (int w = 0; w < kStepWords; ++w) st[w] = sm_steps[wave][(m16 >> 2) * 8 + u * 4 + (m16 & 3)][w];
#pragma unroll
        for (int c = 0; c < NC; ++c) c4 = mfma16x16<MT>(values8(x.k[u][c], step_twice(st[c >> 2], c & 3)), q[c], c4);
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) c4 = mfma16x16<DT>(x.k[u][c], q[c], c4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[u * 4 + i] = c4[i];
    }
    if constexpr (k4 && DT == SLORA_BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] *= q_row;
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
    const float ms = (m == -INFINITY ? 0.f : m) - kWeightLog2<MT>;
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
    for (int i = 0; i < 4; ++i) {
      if constexpr (kTwo) split2<MT>(s[2 * i], s[2 * i + 1], &p[i], &rest[i]);
      else p[i] = round2<MT>(s[2 * i], s[2 * i + 1]);
    }
    const uint4 pb = make_uint4(p[0], p[1], p[2], p[3]);
    const uint4 rb = kTwo ? make_uint4(rest[0], rest[1], rest[2], rest[3]) : pb;
    uint32_t st[kStepWords][8];
    if constexpr (k4) {
#pragma unroll
      for (int w = 0; w < kStepWords; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) st[w][i] = sm_steps[wave][32 + g * 8 + i][w];
    }
#pragma unroll
    for (int h = 0; h < VH; ++h) {
      // two keys' codes of a dimension in a byte, even and odd dimensions, and the two steps
      uint32_t even[4], odd[4];
      half2_t step[4];
      if constexpr (k4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x0 = x.v[2 * i][h], x1 = x.v[2 * i + 1][h];
          even[i] = (x0 & 0x0f0f0f0fu) | (x1 << 4 & 0xf0f0f0f0u);
          odd[i] = (x0 >> 4 & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u);
          const int w = h < kStepWords ? h : 0;
          step[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(st[w][2 * i + 1], st[w][2 * i], v_step) << 7);
        }
      }
#pragma unroll
      for (int e = 0; e < VD; ++e) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (k4) {
            b[i] = values2(e & 1 ? odd[i] : even[i], e >> 1, step[i]);
          } else {
            const int w = e >> 1;
            b[i] = e & 1 ? pair_hi(x.v[2 * i][h][w], x.v[2 * i + 1][h][w])
                         : pair_lo(x.v[2 * i][h][w], x.v[2 * i + 1][h][w]);
          }
        }
        const uint4 v8 = make_uint4(b[0], b[1], b[2], b[3]);
        acc[h][e] = mfma16x16<MT>(v8, pb, kTwo ? mfma16x16<MT>(v8, rb, acc[h][e]) : acc[h][e]);
      }
    }
  };
  if (n_tiles > 0) {
    Tile<NC, BITS> x0, x1;
    put_addr(0, page_of(0), x0);
    int32_t next = page_of(1);
    fence();
    fetch(0, x0);
    auto step = [&](int t, Tile<NC, BITS>& cur, Tile<NC, BITS>& nxt) {
      if (t + 1 < n_tiles) {
        fence();
        put_addr(t + 1, next, nxt);
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
    if (a.lse && g == 0) a.lse[(int64_t)r * heads_q + head] = seen.bad ? NAN : log_sum<MT>(m, l);
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
      if (a.lse && d == 0) a.lse[(int64_t)r * heads_q + hq] = seen.bad ? NAN : log_sum<MT>(mt, lt);
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
    if (a.lse && lane == 0) a.lse[(int64_t)r * heads_q + hq] = log_sum<MT>(mt, lt);
  }
}

}  // namespace
}  // namespace slora
