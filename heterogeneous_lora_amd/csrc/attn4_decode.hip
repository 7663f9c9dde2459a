// Attention of one new token per request over a cache in 4 bits (slora_attn4_decode).
//
//   s_j = q . k_j (scaled, capped, biased),  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Bound by the bytes of K and V: 68 a vector of 128 dimensions. Products and softmax are those of
// attn_decode.hip, in f16 (step times level is exact there); codes become values on their way to
// the matrix instructions, 2 instructions for 2 of them.
//
// With few keys (Decode4) the kernel is attn_decode.hip's, a wave a head, chunks and their join as
// there. With many it would wait for its loads' addresses: a head's vector is half a line, 16 keys'
// words in a register are 64 accesses of the address unit, and tokens' rows begin anywhere. So
// attn4_decode_kernel
// - takes neighbouring heads one after the other for the same 32 keys, as many as make up to 16 rows
//   with the query heads that share them: rows of the matrix instructions that a single head leaves
//   empty hold the other heads' scores and results. Of the products with a head's K its own rows'
//   scores are kept; for those with its V the other rows' weights are zero;
// - reads straight to LDS, 4 lanes a key, several pieces ahead (register loads in the operands'
//   order: 952 us for 512 requests of 40 heads, 2 heads' pieces in flight 920);
// - gives every workgroup one span of all requests' keys, of one length (a chunk of a request to a
//   workgroup, 2048 in all: 773 us).
//
// 512 requests of 64 to 2048 keys, 40 heads of 128: 0.69 ms (4.3 TB/s); three of 100000 to 131072
// keys, 64 query heads on 8: 115 us; 64 with a window of 1024: 25 us.
#include "attn4_dev.h"
#include "attn_decode_dev.h"

namespace slora {
namespace {

// NC: the head's groups of 32 dimensions. ST: runs of 32 keys a wave takes at once (Decode4).
template <int NC, int ST>
struct SpanShape {
  static constexpr int VD = NC <= 2 ? 4 : 8;  // dimensions of V a lane takes (16 lanes cover it in VH turns)
  static constexpr int VH = NC <= 4 ? 1 : 2;
  static constexpr int kStepBytes = NC <= 2 ? NC : NC <= 4 ? 4 : 8;
  static constexpr int kStepWords = NC <= 4 ? 1 : 2;
  static constexpr int kKeys = 32 * ST;  // of a wave's tile
  // A piece is a head's codes of 32 keys. Two workgroups a CU leave a wave 20 KB of LDS; pieces on
  // their way while one is worked on:
  static constexpr int kPiece = 2048 * ((NC + 3) / 4), kLoads = kPiece / 1024;
  static constexpr int kAhead = NC > 4 ? 2 : ST == 1 ? 6 : 4, kRing = kAhead + 1;
  // a key's steps, of K or V, in LDS; a tile's
  static constexpr int kKeySteps = 64 / ST, kSteps = kKeys * kKeySteps;
  static constexpr int kBytes = kRing * kPiece + 2 * kSteps;
};

// Place of a tile's key in LDS, among 32: so that the 16 keys that a K operand takes lie together,
// and the 4 of which 16 lanes each take a word of V on different banks.
__device__ __forceinline__ int slot_of(int key) { return (key & 7) * 4 + (key >> 3); }
__device__ __forceinline__ int key_of_slot(int slot) { return (slot & 3) * 8 + (slot >> 2); }

// Whether some byte of w is above kMaxStep: a step that is no number.
__device__ __forceinline__ bool bad_step(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x1d1d1d1du) & w & 0x80808080u;
}
__device__ __forceinline__ uint32_t without_bad(uint32_t w) {
  const uint32_t bad = ((w & 0x7f7f7f7fu) + 0x1d1d1d1du) & w & 0x80808080u;
  return w & ~((bad >> 7) * 255u);
}

// A workgroup's share of the call: all requests' keys, in rounds (one at least for each request),
// one after the other and cut into spans of one length.
struct Span {
  int r;              // its first request, -1: none
  int32_t off;        // the round of that request it begins with
  int64_t length;     // rounds of a span
};
__device__ __forceinline__ int32_t rounds_of(const AttnArgs& a, int32_t seq, int32_t prefix, int round_log2) {
  return max((seen_by(a, seq, prefix).keys.count + (1 << round_log2) - 1) >> round_log2, 1);
}
// A lane takes HOLD requests at a time, all their loads in flight at once, and keeps them where one
// turn covers the call.
template <int HOLD>
__device__ __forceinline__ Span find_span(const AttnArgs& a, int lane, int x, int round_log2) {
  constexpr int kTurn = 64 * HOLD;
  int32_t rounds[HOLD];
  auto load = [&](int r0) {
    int32_t seq[HOLD], prefix[HOLD];
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
      const int r = min(r0 + lane * HOLD + k, a.n_req - 1);
      seq[k] = a.seq[r];
      prefix[k] = a.prefix ? a.prefix[r] : 0;
    }
    int64_t sum = 0;
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
      rounds[k] = r0 + lane * HOLD + k < a.n_req ? rounds_of(a, seq[k], prefix[k], round_log2) : 0;
      sum += rounds[k];
    }
    return sum;
  };
  int64_t mine = 0, total = 0;
  for (int r0 = 0; r0 < a.n_req; r0 += kTurn) total += mine = load(r0);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  const int64_t length = (total + a.spans - 1) / a.spans, start = length * x;
  if (start >= total) return {-1, 0, 0};
  int64_t before = 0;
  for (int r0 = 0;; r0 += kTurn) {
    if (a.n_req > kTurn) mine = load(r0);
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t y = __shfl_up(sum, d);
      sum += lane >= d ? y : 0;
    }
    const uint64_t hit = __ballot(start < before + sum);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      int64_t at = before + sum - mine;  // of lane l's requests; the other lanes' result is not read
      int r = r0 + lane * HOLD;
#pragma unroll
      for (int k = 0; k + 1 < HOLD; ++k)
        if (start >= at + rounds[k] && r == r0 + lane * HOLD + k) {
          at += rounds[k];
          ++r;
        }
      return {__builtin_amdgcn_readlane(r, l), __builtin_amdgcn_readlane((int)(start - at), l), length};
    }
    before += __shfl(sum, 63);
  }
}

template <int DT, int NC, int ST>
__global__ __launch_bounds__(kWaves * 64, 2) void attn4_decode_kernel(AttnArgs a) {
  using S = SpanShape<NC, ST>;
  constexpr int VD = S::VD, VH = S::VH, kStepWords = S::kStepWords, kKeys = S::kKeys, kPiece = S::kPiece;
  constexpr int MT = SLORA_F16;                // the products' type
  constexpr bool kTwo = DT == SLORA_F16;       // weights as two values each
  // [wave]: pieces of codes, steps; then the join's floats
  extern __shared__ __attribute__((aligned(16))) uint8_t sm[];
  __shared__ uint64_t sm_addr[kWaves][ST][64], sm_step_addr[kWaves][2][kKeys];  // [K's slots, then V's]
  __shared__ int32_t sm_page[kWaves][ST][64];
  __shared__ float sm_m[kWaves][kRows], sm_l[kWaves][kRows];

  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m16 = lane & 15, g = lane >> 4;
  // a workgroup: 1, 2 or 4 units of heads, its waves in turn on the tiles of each
  const int units_log2 = a.wg_units >> 1, wg_units = a.wg_units;
  const int phases = kWaves >> units_log2, phase = wave >> units_log2;
  const int round_log2 = 7 - units_log2 + (ST >> 1), round = 1 << round_log2;  // phases * kKeys
  // a span's workgroups go to one XCD, where they share what lines they share
  const int xcd_log2 = a.xcd_log2;
  const int x = ((int)blockIdx.y << xcd_log2) + ((int)blockIdx.x & ((1 << xcd_log2) - 1));
  const Span span = a.n_req <= 64 ? find_span<1>(a, lane, x, round_log2) : find_span<8>(a, lane, x, round_log2);
  if (span.r < 0) return;
  // a unit: wave_heads KV heads, or 16 rows of one
  const int row_groups = (a.group + kRows - 1) / kRows, unit0 = (int)(blockIdx.x >> xcd_log2) << units_log2;
  struct Unit {
    int kv0, row0, heads, rows;
    __device__ int cols() const { return heads * rows; }
  };
  auto unit_of = [&](int unit) {
    const int u = row_groups == 1 ? unit : unit / row_groups;
    Unit x;
    x.kv0 = u * a.wave_heads;
    x.row0 = (unit - u * row_groups) * kRows;
    x.heads = max(min(a.wave_heads, a.hk - x.kv0), 0);  // (none: a wave too many)
    x.rows = min(a.group - x.row0, kRows);
    return x;
  };
  auto query_head = [&](const Unit& u, int c) { return (u.kv0 + c / u.rows) * a.group + u.row0 + c % u.rows; };
  const Unit mine = unit_of(unit0 + (wave & (wg_units - 1)));
  const int kv0 = mine.kv0, heads = mine.heads, rows = mine.rows, cols = mine.cols();
  // this lane's row: of head my_head of the wave's, of query head my_q
  const int my_head = m16 / rows, my_q = heads ? query_head(mine, min(m16, cols - 1)) : 0;
  const float slope = a.slopes ? a.slopes[my_q] * kLog2e : 0.f;

  // The part of a request that is worked on: keys begin .. end of those it sees.
  int r = span.r;
  Seen seen;
  int begin, end, first_key, n_tiles;
  const int32_t* table;  // (lane l looks up slot l % 32 of a run: its K page, l < 32, or V page)
  uint4 q[NC];           // as the B operand: lane l holds dimensions 32 c + 8 (l / 16) .. + 7 of row l % 16
  float q_row = 1.f;     // bf16: what the row is divided by to be in f16
  f32x4 acc[VH][VD];
  float m, l;
  uint32_t bad_groups;  // of the row's head: some V that it sees is no number there
  auto begin_part = [&](int32_t off, int32_t rounds) {
    begin = off << round_log2;
    end = min(begin + (rounds << round_log2), seen.keys.count);
    first_key = begin + phase * kKeys;
    n_tiles = heads && end > first_key ? (end - first_key + round - 1) >> round_log2 : 0;
    table = (lane < 32 ? a.kt : a.vt) + (int64_t)r * a.max_blocks;
    const uint16_t* qp = a.q + (int64_t)r * a.q_ts + (int64_t)my_q * a.q_hs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = c * 32 + g * 8;
      q[c] = ld16(c + 1 < NC || d < a.D ? qp + d : kAttnFill.zero);
    }
    if constexpr (DT == SLORA_BF16) {
      float most = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) most = fmaxf(most, largest_bf16(q[c]));
      const int up = f16_shift(max32(max16(most)));
      q_row = ldexpf(1.f, -up);
#pragma unroll
      for (int c = 0; c < NC; ++c) q[c] = bf16_to_f16(q[c], up);
    }
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
      for (int e = 0; e < VD; ++e) acc[h][e] = {0.f, 0.f, 0.f, 0.f};
    m = -INFINITY;
    l = 0.f;
    bad_groups = 0;
  };
  // addresses and steps are written and read by the lanes of one wave, in order
  auto fence = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); __builtin_amdgcn_wave_barrier(); };
  // Piece p: head p / ST, run p % ST. No fewer than are on their way at once (those past the heads
  // are the last one's again, and not used).
  const int n_used = heads * ST, n_pieces = max(n_used, S::kAhead);
  const int step0 = kv0 * S::kStepBytes, skip = step0 & 15;  // the first head's steps begin inside 16 bytes
  const int step_units = (skip + heads * S::kStepBytes + 15) >> 4;
  uint8_t* const codes = sm + wave * S::kBytes;
  uint8_t* const steps = codes + S::kRing * kPiece;
  const uint32_t lds_codes = lds_offset(codes), lds_steps = lds_offset(steps), lds_page = lds_offset(&sm_page[wave][0][0]);
  // Everything that is read comes straight to LDS, 16 bytes a lane (page ids 4), and is waited for
  // by how many loads may still be on their way: they arrive in order.
  auto tile_begin = [&](int t) { return first_key + t * round; };
  auto index_of = [&](int t, int j) { return tile_begin(t) + j * 32 + key_of_slot(lane & 31); };
  auto load_pages = [&](int t) {
#pragma unroll
    for (int j = 0; j < ST; ++j) {
      const int32_t key = seen.keys.key(min(index_of(t, j), end - 1));
      load_word_to_lds((uint64_t)(table + div_tpp(a, (uint32_t)key)), lds_page + j * 256);
    }
  };
  // Addresses of a tile's keys (past the last one: the last one's, with steps of 0).
  auto put_addr = [&](int t) {
#pragma unroll
    for (int j = 0; j < ST; ++j) {
      const int i = index_of(t, j);
      const Key4 k = key4_addr(a, sm_page[wave][j][lane], seen.keys.key(min(i, end - 1)), 0);
      sm_addr[wave][j][lane] = k.good ? k.codes + (uint32_t)(kv0 * 16 * NC) : (uint64_t)kNoCodes;
      sm_step_addr[wave][lane >> 5][j * 32 + (lane & 31)] = i >= end ? fill_addr<DT>(true)
                                                            : k.good ? k.steps + (uint32_t)(step0 - skip)
                                                                     : (uint64_t)kAttnFill.nan_steps;
    }
    fence();
  };
  // A tile's steps of K (v 0) or V (1), those of the heads in units of 16 bytes.
  auto load_steps = [&](int v) {
    constexpr int kLanes = S::kKeySteps / 16;  // of a key
    const int unit = min(lane % kLanes, step_units - 1) * 16;
#pragma unroll
    for (int n = 0; n < S::kSteps / 1024; ++n)
      load_to_lds(sm_step_addr[wave][v][(n * 64 + lane) / kLanes] + unit, lds_steps + v * S::kSteps + n * 1024);
  };
  // A piece of K or V: 4 lanes a key.
  auto load_piece = [&](int p, int v, int place) {
    const uint64_t* ad = sm_addr[wave][p % ST] + v * 32 + (lane >> 2);
    const uint32_t head = (uint32_t)min(p / ST, heads - 1) * (16 * NC);
#pragma unroll
    for (int n = 0; n < S::kLoads; ++n)
      load_to_lds(ad[n % 2 * 16] + head + min((n / 2 * 4 + (lane & 3)) * 16, 16 * NC - 16),
                  lds_codes + place * kPiece + n * 1024);
  };
  auto steps_at = [&](int v, int j, int h, int slot) {
    return steps + v * S::kSteps + (j * 32 + slot) * S::kKeySteps + skip + h * S::kStepBytes;
  };
  const int k_slot = (m16 & 3) * 4 + (m16 >> 2);  // of the first 16 keys' operand; 16 on for the other
  int k_at[NC];                                   // the lane's words of a key of K in a piece
#pragma unroll
  for (int c = 0; c < NC; ++c) k_at[c] = ((g * NC + c) >> 4) * 2048 + ((g * NC + c) & 15) * 4;
  // The lane's dimensions of V: word (or half of one) m16 of a key's codes, 16 on in the next turn
  // (past the head's groups any will do: what they make is dropped).
  auto v_word = [&](int h, int row) { return VD == 8 ? h * 16 + row : row >> 1; };
  int v_at[VH], v_group[VH];
#pragma unroll
  for (int h = 0; h < VH; ++h) {
    const int x = min(v_word(h, m16), 4 * NC - 1);
    v_at[h] = (x >> 4) * 2048 + (x & 15) * 4 + (VD == 8 ? 0 : (m16 & 1) * 2);
    v_group[h] = x % NC;
  }
  // The first dimension that row `row` of turn h stands for, and its group.
  auto dim_of = [&](int h, int row) {
    const int x = v_word(h, row);
    return x < 4 * NC ? x % NC * 32 + x / NC * 8 + (VD == 8 ? 0 : (row & 1) * 4) : 256;
  };
  float s[ST][8] = {};
  auto scores = [&](int head, int j, int place) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* x = codes + place * kPiece + (u * 16 + k_slot) * 64;
      const uint8_t* y = steps_at(0, j, head, u * 16 + k_slot);
      uint32_t st[kStepWords], w[NC];
      if constexpr (NC == 1) st[0] = *y;
      else if constexpr (NC == 2) st[0] = *(const uint16_t*)y;
      else {
#pragma unroll
        for (int i = 0; i < kStepWords; ++i) st[i] = ((const uint32_t*)y)[i];
      }
      if constexpr (NC == 4) {
        const uint4 z = *(const uint4*)(x + g * 16);
        w[0] = z.x; w[1] = z.y; w[2] = z.z; w[3] = z.w;
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) w[c] = *(const uint32_t*)(x + k_at[c]);
      }
      f32x4 c4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) c4 = mfma16x16<MT>(values8(w[c], step_twice(st[c >> 2], c & 3)), q[c], c4);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][u * 4 + i] = my_head == head ? c4[i] : s[j][u * 4 + i];
    }
  };
  uint32_t w[ST][4], rest[ST][4];
  auto weights = [&](int t) {
    const int i0 = tile_begin(t) + g * 8;
    float x[ST][8];
#pragma unroll
    for (int j = 0; j < ST; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = s[j][i] * q_row;
    auto each_score = [&](auto f) {
#pragma unroll
      for (int j = 0; j < ST; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = f(x[j][i], i0 + j * 32 + i);
    };
    if (a.cap_out > kNearCap * kLog2e) each_score([&](float y, int) { return capped(a, y); });
    else if (a.cap_out != 0.f) each_score([&](float y, int) { return capped_near(a, y); });
    else each_score([&](float y, int) { return y * a.scale2; });
    if (a.slopes) each_score([&](float y, int i) { return y + slope * (float)(seen.keys.key(i) - (seen.n - 1)); });
    if (tile_begin(t) + kKeys > end) each_score([&](float y, int i) { return i < end ? y : -INFINITY; });
    float mx = x[0][0];
    each_score([&](float y, int) {
      mx = fmaxf(mx, y);
      return y;
    });
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
    each_score([&](float y, int) {
      y = __builtin_amdgcn_exp2f(y - ms);
      l += y;
      return y;
    });
    // f16 results: two values a weight, as one would bring as much error as the result's own
    // rounding; bf16's has bits to spare.
#pragma unroll
    for (int j = 0; j < ST; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kTwo) split2<MT>(x[j][2 * i], x[j][2 * i + 1], &w[j][i], &rest[j][i]);
        else w[j][i] = round2<MT>(x[j][2 * i], x[j][2 * i + 1]);
      }
  };
  auto add_values = [&](int head, int j, int place) {
    const bool mine = my_head == head;
    auto of_head = [&](const uint32_t (&y)[4]) { return make_uint4(mine ? y[0] : 0, mine ? y[1] : 0, mine ? y[2] : 0, mine ? y[3] : 0); };
    const uint4 b = of_head(w[j]);
    uint4 b_rest;
    if constexpr (kTwo) b_rest = of_head(rest[j]);
    const uint8_t* x = codes + place * kPiece + g * 64;     // key i of the lane's 8: slot 4 i + g
    const uint8_t* y = steps_at(1, j, head, g);
#pragma unroll
    for (int h = 0; h < VH; ++h) {
      // two keys' codes of a dimension in a byte, even and odd dimensions, and the two steps
      uint32_t even[4], odd[4];
      half2_t step[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t c[2], st[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t* z = x + (2 * i + e) * 256 + v_at[h];
          c[e] = VD == 8 ? *(const uint32_t*)z : *(const uint16_t*)z;
          st[e] = y[(2 * i + e) * 4 * S::kKeySteps + v_group[h]];
        }
        even[i] = (c[0] & 0x0f0f0f0fu) | (c[1] << 4 & 0xf0f0f0f0u);
        odd[i] = (c[0] >> 4 & 0x0f0f0f0fu) | (c[1] & 0xf0f0f0f0u);
        step[i] = __builtin_bit_cast(half2_t, st[0] << 7 | st[1] << 23);
      }
#pragma unroll
      for (int e = 0; e < VD; ++e) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = values2(e & 1 ? odd[i] : even[i], e >> 1, step[i]);
        const uint4 v8 = make_uint4(v[0], v[1], v[2], v[3]);
        if constexpr (kTwo) acc[h][e] = mfma16x16<MT>(v8, b_rest, acc[h][e]);
        acc[h][e] = mfma16x16<MT>(v8, b, acc[h][e]);
      }
    }
  };
  // A step of V that is no number would reach the other heads' rows (0 times a NaN): such steps are
  // noted for the rows of their head and made 0.
  auto take_bad = [&] {
    uint4* const vecs = (uint4*)(steps + S::kSteps);
    constexpr int kVecs = S::kSteps / 1024;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint4 x = vecs[i * 64 + lane];
      bad = bad || bad_step(x.x) || bad_step(x.y) || bad_step(x.z) || bad_step(x.w);
    }
    if (!__any(bad)) return;
#pragma unroll 1
    for (int i = 0; i < kKeys; ++i) {
      const uint8_t* y = steps_at(1, i >> 5, min(my_head, heads - 1), i & 31);
      for (int c = 0; c < NC; ++c) bad_groups |= y[c] > kMaxStep ? 1u << c : 0u;
    }
    fence();
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint4 x = vecs[i * 64 + lane];
      vecs[i * 64 + lane] = make_uint4(without_bad(x.x), without_bad(x.y), without_bad(x.z), without_bad(x.w));
    }
    fence();
  };

  // Loads arrive in the order they were asked for. A piece is there when kAhead - 1 pieces' loads
  // are on their way, and with it what was asked for before it: a tile's steps of K before its
  // first piece, of V (and the next tile's page ids) before kAhead of its pieces of K.
  auto work = [&] {
    if (n_tiles <= 0) return;
    load_pages(0);
    landed();
    put_addr(0);
    load_steps(0);
    for (int i = 0; i < S::kAhead; ++i) load_piece(i, 0, i);
    int place = 0, place_next = S::kAhead;  // of the piece worked on, of the one that is loaded
    auto after = [](int x) { return x == S::kAhead ? 0 : x + 1; };
    auto wait = [] { some_landed<(S::kAhead - 1) * S::kLoads>(); };
    for (int t = 0; t < n_tiles; ++t) {
      load_steps(1);
      load_pages(t + 1);
      auto k_step = [&](int p, int head, int j) {
        wait();
        const int next = p + S::kAhead;
        if (next < n_pieces) load_piece(next, 0, place_next);
        else load_piece(next - n_pieces, 1, place_next);
        if (head < heads) scores(head, j, place);
        place = after(place);
        place_next = after(place_next);
        __builtin_amdgcn_sched_barrier(0);
      };
      for (int p = 0; p < n_pieces; p += ST)
#pragma unroll
        for (int j = 0; j < ST; ++j) k_step(p + j, p / ST, j);
      weights(t);
      wait();
      take_bad();
      auto v_step = [&](int p, int head, int j) {
        wait();
        const int next = p + S::kAhead;
        if (next == n_pieces) {  // (past the last tile: its last key again)
          put_addr(t + 1);
          load_steps(0);
        }
        if (next < n_pieces) load_piece(next, 1, place_next);
        else load_piece(next - n_pieces, 0, place_next);
        if (head < heads) add_values(head, j, place);
        place = after(place);
        place_next = after(place_next);
        __builtin_amdgcn_sched_barrier(0);
      };
      for (int p = 0; p < n_pieces; p += ST)
#pragma unroll
        for (int j = 0; j < ST; ++j) v_step(p + j, p / ST, j);
    }
  };
  const int heads_q = a.hk * a.group;
  auto finish = [&](bool whole, int place) {
    if (bad_groups) {
#pragma unroll
      for (int h = 0; h < VH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = dim_of(h, g * 4 + i);
          // (the groups are this row's: lanes of its column)
          if (d < 256 && bad_groups >> (d >> 5) & 1) {
#pragma unroll
            for (int e = 0; e < VD; ++e) acc[h][e][i] = NAN;
          }
        }
    }

    l = sum32(sum16(l));
    landed();  // (what was loaded past the last tile)
    if (phases == 1 && whole) {  // rows of this wave's alone: straight from the registers
      if (m16 >= cols) return;
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      uint16_t* o = a.out + (int64_t)r * a.o_ts + (int64_t)my_q * a.o_hs;
#pragma unroll
      for (int h = 0; h < VH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = dim_of(h, g * 4 + i);
          if (d >= a.D) continue;
          uint32_t x[VD / 2];
#pragma unroll
          for (int e = 0; e < VD; e += 2)
            x[e / 2] = round2<DT>(seen.bad ? NAN : l == 0.f ? 0.f : acc[h][e][i] * inv,
                                  seen.bad ? NAN : l == 0.f ? 0.f : acc[h][e + 1][i] * inv);
          if constexpr (VD == 8) st16(o + d, make_uint4(x[0], x[1], x[2], x[3]));
          else *reinterpret_cast<uint2*>(o + d) = make_uint2(x[0], x[1]);
        }
      if (a.lse && g == 0) a.lse[(int64_t)r * heads_q + my_q] = seen.bad ? NAN : log_sum<MT>(m, l);
      return;
    }
    // Join the waves of a unit. Rows are 4 floats apart from a multiple of 8, so the 16 rows' stores
    // meet no bank twice.
    __syncthreads();  // every wave is done with its steps
    float* const sm_out = (float*)sm;  // [wave][row][D + 4]
    const int stride = a.D + 4, most_cols = min(a.wave_heads * a.group, kRows);
    if (g == 0) {
      sm_m[wave][m16] = m;
      sm_l[wave][m16] = l;
    }
    if (m16 < cols) {
      float* o = sm_out + (wave * most_cols + m16) * stride;
#pragma unroll
      for (int h = 0; h < VH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = dim_of(h, g * 4 + i);
          if (d < a.D) {
#pragma unroll
            for (int e = 0; e < VD; e += 4)
              *reinterpret_cast<float4*>(o + d + e) = make_float4(acc[h][e][i], acc[h][e + 1][i], acc[h][e + 2][i], acc[h][e + 3][i]);
          }
        }
    }
    __syncthreads();
    // A part's result: [place][query head][m, l, out].
    const int64_t part_row = a.D + 2;
    const int pairs = a.D / 2;
    for (int j = 0; j < wg_units; ++j) {
      const Unit u = unit_of(unit0 + j);
      for (int i = tid; i < u.cols() * pairs; i += kWaves * 64) {
        const int c = i / pairs, d = (i - c * pairs) * 2, hq = query_head(u, c);
        float mt = -INFINITY, lt = 0.f, x = 0.f, y = 0.f;
        for (int k = j; k < kWaves; k += wg_units) mt = fmaxf(mt, sm_m[k][c]);
        for (int k = j; k < kWaves; k += wg_units) {
          const float f = part_weight(sm_m[k][c], mt);
          const float2 o = *reinterpret_cast<const float2*>(sm_out + (k * most_cols + c) * stride + d);
          lt += f * sm_l[k][c];
          x += f * o.x;
          y += f * o.y;
        }
        if (whole) {
          const float inv = lt == 0.f ? 0.f : 1.0f / lt;
          *reinterpret_cast<uint32_t*>(a.out + (int64_t)r * a.o_ts + (int64_t)hq * a.o_hs + d) =
              round2<DT>(seen.bad ? NAN : lt == 0.f ? 0.f : x * inv, seen.bad ? NAN : lt == 0.f ? 0.f : y * inv);
          if (a.lse && d == 0) a.lse[(int64_t)r * heads_q + hq] = seen.bad ? NAN : log_sum<MT>(mt, lt);
        } else {
          float* part = a.part + ((int64_t)place * heads_q + hq) * part_row;
          *reinterpret_cast<float2*>(part + 2 + d) = make_float2(x, y);
          if (d == 0) *reinterpret_cast<float2*>(part) = make_float2(mt, lt);
        }
      }
    }
    __syncthreads();  // (the next part's pieces go where the rows are)
  };

  int32_t off = span.off, seq = a.seq[r], prefix = a.prefix ? a.prefix[r] : 0;
  for (int64_t left = span.length;;) {
    seen = seen_by(a, seq, prefix);
    const int32_t rounds = rounds_of(a, seq, prefix, round_log2), take = (int32_t)min((int64_t)(rounds - off), left);
    const bool whole = take == rounds;
    if (off == 0 && unit0 == 0 && tid == 0)
      a.cut[r] = make_int2(x, whole ? 1 : (int)((rounds - take + span.length - 1) / span.length) + 1);
    left -= take;
    const bool more = left > 0 && r + 1 < a.n_req;
    if (more) {  // (on their way while this part is worked on)
      seq = a.seq[r + 1];
      prefix = a.prefix ? a.prefix[r + 1] : 0;
    }
    begin_part(off, take);
    work();
    finish(whole, 2 * x + (off == 0));
    if (!more) return;
    ++r;
    off = 0;
  }
}

// Results of requests that were cut, from their parts' in order. W waves a row, in a launch of its
// own: a part holds a request's heads all at once, so the workgroup that finished last would have
// all rows to join.
constexpr int kJoinAhead = 4;  // parts whose loads are in flight
template <int DT, int W>
__global__ __launch_bounds__(W * 64) void attn4_join_kernel(AttnArgs a) {
  __shared__ float2 sm_out[W][2][64];
  __shared__ float sm_l[W];
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = (int)blockIdx.y, heads_q = a.hk * a.group;
  const int first = a.cut[r].x, n = a.cut[r].y;
  if (n <= 1) return;
  const int64_t part_row = a.D + 2;
  // the first span ends with the request, the others begin with it
  auto part_of = [&](int c, int hq) { return a.part + ((int64_t)(2 * (first + c) + (c == 0)) * heads_q + hq) * part_row; };
  const int e1 = min(lane * 2, a.D - 2), e2 = min(lane * 2 + 128, a.D - 2);
  for (int hq = (int)blockIdx.x; hq < heads_q; hq += (int)gridDim.x) {
    float mt = -INFINITY;
    for (int c = lane; c < n; c += 64) mt = fmaxf(mt, *part_of(c, hq));
    mt = max32(max16(mt));
    for (int d = 8; d; d >>= 1) mt = fmaxf(mt, __shfl_xor(mt, d));
    float2 o1 = make_float2(0.f, 0.f), o2 = o1;
    float l = 0.f;
    for (int c0 = wave * kJoinAhead; c0 < n; c0 += W * kJoinAhead) {
      float2 ml[kJoinAhead], x1[kJoinAhead], x2[kJoinAhead];
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) {
        const float* p = part_of(min(c0 + i, n - 1), hq);
        ml[i] = *reinterpret_cast<const float2*>(p);
        x1[i] = *reinterpret_cast<const float2*>(p + 2 + e1);
        if (a.D > 128) x2[i] = *reinterpret_cast<const float2*>(p + 2 + e2);
      }
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) {
        if (c0 + i >= n) break;
        const float f = part_weight(ml[i].x, mt);
        l += f * ml[i].y;
        o1.x += f * x1[i].x;
        o1.y += f * x1[i].y;
        if (a.D > 128) {
          o2.x += f * x2[i].x;
          o2.y += f * x2[i].y;
        }
      }
    }
    if (W > 1) {
      sm_out[wave][0][lane] = o1;
      sm_out[wave][1][lane] = o2;
      if (lane == 0) sm_l[wave] = l;
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int k = 1; k < W; ++k) {
          l += sm_l[k];
          o1.x += sm_out[k][0][lane].x;
          o1.y += sm_out[k][0][lane].y;
          o2.x += sm_out[k][1][lane].x;
          o2.y += sm_out[k][1][lane].y;
        }
      }
      __syncthreads();
      if (wave) continue;
    }
    const float inv = 1.0f / l;
    uint16_t* out = a.out + (int64_t)r * a.o_ts + (int64_t)hq * a.o_hs;
    // (a row with scores of minus infinity alone is 0, also where a V is no number)
    auto put = [&](int d, float2 o) {
      if (d < a.D) *reinterpret_cast<uint32_t*>(out + d) = l == 0.f ? 0u : round2<DT>(o.x * inv, o.y * inv);
    };
    put(lane * 2, o1);
    put(lane * 2 + 128, o2);
    if (a.lse && lane == 0) a.lse[(int64_t)r * heads_q + hq] = log_sum<SLORA_F16>(mt, l);
  }
}

template <int DT, int NC, int ST>
hipError_t launch_st(AttnArgs a, hipStream_t s, const LaunchEvents& ev) {
  using S = SpanShape<NC, ST>;
  const int units = (a.hk + a.wave_heads - 1) / a.wave_heads * ((a.group + kRows - 1) / kRows);
  const int wgs = (units + a.wg_units - 1) / a.wg_units;
  a.xcd_log2 = 3;  // (there are a multiple of 8)
  const int heads_q = a.hk * a.group;
  if ((int64_t)a.spans * wgs * kWaves * 64 >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)wgs << a.xcd_log2, (unsigned)(a.spans >> a.xcd_log2));
  const int cols = a.wave_heads * a.group < kRows ? a.wave_heads * a.group : kRows;
  const size_t join = sizeof(float) * kWaves * cols * (a.D + 4), pieces = kWaves * S::kBytes;
  const size_t lds = join > pieces ? join : pieces;
  if (lds > 48 * 1024) {  // with the static part past the 64 KiB a launch has by default
    const hipError_t e = hipFuncSetAttribute((const void*)attn4_decode_kernel<DT, NC, ST>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  const bool cut = a.max_len > kWaves / a.wg_units * S::kKeys && a.spans > 1;  // some request may be
  hipExtLaunchKernelGGL((attn4_decode_kernel<DT, NC, ST>), grid, dim3(kWaves * 64), lds, s, ev.start,
                        cut ? nullptr : ev.stop, 0, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !cut) return e;
  const dim3 rows((unsigned)(heads_q < 64 ? heads_q : 64), (unsigned)a.n_req);
  if ((int64_t)a.n_req * heads_q >= 4096)
    hipExtLaunchKernelGGL((attn4_join_kernel<DT, 1>), rows, dim3(64), 0, s, nullptr, ev.stop, 0, a);
  else
    hipExtLaunchKernelGGL((attn4_join_kernel<DT, 16>), rows, dim3(1024), 0, s, nullptr, ev.stop, 0, a);
  return hipGetLastError();
}

template <int DT, int NC>
hipError_t launch_nc(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  if constexpr (NC <= 4) {
    if (a.wave_runs == 4) return launch_st<DT, NC, 4>(a, s, ev);
  }
  return a.wave_runs == 2 ? launch_st<DT, NC, 2>(a, s, ev) : launch_st<DT, NC, 1>(a, s, ev);
}

template <int DT, int NC>
hipError_t launch_few_nc(const AttnArgs& a, dim3 grid, hipStream_t s, const LaunchEvents& ev) {
  const int rows = a.group < kRows ? a.group : kRows;
  const size_t lds = sizeof(float) * kWaves * rows * (a.D + 4);
  if (lds > 48 * 1024) {  // with the static part past the 64 KiB a launch has by default
    const hipError_t e = hipFuncSetAttribute((const void*)attn_decode_kernel<DT, NC, 4>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipExtLaunchKernelGGL((attn_decode_kernel<DT, NC, 4>), grid, dim3(kWaves * 64), lds, s, ev.start, ev.stop, 0, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_few(AttnArgs a, hipStream_t s, const LaunchEvents& ev) {
  const int units = a.hk / a.wg_heads * ((a.group + kRows - 1) / kRows);
  // No request has more chunks than rounds of keys.
  const int64_t round = kTile * (kWaves / a.wg_heads);
  const int64_t most = (a.max_len + round - 1) / round, all = (int64_t)a.n_req * (most > 1 ? most : 1);
  const int64_t chunks = all < (int64_t)a.n_req + a.chunks ? all : (int64_t)a.n_req + a.chunks;
  a.xcd_log2 = chunks >= 32 ? 3 : 0;
  const int64_t rounds = (chunks + (1 << a.xcd_log2) - 1) >> a.xcd_log2;
  if ((rounds << a.xcd_log2) * units * kWaves * 64 >= kMaxThreads) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)units << a.xcd_log2, (unsigned)rounds);
  switch (a.kv4.groups) {
    case 1: return launch_few_nc<DT, 1>(a, grid, s, ev);
    case 2: return launch_few_nc<DT, 2>(a, grid, s, ev);
    case 3: return launch_few_nc<DT, 3>(a, grid, s, ev);
    case 4: return launch_few_nc<DT, 4>(a, grid, s, ev);
    case 5: return launch_few_nc<DT, 5>(a, grid, s, ev);
    case 6: return launch_few_nc<DT, 6>(a, grid, s, ev);
    case 7: return launch_few_nc<DT, 7>(a, grid, s, ev);
    default: return launch_few_nc<DT, 8>(a, grid, s, ev);
  }
}

template <int DT>
hipError_t launch_dt(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  if (a.spans == 0) return launch_few<DT>(a, s, ev);
  switch (a.kv4.groups) {
    case 1: return launch_nc<DT, 1>(a, s, ev);
    case 2: return launch_nc<DT, 2>(a, s, ev);
    case 3: return launch_nc<DT, 3>(a, s, ev);
    case 4: return launch_nc<DT, 4>(a, s, ev);
    case 5: return launch_nc<DT, 5>(a, s, ev);
    case 6: return launch_nc<DT, 6>(a, s, ev);
    case 7: return launch_nc<DT, 7>(a, s, ev);
    default: return launch_nc<DT, 8>(a, s, ev);
  }
}

}  // namespace

hipError_t launch_attn4_decode(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
