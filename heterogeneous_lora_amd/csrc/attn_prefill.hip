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
// The next tile's products run beside this tile's weights, and this tile's values beside the
// next one's scores, so that the matrix and the vector units of a wave both have work.
//
// Pages are gathered straight into LDS (global_load_lds, 16 bytes a lane), one tile ahead
// of the products, a load between two of them; the addresses of a tile's keys are made a tile
// earlier, its page ids read another earlier. A tile's rows lie as in the page, in 16-byte units whose places
// within a row are xored with bits of the row's number: K is read a row to a lane
// (ds_read_b128), V four keys x 16 dimensions to 16 lanes, turned on the way
// (ds_read_b64_tr_b16), both without bank conflicts (counted: none). Two workgroups share a
// CU, so that one has work while the other waits.
//
// Two prompts of 8000 tokens after 7000-8192 cached, 32 query heads on 8 KV heads of 128,
// bf16: 3.2 ms (970 TFLOP/s), with softcap 3.6 ms (860; it triples the transcendentals). A
// library product of 8192^3 reaches 1262 on the same card. 64 prompts of 8 to 512 tokens, 32
// heads of 128: 187 us.
#include "attn_dev.h"

namespace slora {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWaveRows = 32;
constexpr int kTileM = 128;           // rows of a workgroup
constexpr int kAhead = 4;              // fragments read ahead of their products
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
  // Unit c of row `key` lies at place c ^ k_swap(key) (K) or c ^ v_swap(key) (V) of the row:
  // LDS has 16 units a bank row, K is read one unit of 16 rows at a time, V four units of 4
  // rows.
  __device__ static __forceinline__ int k_swap(int key) {
    return CH == 12 ? key >> 2 & 3 : CH % 16 ? key >> 1 & 7 : key & 15;
  }
  __device__ static __forceinline__ int v_swap(int key) {
    return CH == 12 ? 0 : CH % 16 ? (key >> 1 & 1) * 4 : (key & 3) * 4;
  }
};

struct RowTile {
  int r;                   // request, -1: none
  int tile;                // row tile of the request
  int chunk, chunks;       // which part of the tile's keys, of how many
  int extra;               // chunks past one a tile, over all tiles before this one
  int q0, n_new, n, prefix;  // the request's first new token, new tokens, seq_len, prefix_len
};

// The x-th chunk over all row tiles. Where the tiles alone do not fill the device, requests
// with more keys than others are cut into chunks, so that the call makes some a.chunks more
// of them per KV head. What the kernel needs of the request comes from the same pass: a
// second round of loads would cost a short prompt more than its products.
constexpr int kMinChunk = 512;  // keys: some 20 us of products, what joining 16 chunks costs
__device__ __forceinline__ RowTile find_tile(const AttnArgs& a, int lane, int x) {
  int q0 = 0, n_new = 0, n = 0, prefix = 0, tiles = 0, sees = 0;
  auto load = [&](int r0) {
    const int r = min(r0 + lane, a.n_req - 1);
    q0 = min(max(a.q_offsets[r], 0), a.n_tok);
    n_new = max(min(max(a.q_offsets[r + 1], 0), a.n_tok) - q0, 0);
    n = a.seq[r];
    prefix = a.prefix ? a.prefix[r] : 0;
    tiles = r0 + lane < a.n_req ? (int)(((int64_t)n_new * a.group + kTileM - 1) / kTileM) : 0;
    // keys of its last tile, about
    sees = n < 0 || n > a.max_len ? 0 : a.window ? (int)min((int64_t)n, (int64_t)a.window + max(prefix, 0) + kTileM) : n;
  };
  load(0);
  float length = 1e30f;
  if (a.chunks) {
    float work = (float)tiles * (float)sees;
    for (int r0 = 64; r0 < a.n_req; r0 += 64) {
      load(r0);
      work += (float)tiles * (float)sees;
    }
    length = fmaxf(wave_sum(work) / (float)a.chunks, (float)kMinChunk);
    if (a.n_req > 64) load(0);
  }
  int before = 0, extra = 0;
  for (int r0 = 0;;) {
    const int chunks = (int)fmaxf((float)sees / length + 0.5f, 1.f);
    const int mine = tiles * chunks, sum = running_sum(mine), extra_mine = mine - tiles, extra_sum = running_sum(extra_mine);
    const uint64_t hit = __ballot(x < before + sum);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      const int c = of(chunks), i = x - before - of(sum - mine), t = c == 1 ? i : i / c;
      // later tiles of a request see more keys: they go first
      return {r0 + l, of(tiles) - 1 - t, i - t * c, c, extra + of(extra_sum - extra_mine) + t * (c - 1),
              of(q0), of(n_new), of(n), of(prefix)};
    }
    before += __builtin_amdgcn_readlane(sum, 63);
    extra += __builtin_amdgcn_readlane(extra_sum, 63);
    r0 += 64;
    if (r0 >= a.n_req) return {-1, 0, 0, 1, 0, 0, 0, 0, 0};
    load(r0);
  }
}

// The halves of a dword of two storage values that hold an infinity or NaN; the rest 0.
template <int DT>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t e = DT == SLORA_F16 ? 0x7C00u : 0x7F80u;
  const uint32_t lo = (w & e) == e ? 0xffffu : 0u, hi = (w & e << 16) == e << 16 ? 0xffff0000u : 0u;
  return w & (lo | hi);
}
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 magnitudes(uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7fff7fffu); }
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

// 16 bytes `off` past an LDS offset (a constant `off` is the instruction's).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(3))) char lds_bytes;
__device__ __forceinline__ uint4 read_lds(uint32_t at, int off) {
  return __builtin_bit_cast(uint4, *(const __attribute__((address_space(3))) u32x4*)((lds_bytes*)(uintptr_t)at + off));
}
// Four 16-bit values of this lane's column (16 lanes: 4 rows of 16 values, 4 to a lane).
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 read_turned(uint32_t at, int off) {
  return __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)((lds_bytes*)(uintptr_t)at + off)));
}

// What a score passes through between the two products. kPlain: the scale alone, taken in
// the subtraction of the maximum. kCap: softcap. kBias, kBiasCap: a bias that depends on
// distance after them, and scales of zero or below (which would turn a masked -infinity).
// kWideCap: a softcap above kNearCap, with or without them, in the form that holds there (long
// prompts without a bias 5022 us, kCap 3748: two forms a score, and 19 registers that spill).
enum Mode { kPlain, kCap, kBias, kBiasCap, kWideCap };

// Two workgroups a CU leave a wave 256 registers: heads up to 192 fit (192: 2.4 ms against 3.8
// with one workgroup), 256 would spill (9.4 ms against 4.6).
template <int DT, int NC, int MODE>
__global__ __launch_bounds__(kThreads, NC <= 6 ? 2 : 1) void attn_prefill_kernel(AttnArgs a) {
  using S = Shape<NC>;
  constexpr int BN = S::BN, KT = S::KT, CH = S::CH;
  __shared__ uint4 sm_k[2][S::kUnits];
  __shared__ uint4 sm_v[2][S::kUnits];
  __shared__ uint64_t sm_addr[2][2 * BN];
  __shared__ uint32_t sm_flag[4];  // tile t (mod 4) has infinities or NaN in V that some row must not see

  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m32 = lane & 31, h = lane >> 5;
  const int tile_x = a.hk == 1 ? (int)blockIdx.x : (int)(__umulhi(blockIdx.x, a.hk_magic) >> a.hk_shift);
  const int kv_head = (int)blockIdx.x - tile_x * a.hk;
  const RowTile rt = find_tile(a, lane, tile_x);
  const int r = rt.r, row_tile = rt.tile, q0 = rt.q0, n_new = rt.n_new;
  if (r < 0) return;
  const bool bad = rt.n < 0 || rt.n > a.max_len;
  const int32_t n = bad ? 0 : rt.n;
  const int first_pos = n - n_new;
  const int prefix = min(max(rt.prefix, 0), n);

  // Row i of the tile: token tok0 + (head0 + i) / group, query head (head0 + i) % group.
  const int rows = (int)min((int64_t)n_new * a.group - (int64_t)row_tile * kTileM, (int64_t)kTileM);
  const int tile_q = (int)div_group(a, (uint32_t)row_tile), tile_r = row_tile - tile_q * a.group;
  const int tok0 = tile_q * kTileM + (int)div_group(a, (uint32_t)(tile_r * kTileM));
  const int head0 = tile_r * kTileM - (tok0 - tile_q * kTileM) * a.group;
  auto pos_of = [&](int i) { return first_pos + tok0 + (int)div_group(a, (uint32_t)(head0 + min(i, rows - 1))); };
  // this lane's row
  const int my_row = wave * kWaveRows + m32;
  const int pos = pos_of(my_row), tok = pos - first_pos;
  const int head = kv_head * a.group + head0 + min(my_row, rows - 1) - (tok - tok0) * a.group;
  const int wave_p1 = pos_of(wave * kWaveRows + kWaveRows - 1);
  const int wg_p0 = first_pos + tok0, wg_p1 = pos_of(kTileM - 1);
  const Keys keys = n > 0 ? keys_of(a, prefix, n, wg_p0, wg_p1, BN) : Keys{0, 0, 0};
  // this chunk's tiles of keys
  const int all_tiles = (keys.count + BN - 1) / BN, per_chunk = rt.chunks == 1 ? all_tiles : (all_tiles + rt.chunks - 1) / rt.chunks;
  const int first_tile = min(rt.chunk * per_chunk, all_tiles), n_tiles = min(first_tile + per_chunk, all_tiles);
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
  float slope = MODE >= kBias && a.slopes ? a.slopes[head] * kLog2e : 0.f;
  // Scores are s * mul, or s * mul + cap: with softcap s is the reciprocal 1 / (e^(2 x / cap) +
  // 1) in cap tanh(x / cap) = cap - 2 cap s.
  const float mul = MODE == kPlain ? a.scale2 : MODE == kCap ? -2.0f * a.cap_out : 1.f;

  f32x16 acc[NC];
#pragma unroll
  for (int d = 0; d < NC; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  // Addresses of a tile's keys: threads [0, BN) K, [BN, 2 BN) V, the others the same again.
  // The products take K one tile ahead of V, so tile t's turn brings V of tile t + 1 and K of
  // tile t + 2: place t & 1 holds the addresses for turn t, K's of one tile further on.
  // (The loop has no branch that lanes could disagree on, one body, and no other place that
  // changes the accumulators: otherwise the compiler keeps a second set of them, and every
  // tile pays for copies between the two.)
  const int my_key = tid % BN, is_v = tid / BN % 2;
  const uint64_t zeros = settled(fill_addr<DT>(true)), nans = settled(fill_addr<DT>(false));
  const int32_t* table = (is_v ? a.vt : a.kt) + (int64_t)r * a.max_blocks;
  auto index_of = [&](int turn) { return (turn + 2 - is_v) * BN + my_key; };  // V at turn -2: below 0
  auto key_of = [&](int turn) { return keys.key(max(min(index_of(turn), keys.count - 1), 0)); };
  auto page_of = [&](int turn) -> int32_t { return table[div_tpp(a, (uint32_t)key_of(turn))]; };
  auto put_addr = [&](int turn, int32_t page) {
    const int i = index_of(turn);
    const uint64_t p = settled(key_addr(a, page, key_of(turn), h_off, nans));
    sm_addr[turn & 1][tid % (2 * BN)] = i < keys.count ? p : zeros;
  };
  const uint32_t lds_k = lds_offset(sm_k) + wave * 1024, lds_v = lds_offset(sm_v) + wave * 1024;
  // One of a turn's loads: K's first, then V's. K's units past the head are zeros (their q is
  // 0, but 0 times an infinity is not); V's make dimensions that are dropped, so any will do.
  auto row_of = [&](int turn, int u) {
    return sm_addr[turn & 1][(u < S::kLoads ? 0 : BN) + (tid + u % S::kLoads * kThreads) / CH];
  };
  auto fetch = [&](int turn, int u, uint64_t row) {
    const int i = tid + u % S::kLoads * kThreads, key = i / CH;
    if (u < S::kLoads) {
      const int d = (i % CH ^ S::k_swap(key)) * 8;
      load_to_lds(settled(d < a.D ? row + d * 2 : zeros), lds_k + ((turn & 1) * S::kUnits + u * kThreads) * 16);
    } else {
      const int d = (i % CH ^ S::v_swap(key)) * 8;
      load_to_lds(row + min(d, a.D - 8) * 2, lds_v + (((turn + 1) & 1) * S::kUnits + (u - S::kLoads) * kThreads) * 16);
    }
  };
  auto fetch_all = [&](int turn, int from, int to) {
#pragma unroll
    for (int u = from; u < to; ++u) fetch(turn, u, settled(row_of(turn, u)));
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
  if (first_tile < n_tiles) {  // turn t - 2 brings K of tile t, turn t - 1 V of tile t and K of tile t + 1
    const int t = first_tile;
    int32_t first = page_of(t - 2), second = page_of(t - 1);
    next = page_of(t);
    put_addr(t - 2, first);
    put_addr(t - 1, second);
    __syncthreads();
    fetch_all(t - 2, 0, S::kLoads);
    fetch_all(t - 1, 0, 2 * S::kLoads);
    landed();
    __syncthreads();
    put_addr(t, settled(next));
    next = page_of(t + 1);
  }

  const int k_row = (m32 & ~12) | (m32 & 4) << 1 | (m32 & 8) >> 1;
  const int v_key = h * 8 + (lane >> 2 & 3), v_c = (lane >> 4 & 1) * 2 + (lane >> 1 & 1), v_in = (lane & 1) * 4;
  // Fragments: K's rows (the products of a tile are numbered c, kt), V's dimensions (d, kt,
  // u). One xor and one addition make the address of a c's or d's; the rest is in the
  // instructions. (Kept in registers, the addresses would be spilled.)
  constexpr int kSteps = KT * NC * 2, kPairs = KT * 8, kRow = CH * 16;
  // a step's share of the pairs of weights (or scores) and of the loads, at most
  constexpr int kPairsStep = (kPairs + kSteps - 1) / kSteps, kLoadsStep = (2 * S::kLoads + kSteps - 1) / kSteps;
  const uint32_t k_base = lds_offset(sm_k) + k_row * kRow, k_xor = (h ^ S::k_swap(k_row)) * 16;
  const uint32_t v_base = lds_offset(sm_v) + v_key * kRow + v_c * 16 + v_in * 2, v_xor = S::v_swap(v_key) * 16;
  uint32_t frag_at = 0;
  auto k_frag = [&](uint32_t place, int i) {
    if (i % KT == 0) frag_at = (k_xor ^ i / KT * 32) + place;
    return read_lds(frag_at, i % KT * 32 * kRow);
  };
  auto v_frag = [&](uint32_t place, int i) {
    if (i % (KT * 2) == 0) frag_at = (v_xor ^ i / (KT * 2) * 64) + place;
    const int off = i % (KT * 2) * 16 * kRow;
    const uint2 x = read_turned(frag_at, off), y = read_turned(frag_at, off + 4 * kRow);
    return make_uint4(x.x, x.y, y.x, y.y);
  };
  // Scores 2 j and 2 j + 1 of a lane, from the products. Register i of product kt: index t *
  // BN + kt * 32 + 16 (i / 8) + 8 h + i % 8 of the run.
  auto score_pair = [&](float far, f32x16 (&s)[KT], int j) {  // far: of register 0, key - position
    const int kt = j / 8;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = j % 8 * 2 + e;
      float x = s[kt][i];
      if (MODE == kCap) x = __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x * a.cap_in) + 1.0f);
      else if (MODE == kBiasCap) x = capped_near(a, x);
      else if (MODE == kWideCap) x = capped(a, x);
      else if (MODE == kBias) x *= a.scale2;
      if (MODE >= kBias) x = __builtin_fmaf(slope, far + (float)(kt * 32 + 16 * (i / 8) + i % 8), x);
      s[kt][i] = x;
    }
  };
  // (a tile lies on one side of the hole behind the prefix)
  auto far_of = [&](int t) { return MODE >= kBias ? (float)(keys.key(t * BN) + 8 * h - pos) : 0.f; };
  // -infinity for what the row must not see of a border tile.
  auto mask = [&](int t, f32x16 (&s)[KT]) {
    const int at = t * BN + 8 * h, hi = see_hi - at, lo = see_lo - at, pre = prefix - at;
    const float out = MODE == kCap ? INFINITY : -INFINITY;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = kt * 32 + 16 * (i / 8) + i % 8;
        s[kt][i] = (((k <= hi) & (k >= lo)) | (k < pre)) ? s[kt][i] : out;
      }
  };
  auto maximum = [&](const f32x16 (&s)[KT]) {
    float x = s[0][0];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) x = MODE == kCap ? fminf(x, s[kt][i]) : fmaxf(x, s[kt][i]);
    return MODE == kCap ? __builtin_fmaf(-max32(-x), mul, a.cap_out) : max32(x) * mul;
  };
  // Weights 2 j and 2 j + 1, their part of the sum and of the B operand. They are rounded to the
  // storage type once, the usual trade: as sums of two values, with two products each, long
  // prompts take 4683 us against 3666 and 64 short ones 215 against 188.
  auto weight_pair = [&](const f32x16 (&s)[KT], float ms, uint32_t (&p)[KT * 8], int j) {
    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j / 8][j % 8 * 2], mul, ms));
    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j / 8][j % 8 * 2 + 1], mul, ms));
    l += x;
    l += y;
    p[j] = round2<DT>(x, y);
  };

  // Tiles this wave's rows see: those below w_tiles.
  int w_tiles = n_tiles;
  while (w_tiles > first_tile) {
    const int j0 = keys.key((w_tiles - 1) * BN);
    if (j0 <= wave_p1 || j0 < prefix) break;
    --w_tiles;
  }
  // q is waited for here: a wait inside the loop would be one for the tiles on their way.
#pragma unroll
  for (int c = 0; c < NC * 2; ++c) q[c] = __builtin_bit_cast(uint4, settled(__builtin_bit_cast(u32x4, q[c])));
  slope = settled(slope);
  f32x16 s[KT];
  float mx = -INFINITY;
  if (w_tiles > first_tile) {
    const uint32_t place = k_base + (first_tile & 1) * S::kUnits * 16;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[kt][i] = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) s[i % KT] = mfma32x32<DT>(k_frag(place, i), q[i / KT], s[i % KT]);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) score_pair(far_of(first_tile), s, j);
    if (!all_seen(first_tile, wg_p0, wg_p1)) mask(first_tile, s);
    mx = maximum(s);
  }
  bool cleared = false;  // some tile held an infinity or NaN
  for (int t = first_tile; t < n_tiles; ++t) {
    landed();              // this wave's share of K of tile t + 1 and V of tile t
    next = settled(next);  // (waited for here, not behind the loads below)
    // A tile on some row's border. A weight of zero does not keep an infinity or NaN in V
    // out of a product, so these are taken out of such a tile and dealt with at the end.
    // Every thread looks at what it loaded; no ordinary tile costs more.
    const bool edge = !all_seen(t, wg_p0, wg_p1);
    uint4* const vt = sm_v[t & 1];
    if (edge) {
      u16x2 top = {0, 0};
#pragma unroll
      for (int u = 0; u < S::kLoads; ++u) {
        const uint4 w = vt[tid + u * kThreads];
        top = __builtin_elementwise_max(top, magnitudes(w.x));
        top = __builtin_elementwise_max(top, magnitudes(w.y));
        top = __builtin_elementwise_max(top, magnitudes(w.z));
        top = __builtin_elementwise_max(top, magnitudes(w.w));
      }
      if (__any(not_finite<DT>(__builtin_bit_cast(uint32_t, top)) != 0)) sm_flag[t & 3] = 1;
    }
    __syncthreads();  // everyone's share; and everyone is done with the places about to be filled
    if (edge || cleared) sm_flag[(t + 2) & 3] = 0;
    if (edge && __builtin_amdgcn_readfirstlane(sm_flag[t & 3])) {
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
    if (t >= w_tiles) {
      fetch_all(t, 0, 2 * S::kLoads);
      put_addr(t + 1, next);
      next = page_of(t + 2);
      continue;
    }
    // The maximum is moved only when it has grown by kRescale: until then the weights
    // reach 2^kRescale (times 2^kWeightLog2, which f16 holds).
    if (__any(mx > m + kRescale)) {
      const float mn = fmaxf(m, mx);
      const float f = part_weight(m, mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < NC; ++d) acc[d] *= f;
    }
    // Two stretches of matrix work, each beside vector work that does not need it: the next
    // tile's products beside this one's weights, this tile's values beside the next one's
    // scores. Step by step in this order (the compiler's own puts a fragment's load right
    // before its product, and waits for each): fragments are read kAhead products early.
    f32x16 sn[KT];
    uint32_t p[KT * 8];
    const float ms = (MODE == kCap ? a.cap_out : 0.f) + kWeightLog2<DT> - (m == -INFINITY ? 0.f : m);
    const bool edge_next = !all_seen(t + 1, wg_p0, wg_p1);
    const float far = far_of(t + 1);
    const uint32_t k_place = k_base + ((t + 1) & 1) * S::kUnits * 16, v_place = v_base + (t & 1) * S::kUnits * 16;
    uint4 frag[kSteps];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) sn[kt][i] = 0.f;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) frag[i] = k_frag(k_place, i);
    uint64_t row = row_of(t, 0);
    // A wave with products to issue goes before one at a tile's border (long prompts -2%).
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
    uint4 vfrag[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i + kAhead < kSteps) frag[i + kAhead] = k_frag(k_place, i + kAhead);
      else vfrag[i + kAhead - kSteps] = v_frag(v_place, i + kAhead - kSteps);
#pragma unroll
      for (int e = 0; e < kLoadsStep; ++e) {
        const int u = i * 2 * S::kLoads / kSteps + e;
        if (u < (i + 1) * 2 * S::kLoads / kSteps) {
          fetch(t, u, row);
          if (u + 1 < 2 * S::kLoads) row = row_of(t, u + 1);
        }
      }
      sn[i % KT] = mfma32x32<DT>(frag[i], q[i / KT], sn[i % KT]);
#pragma unroll
      for (int e = 0; e < kPairsStep; ++e) {
        const int j = i * kPairs / kSteps + e;
        if (j < (i + 1) * kPairs / kSteps) weight_pair(s, ms, p, j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i + kAhead < kSteps) vfrag[i + kAhead] = v_frag(v_place, i + kAhead);
      if (i == kSteps / 2) put_addr(t + 1, next);
      if (i == kSteps - 1) next = page_of(t + 2);
      const int b = i % (KT * 2) * 4, d = i / (KT * 2);
      acc[d] = mfma32x32<DT>(vfrag[i], make_uint4(p[b], p[b + 1], p[b + 2], p[b + 3]), acc[d]);
#pragma unroll
      for (int e = 0; e < kPairsStep; ++e) {
        const int j = i * kPairs / kSteps + e;
        if (j < (i + 1) * kPairs / kSteps) score_pair(far, sn, j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    // (the compiler would move the sum and the scores behind the branch)
    l = settled(l);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) sn[kt] = settled(sn[kt]);
    if (edge_next) mask(t + 1, sn);
    mx = maximum(sn);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) s[kt] = sn[kt];
  }
  landed();  // (tiles past the last, fetched as zeros)
  // The infinities and NaN taken out, to the rows that see them: they decide these rows'
  // results, whatever their weight.
  if (cleared) {
    const int32_t* vt = a.vt + (int64_t)r * a.max_blocks;
#pragma unroll 1
    for (int i = first_tile * BN; i < n_tiles * BN; ++i) {
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
  if (rt.chunks > 1) {
    // A chunk's result goes to the workspace as the lanes hold it, pairs of values 64 lanes
    // wide, and the workgroup that finishes last adds the others' to its own. Parts are
    // numbered 2 extra + chunk: a cut tile has at most twice its extra chunks.
    float* const mine = a.part + (((int64_t)(2 * rt.extra) * a.hk + kv_head) * a.part_waves + wave) * part_floats(NC) + lane * 2;
    const int64_t part_step = (int64_t)a.hk * a.part_waves * part_floats(NC);
    const bool used = wave * kWaveRows < rows;  // (then wave < part_waves)
    if (used) {
      float* to = mine + rt.chunk * part_step;
      put_pair(to, m, l);
#pragma unroll
      for (int d = 0; d < NC; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 2) put_pair(to + (1 + d * 8 + i / 2) * 128, acc[d][i], acc[d][i + 1]);
    }
    landed();
    __syncthreads();
    if (tid == 0) {
      int32_t* counter = a.counters + rt.extra * a.hk + kv_head;
      const int32_t done = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      sm_flag[0] = done == rt.chunks - 1;
      if (done == rt.chunks - 1) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
    }
    __syncthreads();
    if (!__builtin_amdgcn_readfirstlane(sm_flag[0]) || !used) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    // In the chunks' order, so that the result does not depend on which one was last.
    float mt = -INFINITY;
    for (int c = 0; c < rt.chunks; ++c) mt = fmaxf(mt, mine[c * part_step]);
    m = mt;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < NC; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
#pragma unroll 1
    for (int c = 0; c < rt.chunks; ++c) {
      const float* from = mine + c * part_step;
      const float f = part_weight(from[0], mt);
      l += f * from[1];
#pragma unroll
      for (int d = 0; d < NC; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 x = *reinterpret_cast<const float2*>(from + (1 + d * 8 + i / 2) * 128);
          acc[d][i] += f * x.x;
          acc[d][i + 1] += f * x.y;
        }
    }
  }
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
    a.lse[(int64_t)(q0 + tok) * (a.hk * a.group) + head] = bad ? NAN : log_sum<DT>(m, l);
}

template <int DT, int MODE>
hipError_t launch_mode(const AttnArgs& a, hipStream_t s, const LaunchEvents& ev) {
  const int64_t tiles = ((int64_t)a.n_tok * a.group + kTileM - 1) / kTileM + a.n_req + a.chunks;
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
  const bool cap = a.cap_out != 0.f, bias = a.slopes || !(a.scale2 > 0.f);
  if (a.cap_out > kNearCap * kLog2e) return launch_mode<DT, kWideCap>(a, s, ev);
  return bias && cap ? launch_mode<DT, kBiasCap>(a, s, ev)
         : bias      ? launch_mode<DT, kBias>(a, s, ev)
         : cap       ? launch_mode<DT, kCap>(a, s, ev)
                     : launch_mode<DT, kPlain>(a, s, ev);
}

}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& a, int32_t dtype, hipStream_t s, const LaunchEvents& ev) {
  return dtype == SLORA_F16 ? launch_dt<SLORA_F16>(a, s, ev) : launch_dt<SLORA_BF16>(a, s, ev);
}

}  // namespace slora
