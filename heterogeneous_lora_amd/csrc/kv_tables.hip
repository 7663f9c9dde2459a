// Block tables, slot maps and positions of a step, built on the GPU from its requests'
// lengths (slora_kv_tables): the S-LoRA overview, section "1. Unified Paging", keeps the
// KV cache on pages of the unified pool; a request's tokens are found through a table of
// its pages.
//
// The page list comes block by block, each block's planes together; a table row holds one
// plane's blocks. So the work is a transposition, bound by the bytes of the list and the
// tables: a workgroup copies runs of 64 blocks (one stretch of the list) to LDS and writes
// each plane's 256 bytes of the row, 16 bytes a lane. Where a request's blocks start in the
// list and its tokens in the step's arrays is the sum of the lengths before it: every
// workgroup adds them up by itself (at most 16384 of them, L2 hits), which takes less time
// than another launch and a hand-over through memory. Short rows, a step's one new block
// or token, take as many lanes as they need, so that all planes are written at once. A
// rebuild of 560 requests x 80 planes (671 MB): 154 us, 4.4 TB/s; one step's new blocks of 256
// requests x 64 planes: 5.5 us.
#include "device_common.h"

namespace slora {
namespace {

constexpr int kThreads = 256;
constexpr int kPlanes = 96;   // planes a workgroup turns at once, at most
constexpr int kBlocks = 64;   // blocks of a tile
constexpr int kLdsInts = kBlocks * (kPlanes | 1);  // rows of an odd stride: no bank conflicts

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

struct Sums {
  int64_t blocks, tokens;
};

__device__ __forceinline__ int64_t div_up(int64_t a, int32_t b) {
  const uint64_t n = (uint64_t)a + (uint32_t)b - 1;
  return (n >> 32) ? (int64_t)(n / (uint32_t)b) : (int64_t)((uint32_t)n / (uint32_t)b);
}

struct Request {
  int64_t past, seq;      // tokens cached before, and after the step
  int64_t first, blocks;  // its blocks [first, blocks) are in the list
};

__device__ __forceinline__ Request request(const slora_kv_step& st, int32_t tpp, int r) {
  Request q;
  q.past = max(st.past_len[r], 0);
  q.seq = q.past + max(st.new_len[r], 0);
  q.blocks = div_up(q.seq, tpp);
  q.first = st.append ? div_up(q.past, tpp) : 0;
  return q;
}

// Sums over requests [0, r) of their list blocks and new tokens, on every thread.
__device__ Sums sums_before(const slora_kv_step& st, int32_t tpp, int r) {
  __shared__ Sums part[kThreads / 64];
  Sums s{0, 0};
  for (int i = (int)threadIdx.x; i < r; i += kThreads) {
    const Request q = request(st, tpp, i);
    s.blocks += q.blocks - q.first;
    s.tokens += q.seq - q.past;
  }
  for (int d = 32; d; d >>= 1) {
    s.blocks += __shfl_xor(s.blocks, d);
    s.tokens += __shfl_xor(s.tokens, d);
  }
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = part[0];
  for (int w = 1; w < kThreads / 64; ++w) {
    s.blocks += part[w].blocks;
    s.tokens += part[w].tokens;
  }
  return s;
}

// A value that is the same on every thread, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Lanes that take one row of n elements: a power of two up to 64.
__device__ __forceinline__ int row_lanes_log2(int n) { return n >= 64 ? 6 : n <= 1 ? 0 : 32 - __builtin_clz(n - 1); }

// blockIdx.y = request (n_requests: the rows past the step's tokens), blockIdx.x = its
// share of the row's tiles, blockIdx.z = group of planes.
template <bool APPEND>
__global__ __launch_bounds__(kThreads) void kv_tables_kernel(slora_kv_step st, int64_t n_pages, int32_t tpp, int32_t n_req,
                                                             int32_t max_blocks, int32_t group, uint32_t magic,
                                                             uint32_t shift) {
  __shared__ int32_t tile[kLdsInts];
  const int r = (int)blockIdx.y, tid = (int)threadIdx.x;
  const int p0 = (int)blockIdx.z * group, np = min(st.n_planes - p0, group);
  const int64_t T = st.n_tokens;
  const int sub = (int)blockIdx.x, n_sub = (int)gridDim.x;

  if (r == n_req) {
    const int64_t total = min(sums_before(st, tpp, n_req).tokens, T);
    if (sub == 0 && p0 == 0 && tid == 0) st.q_offsets[n_req] = (int32_t)total;
    for (int64_t t = total + sub * kThreads + tid; t < T; t += n_sub * kThreads) {
      if (p0 == 0) {
        st.token_request[t] = -1;
        st.position[t] = -1;
      }
      for (int p = 0; p < np; ++p) st.slots[(int64_t)(p0 + p) * T + t] = -1;
    }
    return;
  }

  const Request q = request(st, tpp, r);
  // blocks this row deals with: all of it, or the ones the new tokens touch
  const int64_t b_begin = APPEND ? q.past / tpp : 0;
  const int64_t b_used = q.seq > q.past || !APPEND ? min(q.blocks, (int64_t)max_blocks) : b_begin;
  const int64_t b_end = APPEND ? b_used : max_blocks;
  const int stride = np | 1;
  const int64_t tile0 = b_begin + (int64_t)sub * kBlocks;
  if (sub != 0 && tile0 >= b_end) return;
  // 16-byte stores where the rows allow them (a tile begins at a multiple of 64 blocks)
  const bool wide = !APPEND && max_blocks % 4 == 0 && ((uintptr_t)st.tables & 15) == 0;

  // Rows past the request's blocks are -1 and need no sums.
  const bool any_used = sub == 0 || tile0 < b_used;
  Sums before{0, 0};
  if (any_used) before = sums_before(st, tpp, r);
  const int64_t t_first = before.tokens;
  if (sub == 0 && p0 == 0 && tid == 0) {
    st.seq_len[r] = (int32_t)min(q.seq, (int64_t)INT32_MAX);
    st.q_offsets[r] = (int32_t)min(t_first, T);
  }

  // A tile's page ids: entry i is block i / group's id of plane i % group.
  const int64_t list0 = uniform(before.blocks) - q.first;
  auto block_of = [&](int i) { return group == 1 ? i : (int)(__umulhi((uint32_t)i, magic) >> shift); };
  auto used_from = [&](int64_t b0) { return (int)max(min(min(b0 + kBlocks, b_end), b_used) - b0, (int64_t)0); };
  // A rebuild reads them a tile ahead of the rows being written, kHold to a thread, all
  // loads in flight at once (an id past the tile or the list reads the last one).
  constexpr int kHold = kBlocks * kPlanes / kThreads;
  int32_t held[kHold];
  auto read = [&](int64_t b0) {
    const int n_used = used_from(b0);
    const int64_t at0 = (list0 + b0) * st.n_planes + p0, left = st.n_page_ids - at0;
    if (n_used == 0 || left <= 0) return;
    const int last = (int)min((int64_t)((n_used - 1) * st.n_planes + np), left) - 1;
    const int32_t* from = st.pages + at0;
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
      const int i = tid + u * kThreads, b = block_of(i);
      held[u] = from[min(b * st.n_planes + i - b * group, last)];
    }
  };
  if (!APPEND) read(tile0);
  for (int64_t b0 = tile0; b0 < b_end; b0 += (int64_t)n_sub * kBlocks) {
    const int n = (int)(min(b0 + kBlocks, b_end) - b0), n_used = used_from(b0);
    if (n_used > 0) {
      const int64_t at0 = (list0 + b0) * st.n_planes + p0, left = st.n_page_ids - at0;
      __syncthreads();  // the previous tile has been read
      if (APPEND) {
        for (int i = tid; i < n_used * group; i += kThreads) {
          const int b = block_of(i), p = i - b * group;
          if (p >= np) continue;
          int32_t page = -1;
          if (b0 + b >= q.first) {
            const int64_t off = (int64_t)b * st.n_planes + p;
            if (off < left) page = st.pages[at0 + off];
          } else {  // the block the step before left part full
            page = st.tables[((int64_t)(p0 + p) * n_req + r) * max_blocks + b0 + b];
          }
          tile[b * stride + p] = page;
        }
      } else {
#pragma unroll
        for (int u = 0; u < kHold; ++u) {
          const int i = tid + u * kThreads, b = block_of(i), p = i - b * group;
          if (b < n_used && p < np) tile[b * stride + p] = (int64_t)b * st.n_planes + p < left ? held[u] : -1;
        }
      }
      __syncthreads();
      if (!APPEND) read(b0 + (int64_t)n_sub * kBlocks);
    }
    // table rows: from the tile, -1 past the request's blocks
    if (wide) {
      for (int p = tid >> 4; p < np; p += kThreads >> 4) {
        const int b = (tid & 15) * 4;
        if (b >= n) continue;
        i32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = b + e < n_used ? tile[(b + e) * stride + p] : -1;
        // Past the caches, where the ids of the tiles to come are kept instead (560 requests
        // x 80 planes, 413 MB of tables: 154 us against 160).
        __builtin_nontemporal_store(x, reinterpret_cast<i32x4*>(st.tables + ((int64_t)(p0 + p) * n_req + r) * max_blocks + b0 + b));
      }
    } else {
      const int w0 = (int)max(q.first - b0, (int64_t)0);  // append: the part-full block stays
      const int log2 = row_lanes_log2(n - w0), lanes = 1 << log2;
      for (int p = tid >> log2; p < np; p += kThreads >> log2) {
        int32_t* row = st.tables + ((int64_t)(p0 + p) * n_req + r) * max_blocks + b0;
        for (int b = w0 + (tid & (lanes - 1)); b < n; b += lanes) row[b] = b < n_used ? tile[b * stride + p] : -1;
      }
    }
    // slots, positions and ids of the new tokens on these blocks
    const int64_t s0 = max(b0 * tpp, q.past), s1 = min((b0 + n_used) * (int64_t)tpp, q.seq);
    const int64_t at = t_first + s0 - q.past;
    const int n_tok = (int)max(min(s1 - s0, T - at), (int64_t)0);
    const int log2 = row_lanes_log2(n_tok), lanes = 1 << log2;
    for (int p = tid >> log2; p < np; p += kThreads >> log2) {
      for (int i = tid & (lanes - 1); i < n_tok; i += lanes) {
        const int64_t pos = s0 + i;
        const int64_t blk = (uint32_t)pos / (uint32_t)tpp;  // pos < 2^32
        const int32_t page = tile[(int)(blk - b0) * stride + p];
        const bool ok = page >= 0 && page < n_pages;
        st.slots[(int64_t)(p0 + p) * T + at + i] = ok ? (int64_t)page * tpp + (pos - blk * tpp) : -1;
        if (p0 + p == 0) {
          st.token_request[at + i] = r;
          st.position[at + i] = (int32_t)min(pos, (int64_t)INT32_MAX);
        }
      }
    }
  }

  // tokens past the table have no slot
  const int64_t limit = (int64_t)max_blocks * tpp;
  if (sub == 0 && q.seq > limit) {
    const int64_t from = max(q.past, limit), at = t_first + from - q.past;
    const int64_t n_tok = min(q.seq - from, T - at);
    for (int64_t i = tid; i < n_tok; i += kThreads) {
      if (p0 == 0) {
        st.token_request[at + i] = r;
        st.position[at + i] = (int32_t)min(from + i, (int64_t)INT32_MAX);
      }
      for (int p = 0; p < np; ++p) st.slots[(int64_t)(p0 + p) * T + at + i] = -1;
    }
  }
}

}  // namespace

hipError_t launch_kv_tables(const slora_kv& kv, const slora_kv_step& st, hipStream_t s,
                            const LaunchEvents& ev) {
  const int groups = (st.n_planes + kPlanes - 1) / kPlanes, group = (st.n_planes + groups - 1) / groups;
  uint32_t magic, shift;
  divisor(group, &magic, &shift);
  // Shares of a row: enough workgroups to fill the device, no more than a row has tiles (an
  // append: than the step's tokens could fill).
  const int64_t rows = (int64_t)(kv.n_requests + 1) * groups;
  int64_t sub = (2048 + rows - 1) / rows;
  int64_t blocks = kv.max_blocks;
  if (st.append && blocks > st.n_tokens / kv.tokens_per_page + 2) blocks = st.n_tokens / kv.tokens_per_page + 2;
  const int64_t tiles = (blocks + kBlocks - 1) / kBlocks;
  if (sub > tiles) sub = tiles;
  if (sub < 1) sub = 1;
  hipExtLaunchKernelGGL(st.append ? kv_tables_kernel<true> : kv_tables_kernel<false>,
                        dim3((unsigned)sub, (unsigned)(kv.n_requests + 1), (unsigned)groups), dim3(kThreads), 0, s,
                        ev.start, ev.stop, 0, st, kv.n_pages, kv.tokens_per_page, kv.n_requests, kv.max_blocks, group,
                        magic, shift);
  return hipGetLastError();
}

}  // namespace slora
