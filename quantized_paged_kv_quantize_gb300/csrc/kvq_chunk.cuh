// kvq_chunk.cuh -- what the chunk attention kernels share: their arguments, the
// search for a CTA's rows in the ragged batch, the rule of which tokens a row
// sees, and the launchers.
#pragma once

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

struct ChunkArgs {
  const uint8_t* pool;
  const void* q;                // [total_q][Hq][D]
  const int32_t* cu_q;          // [B + 1]
  const int32_t* block_table;   // [B][max_pages]
  const int32_t* seq_lens;      // [B]
  const int32_t* prefix_lens;   // [B] or null
  const float* slopes;          // [Hq] or null
  void* out;                    // [total_q][Hq][D]
  float* ws_o;                  // [total_q][Hq][splits][D]
  float* ws_ml;                 // [total_q][Hq][splits][2]
  int total_q, B, Hq, Hkv, G, num_pages, max_pages, max_q_len, max_seq_len;
  int window;      // 0: none
  int num_splits;  // parts of a row tile's token range, one CTA each
  int out_f32;
  float scale;     // of q . k
  float cap;       // 0: none
  size_t block_bytes;
  Span out_span, ws_span;
};

// A CTA's rows: rows r0 .. r0 + count - 1 of a sequence's chunk for one kv
// head, row r being query r / G under head r % G of the group.
struct RowTile {
  int seq;       // -1: no such tile
  int q0, m, n;  // first query row of the chunk, its queries, the sequence's tokens
  int prefix;    // tokens that every query of the sequence sees
  int r0, count;
};

// Upper bound of the row tiles of a batch: sum over its sequences of
// ceil(m G / rows) <= total_q G / rows + (sequences with a query).
inline long long chunk_tile_bound(int total_q, int B, int G, int rows) {
  return (long long)total_q * G / rows + (total_q < B ? total_q : B);
}

// Tile `index` of the batch, counted sequence by sequence, each chunk from its
// last rows (the longest contexts) to its first.  All lanes of a warp call it.
// A sequence whose cu_q entries are not an ascending range of at most
// max_q_len rows inside the batch is flagged (by the CTAs with `flag`) and has
// no tiles; a seq_len outside its bounds is flagged and clamped.
__device__ __forceinline__ RowTile find_tile(const ChunkArgs& a, int index, int rows, bool flag) {
  const int lane = threadIdx.x & 31;
  RowTile t{-1, 0, 0, 0, 0, 0, 0};
  const int lim = (int)min((long long)a.max_seq_len, (long long)a.max_pages * 16);
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int q0 = 0, m = 0, tiles = 0, n = 0, prefix = 0;
    if (b < a.B) {  // (all loads at once)
      q0 = __ldg(a.cu_q + b);
      const int q1 = __ldg(a.cu_q + b + 1);
      n = __ldg(a.seq_lens + b);
      if (a.prefix_lens) prefix = __ldg(a.prefix_lens + b);
      if (q0 < 0 || q1 < q0 || q1 > a.total_q || q1 - q0 > a.max_q_len) {
        if (flag) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_QUERY_RANGE);
      } else {
        m = q1 - q0;
        tiles = (int)(((long long)m * a.G + rows - 1) / rows);
      }
      if (n > lim || n < 0) {
        if (flag && m > 0) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_SEQ_LEN);
        n = n < 0 ? 0 : lim;
      }
    }
    int upto = tiles;  // inclusive prefix sum over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const bool mine = index >= before + upto - tiles && index < before + upto;
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    if (who && t.seq < 0) {
      const int src = __ffs(who) - 1;
      t.seq = b0 + src;
      t.q0 = __shfl_sync(0xffffffffu, q0, src);
      t.m = __shfl_sync(0xffffffffu, m, src);
      t.n = __shfl_sync(0xffffffffu, n, src);
      t.prefix = max(0, min(__shfl_sync(0xffffffffu, prefix, src), t.n));
      const int k = before + __shfl_sync(0xffffffffu, upto, src) - 1 - index;  // from the chunk's first rows
      t.r0 = k * rows;
      t.count = (int)min((long long)rows, (long long)t.m * a.G - t.r0);
      if (!flag) break;  // (a flagging warp looks at every sequence)
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return t;
}

// The KV tiles (of `kt` tokens) that some row of a CTA sees, as up to two runs
// of tile numbers: the prefix's, then the causal (and windowed) ones.
struct TokenRange {
  int p_min, p_max;   // positions of the CTA's first and last query
  int lowest;         // first token of the window of the CTA's first query (0 without a window)
  int prefix;         // tokens below it are seen by every row (at a position >= 0)
  int first, second;  // tiles of the first run (from 0); first tile of the second run
  int tiles;          // in all
  // a page of the tiles that lies wholly between the prefix and the windows: not seen by any row, and not read
  // (it may have been given up)
  __device__ __forceinline__ bool unseen(int page) const { return page * 16 + 16 <= lowest && page * 16 >= prefix; }
  __device__ __forceinline__ int tile(int i) const { return i < first ? i : second + (i - first); }
};
__device__ __forceinline__ TokenRange token_range(const ChunkArgs& a, const RowTile& t, int kt) {
  TokenRange r;
  r.p_min = t.n - t.m + t.r0 / a.G;
  r.p_max = t.n - t.m + (t.r0 + t.count - 1) / a.G;
  r.prefix = t.prefix;
  r.lowest = a.window > 0 ? max(0, max(r.p_min, 0) - a.window + 1) : 0;
  if (r.p_max < 0) {  // more queries than tokens: these see nothing
    r.first = r.second = r.tiles = 0;
    return r;
  }
  const int hi = (r.p_max + kt) / kt;  // tiles up to the last query's own token
  const int lo = r.lowest / kt;
  r.first = min((r.prefix + kt - 1) / kt, lo);
  r.second = lo;
  r.tiles = r.first + max(hi, (r.prefix + kt - 1) / kt) - lo;
  return r;
}
// Whether every row of the CTA sees every token of [t0, t0 + kt).
__device__ __forceinline__ bool all_see(const ChunkArgs& a, const TokenRange& r, int t0, int kt) {
  if (r.p_min < 0) return false;
  return t0 + kt <= r.prefix || (t0 + kt <= r.p_min + 1 && (a.window == 0 || t0 > r.p_max - a.window));
}
// One row's tokens: t in [lo, hi) or t < prefix.
struct RowSees {
  int lo, hi, prefix;
  __device__ __forceinline__ bool operator()(int t) const { return (t >= lo && t < hi) || t < prefix; }
};
__device__ __forceinline__ RowSees row_sees(const ChunkArgs& a, const TokenRange& r, int pos, bool real) {
  if (!real || pos < 0) return {0, 0, 0};
  return {a.window > 0 ? max(0, pos - a.window + 1) : 0, pos + 1, r.prefix};
}

// Merge of the splits of the row tiles (kvq_chunk.cu); `rows`: of a tile.
cudaError_t launch_chunk_combine(const kvq_cache* c, const ChunkArgs& a, int rows, cudaStream_t stream);

// The tcgen05 kernel (kvq_chunk_umma.cu): rows of a CTA, and the launch.
constexpr int kUmmaRows = 256;
cudaError_t launch_chunk_umma(const kvq_cache* c, const ChunkArgs& a, cudaStream_t s);

}  // namespace kvq
