// kvq_latent.cuh -- what the latent-cache kernels share: the page's layout, the
// arguments of the attention kernels, the dequantization of sixteen codes, and the
// launchers.
#pragma once

#include "kvq_chunk.cuh"

struct kvq_latent {
  kvq_latent_config cfg;
  uint8_t* base;      // device pool (header at byte 0)
  size_t page_bytes;  // of one page of 16 tokens
};

namespace kvq {

constexpr int kLatentRope = 64;    // rotary channels
constexpr int kLatentHead = 128;   // an expanded head's other key channels, and its values

// A page: codes, then the rotary rows, then the scales.
template <int MODE>
constexpr bool kLatentFour = MODE == KVQ_NVFP4 || MODE == KVQ_NVFP4_4OVER6;
template <int MODE>
constexpr bool kLatentTokenScale = MODE == KVQ_INT8_PER_TOKEN_HEAD || MODE == KVQ_FP8_PER_TOKEN_HEAD;
template <int MODE, int L>
struct LatentPage {
  static constexpr int CODES = kLatentFour<MODE> ? L / 2 : L;  // bytes of a token's codes
  static constexpr int ROPE = 16 * CODES;
  static constexpr int SCALES = ROPE + 16 * kLatentRope * 2;
  static constexpr int BYTES = SCALES + (kLatentFour<MODE> ? L : kLatentTokenScale<MODE> ? 64 : 0);
};
inline size_t latent_page_bytes(int mode, int L) {
  const bool four = mode == KVQ_NVFP4 || mode == KVQ_NVFP4_4OVER6;
  return (size_t)16 * (four ? L / 2 : L) + 16 * kLatentRope * 2 + (four ? L : mode == KVQ_FP8_PER_TENSOR ? 0 : 64);
}
Span latent_pages(const kvq_latent* c);  // the pool without its header

// Sixteen codes as fp16 pairs, exact: one-byte codes from 16 bytes, E2M1 codes from 8
// times their E4M3 block scale (6 significant bits at most).
template <int MODE>
__device__ __forceinline__ void latent_codes16(const uint32_t* w, uint32_t sb, uint32_t* h) {
  if constexpr (kLatentFour<MODE>) {
    const __half s1 = __low2half(u32_as_h2(e4m3x2_to_f16x2(sb & 0xFFu)));
    const __half2 s = __half2half2(s1);
    e2m1x8_to_f16x2x4(w[0], h);
    e2m1x8_to_f16x2x4(w[1], h + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = h2_as_u32(__hmul2(u32_as_h2(h[i]), s));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (MODE == KVQ_INT8_PER_TOKEN_HEAD) {
        const __half2 bias = u32_as_h2(0x64806480u);  // 1024 + (x + 128) - 1152
        const uint32_t v = w[i] ^ 0x80808080u;
        h[2 * i] = h2_as_u32(__hsub2(u32_as_h2(prmt(v, 0x64646464u, 0x4140u)), bias));
        h[2 * i + 1] = h2_as_u32(__hsub2(u32_as_h2(prmt(v, 0x64646464u, 0x4342u)), bias));
      } else {
        h[2 * i] = e4m3x2_to_f16x2(w[i] & 0xFFFFu);
        h[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
      }
    }
  }
}

// Arguments of the attention kernels.  Of ChunkArgs: absorbed, all heads share one key
// head (Hkv = 1, G = Hq); expanded, each has its own (Hkv = Hq, G = 1).
struct LatentArgs : ChunkArgs {
  int causal;
  // The tcgen05 kernel's CTAs where row tiles are split: CTA c leaves its rows' partials at
  // ws_o [c][rows][L] and ws_ml [c][rows][2], and (first CTA, parts) of row tile i < ctas is at
  // map[i].
  // 0: a CTA takes a whole row tile.
  int ctas;
  int2* map;
  float* lse;  // [total_q][Hq] or null
  Span lse_span;
  // expanded
  const int32_t* cu_k;
  const void* k;
  const void* k_rope;
  const void* v;
  long long k_stride, k_head_stride, v_stride, v_head_stride, k_rope_stride;
  int total_k;
  int group;  // heads whose CTAs run together
};

// The rows of a CTA.  Expanded: a sequence's tokens are its range of cu_k.
template <bool EXPANDED>
__device__ __forceinline__ RowTile latent_tile(const LatentArgs& a, int index, int rows, bool flag) {
  if constexpr (!EXPANDED) {
    return find_tile(a, index, rows, flag);
  } else {
    return find_tile(
        a, index, rows, flag, a.max_seq_len, [&](int b) { return (int)max(0ll, min((long long)a.max_seq_len, (long long)__ldg(a.cu_k + b + 1) - __ldg(a.cu_k + b))); },
        [&](int b, bool f) {
          const int k0 = __ldg(a.cu_k + b), k1 = __ldg(a.cu_k + b + 1);
          const bool bad = k0 < 0 || k1 < k0 || k1 > a.total_k || k1 - k0 > a.max_seq_len;  // (k1 - k0: after k0 >= 0 and k1 >= k0)
          if (bad && f) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_QUERY_RANGE);
          return bad;
        });
  }
}
// Tokens that row rr of a sequence's chunk sees (from its first), 0 and up.
__device__ __forceinline__ int latent_sees(const LatentArgs& a, const RowTile& t, int rr) {
  return a.causal ? max(0, t.n - t.m + rr / a.G + 1) : t.n;
}
// Row of q, out and the partials that row rr of a tile's sequence is.
__device__ __forceinline__ long long latent_row(const LatentArgs& a, const RowTile& t, int kvh, int rr) {
  return (long long)(t.q0 + rr / a.G) * a.Hq + kvh * a.G + rr % a.G;
}

// A CTA's part of a row tile.
struct LatentPart {
  RowTile t;
  int tile;         // the row tile's number, as find_tile counts
  int part, parts;  // of its token range
  int first;        // the CTA of its part 0
};
// CTA `cta` of a.ctas: each sequence's range is cut into parts of at most T tiles of 128 tokens,
// with the smallest T for which the batch has no more parts than CTAs.  (The host has bounds
// of the lengths only; equal counts of parts, for any lengths, left CTAs with a few tiles
// beside others with many.)  One warp; seqs: shared memory for (row tiles, token tiles) of
// kLatentSeqs sequences.
constexpr int kLatentSeqs = 512;
__device__ __forceinline__ LatentPart latent_part(const LatentArgs& a, int cta, int rows, bool flag, int2* seqs) {
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int lim = (int)min((long long)a.max_seq_len, (long long)a.max_pages * 16);
  LatentPart p{{-1, 0, 0, 0, 0, 0, 0}, 0, 0, 1, 0};
  int most = 1;
  for (int b = lane; b < a.B; b += 32) {
    const int q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1), n = __ldg(a.seq_lens + b);
    int2 s = make_int2(0, 1);
    if (q0 < 0 || q1 < q0 || q1 > a.total_q || q1 - q0 > a.max_q_len) {
      if (flag) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_QUERY_RANGE);
    } else if (q1 > q0) {
      if (flag && (n > lim || n < 0)) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_SEQ_LEN);
      s.x = (int)(((long long)(q1 - q0) * a.G + rows - 1) / rows);
      s.y = max(1, (max(0, min(n, lim)) + 127) / 128);
      most = max(most, s.y);
    }
    seqs[b] = s;
  }
  __syncwarp();
  const int cap = a.ctas + 1;
  auto parts = [&](int2 s, int T) { return min(cap, (s.y + T - 1) / T); };
  int lo = 1, hi = __reduce_max_sync(kAll, most);
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    int sum = 0;
    for (int b = lane; b < a.B; b += 32) sum += seqs[b].x * parts(seqs[b], mid);
    if (__reduce_add_sync(kAll, sum) <= a.ctas) hi = mid;
    else lo = mid + 1;
  }
  int before = 0, tiles_before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    const int2 s = b < a.B ? seqs[b] : make_int2(0, 1);
    const int n = parts(s, lo);
    int upto = s.x * n, tiles = s.x;  // inclusive prefix sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kAll, upto, o), y = __shfl_up_sync(kAll, tiles, o);
      if (lane >= o) {
        upto += x;
        tiles += y;
      }
    }
    const uint32_t who = __ballot_sync(kAll, cta >= before + upto - s.x * n && cta < before + upto);
    if (who) {
      const int src = __ffs(who) - 1;
      const int R = __shfl_sync(kAll, s.x, src), start = before + __shfl_sync(kAll, upto, src);
      p.parts = __shfl_sync(kAll, n, src);
      const int at = cta - (start - R * p.parts), k = at / p.parts;  // row tiles from the chunk's last rows
      p.part = at % p.parts;
      p.first = cta - p.part;
      p.tile = tiles_before + __shfl_sync(kAll, tiles, src) - R + k;
      p.t.seq = b0 + src;
      p.t.q0 = __ldg(a.cu_q + p.t.seq);
      p.t.m = __ldg(a.cu_q + p.t.seq + 1) - p.t.q0;
      p.t.n = max(0, min(__ldg(a.seq_lens + p.t.seq), lim));
      p.t.r0 = (R - 1 - k) * rows;
      p.t.count = (int)min((long long)rows, (long long)p.t.m * a.G - p.t.r0);
      break;
    }
    before += __shfl_sync(kAll, upto, 31);
    tiles_before += __shfl_sync(kAll, tiles, 31);
  }
  return p;
}

struct LatentPlan {
  int num_splits = 1;  // at most so many parts of a row tile
  int ctas = 0;        // of the tcgen05 kernel, where it splits
  size_t workspace_bytes = 0;
};
// rows: query rows of a CTA of the tcgen05 kernel, from the largest chunk
inline int latent_umma_rows(int max_q_len, int Hq) {
  const long long most = (long long)max_q_len * Hq;
  return most <= 16 ? 16 : most <= 32 ? 32 : 64;
}
LatentPlan plan_latent(const kvq_latent* c, int total_q, int num_seqs, int num_q_heads, int max_q_len, int max_seq_len,
                       int out_dtype);
cudaError_t launch_latent_attention(const kvq_latent* c, const LatentPlan& p, LatentArgs& a, cudaStream_t s);
cudaError_t launch_latent_prompt(const kvq_latent* c, LatentArgs& a, cudaStream_t s);
cudaError_t launch_latent_umma(const kvq_latent* c, const LatentArgs& a, cudaStream_t s);         // absorbed
cudaError_t launch_latent_prompt_umma(const kvq_latent* c, const LatentArgs& a, cudaStream_t s);  // expanded
cudaError_t launch_latent_write(const kvq_latent* c, const kvq_latent_rows& r, cudaStream_t s);
cudaError_t launch_latent_read(const kvq_latent* c, const int32_t* slots, int num_tokens, void* latent_out, void* rope_out,
                               int out_dtype, cudaStream_t s);

}  // namespace kvq
