// kvq_chunk.cu -- attention of ragged chunks of new tokens over the packed
// paged cache (kvq_chunk_attention): the plan, the merge of split token ranges,
// and the mma.sync kernel that takes fp32 queries or outputs and head_dim 32.
//
// For query i of a sequence's m new tokens, at position p = n - m + i:
//   s_t = scale q . k_t,  s_t = cap tanh(s_t / cap),  s_t -= slope_h |p - t|
//   o = sum_t softmax(s)_t v_t over t <= p (and t > p - window) or t < prefix
// k_t, v_t are codes times scales; codes are exact in fp16, so both products
// run on them and the scales go to the fp32 scores and into P.
//
// mma.sync kernel: a CTA of four warps takes 64 rows (query x head of a kv
// head's group, 16 a warp) and walks over KT-token tiles.  The CTA's threads
// bring a tile's packed words into registers one tile ahead, write the codes as
// fp16 rows to shared memory, and each warp multiplies them with its rows:
// S = Q K^T, online softmax in base 2 with the running maximum and sum in fp32,
// O += P V with fp32 accumulators.  fp32 queries enter as an fp16 hi + lo pair
// under a power of two per row, P always does (22 bits of each weight), so the
// result keeps fp32 grade.  The maximum is that of the score plus the exponent of
// the value's scale, over the tokens that the row sees: its largest P (a weight
// times a value scale) then lies between 2^(kTop - 1) and 2^(kTop + 1) whatever the
// magnitudes (it is rounded up to a whole number, so that no rescale rounds), and one below fp16's range is off by 2^-38 of the largest at most.
// Bound by the matrix and conversion instructions, which the pairs double: three int8
// prompts of 700 to 2048 tokens with 32 fp32 heads of 128 take 480 us (42 GFLOP of the
// formula); four chunks of 60 to 300 tokens with heads of 32, 18 us, mostly latency.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kvq_chunk.cuh"
#include "kvq_unpack.cuh"

namespace kvq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16 * kWarps;

constexpr float kTop = 14.0f;      // log2 of a row's largest P

template <int D>
constexpr int kTile = D == 128 ? 32 : 64;  // tokens

__device__ __forceinline__ void ldsm4(uint32_t* r, const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
// x = hi + lo in fp16 (the remainder of the first rounding is exact in fp32)
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  hi = h2_as_u32(h);
  lo = h2_as_u32(__floats2half2_rn(x0 - f.x, x1 - f.y));
}
// floor(log2 x) of a positive x, kept to exponents whose powers are normal both ways
__device__ __forceinline__ int exponent(float x) {
  return max(-126, min(126, (int)((__float_as_uint(x) >> 23) & 0xFFu) - 127));
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

template <int MODE, int D, bool QF32>
__global__ void __launch_bounds__(kThreads) chunk_mma_kernel(const __grid_constant__ ChunkArgs a) {
  constexpr int KT = kTile<D>, ST = D + 8;  // smem row stride (halves): 16-byte chunks of 8 rows hit 8 bank groups
  constexpr int J = D / 8, U = KT * J / kThreads;  // 8-channel units per row; units per thread and side
  constexpr bool PT = kPerTokenScale<MODE>;
  __shared__ __align__(16) __half ks[KT * ST], vs[KT * ST];
  __shared__ float kscale[KT], vscale[KT], vexp[KT];  // vexp: floor(log2 vscale)
  __shared__ RowTile tile_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int kvh = blockIdx.y, split = blockIdx.z;
  if (warp == 0) {
    const RowTile t = find_tile(a, blockIdx.x, kRows, blockIdx.x == 0 && kvh == 0 && split == 0);
    if (lane == 0) tile_s = t;
  }
  __syncthreads();
  const RowTile t = tile_s;
  if (t.seq < 0) return;
  const TokenRange tr = token_range(a, t, KT);
  const int i0 = (int)((long long)tr.tiles * split / a.num_splits);
  const int i1 = (int)((long long)tr.tiles * (split + 1) / a.num_splits);

  // this thread's rows g, g + 8 of its warp's 16
  int pos[2], hq[2];
  long long qrow[2];
  bool real[2];
  float slope[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = 16 * warp + g + 8 * u;
    real[u] = r < t.count;
    const int rr = t.r0 + (real[u] ? r : 0);
    pos[u] = t.n - t.m + rr / a.G;
    hq[u] = kvh * a.G + rr % a.G;
    qrow[u] = (long long)(t.q0 + rr / a.G) * a.Hq + hq[u];
    slope[u] = a.slopes ? __ldg(a.slopes + hq[u]) * kLog2e : 0.0f;
  }
  const RowSees sees[2] = {row_sees(a, tr, pos[0], real[0]), row_sees(a, tr, pos[1], real[1])};

  // Q as A fragments
  uint32_t qh[D / 16][4], ql[QF32 ? D / 16 : 1][4];
  float qfac[2] = {1.0f, 1.0f};
  if constexpr (QF32) {
    const float* q = static_cast<const float*>(a.q);
    float mx[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      for (int d = 2 * tq; d < D; d += 8) {
        const float2 x = __ldg(reinterpret_cast<const float2*>(q + qrow[u] * D + d));
        mx[u] = fmaxf(mx[u], fmaxf(fabsf(x.x), fabsf(x.y)));
      }
      mx[u] = warp_max_xor(mx[u], 1, 2);
      const int e = mx[u] > 0.0f ? exponent(mx[u]) : 0;
      mx[u] = pow2(-e);
      qfac[u] = pow2(e);
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int u = f & 1, d = 16 * j + 2 * tq + 8 * (f >> 1);
        const float2 x = __ldg(reinterpret_cast<const float2*>(q + qrow[u] * D + d));
        split2(x.x * mx[u], x.y * mx[u], qh[j][f], ql[j][f]);
      }
  } else {
    const __half* q = static_cast<const __half*>(a.q);
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int f = 0; f < 4; ++f)
        qh[j][f] = __ldg(reinterpret_cast<const uint32_t*>(q + qrow[f & 1] * D + 16 * j + 2 * tq + 8 * (f >> 1)));
  }

  float kfac = a.scale, vfac = 1.0f;
  if constexpr (!PT) {
    kfac *= *reinterpret_cast<const float*>(a.pool + kHdrKScaleOffset);
    vfac = *reinterpret_cast<const float*>(a.pool + kHdrVScaleOffset);
  }
  const float rcap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;

  // packed words of tile i: thread's units u = tid + 128 r -> token u / J, channels 8 (u % J) ..
  Packed8 pk[U], pv[U];
  float psc = 0.0f;    // per-token scale of token tid % KT, keys for tid < KT, values above
  bool there = false;  // that token is in the cache
  auto page_of = [&](int tok) -> int {  // the token's page, -1 past the sequence or out of the pool
    if (tok >= t.n || tr.unseen(tok >> 4)) return -1;
    const int pid = __ldg(a.block_table + (long long)t.seq * a.max_pages + (tok >> 4));
    if (pid < 0 || pid >= a.num_pages) {
      set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_PAGE_RANGE);
      return -1;
    }
    return pid;
  };
  auto block = [&](int pid) { return a.pool + kHeaderBytes + ((size_t)pid * a.Hkv + kvh) * a.block_bytes; };
  auto fetch = [&](int i) {
    const int t0 = tr.tile(i) * KT;
#pragma unroll
    for (int r = 0; r < U; ++r) {
      const int u = tid + kThreads * r, tok = t0 + u / J, j = u % J, pid = page_of(tok);
      pk[r] = pv[r] = Packed8{make_uint2(0u, 0u), 0u};  // an absent token: zero codes and scales
      if (pid >= 0) {
        pk[r] = load_packed8<MODE, D, 0>(block(pid), tok & 15, j);
        pv[r] = load_packed8<MODE, D, 1>(block(pid), tok & 15, j);
      }
    }
    psc = 0.0f;
    if (tid < 2 * KT) {
      const int tok = t0 + tid % KT, pid = page_of(tok);
      there = pid >= 0;
      if constexpr (PT) {
        if (there)
          psc = __ldg(reinterpret_cast<const float*>(block(pid) + (MODE == KVQ_INT4_PER_TOKEN_HEAD ? 16 * D : 32 * D) +
                                                     (tid < KT ? 0 : 64)) + (tok & 15));
      }
    }
  };

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  float m[2] = {kLowest, kLowest}, l[2] = {0.0f, 0.0f};

  if (i0 < i1) fetch(i0);
  for (int i = i0; i < i1; ++i) {
    const int t0 = tr.tile(i) * KT;
    __syncthreads();  // the previous tile has been read
#pragma unroll
    for (int r = 0; r < U; ++r) {
      const int u = tid + kThreads * r, tok = u / J, j = u % J;
      uint32_t h[4];
      codes8<MODE, 0>(pk[r], tok & 15, h);
      *reinterpret_cast<uint4*>(ks + tok * ST + 8 * j) = make_uint4(h[0], h[1], h[2], h[3]);
      codes8<MODE, 1>(pv[r], tok & 15, h);
      *reinterpret_cast<uint4*>(vs + tok * ST + 8 * j) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    if (tid < 2 * KT) {
      float* sc = tid < KT ? kscale : vscale;
      const int k = tid % KT;
      // an absent token (past the sequence, a missing page) is marked by a negative key scale
      sc[k] = tid < KT && !there ? -1.0f : PT ? psc : 1.0f;
      if (PT && tid >= KT) vexp[k] = scale_exponent(psc);
    }
    __syncthreads();
    if (i + 1 < i1) fetch(i + 1);

    // ---- S = Q K^T
    float s[KT / 8][4];
#pragma unroll
    for (int n = 0; n < KT / 8; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 16; j += 2) {
        uint32_t b[4];
        ldsm4(b, ks + (8 * n + (lane & 7)) * ST + 16 * j + 8 * (lane >> 3));
        mma16816(s[n], qh[j], b[0], b[1]);
        mma16816(s[n], qh[j + 1], b[2], b[3]);
        if constexpr (QF32) {
          mma16816(s[n], ql[j], b[0], b[1]);
          mma16816(s[n], ql[j + 1], b[2], b[3]);
        }
      }
    }

    // ---- scores in log2 units, the row's maximum
    const bool masked = !all_see(a, tr, t0, KT);
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < KT / 8; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int u = e >> 1, k = 8 * n + 2 * tq + (e & 1), tok = t0 + k;
        const float sc = kscale[k];
        float x = s[n][e] * (qfac[u] * (kfac * sc));
        if (a.cap > 0.0f) x = a.cap * tanhf(x * rcap);
        x = x * kLog2e;
        if (a.slopes) x -= slope[u] * fabsf((float)(pos[u] - tok));
        if (sc < 0.0f || (masked && !sees[u](tok))) x = -INFINITY;
        s[n][e] = x;
        mx[u] = fmaxf(mx[u], PT ? x + vexp[k] : x);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      mx[u] = fmaxf(ceilf(warp_max_xor(mx[u], 1, 2)), m[u]);  // whole: the rescale is exact
      const float al = ex2(m[u] - mx[u]);
      l[u] *= al;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][2 * u] *= al;
        o[n][2 * u + 1] *= al;
      }
      m[u] = mx[u];
    }

    // ---- P (times the value scale), split in fp16, and O += P V
    uint32_t ph[KT / 16][4], pl[KT / 16][4];
#pragma unroll
    for (int j = 0; j < KT / 16; ++j) {
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int n = 2 * j + (f >> 1), u = f & 1;
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = s[n][2 * u + e];
          p[e] = ex2(x - (m[u] - kTop));
          l[u] += p[e];
          // a weight of zero stays zero whatever the scale of a token that is not seen
          if constexpr (PT) p[e] = x == -INFINITY ? 0.0f : p[e] * vscale[8 * n + 2 * tq + e];
        }
        split2(p[0], p[1], ph[j][f], pl[j][f]);
      }
    }
    // The products cut their sums off, up to 2^-23 of O at each.  Over a range of more than
    // 2048 tokens a tile's are summed from zero and added to O with rounding (1024 queries
    // over 32768 tokens: 7e-7 instead of 1e-5 of the result, 6% slower); in a shorter one
    // the cuts come to 128 x 2^-23 where all values have one sign, and 1e-6 as a rule.
    auto pv = [&](auto anew) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        float c0[4] = {}, c1[4] = {};
        float *x0 = anew ? c0 : o[2 * n], *x1 = anew ? c1 : o[2 * n + 1];
#pragma unroll
        for (int j = 0; j < KT / 16; ++j) {
          uint32_t b[4];
          ldsm4_t(b, vs + (16 * j + (lane & 15)) * ST + 16 * n + 8 * (lane >> 4));
          mma16816(x0, ph[j], b[0], b[1]);
          mma16816(x1, ph[j], b[2], b[3]);
          mma16816(x0, pl[j], b[0], b[1]);
          mma16816(x1, pl[j], b[2], b[3]);
        }
        if (anew) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[2 * n][e] += c0[e];
            o[2 * n + 1][e] += c1[e];
          }
        }
      }
    };
    if ((i1 - i0) * KT > 2048) pv(std::true_type{});
    else pv(std::false_type{});
  }

#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] += __shfl_xor_sync(kFull, l[u], 1);
    l[u] += __shfl_xor_sync(kFull, l[u], 2);
    if (!real[u]) continue;
    const float f = vfac;  // (1 with per-token scales)
    if (a.num_splits == 1) {
      const float r = f / l[u];  // (a NaN score makes its row NaN; no token seen: 0)
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        const long long at = qrow[u] * D + 8 * n + 2 * tq;
        const float x = l[u] == 0.0f ? 0.0f : o[n][2 * u] * r, y = l[u] == 0.0f ? 0.0f : o[n][2 * u + 1] * r;
        if (a.out_f32) st_chk(reinterpret_cast<float2*>(static_cast<float*>(a.out) + at), make_float2(x, y), a.out_span, a.pool);
        else st_chk(reinterpret_cast<__half2*>(static_cast<__half*>(a.out) + at), __floats2half2_rn(x, y), a.out_span, a.pool);
      }
    } else {
      const long long pi = qrow[u] * a.num_splits + split;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        st_chk(reinterpret_cast<float2*>(a.ws_o + pi * D + 8 * n + 2 * tq), make_float2(o[n][2 * u] * f, o[n][2 * u + 1] * f),
               a.ws_span, a.pool);
      if (tq == 0) st_chk(reinterpret_cast<float2*>(a.ws_ml + 2 * pi), make_float2(l[u] == 0.0f ? -INFINITY : m[u], l[u]),
                          a.ws_span, a.pool);
    }
  }
}

// Merge of the splits: a warp per row (query x head) of a row tile, D / 32 channels
// a lane, eight partials in flight.  A split without tokens has m = -inf, and its
// partial is not read.  A CTA takes `span` rows: eight, or more where there are
// many rows, to find its tile once for them.
constexpr int kCombineWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kCombineWarps) chunk_combine_kernel(const __grid_constant__ ChunkArgs a, int rows, int span) {
  constexpr int C = D / 32;
  __shared__ RowTile tile_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kvh = blockIdx.y;
  pdl_wait_primary();
  if (warp == 0) {
    const RowTile t = find_tile(a, blockIdx.x, rows, false);
    if (lane == 0) tile_s = t;
  }
  __syncthreads();
  const RowTile t = tile_s;
  if (t.seq < 0) return;
  const int end = min(t.count, ((int)blockIdx.z + 1) * span);
  for (int r = blockIdx.z * span + warp; r < end; r += kCombineWarps) {
    const int rr = t.r0 + r;
    const long long row = (long long)(t.q0 + rr / a.G) * a.Hq + kvh * a.G + rr % a.G;
    const float2 v = lane < a.num_splits ? reinterpret_cast<const float2*>(a.ws_ml)[row * a.num_splits + lane]
                                         : make_float2(-INFINITY, 0.0f);  // at most 32 splits
    const float M = warp_max_xor(v.x, 1, 16);
    const float w = v.x == -INFINITY ? 0.0f : exp2f(v.x - M);
    float L = v.y * w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) L += __shfl_xor_sync(kFull, L, o);
    float acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.0f;
    for (int s0 = 0; s0 < a.num_splits; s0 += 8) {
      float x[8][C], ws[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        ws[u] = __shfl_sync(kFull, w, (s0 + u) & 31);  // (zero past the splits)
        const float* src = a.ws_o + (row * a.num_splits + s0 + u) * D + C * lane;
#pragma unroll
        for (int c = 0; c < C; ++c) x[u][c] = s0 + u < a.num_splits && ws[u] != 0.0f ? src[c] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] += ws[u] * x[u][c];
    }
    const float f = 1.0f / L;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float x = L == 0.0f ? 0.0f : acc[c] * f;
      const long long at = row * D + C * lane + c;
      if (a.out_f32) st_chk(static_cast<float*>(a.out) + at, x, a.out_span, a.pool);
      else st_chk(static_cast<__half*>(a.out) + at, __float2half_rn(x), a.out_span, a.pool);
    }
  }
}

template <int D, bool QF32>
cudaError_t launch_mma(int mode, const ChunkArgs& a, dim3 grid, cudaStream_t s) {
  switch (mode) {
    case KVQ_FP8_PER_TENSOR: chunk_mma_kernel<KVQ_FP8_PER_TENSOR, D, QF32><<<grid, kThreads, 0, s>>>(a); break;
    case KVQ_INT8_PER_TOKEN_HEAD: chunk_mma_kernel<KVQ_INT8_PER_TOKEN_HEAD, D, QF32><<<grid, kThreads, 0, s>>>(a); break;
    case KVQ_FP8_PER_TOKEN_HEAD: chunk_mma_kernel<KVQ_FP8_PER_TOKEN_HEAD, D, QF32><<<grid, kThreads, 0, s>>>(a); break;
    case KVQ_NVFP4:
    case KVQ_NVFP4_4OVER6: chunk_mma_kernel<KVQ_NVFP4, D, QF32><<<grid, kThreads, 0, s>>>(a); break;
    case KVQ_INT4_PER_TOKEN_HEAD: chunk_mma_kernel<KVQ_INT4_PER_TOKEN_HEAD, D, QF32><<<grid, kThreads, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_combine(const kvq_cache* c, const ChunkArgs& a, int rows, cudaStream_t stream) {
  const int most = (int)std::min<long long>(rows, (long long)a.max_q_len * a.G);  // rows of a tile
  cudaLaunchConfig_t cfg = {};
  const int span = (long long)a.total_q * a.Hq >= 64ll * kCombineWarps * num_sms() ? 64 : kCombineWarps;
  cfg.gridDim = dim3((unsigned)chunk_tile_bound(a.total_q, a.B, a.G, rows), a.Hkv, (most + span - 1) / span);
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = c->cfg.head_dim == 128 ? cudaLaunchKernelEx(&cfg, chunk_combine_kernel<128>, a, rows, span)
                                         : cudaLaunchKernelEx(&cfg, chunk_combine_kernel<32>, a, rows, span);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The tcgen05 kernel takes fp16 in and out at head_dim 128.
bool chunk_on_umma(const kvq_cache* c, int out_dtype) {
  return c->cfg.head_dim == 128 && c->cfg.io_dtype == KVQ_F16 && out_dtype == KVQ_F16;
}

// Splits of the token ranges.  The lengths are on the device: every tile of rows is
// taken to see max_seq_len tokens (a window bounds what it sees).  A plan of s splits is
// estimated at
//   ceil(units s / slots) waves x (token tiles / s + cost of a CTA)
// as for the decode kernels; more splits than one are worth their partials'
// way through memory only where a wave is not full or its last one is ragged.
int chunk_parts(bool umma, int D, int G, int Hkv, int total_q, int num_seqs, int max_q_len, int max_seq_len, int window,
                bool has_prefix) {
  const int rows = umma ? kUmmaRows : kRows;
  // tokens a CTA takes at a time: the tcgen05 kernel runs two tiles at once for up to 128 rows
  const int kt = !umma ? (D == 128 ? kTile<128> : kTile<32>) : (long long)max_q_len * G <= 128 ? 256 : 128;
  const long long slots = (umma ? 1ll : 4ll) * num_sms();  // CTAs side by side
  const long long cost_cta = !umma && D == 128 ? 8 : 4;    // start-up, merge and partials of a CTA, in such tiles
  long long len = max_seq_len;
  if (window > 0 && !has_prefix) len = std::min<long long>(len, (long long)window + max_q_len + kt);
  const long long tiles = (len + kt - 1) / kt;
  const long long per_seq = ((long long)max_q_len * G + rows - 1) / rows;
  long long units = ((long long)total_q * G + rows - 1) / rows + num_seqs / 2;
  units = std::min(units, per_seq * num_seqs) * Hkv;
  long long best = -1;
  int parts = 1;
  for (long long s = 1; s <= 32 && s <= std::max(1ll, tiles); ++s) {
    const long long cost = (units * s + slots - 1) / slots * ((tiles + s - 1) / s + cost_cta);
    if (best < 0 || cost < best) {
      best = cost;
      parts = (int)s;
    }
  }
  return parts;
}

// The splits are those of the kernel that the output's type chooses; the workspace, which
// a caller asks for without naming that type, serves the other one too.
ChunkPlan plan_chunk(const kvq_cache* c, int total_q, int num_seqs, int num_q_heads, int max_q_len, int max_seq_len,
                     int window, bool has_prefix, int out_dtype) {
  ChunkPlan p;
  const int D = c->cfg.head_dim, Hkv = c->cfg.num_kv_heads;
  if (max_q_len <= 1 && num_seqs <= 65535) {  // single tokens: the decode kernels (one grid row per sequence)
    int len = max_seq_len;
    if (window > 0 && !has_prefix) len = (int)std::min<long long>(len, (long long)window + 15);
    p.single = true;
    p.decode = plan_decode(c, num_seqs, num_q_heads, len);
    p.num_splits = p.decode.num_splits;
    p.workspace_bytes = p.decode.workspace_bytes;
    return p;
  }
  auto parts = [&](int out) {
    return chunk_parts(chunk_on_umma(c, out), D, num_q_heads / Hkv, Hkv, total_q, num_seqs, max_q_len, max_seq_len, window,
                       has_prefix);
  };
  p.num_splits = parts(out_dtype);
  const int most = std::max(parts(KVQ_F16), parts(KVQ_F32));
  if (most > 1) p.workspace_bytes = (size_t)total_q * num_q_heads * most * (D + 2) * sizeof(float);
  return p;
}

cudaError_t launch_chunk(const kvq_cache* c, const ChunkPlan& plan, const ChunkCall& k, cudaStream_t stream) {
  if (plan.single)
    return launch_decode(c, plan.decode, k.q, k.block_table, k.max_pages, k.seq_lens, k.num_seqs, k.num_q_heads,
                         k.max_seq_len, k.scale, k.out, k.out_dtype, k.workspace, stream, nullptr, 1, &k);
  ChunkArgs a;
  a.pool = c->base;
  a.q = k.q;
  a.cu_q = k.cu_q;
  a.block_table = k.block_table;
  a.seq_lens = k.seq_lens;
  a.prefix_lens = k.prefix_lens;
  a.slopes = k.slopes;
  a.out = k.out;
  const int D = c->cfg.head_dim;
  const size_t rows = (size_t)k.total_q * k.num_q_heads;
  a.ws_o = static_cast<float*>(k.workspace);
  a.ws_ml = plan.num_splits > 1 ? a.ws_o + rows * plan.num_splits * D : nullptr;
  a.total_q = k.total_q;
  a.B = k.num_seqs;
  a.Hq = k.num_q_heads;
  a.Hkv = c->cfg.num_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.num_pages = c->cfg.num_pages;
  a.max_pages = k.max_pages;
  a.max_q_len = k.max_q_len;
  a.max_seq_len = k.max_seq_len;
  a.window = k.window;
  a.num_splits = plan.num_splits;
  a.out_f32 = k.out_dtype == KVQ_F32;
  a.scale = k.scale;
  a.cap = k.cap;
  a.block_bytes = c->block_bytes;
  uint8_t* o = static_cast<uint8_t*>(k.out);
  a.out_span = Span{o, o + rows * D * (a.out_f32 ? 4 : 2)};
  uint8_t* w = static_cast<uint8_t*>(k.workspace);
  a.ws_span = Span{w, w ? w + plan.workspace_bytes : nullptr};
  if (chunk_on_umma(c, k.out_dtype)) {
    cudaError_t e = launch_chunk_umma(c, a, stream);
    if (e != cudaSuccess || a.num_splits == 1) return e;
    return launch_chunk_combine(c, a, kUmmaRows, stream);
  }
  const dim3 grid((unsigned)chunk_tile_bound(a.total_q, a.B, a.G, kRows), a.Hkv, a.num_splits);
  const bool qf32 = c->cfg.io_dtype == KVQ_F32;
  const int mode = c->cfg.mode;
  cudaError_t e = D == 128 ? (qf32 ? launch_mma<128, true>(mode, a, grid, stream) : launch_mma<128, false>(mode, a, grid, stream))
                : D == 32  ? (qf32 ? launch_mma<32, true>(mode, a, grid, stream) : launch_mma<32, false>(mode, a, grid, stream))
                           : cudaErrorInvalidValue;
  if (e != cudaSuccess || a.num_splits == 1) return e;
  return launch_chunk_combine(c, a, kRows, stream);
}

}  // namespace kvq
