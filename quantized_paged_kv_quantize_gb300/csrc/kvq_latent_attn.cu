// kvq_latent_attn.cu -- latent attention in fp32 throughout, absorbed and expanded, the
// merge of split ranges, and the plan.
//
// Mathematics.  For a query row q (absorbed: L + 64 values against [c_t, r_t], and the
// latents c_t are the values too; expanded: 192 values against [k_t, r_t], and v_t):
//   s_t = scale q . key_t,  out = sum 2^(y_t - m) value_t / sum 2^(y_t - m),  y = s log2(e)
// with the running maximum m and sum l of one pass over the tokens.
//
// The kernel here takes what the tensor cores would round: fp32 queries or fp32 outputs.
// A CTA has 32 rows and walks over tiles of 32 tokens, dequantized to fp32 in shared
// memory.  Products are fp32 multiply-adds, two rows by two tokens a thread for the
// scores (shared-memory reads bound it: 4 loads of 16 bytes to 16 multiply-adds), and
// 32 rows by L / 256 channels a thread for the values.
// Bound by the multiply-adds and their shared-memory reads.
// Measured: 2048 queries of 128 heads over 8192 keys, expanded, 65.9 ms (18 TFLOP/s; the tensor cores,
// with fp16 weights, take 0.83 ms).
#include <cuda_fp16.h>

#include <algorithm>

#include "kvq_latent.cuh"

namespace kvq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256, kRows = 32, kTok = 32;

template <int DK>
struct PlainSmem {
  static constexpr int STRIDE = DK + 4;  // floats; the pad spreads the rows over the banks
  static constexpr int Q = 0, K = Q + kRows * STRIDE, S = K + kTok * STRIDE, P = S + kRows * (kTok + 1), A = P + kTok * kRows,
                       FLOATS = A + 2 * kRows;
  static constexpr size_t BYTES = FLOATS * sizeof(float);
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* f);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float* f) {
  const float4 u = __ldg(reinterpret_cast<const float4*>(p));
  f[0] = u.x;
  f[1] = u.y;
  f[2] = u.z;
  f[3] = u.w;
}
template <>
__device__ __forceinline__ void load4<__half>(const __half* p, float* f) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  const float2 a = __half22float2(u32_as_h2(u.x)), b = __half22float2(u32_as_h2(u.y));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

// MODE 0: expanded.  L: the latent width (absorbed), 128 (expanded).
template <int MODE, typename T, int L>
__global__ void __launch_bounds__(kThreads) latent_plain_kernel(const __grid_constant__ LatentArgs a) {
  constexpr bool EXP = MODE == 0;
  constexpr int DK = L + kLatentRope;
  // (expanded: the tile's values follow the keys, in the place of a second tile)
  using S = PlainSmem<EXP ? DK + kLatentHead : DK>;
  constexpr int ST = S::STRIDE;
  constexpr int CH = L >= 256 ? L / 256 : 1;           // channels of a thread
  constexpr int RG = kThreads * CH / L, RP = kRows / RG;  // row groups, rows of a thread
  extern __shared__ __align__(16) float sm[];
  float *qs = sm + S::Q, *ks = sm + S::K, *ss = sm + S::S, *ps = sm + S::P, *al = sm + S::A, *ls = al + kRows;
  const float* vs = EXP ? ks + DK : ks;
  __shared__ RowTile tile_s;
  __shared__ int there_s[2];  // page ids of the tile
  const int tid = threadIdx.x, lane = tid & 31, kvh = blockIdx.y, split = blockIdx.z;
  if (tid < 32) {
    const RowTile t = latent_tile<EXP>(a, blockIdx.x, kRows, blockIdx.x == 0 && kvh == 0 && split == 0);
    if (lane == 0) tile_s = t;
  }
  __syncthreads();
  const RowTile t = tile_s;
  if (t.seq < 0) return;
  const int most = latent_sees(a, t, t.r0 + t.count - 1);  // tokens that the last row sees
  const int tiles = (most + kTok - 1) / kTok;
  const int i0 = (int)((long long)tiles * split / a.num_splits), i1 = (int)((long long)tiles * (split + 1) / a.num_splits);

  for (int it = tid; it < kRows * (DK / 4); it += kThreads) {
    const int r = it / (DK / 4), c = it % (DK / 4) * 4;
    float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r < t.count) load4(static_cast<const T*>(a.q) + latent_row(a, t, kvh, t.r0 + r) * DK + c, f);
    *reinterpret_cast<float4*>(qs + r * ST + c) = make_float4(f[0], f[1], f[2], f[3]);
  }
  float acc[CH][RP];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int r = 0; r < RP; ++r) acc[c][r] = 0.0f;
  // softmax: eight threads a row, four tokens each
  const int srow = tid >> 3, sub = tid & 7;
  const int sees = srow < t.count ? latent_sees(a, t, t.r0 + srow) : 0;
  float m = kLowest, l = 0.0f;
  const float st = EXP ? 1.0f : *reinterpret_cast<const float*>(a.pool + kHdrKScaleOffset);
  const float to_log2 = a.scale * kLog2e;
  const int k0 = EXP ? __ldg(a.cu_k + t.seq) : 0;

  for (int i = i0; i < i1; ++i) {
    const int t0 = i * kTok;
    __syncthreads();  // the last tile has been read
    if (!EXP && tid < 2) {
      int id = -1;
      if (t0 + 16 * tid < most) {
        id = __ldg(a.block_table + (long long)t.seq * a.max_pages + 2 * i + tid);
        if (id < 0 || id >= a.num_pages) {
          set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_PAGE_RANGE);
          id = -1;
        }
      }
      there_s[tid] = id;
    }
    __syncthreads();
    if constexpr (EXP) {
      constexpr int W = (DK + kLatentHead) / 4;
      for (int it = tid; it < kTok * W; it += kThreads) {
        const int r = it / W, c = it % W * 4;
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (t0 + r < most) {
          const long long row = k0 + t0 + r;
          if (c < L) load4(static_cast<const T*>(a.k) + row * a.k_stride + kvh * a.k_head_stride + c, f);
          else if (c < DK) load4(static_cast<const T*>(a.k_rope) + row * a.k_rope_stride + c - L, f);
          else load4(static_cast<const T*>(a.v) + row * a.v_stride + kvh * a.v_head_stride + c - DK, f);
        }
        *reinterpret_cast<float4*>(ks + r * ST + c) = make_float4(f[0], f[1], f[2], f[3]);
      }
    } else {
      using PG = LatentPage<MODE, L>;
      constexpr int W = L / 16 + kLatentRope / 16;
      for (int it = tid; it < kTok * W; it += kThreads) {
        const int r = it / W, c = it % W, id = there_s[r >> 4];
        const bool in = id >= 0 && t0 + r < most;
        const uint8_t* page = a.pool + kHeaderBytes + (size_t)(in ? id : 0) * a.block_bytes;
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = 0.0f;
        if (in) {
          uint32_t h[8];
          float s = 1.0f;
          if (c < L / 16) {
            uint32_t w[4], sb = 0;
            const uint8_t* p = page + (r & 15) * PG::CODES + c * (PG::CODES * 16 / L);
            if constexpr (kLatentFour<MODE>) {
              const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
              w[0] = u.x;
              w[1] = u.y;
              sb = __ldg(page + PG::SCALES + (r & 15) * (L / 16) + c);
            } else {
              const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
              w[0] = u.x;
              w[1] = u.y;
              w[2] = u.z;
              w[3] = u.w;
            }
            latent_codes16<MODE>(w, sb, h);
            s = kLatentTokenScale<MODE> ? __ldg(reinterpret_cast<const float*>(page + PG::SCALES) + (r & 15)) : st;
          } else {
            const uint4* p = reinterpret_cast<const uint4*>(page + PG::ROPE + (r & 15) * kLatentRope * 2) + 2 * (c - L / 16);
            const uint4 u = __ldg(p), v = __ldg(p + 1);
            h[0] = u.x;
            h[1] = u.y;
            h[2] = u.z;
            h[3] = u.w;
            h[4] = v.x;
            h[5] = v.y;
            h[6] = v.z;
            h[7] = v.w;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 x = __half22float2(u32_as_h2(h[e]));
            f[2 * e] = x.x * s;
            f[2 * e + 1] = x.y * s;
          }
        }
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<float4*>(ks + r * ST + 16 * c + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
      }
    }
    __syncthreads();
    {  // scores: rows ty, ty + 16 and tokens tx, tx + 16
      const int ty = tid >> 4, tx = tid & 15;
      float s[2][2] = {};
#pragma unroll 4
      for (int c = 0; c < DK; c += 4) {
        float4 x[2], y[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[u] = *reinterpret_cast<const float4*>(qs + (ty + 16 * u) * ST + c);
          y[u] = *reinterpret_cast<const float4*>(ks + (tx + 16 * u) * ST + c);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            s[u][v] = fmaf(x[u].x, y[v].x, s[u][v]);
            s[u][v] = fmaf(x[u].y, y[v].y, s[u][v]);
            s[u][v] = fmaf(x[u].z, y[v].z, s[u][v]);
            s[u][v] = fmaf(x[u].w, y[v].w, s[u][v]);
          }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) ss[(ty + 16 * u) * (kTok + 1) + tx + 16 * v] = s[u][v];
    }
    __syncthreads();
    {
      float y[4], mx = kLowest;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = sub + 8 * e;
        y[e] = ss[srow * (kTok + 1) + k] * to_log2;
        if (t0 + k >= sees || (!EXP && there_s[k >> 4] < 0)) y[e] = -INFINITY;
        mx = fmaxf(mx, y[e]);
      }
      mx = fmaxf(m, warp_max_xor(mx, 1, 4));
      const float f = exp2f(m - mx);  // (1 while nothing is seen)
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = exp2f(y[e] - mx);
        sum += p;
        ps[(sub + 8 * e) * kRows + srow] = p;
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
      l = l * f + sum;
      m = mx;
      if (sub == 0) al[srow] = f;
    }
    __syncthreads();
    {
      const int c0 = tid % (L / CH), rg = tid / (L / CH);
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const float f = al[rg * RP + r];
#pragma unroll
        for (int c = 0; c < CH; ++c) acc[c][r] *= f;
      }
#pragma unroll 2
      for (int k = 0; k < kTok; ++k) {
        float v[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) v[c] = vs[k * ST + c0 + c * (L / CH)];
#pragma unroll
        for (int r = 0; r < RP; r += 4) {
          const float4 p = *reinterpret_cast<const float4*>(ps + k * kRows + rg * RP + r);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            acc[c][r] = fmaf(p.x, v[c], acc[c][r]);
            acc[c][r + 1] = fmaf(p.y, v[c], acc[c][r + 1]);
            acc[c][r + 2] = fmaf(p.z, v[c], acc[c][r + 2]);
            acc[c][r + 3] = fmaf(p.w, v[c], acc[c][r + 3]);
          }
        }
      }
    }
  }
  __syncthreads();
  if (sub == 0) {
    ls[srow] = l;
    if (srow < t.count) {
      const long long row = latent_row(a, t, kvh, t.r0 + srow);
      if (a.num_splits > 1)
        st_chk(reinterpret_cast<float2*>(a.ws_ml) + row * a.num_splits + split, make_float2(l == 0.0f ? -INFINITY : m, l), a.ws_span,
               a.pool);
      else if (a.lse)
        st_chk(a.lse + row, l == 0.0f ? -INFINITY : (m + log2f(l)) * (1.0f / kLog2e), a.lse_span, a.pool);
    }
  }
  __syncthreads();
  const int c0 = tid % (L / CH), rg = tid / (L / CH);
#pragma unroll
  for (int r = 0; r < RP; ++r) {
    const int row_of = rg * RP + r;
    if (row_of >= t.count) continue;
    const long long row = latent_row(a, t, kvh, t.r0 + row_of);
    const float sum = ls[row_of];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = c0 + c * (L / CH);
      if (a.num_splits > 1) {
        st_chk(a.ws_o + (row * a.num_splits + split) * L + at, acc[c][r], a.ws_span, a.pool);
        continue;
      }
      const float x = sum == 0.0f ? 0.0f : acc[c][r] / sum;
      if (a.out_f32) st_chk(static_cast<float*>(a.out) + row * L + at, x, a.out_span, a.pool);
      else st_chk(static_cast<__half*>(a.out) + row * L + at, __float2half_rn(x), a.out_span, a.pool);
    }
  }
}

template <int MODE, typename T, int L>
cudaError_t launch_plain(const LatentArgs& a, cudaStream_t s) {
  auto kern = latent_plain_kernel<MODE, T, L>;
  constexpr size_t smem = PlainSmem<MODE == 0 ? L + kLatentRope + kLatentHead : L + kLatentRope>::BYTES;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)chunk_tile_bound(a.total_q, a.B, a.G, kRows), a.Hkv, a.num_splits);
  kern<<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int L>
cudaError_t launch_plain_mode(int mode, const LatentArgs& a, cudaStream_t s) {
  switch (mode) {
    case KVQ_FP8_PER_TENSOR: return launch_plain<KVQ_FP8_PER_TENSOR, T, L>(a, s);
    case KVQ_INT8_PER_TOKEN_HEAD: return launch_plain<KVQ_INT8_PER_TOKEN_HEAD, T, L>(a, s);
    case KVQ_FP8_PER_TOKEN_HEAD: return launch_plain<KVQ_FP8_PER_TOKEN_HEAD, T, L>(a, s);
    case KVQ_NVFP4:
    case KVQ_NVFP4_4OVER6: return launch_plain<KVQ_NVFP4, T, L>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

// ---------------------------------------------------------------- merge of split ranges
// A warp per row of a row tile: with (m_s, l_s) of its parts, M = max m_s,
// out = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s.  A part without tokens has m = -inf
// and is not read.  Bound by the partials' way through memory, eight loads of 16 bytes
// in flight a lane.
constexpr int kMaxParts = 512;
template <int L>
__global__ void __launch_bounds__(kThreads) latent_combine_kernel(const __grid_constant__ LatentArgs a, int rows) {
  constexpr int N4 = L / 128;  // 16-byte groups of a lane
  __shared__ RowTile tile_s;
  __shared__ float w_s[kThreads / 32][kMaxParts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait_primary();
  if (warp == 0) {
    const RowTile t = find_tile(a, blockIdx.x, rows, false);
    if (lane == 0) tile_s = t;
  }
  __syncthreads();
  const RowTile t = tile_s;
  const int r = blockIdx.y * (kThreads / 32) + warp;
  if (t.seq < 0 || r >= t.count) return;
  const long long row = latent_row(a, t, 0, t.r0 + r);
  // part s of this row is partial first + s step
  long long first = row * a.num_splits;
  int parts = a.num_splits, step = 1;
  if (a.ctas) {
    const int2 m = a.map[blockIdx.x];
    if (m.y == 1) return;  // (written whole)
    first = (long long)m.x * rows + r;
    parts = m.y;
    step = rows;
  }
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + first;
  float M = -INFINITY;
  for (int s = lane; s < parts; s += 32) M = fmaxf(M, ml[(long long)s * step].x);
  M = warp_max_xor(M, 1, 16);
  float sum = 0.0f;
  for (int s = lane; s < parts; s += 32) {
    const float2 v = ml[(long long)s * step];
    const float w = v.x == -INFINITY ? 0.0f : exp2f(v.x - M);  // (a NaN stays)
    w_s[warp][s] = w;
    sum += w * v.y;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
  __syncwarp();
  float4 acc[N4];
#pragma unroll
  for (int c = 0; c < N4; ++c) acc[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int U = 8 / N4;
  for (int s0 = 0; s0 < parts; s0 += U) {
    float4 x[U][N4];
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = s0 + u < parts ? w_s[warp][s0 + u] : 0.0f;
      const float4* src = reinterpret_cast<const float4*>(a.ws_o + (first + (long long)(s0 + u) * step) * L) + lane;
#pragma unroll
      for (int c = 0; c < N4; ++c) x[u][c] = w[u] != 0.0f ? src[32 * c] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < N4; ++c) {
        acc[c].x = fmaf(w[u], x[u][c].x, acc[c].x);
        acc[c].y = fmaf(w[u], x[u][c].y, acc[c].y);
        acc[c].z = fmaf(w[u], x[u][c].z, acc[c].z);
        acc[c].w = fmaf(w[u], x[u][c].w, acc[c].w);
      }
  }
  const float f = 1.0f / sum;
#pragma unroll
  for (int c = 0; c < N4; ++c) {
    const float4 x = sum == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                 : make_float4(acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f);
    const long long at = row * L + 4 * lane + 128 * c;
    if (a.out_f32) st_chk(reinterpret_cast<float4*>(static_cast<float*>(a.out) + at), x, a.out_span, a.pool);
    else
      st_chk(reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at),
             make_uint2(h2_as_u32(__floats2half2_rn(x.x, x.y)), h2_as_u32(__floats2half2_rn(x.z, x.w))), a.out_span, a.pool);
  }
  if (lane == 0 && a.lse)
    st_chk(a.lse + row, sum == 0.0f ? -INFINITY : (M + log2f(sum)) * (1.0f / kLog2e), a.lse_span, a.pool);
}

cudaError_t launch_combine(const kvq_latent* c, const LatentArgs& a, int rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int most = (int)std::min<long long>(rows, (long long)a.max_q_len * a.G);  // rows of a tile
  cfg.gridDim = dim3((unsigned)chunk_tile_bound(a.total_q, a.B, a.G, rows), (most + kThreads / 32 - 1) / (kThreads / 32));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = c->cfg.latent_dim == 512 ? cudaLaunchKernelEx(&cfg, latent_combine_kernel<512>, a, rows)
                                           : cudaLaunchKernelEx(&cfg, latent_combine_kernel<256>, a, rows);
  return e != cudaSuccess ? e : cudaGetLastError();
}

bool on_umma(const kvq_latent* c, bool out_f32) { return c->cfg.io_dtype == KVQ_F16 && !out_f32; }

// Parts of a row tile's token range in the fp32 kernel.  The lengths are on the device: every
// tile is taken to see max_seq_len tokens.  One CTA on an SM; a plan of s parts is
// estimated at ceil(units s / SMs) waves x (token tiles / s + the cost of a CTA's start
// and end, in tiles) plus the merge of s partials.
int plain_parts(int Hq, int total_q, int num_seqs, int max_q_len, int max_seq_len) {
  const long long sms = num_sms(), cost_cta = 4;
  const long long tiles = ((long long)max_seq_len + kTok - 1) / kTok;
  const long long per_seq = ((long long)max_q_len * Hq + kRows - 1) / kRows;
  const long long units = std::min(((long long)total_q * Hq + kRows - 1) / kRows + num_seqs / 2, per_seq * num_seqs);
  long long best = -1;
  int parts = 1;
  for (long long s = 1; s <= 128 && s <= std::max(1ll, tiles); ++s) {
    const long long cost = (units * s + sms - 1) / sms * ((tiles + s - 1) / s + cost_cta) * 8 + s;
    if (best < 0 || cost < best) {
      best = cost;
      parts = (int)s;
    }
  }
  return parts;
}
// CTAs of the tcgen05 kernel: whole waves, for parts of the ranges, unless there are several
// waves of row tiles or nothing to split.
constexpr int kSplitWaves = 3;
int umma_ctas(int Hq, int total_q, int num_seqs, int max_q_len, int max_seq_len) {
  const int rows = latent_umma_rows(max_q_len, Hq);
  const long long per_seq = ((long long)max_q_len * Hq + rows - 1) / rows, sms = num_sms();
  const long long tiles = std::min(chunk_tile_bound(total_q, num_seqs, Hq, rows), per_seq * num_seqs);
  if (max_seq_len <= 128 || tiles > kSplitWaves * sms || num_seqs > kLatentSeqs) return 0;
  return (int)std::min((tiles + sms - 1) / sms * sms, (long long)kMaxParts);
}

void spans(LatentArgs& a, int width) {
  const size_t rows = (size_t)a.total_q * a.Hq;
  uint8_t* o = static_cast<uint8_t*>(a.out);
  a.out_span = Span{o, o + rows * width * (a.out_f32 ? 4 : 2)};
  uint8_t* l = reinterpret_cast<uint8_t*>(a.lse);
  a.lse_span = Span{l, l ? l + rows * 4 : nullptr};
}

}  // namespace

// The parts are those of the kernel that the output's type chooses; the workspace, which
// a caller asks for without naming that type, serves the other one too.
LatentPlan plan_latent(const kvq_latent* c, int total_q, int num_seqs, int num_q_heads, int max_q_len, int max_seq_len,
                       int out_dtype) {
  LatentPlan p;
  if (total_q == 0 || num_seqs == 0 || max_q_len == 0) return p;
  const int plain = plain_parts(num_q_heads, total_q, num_seqs, max_q_len, max_seq_len);
  const size_t row = (c->cfg.latent_dim + 2) * sizeof(float);
  if (plain > 1) p.workspace_bytes = (size_t)total_q * num_q_heads * plain * row;
  p.num_splits = plain;
  if (c->cfg.io_dtype == KVQ_F16) {
    const int rows = latent_umma_rows(max_q_len, num_q_heads);
    const int ctas = umma_ctas(num_q_heads, total_q, num_seqs, max_q_len, max_seq_len);
    if (ctas) p.workspace_bytes = std::max(p.workspace_bytes, (size_t)ctas * (rows * row + sizeof(int2)));
    if (on_umma(c, out_dtype == KVQ_F32)) {
      p.ctas = ctas;
      p.num_splits = ctas ? std::min(ctas, (max_seq_len + 127) / 128) : 1;
    }
  }
  return p;
}

cudaError_t launch_latent_attention(const kvq_latent* c, const LatentPlan& p, LatentArgs& a, cudaStream_t s) {
  const int L = c->cfg.latent_dim, mode = c->cfg.mode;
  const bool umma = on_umma(c, a.out_f32);
  const int rows = umma ? latent_umma_rows(a.max_q_len, a.Hq) : kRows;
  a.num_splits = umma ? 1 : p.num_splits;
  a.ctas = p.ctas;
  const size_t partials = umma ? (size_t)p.ctas * rows : (size_t)a.total_q * a.Hq * a.num_splits;
  a.ws_ml = a.ws_o + partials * L;  // (not used where nothing is split)
  a.map = reinterpret_cast<int2*>(a.ws_ml + 2 * partials);
  spans(a, L);
  cudaError_t e;
  if (umma) e = launch_latent_umma(c, a, s);
  else if (c->cfg.io_dtype == KVQ_F32)
    e = L == 512 ? launch_plain_mode<float, 512>(mode, a, s) : launch_plain_mode<float, 256>(mode, a, s);
  else e = L == 512 ? launch_plain_mode<__half, 512>(mode, a, s) : launch_plain_mode<__half, 256>(mode, a, s);
  if (e != cudaSuccess || (a.num_splits == 1 && !a.ctas)) return e;
  return launch_combine(c, a, rows, s);
}

cudaError_t launch_latent_prompt(const kvq_latent* c, LatentArgs& a, cudaStream_t s) {
  a.num_splits = 1;
  spans(a, kLatentHead);
  if (on_umma(c, a.out_f32)) return launch_latent_prompt_umma(c, a, s);
  return c->cfg.io_dtype == KVQ_F32 ? launch_plain<0, float, kLatentHead>(a, s) : launch_plain<0, __half, kLatentHead>(a, s);
}

}  // namespace kvq
