// kvq_latent_write.cu -- the write and the read-back of a latent cache.
//
// kvq_latent_write.  For a token's latent row x (L values), weights w, and for the rotary
// parts of its key and of its queries' heads:
//   c = x w / sqrt(mean(x^2) + eps),   z_a = y_a cos - y_b sin,  z_b = y_b cos + y_a sin
// each rounded once to the io type, correctly (a last-bit change of a latent moves some
// codes by a whole step; kvq_rope.cu says how the rotation is rounded).  A latent row is
// normed in double-word fp32 throughout, good to about 2^-44 and rounded once: there is one
// such row to a token, beside the queries' heads.  Codes come from the rounded row by the
// arithmetic of the other write kernels (kvq_quant.cuh).
//
// Bound by memory for many tokens (the queries' rotary parts, in and out, are most of it),
// by latency for few.  One launch: the first CTAs take latent rows, a warp each, with L / 32
// values a lane; the others take rotary rows, 64 values in 8 lanes (fp16) or 16 (fp32), a
// group of lanes walking over some heads of one token, so that the token's cosines and sines
// are read once for them; the key is one head more.  Measured: 8191 tokens of 64 heads into an
// fp8 cache 48 us (68% of the issue slots, mostly the rotation; 3.1 TB/s of rows in and out);
// 40 tokens 3.7 us.
//
// kvq_latent_read.  code x scale in fp32, rounded once.  Bound by memory, mostly the dense
// rows out.  A warp takes four tokens: their rotary rows are one 16-byte load a lane, their
// codes one 16-code load a lane and token (L = 512), all in flight before the first store.
// Measured: 65521 nvfp4 tokens of 512 channels 22.4 us (4.6 TB/s).
#include <cuda_fp16.h>

#include "kvq_latent.cuh"
#include "kvq_rotate.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;

struct LatentWriteArgs {
  WriteArgs w;  // pool, slots (null: no cache write), num_tokens, num_pages, pool_span
  const void* latent;
  const void* k_rope;
  const void* q_rope;
  void* q_rope_out;
  long long latent_stride, k_rope_stride, q_stride, q_head_stride, q_out_stride, q_out_head_stride;
  const void* weight;
  const int32_t* positions;
  const float* cos_sin;
  void* latent_out;
  void* k_rope_out;
  int heads;  // rotary rows of a token: the queries' heads, then its key
  int max_position, interleaved;
  float eps;
  int latent_ctas, chunk;  // CTAs that take latent rows; heads of a group
  Span q_span, latent_span, rope_span;
};

template <typename T>
__device__ __forceinline__ void narrow_out(T* p, const float* f, const Span& span, const uint8_t* pool) {
  st_chk(reinterpret_cast<uint4*>(p), narrow16<T>(f), span, pool);
}

// The token's position, or -1 where it is not to be written.
__device__ __forceinline__ int position_of(const LatentWriteArgs& a, long long token, bool flag) {
  if (token >= a.w.num_tokens) return -1;
  const int p = __ldg(a.positions + token);
  if (p >= 0 && p < a.max_position) return p;
  if (flag) set_error(a.w.pool, KVQ_DEVERR_POSITION);
  return -1;
}
// Its page in the pool and its row there; null where nothing is written.
__device__ __forceinline__ uint8_t* page_of(const LatentWriteArgs& a, long long token, int& off, bool flag) {
  if (!a.w.slots) return nullptr;
  const int slot = __ldg(a.w.slots + token);
  if (slot < 0) return nullptr;
  if ((slot >> 4) >= a.w.num_pages) {
    if (flag) set_error(a.w.pool, KVQ_DEVERR_SLOT_RANGE);
    return nullptr;
  }
  off = slot & 15;
  return a.w.pool + kHeaderBytes + (size_t)(slot >> 4) * a.w.block_bytes;
}

// One latent row by a warp: lane j holds values (32 r + j) VEC .. of it, r < NL.
template <int MODE, typename T, int L>
__device__ __forceinline__ void latent_row_of(const LatentWriteArgs& a, long long token, int lane) {
  constexpr int VEC = 16 / (int)sizeof(T), NL = L / (32 * VEC), V = NL * VEC;
  if (position_of(a, token, lane == 0) < 0) return;
  const T* src = static_cast<const T*>(a.latent) + token * a.latent_stride;
  float x[V];
#pragma unroll
  for (int r = 0; r < NL; ++r)
    widen16<T>(*reinterpret_cast<const uint4*>(src + (32 * r + lane) * VEC), x + r * VEC);
  if (a.weight) {
    float2 p[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = make_float2(x[2 * i], x[2 * i + 1]);
    DW ms = mean_square_dw<L, V>(p, a.eps);
    float by = 1.0f;
    if (sizeof(T) == 4 && !(ms.h >= 0x1p-80f && ms.h <= 0x1p96f)) {  // (the whole warp)
      // low words would leave fp32: the row is normed times a power of two
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, fabsf(x[i]));
      top = group_max<32>(top);
      const int e = max((int)(__float_as_uint(top) >> 23) - 127,
                        a.eps > 0.0f ? ((int)(__float_as_uint(a.eps) >> 23) - 127) >> 1 : -126);
      if (isfinite(top)) by = __int_as_float((127 - max(-126, min(126, e))) << 23);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) p[i] = make_float2(p[i].x * by, p[i].y * by);
      ms = mean_square_dw<L, V>(p, a.eps * by * by);
    }
    const DW rs = rsqrt_dw(ms);
    constexpr bool F16 = sizeof(T) == 2;
#pragma unroll
    for (int r = 0; r < NL; ++r) {
      float w[VEC];
      widen16<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.weight) + (32 * r + lane) * VEC)), w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const DW y = two_prod(x[r * VEC + i] * by, w[i]);  // (fp16: exact, no low word)
        float v = rotate_dw<F16>(y, y, 1.0f, 0.0f, false, rs);
        if (!isfinite(v)) v = rotate_plain(y.h, y.h, 1.0f, 0.0f, false, rs.h);
        x[r * VEC + i] = v;
      }
    }
    if (F16) {  // the row as the io type holds it
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = __half2float(__float2half_rn(x[i]));
    }
  }
  if (a.latent_out) {
#pragma unroll
    for (int r = 0; r < NL; ++r)
      narrow_out<T>(static_cast<T*>(a.latent_out) + token * L + (32 * r + lane) * VEC, x + r * VEC, a.latent_span, a.w.pool);
  }
  int off = 0;
  uint8_t* page = page_of(a, token, off, lane == 0);
  using PG = LatentPage<MODE, L>;
  const float2 nz = dup2(a.w.neg_zero);
  if constexpr (kLatentFour<MODE>) {
    const TensorScale ts = TensorScale::make<MODE>(a.w, 0);
#pragma unroll
    for (int r = 0; r < NL; ++r) {
      uint32_t w[1], sb;
      nvfp4_codes<VEC, 16 / VEC, MODE == KVQ_NVFP4_4OVER6>(x + r * VEC, ts.st, ts.qs, ts.q4, nz, w[0], sb);
      const int at = (32 * r + lane) * VEC;
      if (page) {
        store_bytes_chk<VEC / 2>(page + (size_t)off * PG::CODES + at / 2, w, a.w);
        if (at % 16 == 0) st_chk(page + PG::SCALES + (size_t)off * (L / 16) + at / 16, static_cast<uint8_t>(sb), a.w.pool_span, a.w.pool);
      }
    }
  } else {
    float s;
    if constexpr (MODE == KVQ_FP8_PER_TENSOR) {
      s = *reinterpret_cast<const float*>(a.w.pool + kHdrKScaleOffset);
    } else {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) amax = fmaxf(amax, fabsf(x[i]));
      amax = fmaxf(group_max<32>(amax), 1e-8f);
      s = MODE == KVQ_INT8_PER_TOKEN_HEAD ? div_const(amax, 127.0f, kRcp127) : div_const(amax, 448.0f, kRcp448);
    }
    const QDiv q(s);
#pragma unroll
    for (int r = 0; r < NL; ++r) {
      uint32_t w[VEC / 4];
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float* y = x + r * VEC + i;
        if constexpr (MODE == KVQ_INT8_PER_TOKEN_HEAD) w[i / 4] = q.int8x4(y, nz);
        else w[i / 4] = q.e4m3x2(y[1], y[0]) | (q.e4m3x2(y[3], y[2]) << 16);
      }
      if (page) store_bytes_chk<VEC>(page + (size_t)off * PG::CODES + (32 * r + lane) * VEC, w, a.w);
    }
    if (kLatentTokenScale<MODE> && page && lane == 0)
      st_chk(reinterpret_cast<float*>(page + PG::SCALES) + off, s, a.w.pool_span, a.w.pool);
  }
}

// Rotary rows: group g of TPR lanes, `chunk` heads of a token from h0.
template <int MODE, typename T, int L>
__device__ __forceinline__ void rotary_rows_of(const LatentWriteArgs& a, int index) {
  constexpr int D = kLatentRope, VEC = 16 / (int)sizeof(T), TPR = D / VEC, TOK = kThreads / TPR;
  const int g = threadIdx.x / TPR, j = threadIdx.x % TPR;
  const int chunks = (a.heads + a.chunk - 1) / a.chunk;
  const long long token = (long long)(index / chunks) * TOK + g;
  const int h0 = index % chunks * a.chunk, h1 = min(a.heads, h0 + a.chunk);
  const int pos = position_of(a, token, false);  // (flagged with the latent rows)
  const bool in = pos >= 0;
  Rotation<VEC> rot;
  load_rotation<VEC>(rot, a.cos_sin + (long long)(in ? pos : 0) * D, D, a.interleaved != 0, j, in);
  float2 one[VEC / 2];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) one[i] = make_float2(1.0f, 1.0f);
  const T* kr = static_cast<const T*>(a.k_rope) + (in ? token : 0) * a.k_rope_stride + j * VEC;
  const T* q = static_cast<const T*>(a.q_rope) + (in ? token : 0) * a.q_stride + j * VEC;
  T* q_out = static_cast<T*>(a.q_rope_out) + (in ? token : 0) * a.q_out_stride + j * VEC;
  auto load = [&](int h) {
    if (!in || h >= h1) return make_uint4(0u, 0u, 0u, 0u);
    return *reinterpret_cast<const uint4*>(h == a.heads - 1 ? kr : q + h * a.q_head_stride);
  };
  uint4 next = load(h0);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const uint4 raw = next;
    next = load(h + 1);
    float f[VEC];
    widen16<T>(raw, f);
    float2 x[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) x[i] = make_float2(f[2 * i], f[2 * i + 1]);
    const uint4 out = rotate_row<D>(x, one, false, 0.0f, rot, dup2(a.w.neg_zero));
    if (!in) continue;
    if (h < a.heads - 1) {
      st_chk(reinterpret_cast<uint4*>(q_out + h * a.q_out_head_stride), out, a.q_span, a.w.pool);
      continue;
    }
    if (a.k_rope_out)
      st_chk(reinterpret_cast<uint4*>(static_cast<T*>(a.k_rope_out) + token * D + j * VEC), out, a.rope_span, a.w.pool);
    int off = 0;
    uint8_t* page = page_of(a, token, off, false);
    if (page) {
      uint8_t* dst = page + LatentPage<MODE, L>::ROPE + (off * D + j * VEC) * 2;
      if constexpr (sizeof(T) == 2) {
        st_chk(reinterpret_cast<uint4*>(dst), out, a.w.pool_span, a.w.pool);
      } else {
        float z[VEC];
        widen16<T>(out, z);
        st_chk(reinterpret_cast<uint2*>(dst),
               make_uint2(h2_as_u32(__floats2half2_rn(z[0], z[1])), h2_as_u32(__floats2half2_rn(z[2], z[3]))), a.w.pool_span,
               a.w.pool);
      }
    }
  }
}

template <int MODE, typename T, int L>
__global__ void __launch_bounds__(kThreads) latent_write_kernel(const __grid_constant__ LatentWriteArgs a) {
  if ((int)blockIdx.x < a.latent_ctas)
    latent_row_of<MODE, T, L>(a, (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32, threadIdx.x & 31);
  else
    rotary_rows_of<MODE, T, L>(a, (int)blockIdx.x - a.latent_ctas);
}

template <int MODE, typename T, int L>
cudaError_t launch(LatentWriteArgs& a, cudaStream_t s) {
  constexpr int TOK = kThreads / (kLatentRope / (16 / (int)sizeof(T)));
  a.latent_ctas = (int)((a.w.num_tokens + kThreads / 32 - 1) / (kThreads / 32));
  // Heads of a group: more share a token's table row, fewer give more CTAs; doubled
  // while six CTAs per SM are left.
  const long long groups = (a.w.num_tokens + TOK - 1) / TOK;
  auto chunks = [&](int c) { return (a.heads + c - 1) / c; };
  a.chunk = 2;
  while (a.chunk < 32 && groups * chunks(2 * a.chunk) >= 6 * num_sms()) a.chunk *= 2;
  const long long grid = a.latent_ctas + groups * chunks(a.chunk);
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  latent_write_kernel<MODE, T, L><<<(unsigned)grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int L>
cudaError_t launch_mode(int mode, LatentWriteArgs& a, cudaStream_t s) {
  switch (mode) {
    case KVQ_FP8_PER_TENSOR: return launch<KVQ_FP8_PER_TENSOR, T, L>(a, s);
    case KVQ_INT8_PER_TOKEN_HEAD: return launch<KVQ_INT8_PER_TOKEN_HEAD, T, L>(a, s);
    case KVQ_FP8_PER_TOKEN_HEAD: return launch<KVQ_FP8_PER_TOKEN_HEAD, T, L>(a, s);
    case KVQ_NVFP4: return launch<KVQ_NVFP4, T, L>(a, s);
    case KVQ_NVFP4_4OVER6: return launch<KVQ_NVFP4_4OVER6, T, L>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

// ---------------------------------------------------------------- reading back
struct LatentReadArgs {
  const uint8_t* pool;
  const int32_t* slots;
  long long num_tokens;
  int num_pages;
  size_t page_bytes;
  void* latent;  // either may be null
  void* rope;
  Span latent_span, rope_span;
};

template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const float* f, const Span& span, const uint8_t* pool) {
#pragma unroll
  for (int i = 0; i < N; i += 16 / (int)sizeof(T)) st_chk(reinterpret_cast<uint4*>(p + i), narrow16<T>(f + i), span, pool);
}

template <int MODE, typename T, int L>
__global__ void __launch_bounds__(kThreads) latent_read_kernel(const __grid_constant__ LatentReadArgs a) {
  using PG = LatentPage<MODE, L>;
  constexpr int TOK = 4, PER = L / 16, ITEMS = TOK * PER / 32;  // 16-code items of a token, of a lane
  constexpr int W = kLatentFour<MODE> ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const long long t0 = ((long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * TOK;
  if (t0 >= a.num_tokens) return;
  int mine = -1;
  if (lane < TOK && t0 + lane < a.num_tokens) {
    mine = __ldg(a.slots + t0 + lane);
    if (mine >= 0 && (mine >> 4) >= a.num_pages) {
      set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_SLOT_RANGE);
      mine = -1;
    }
  }
  auto page = [&](int slot) { return a.pool + kHeaderBytes + (size_t)(slot >> 4) * a.page_bytes; };
  uint32_t w[ITEMS][W];
  float sc[ITEMS];
  uint32_t sb[ITEMS];
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  const float st = MODE == KVQ_FP8_PER_TENSOR || kLatentFour<MODE> ? *reinterpret_cast<const float*>(a.pool + kHdrKScaleOffset) : 1.0f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int item = 32 * i + lane, slot = __shfl_sync(kFull, mine, item / PER), c = item % PER;
    if (slot < 0 || !a.latent) continue;
    const uint8_t* row = page(slot) + (slot & 15) * PG::CODES + c * (W * 4);
    if constexpr (W == 4) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(row));
      w[i][0] = u.x;
      w[i][1] = u.y;
      w[i][2] = u.z;
      w[i][3] = u.w;
      sc[i] = kLatentTokenScale<MODE> ? __ldg(reinterpret_cast<const float*>(page(slot) + PG::SCALES) + (slot & 15)) : st;
    } else {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(row));
      w[i][0] = u.x;
      w[i][1] = u.y;
      sb[i] = __ldg(page(slot) + PG::SCALES + (slot & 15) * (L / 16) + c);
      sc[i] = st;
    }
  }
  const int rslot = __shfl_sync(kFull, mine, lane >> 3);
  if (rslot >= 0 && a.rope)
    r = __ldg(reinterpret_cast<const uint4*>(page(rslot) + PG::ROPE + (rslot & 15) * kLatentRope * 2) + (lane & 7));
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int item = 32 * i + lane, slot = __shfl_sync(kFull, mine, item / PER), c = item % PER;
    if (slot < 0 || !a.latent) continue;
    uint32_t h[8];
    latent_codes16<MODE>(w[i], kLatentFour<MODE> ? sb[i] : 0u, h);
    float f[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 v = __half22float2(u32_as_h2(h[e]));
      f[2 * e] = v.x * sc[i];
      f[2 * e + 1] = v.y * sc[i];
    }
    store_row<T, 16>(static_cast<T*>(a.latent) + (t0 + item / PER) * L + 16 * c, f, a.latent_span, a.pool);
  }
  if (rslot >= 0 && a.rope) {
    float f[8];
    widen16<__half>(r, f);
    store_row<T, 8>(static_cast<T*>(a.rope) + (t0 + (lane >> 3)) * kLatentRope + 8 * (lane & 7), f, a.rope_span, a.pool);
  }
}

template <typename T, int L>
cudaError_t launch_read(int mode, const LatentReadArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.num_tokens + kThreads / 8 - 1) / (kThreads / 8));
  switch (mode) {
    case KVQ_FP8_PER_TENSOR: latent_read_kernel<KVQ_FP8_PER_TENSOR, T, L><<<grid, kThreads, 0, s>>>(a); break;
    case KVQ_INT8_PER_TOKEN_HEAD: latent_read_kernel<KVQ_INT8_PER_TOKEN_HEAD, T, L><<<grid, kThreads, 0, s>>>(a); break;
    case KVQ_FP8_PER_TOKEN_HEAD: latent_read_kernel<KVQ_FP8_PER_TOKEN_HEAD, T, L><<<grid, kThreads, 0, s>>>(a); break;
    case KVQ_NVFP4:
    case KVQ_NVFP4_4OVER6: latent_read_kernel<KVQ_NVFP4, T, L><<<grid, kThreads, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

// The span of rows at p, strides in elements.
Span rows_span(void* p, long long rows, long long stride, long long heads, long long head_stride, long long width, int esize) {
  uint8_t* b = static_cast<uint8_t*>(p);
  return Span{b, b ? b + ((rows - 1) * stride + (heads - 1) * head_stride + width) * esize : nullptr};
}

}  // namespace

cudaError_t launch_latent_write(const kvq_latent* c, const kvq_latent_rows& r, cudaStream_t s) {
  LatentWriteArgs a = {};
  const int L = c->cfg.latent_dim, esize = c->cfg.io_dtype == KVQ_F16 ? 2 : 4;
  a.w.pool = c->base;
  a.w.slots = r.slot_mapping;
  a.w.num_tokens = r.num_tokens;
  a.w.num_pages = c->cfg.num_pages;
  a.w.block_bytes = c->page_bytes;
  a.w.pool_span = latent_pages(c);
  a.latent = r.latent;
  a.k_rope = r.k_rope;
  a.q_rope = r.q_rope;
  a.q_rope_out = r.q_rope_out;
  a.latent_stride = r.latent_stride;
  a.k_rope_stride = r.k_rope_stride;
  a.q_stride = r.q_stride;
  a.q_head_stride = r.q_head_stride;
  a.q_out_stride = r.q_out_stride;
  a.q_out_head_stride = r.q_out_head_stride;
  a.weight = r.latent_weight;
  a.positions = r.positions;
  a.cos_sin = r.cos_sin;
  a.latent_out = r.latent_out;
  a.k_rope_out = r.k_rope_out;
  a.heads = (r.q_rope ? r.num_q_heads : 0) + 1;
  a.max_position = r.max_position;
  a.interleaved = r.interleaved;
  a.eps = r.eps;
  const long long T = r.num_tokens;
  a.q_span = rows_span(r.q_rope_out, T, r.q_out_stride, a.heads - 1, r.q_out_head_stride, kLatentRope, esize);
  a.latent_span = rows_span(r.latent_out, T, L, 1, 0, L, esize);
  a.rope_span = rows_span(r.k_rope_out, T, kLatentRope, 1, 0, kLatentRope, esize);
  const int mode = c->cfg.mode;
  if (esize == 2) return L == 512 ? launch_mode<__half, 512>(mode, a, s) : launch_mode<__half, 256>(mode, a, s);
  return L == 512 ? launch_mode<float, 512>(mode, a, s) : launch_mode<float, 256>(mode, a, s);
}

cudaError_t launch_latent_read(const kvq_latent* c, const int32_t* slots, int num_tokens, void* latent_out, void* rope_out,
                               int out_dtype, cudaStream_t s) {
  LatentReadArgs a = {};
  const int L = c->cfg.latent_dim, esize = out_dtype == KVQ_F16 ? 2 : 4;
  a.pool = c->base;
  a.slots = slots;
  a.num_tokens = num_tokens;
  a.num_pages = c->cfg.num_pages;
  a.page_bytes = c->page_bytes;
  a.latent = latent_out;
  a.rope = rope_out;
  a.latent_span = rows_span(latent_out, num_tokens, L, 1, 0, L, esize);
  a.rope_span = rows_span(rope_out, num_tokens, kLatentRope, 1, 0, kLatentRope, esize);
  const int mode = c->cfg.mode;
  if (esize == 2) return L == 512 ? launch_read<__half, 512>(mode, a, s) : launch_read<__half, 256>(mode, a, s);
  return L == 512 ? launch_read<float, 512>(mode, a, s) : launch_read<float, 256>(mode, a, s);
}

}  // namespace kvq
