// kvq_read.cu -- the values a cache holds at given slots, as dense rows
// (kvq_cache_read): codes times their scales in fp32, rounded once to the
// output type; KVarN rows r_t c_d (scale q + zero) rotated back to the input
// domain by the normalised Walsh-Hadamard transform (its own inverse).
//
// Bound by memory: the packed rows in, the dense rows out (NVFP4 at head_dim
// 128: 144 + 512 bytes per token and kv head), the stores being most of it.  A
// group of D / 8 lanes holds one row's K and V, eight channels a lane, so
// stores are 16 bytes a lane (fp16).  The groups of a CTA take consecutive
// entries of the slot list and the same heads: a page's rows, the scales
// beside them and the token-pair bytes of 4-bit values are then shared by
// neighbouring groups through L1.  Four heads' loads are in flight per thread.
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_unpack.cuh"

namespace kvq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kVec = 8;       // channels per lane
constexpr int kInFlight = 4;  // heads a thread loads before it converts the first

struct ReadArgs {
  const uint8_t* pool;
  const int32_t* slots;
  long long num_tokens;
  int Hkv, num_pages, heads_per_cta;
  size_t block_bytes;
  void* k;  // either may be null
  void* v;
  Span k_span, v_span;
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f, const Span& span, const uint8_t* pool);
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float* f, const Span& span, const uint8_t* pool) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = h2_as_u32(__floats2half2_rn(f[2 * i], f[2 * i + 1]));
  st_chk(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]), span, pool);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* f, const Span& span, const uint8_t* pool) {
  st_chk(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]), span, pool);
  st_chk(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]), span, pool);
}

// Codes (exact in fp16) times their scale, rounded once in fp32.
template <int MODE, int SIDE>
__device__ __forceinline__ void values(const Packed8& p, int off, float st, float* f) {
  uint32_t h[4];
  codes8<MODE, SIDE>(p, off, h);
  const float s = kPerTokenScale<MODE> ? __uint_as_float(p.scale) : st;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(u32_as_h2(h[i]));
    f[2 * i] = t.x * s;
    f[2 * i + 1] = t.y * s;
  }
}

template <int MODE, int D, typename T>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int TPR = D / kVec, TOK = kThreads / TPR;
  const int g = threadIdx.x / TPR, j = threadIdx.x % TPR;
  const long long token = (long long)blockIdx.x * TOK + g;
  if (token >= a.num_tokens) return;
  const int slot = __ldg(a.slots + token);
  if (slot < 0) return;
  const int page = slot >> 4, off = slot & 15;
  if (page >= a.num_pages) {
    if (j == 0 && blockIdx.y == 0) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_SLOT_RANGE);
    return;
  }
  float st[2] = {1.0f, 1.0f};
  if constexpr (MODE == KVQ_FP8_PER_TENSOR || MODE == KVQ_NVFP4) {
    st[0] = *reinterpret_cast<const float*>(a.pool + kHdrKScaleOffset);
    st[1] = *reinterpret_cast<const float*>(a.pool + kHdrVScaleOffset);
  }
  const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(a.Hkv, h0 + a.heads_per_cta);
  for (int hb = h0; hb < h1; hb += kInFlight) {
    Packed8 pk[kInFlight], pv[kInFlight];
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      const int h = min(hb + r, h1 - 1);
      const uint8_t* blk = a.pool + kHeaderBytes + ((size_t)page * a.Hkv + h) * a.block_bytes;
      if (a.k) pk[r] = load_packed8<MODE, D, 0>(blk, off, j);
      if (a.v) pv[r] = load_packed8<MODE, D, 1>(blk, off, j);
    }
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      if (hb + r >= h1) break;
      const long long o = (token * a.Hkv + hb + r) * D + kVec * j;
      float f[8];
      if (a.k) {
        values<MODE, 0>(pk[r], off, st[0], f);
        store8<T>(static_cast<T*>(a.k) + o, f, a.k_span, a.pool);
      }
      if (a.v) {
        values<MODE, 1>(pv[r], off, st[1], f);
        store8<T>(static_cast<T*>(a.v) + o, f, a.v_span, a.pool);
      }
    }
  }
}

// Normalised Walsh-Hadamard transform of a 128-vector held as eight values in
// each of 16 neighbouring lanes: three levels in the lane, four by shuffle.
__device__ __forceinline__ void fwht128x8(float* v, int j) {
#pragma unroll
  for (int st = 1; st < 8; st <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & st)) {
        const float x = v[i], y = v[i + st];
        v[i] = x + y;
        v[i + st] = x - y;
      }
#pragma unroll
  for (int o = 1; o <= 8; o <<= 1) {
    const float sign = (j & o) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(sign, v[i], __shfl_xor_sync(kFull, v[i], o));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= 0.08838834764831845f;  // 1 / sqrt(128)
}

// KVarN: a group of 16 lanes reads kKvTokens entries of the list for one head,
// keeping the page's per-channel key factors (c scale, c zero) and value factors c
// in registers while the page stays the same.  The entries and every token's codes
// and factors are loaded before the first token is transformed.
constexpr int kKvTokens = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads) read_kvarn_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int D = 128, P = 128, TPR = D / kVec, GRP = kThreads / TPR;
  constexpr int META = P * D * 3 / 4;
  const int g = threadIdx.x / TPR, j = threadIdx.x % TPR, h = blockIdx.y, lane = threadIdx.x & 31;
  const long long t0 = ((long long)blockIdx.x * GRP + g) * kKvTokens;
  int slot = -1;
  if (j < kKvTokens && t0 + j < a.num_tokens) slot = __ldg(a.slots + t0 + j);
  if (slot >= 0 && (slot >> 7) >= a.num_pages) {
    if (h == 0) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_SLOT_RANGE);
    slot = -1;
  }
  int sl[kKvTokens];
  uint32_t kw[kKvTokens], vw[kKvTokens];
  float kr[kKvTokens], vs[kKvTokens], vz[kKvTokens], vr[kKvTokens];
  auto block = [&](int s) { return a.pool + kHeaderBytes + ((size_t)(s >> 7) * a.Hkv + h) * a.block_bytes; };
#pragma unroll
  for (int i = 0; i < kKvTokens; ++i) {
    sl[i] = __shfl_sync(kFull, slot, (lane & 16) + i);
    kw[i] = vw[i] = 0u;
    kr[i] = vs[i] = vz[i] = vr[i] = 0.0f;
    if (sl[i] >= 0) {
      const uint8_t* blk = block(sl[i]);
      const int off = sl[i] & 127;
      const float* km = reinterpret_cast<const float*>(blk + META);
      const float* vm = km + 3 * D + P;
      if (a.k) {
        kw[i] = __ldg(reinterpret_cast<const uint32_t*>(blk + off * (D / 2) + kVec / 2 * j));
        kr[i] = __ldg(km + 3 * D + off);
      }
      if (a.v) {
        vw[i] = __ldg(reinterpret_cast<const uint16_t*>(blk + P * D / 2 + off * (D / 4) + kVec / 4 * j));
        vs[i] = __ldg(vm + off);
        vz[i] = __ldg(vm + P + off);
        vr[i] = __ldg(vm + 2 * P + off);
      }
    }
  }
  int held = -1;
  float ks[8], kz[8], vc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) ks[e] = kz[e] = vc[e] = 0.0f;
  // no early exit: every lane takes part in the transform's shuffles
#pragma unroll
  for (int i = 0; i < kKvTokens; ++i) {
    const bool on = sl[i] >= 0;
    if (on && (sl[i] >> 7) != held) {
      held = sl[i] >> 7;
      const float* km = reinterpret_cast<const float*>(block(sl[i]) + META);
      const float* vm = km + 3 * D + P;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const int d = kVec * j + e;
        const float4 s = __ldg(reinterpret_cast<const float4*>(km + d)), z = __ldg(reinterpret_cast<const float4*>(km + D + d));
        const float4 c = __ldg(reinterpret_cast<const float4*>(km + 2 * D + d));
        const float4 u = __ldg(reinterpret_cast<const float4*>(vm + 3 * P + d));
        ks[e] = c.x * s.x; ks[e + 1] = c.y * s.y; ks[e + 2] = c.z * s.z; ks[e + 3] = c.w * s.w;
        kz[e] = c.x * z.x; kz[e + 1] = c.y * z.y; kz[e + 2] = c.z * z.z; kz[e + 3] = c.w * z.w;
        vc[e] = u.x; vc[e + 1] = u.y; vc[e + 2] = u.z; vc[e + 3] = u.w;
      }
    }
    const long long o = ((t0 + i) * a.Hkv + h) * D + kVec * j;
    float f[8];
    if (a.k) {  // uniform
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = kr[i] * fmaf(ks[e], (float)((kw[i] >> (4 * e)) & 15u), kz[e]);
      fwht128x8(f, j);
      if (on) store8<T>(static_cast<T*>(a.k) + o, f, a.k_span, a.pool);
    }
    if (a.v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = vr[i] * vc[e] * fmaf(vs[i], (float)((vw[i] >> (2 * e)) & 3u), vz[i]);
      fwht128x8(f, j);
      if (on) store8<T>(static_cast<T*>(a.v) + o, f, a.v_span, a.pool);
    }
  }
}

template <int MODE, int D, typename T>
cudaError_t launch_rows(ReadArgs& a, cudaStream_t s) {
  constexpr int TOK = kThreads / (D / kVec);
  const long long blocks = (a.num_tokens + TOK - 1) / TOK;
  // all heads of a token in one CTA unless that leaves SMs without work
  a.heads_per_cta = blocks >= 2 * num_sms() ? a.Hkv : kInFlight;
  const int parts = (a.Hkv + a.heads_per_cta - 1) / a.heads_per_cta;
  read_rows_kernel<MODE, D, T><<<dim3((unsigned)blocks, parts), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_read(const kvq_cache* c, ReadArgs& a, cudaStream_t s) {
  const int D = c->cfg.head_dim;
  if (c->cfg.mode == KVQ_KVARN_K4V2_G128) {
    constexpr int TOK = kThreads / (128 / kVec) * kKvTokens;
    read_kvarn_kernel<T><<<dim3((unsigned)((a.num_tokens + TOK - 1) / TOK), a.Hkv), kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  if (D != 32 && D != 128) return cudaErrorInvalidValue;
  switch (c->cfg.mode) {
    case KVQ_FP8_PER_TENSOR: return D == 128 ? launch_rows<KVQ_FP8_PER_TENSOR, 128, T>(a, s) : launch_rows<KVQ_FP8_PER_TENSOR, 32, T>(a, s);
    case KVQ_INT8_PER_TOKEN_HEAD: return D == 128 ? launch_rows<KVQ_INT8_PER_TOKEN_HEAD, 128, T>(a, s) : launch_rows<KVQ_INT8_PER_TOKEN_HEAD, 32, T>(a, s);
    case KVQ_FP8_PER_TOKEN_HEAD: return D == 128 ? launch_rows<KVQ_FP8_PER_TOKEN_HEAD, 128, T>(a, s) : launch_rows<KVQ_FP8_PER_TOKEN_HEAD, 32, T>(a, s);
    case KVQ_NVFP4:  // NVFP4 4over6 shares NVFP4's storage
    case KVQ_NVFP4_4OVER6: return D == 128 ? launch_rows<KVQ_NVFP4, 128, T>(a, s) : launch_rows<KVQ_NVFP4, 32, T>(a, s);
    case KVQ_INT4_PER_TOKEN_HEAD: return D == 128 ? launch_rows<KVQ_INT4_PER_TOKEN_HEAD, 128, T>(a, s) : launch_rows<KVQ_INT4_PER_TOKEN_HEAD, 32, T>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_cache_read(const kvq_cache* c, const int32_t* slots, int num_tokens, void* k_out, void* v_out,
                              int out_dtype, cudaStream_t stream) {
  ReadArgs a;
  a.pool = c->base;
  a.slots = slots;
  a.num_tokens = num_tokens;
  a.Hkv = c->cfg.num_kv_heads;
  a.num_pages = c->cfg.num_pages;
  a.heads_per_cta = a.Hkv;
  a.block_bytes = c->block_bytes;
  a.k = k_out;
  a.v = v_out;
  const size_t n = (size_t)num_tokens * a.Hkv * c->cfg.head_dim * (out_dtype == KVQ_F16 ? 2 : 4);
  uint8_t* k = static_cast<uint8_t*>(k_out);
  uint8_t* v = static_cast<uint8_t*>(v_out);
  a.k_span = Span{k, k ? k + n : nullptr};
  a.v_span = Span{v, v ? v + n : nullptr};
  return out_dtype == KVQ_F16 ? launch_read<__half>(c, a, stream) : launch_read<float>(c, a, stream);
}

}  // namespace kvq
