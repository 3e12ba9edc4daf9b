// kvq_rope.cu -- per-head RMS norm and rotary position embedding of queries
// and keys, and the quantized write of keys and values into their pages, in
// one pass over a projection's output (kvq_norm_rope_write).
//
// For one head row x of D values, weights w, position p:
//   y = x w / sqrt(mean(x^2) + eps)                      (y = x without weights)
//   z_a = y_a cos - y_b sin,  z_b = y_b cos + y_a sin    for the rot/2 pairs (a, b)
// z is rounded once to the io type (queries and the optional keys leave as
// that); keys are quantized from the rounded row, so the pool holds exactly
// what kvq_quantize_write would store for it.
//
// Rounding.  A last-bit change of a key moves some quantized codes by a whole
// step, so the rotated rows are the correctly rounded ones, at close to the
// cost of plain fp32:
//  - fp16 rows: x w is exact in fp32 (22 bits), the pair product-difference
//    loses at most 3u of itself however much cancels (one FMA recovers the
//    rounding of the first product; Kahan's method, see Jeannerod, Louvet and
//    Muller, "Further analysis of Kahan's algorithm for the accurate
//    computation of 2x2 determinants", 2013), and with the plain fp32 sum of
//    squares the result is within 9u of z (u = 2^-24: the sum 4u, the
//    reciprocal root u, the difference 3u, the product u; the bracket is 11u).  Where both ends of
//    that bracket round to the same fp16 value, that is the answer (all but
//    about one value in 600); else
//  - the value is recomputed in double-word fp32 arithmetic (two-sum and
//    two-product, one Newton step for the reciprocal root; Dekker, "A
//    floating-point technique for extending the available precision", 1971),
//    good to about 2^-44, and rounded once (to odd in fp32, then to fp16).
//  fp32 rows always take the double-word form.
// Infinities and NaN go by the formula in plain fp32: their products have no rounding
// error to carry, and a value that is not rotated meets no other.  An fp32 row whose mean
// square leaves [2^-80, 2^96], where the low words of squares and roots would leave fp32,
// is normed times a power of two (a norm is the same for it).
//
// Bound by instruction issue (73% of the slots; DRAM 33%): about 300 instructions
// for two fp16 head rows, a third of them the double-word path that 35% of the
// warps take.  8191 tokens of 64 + 2 x 8 int8 heads: 105 us (3.3 TB/s of the rows in
// and out and the packed bytes).
//
// Layout.  A group of D / VEC lanes holds a head row (16 bytes a lane) and
// walks over a CTA's heads for one token, so the token's cosines and sines
// (fp32, from the caller's table) are read once per token and head chunk
// instead of once per head; the half-split pairs live in two lanes of the
// group and meet by shuffle.
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_rotate.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 1;  // head rows in flight behind the one a thread converts (two: 2% slower)

struct RopeArgs {
  WriteArgs w;  // pool, slots (null: no cache write), geometry
  const void* q;
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* positions;
  const float* cos_sin;  // [max_position][rot]: rot/2 cosines, then rot/2 sines
  int max_position, rot, interleaved;
  const void* wq;  // null: no norm
  const void* wk;
  float eps;
  void* q_out;  // [T][Hq][D]
  void* k_out;  // [T][Hkv][D] or null
  int Hq, chunk, q_chunks, k_chunks;  // heads per CTA; CTAs along y: queries, keys, values
  Span q_span, k_span;
};

template <int MODE, typename T, int D>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr int TPR = D / VEC;
  constexpr int TOK = kThreads / TPR;  // tokens per CTA
  const int g = threadIdx.x / TPR, j = threadIdx.x % TPR;
  const long long token = (long long)blockIdx.x * TOK + g;
  const int part = blockIdx.y;
  const int role = part < a.q_chunks ? 0 : part < a.q_chunks + a.k_chunks ? 1 : 2;  // queries, keys, values
  const int h0 = (part - (role == 0 ? 0 : role == 1 ? a.q_chunks : a.q_chunks + a.k_chunks)) * a.chunk;
  const int heads = role == 0 ? a.Hq : a.w.Hkv;
  const int h1 = min(heads, h0 + a.chunk);
  bool in = token < a.w.num_tokens;
  const int pos = in && a.rot ? __ldg(a.positions + token) : 0;
  if (in && (pos < 0 || pos >= a.max_position)) {
    if (j == 0 && h0 == 0 && role == 0) set_error(a.w.pool, KVQ_DEVERR_POSITION);
    in = false;
  }
  const T* src = static_cast<const T*>(role == 0 ? a.q : role == 1 ? a.k : a.v);
  src += (in ? token : 0) * (role == 0 ? a.q_stride : role == 1 ? a.k_stride : a.v_stride) + j * VEC;

  Rotation<VEC> rot;
  float2 w[VEC / 2];
  const bool norm = role == 0 ? a.wq != nullptr : a.wk != nullptr;
  if (role < 2) {
    load_rotation<VEC>(rot, a.cos_sin + (long long)(in ? pos : 0) * a.rot, a.rot, a.interleaved != 0, j, in);
    float wv[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) wv[i] = 1.0f;
    if (norm) widen16<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(role == 0 ? a.wq : a.wk) + j * VEC)), wv);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) w[i] = make_float2(wv[2 * i], wv[2 * i + 1]);
  }
  int slot = -1;
  TensorScale ts{1.0f, QDiv(1.0f), QDiv(1.0f)};
  if constexpr (MODE != 0) {
    if (in && role > 0) slot = __ldg(a.w.slots + token);
    ts = TensorScale::make<MODE>(a.w, role == 2);
  }

  // The row being converted and the kAhead rows whose loads are in flight.  One
  // copy of the loop's body: unrolled over four heads it outgrew the
  // instruction cache (8191 tokens of 64 + 2 x 8 int8 heads: 407 us).
  auto load = [&](int h) {
    return in && h < h1 ? *reinterpret_cast<const uint4*>(src + (long long)h * D) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 ahead[kAhead];
#pragma unroll
  for (int r = 0; r < kAhead; ++r) ahead[r] = load(h0 + r);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    uint4 raw = ahead[0];
#pragma unroll
    for (int r = 0; r + 1 < kAhead; ++r) ahead[r] = ahead[r + 1];
    ahead[kAhead - 1] = load(h + kAhead);
    float f[VEC];
    if (role == 2) {
      if constexpr (MODE != 0) {
        if constexpr (kFourBit<MODE>) {
          if constexpr (TPR != 16) __syncthreads();  // the previous head's codes have been read
          pair_values_pass<MODE, D, VEC, TPR, TOK, 1, T>(a.w, h, &slot, &raw, j, ts);
        } else {
          widen16<T>(raw, f);
          quantize_row<MODE, D, VEC, TPR>(a.w, h, 1, slot, j, f, ts);
        }
      }
      continue;
    }
    widen16<T>(raw, f);
    float2 x[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) x[i] = make_float2(f[2 * i], f[2 * i + 1]);
    const uint4 out = rotate_row<D>(x, w, norm, a.eps, rot, dup2(a.w.neg_zero));
    if (role == 0) {
      if (in)
        st_chk(reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + (token * a.Hq + h) * D + j * VEC), out, a.q_span,
               a.w.pool);
      continue;
    }
    if (in && a.k_out)
      st_chk(reinterpret_cast<uint4*>(static_cast<T*>(a.k_out) + (token * a.w.Hkv + h) * D + j * VEC), out, a.k_span,
             a.w.pool);
    if constexpr (MODE != 0) {
      widen16<T>(out, f);  // the key as the io type holds it
      quantize_row<MODE, D, VEC, TPR>(a.w, h, 0, slot, j, f, ts);
    }
  }
}

template <int MODE, typename T, int D>
cudaError_t launch(RopeArgs& a, cudaStream_t s) {
  constexpr int TOK = kThreads / (D / (16 / (int)sizeof(T)));
  const long long blocks = (a.w.num_tokens + TOK - 1) / TOK;
  // Heads per CTA: more heads share a token's table rows and weights, fewer give
  // more CTAs; doubled while six CTAs per SM are left (8191 tokens of 64 + 2 x 8
  // int8 heads: 113 us with 8 heads, 105 with up to 32).
  auto chunks = [](int heads, int c) { return (heads + c - 1) / c; };
  a.chunk = 4;
  while (a.chunk < 32 && blocks * (chunks(a.Hq, 2 * a.chunk) + 2 * chunks(a.w.Hkv, 2 * a.chunk)) >= 6 * num_sms()) a.chunk *= 2;
  a.q_chunks = chunks(a.Hq, a.chunk);
  a.k_chunks = (MODE != 0 || a.k_out) ? chunks(a.w.Hkv, a.chunk) : 0;
  const int v_chunks = MODE != 0 ? chunks(a.w.Hkv, a.chunk) : 0;
  norm_rope_kernel<MODE, T, D><<<dim3((unsigned)blocks, a.q_chunks + a.k_chunks + v_chunks), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_mode(int mode, RopeArgs& a, cudaStream_t s) {
  switch (mode) {
    case 0: return launch<0, T, D>(a, s);
    case KVQ_FP8_PER_TENSOR: return launch<KVQ_FP8_PER_TENSOR, T, D>(a, s);
    case KVQ_INT8_PER_TOKEN_HEAD: return launch<KVQ_INT8_PER_TOKEN_HEAD, T, D>(a, s);
    case KVQ_FP8_PER_TOKEN_HEAD: return launch<KVQ_FP8_PER_TOKEN_HEAD, T, D>(a, s);
    case KVQ_NVFP4: return launch<KVQ_NVFP4, T, D>(a, s);
    case KVQ_INT4_PER_TOKEN_HEAD: return launch<KVQ_INT4_PER_TOKEN_HEAD, T, D>(a, s);
    case KVQ_NVFP4_4OVER6: return launch<KVQ_NVFP4_4OVER6, T, D>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_norm_rope_write(const kvq_cache* c, const kvq_norm_rope& r, cudaStream_t stream) {
  RopeArgs a;
  a.w.pool = c->base;
  a.w.k = r.k;
  a.w.v = r.v;
  a.w.slots = r.slot_mapping;
  a.w.num_tokens = r.num_tokens;
  a.w.Hkv = c->cfg.num_kv_heads;
  a.w.P = c->cfg.page_size;
  a.w.log2P = 0;
  while ((1 << a.w.log2P) < a.w.P) ++a.w.log2P;
  a.w.num_pages = c->cfg.num_pages;
  a.w.block_bytes = c->block_bytes;
  a.w.seq_ids = nullptr;
  a.w.tail = nullptr;
  a.w.num_seqs = 0;
  a.w.pool_span = pool_blocks(c);
  a.w.tail_span = Span{nullptr, nullptr};
  a.q = r.q;
  a.k = r.k;
  a.v = r.v;
  a.q_stride = r.q_stride;
  a.k_stride = r.k_stride;
  a.v_stride = r.v_stride;
  a.positions = r.positions;
  a.cos_sin = r.cos_sin;
  a.max_position = r.rot_dim ? r.max_position : 1;
  a.rot = r.rot_dim;
  a.interleaved = r.interleaved;
  a.wq = r.q_weight;
  a.wk = r.k_weight;
  a.eps = r.eps;
  a.q_out = r.q_out;
  a.k_out = r.k_out;
  a.Hq = r.num_q_heads;
  const int D = c->cfg.head_dim;
  const bool f16 = c->cfg.io_dtype == KVQ_F16;
  const size_t row = (size_t)r.num_tokens * D * (f16 ? 2 : 4);
  uint8_t* qo = static_cast<uint8_t*>(r.q_out);
  uint8_t* ko = static_cast<uint8_t*>(r.k_out);
  a.q_span = Span{qo, qo + row * a.Hq};
  a.k_span = Span{ko, ko ? ko + row * a.w.Hkv : nullptr};
  const int mode = r.slot_mapping ? c->cfg.mode : 0;
  if (D == 128) return f16 ? launch_mode<__half, 128>(mode, a, stream) : launch_mode<float, 128>(mode, a, stream);
  if (D == 32) return f16 ? launch_mode<__half, 32>(mode, a, stream) : launch_mode<float, 32>(mode, a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvq
