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
#include "kvq_quant.cuh"

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

// ---- double-word arithmetic (this file is built with -fmad=false)
struct DW {
  float h, l;
};
__device__ __forceinline__ DW two_sum(float a, float b) {
  const float s = a + b, bb = s - a;
  return {s, (a - (s - bb)) + (b - bb)};
}
__device__ __forceinline__ DW two_prod(float a, float b) {
  const float p = a * b;
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ DW quick(float h, float l) {  // |h| >= |l|
  const float s = h + l;
  return {s, l - (s - h)};
}
__device__ __forceinline__ DW add(DW a, DW b) {
  const DW s = two_sum(a.h, b.h);
  return quick(s.h, s.l + (a.l + b.l));
}
// 1 / sqrt(s): one Newton step on the fp32 reciprocal root r,
// r (1 + e/2 + 3 e^2 / 8) with e = 1 - s r^2, the residual kept to ~2^-47.
__device__ __forceinline__ DW rsqrt_dw(DW s) {
  const float r = rsqrtf(s.h);
  if (!(s.h >= 0x1p-120f && s.h <= 0x1p120f)) return {r, 0.0f};  // zero, infinite, NaN or out of the step's range
  const DW h = two_prod(r, r);
  const DW p = two_prod(s.h, h.h);
  const float e = ((1.0f - p.h) - p.l) - (s.h * h.l + s.l * h.h);
  return quick(r, r * (e * (0.5f + 0.375f * e)));
}
// The nearest fp32 value of z, with its last bit set when inexact if it is to
// be rounded again to fp16 (rounding to odd: the second rounding is then the
// rounding of z itself).
template <bool ODD>
__device__ __forceinline__ float round_dw(DW z) {
  const float r = z.h + z.l;
  if (!ODD) return r;
  const float rest = (z.h - r) + z.l;
  uint32_t b = __float_as_uint(r);
  if (rest != 0.0f && !(b & 1u) && r != 0.0f) b += ((rest < 0.0f) == (r < 0.0f)) ? 1u : ~0u;
  return __uint_as_float(b);
}

template <typename T>
__device__ __forceinline__ uint4 narrow16(const float* z);
template <>
__device__ __forceinline__ uint4 narrow16<__half>(const float* z) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = h2_as_u32(__floats2half2_rn(z[2 * i], z[2 * i + 1]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 narrow16<float>(const float* z) {
  return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
}

// A token's rotation of this lane's values, two neighbours to a register pair.
template <int VEC>
struct Rotation {
  float2 c[VEC / 2], s[VEC / 2];  // z = y c + (the pair's other value) s, signs in s
  int partner;                    // half-split: the lane that holds the other half's values
  bool on, pairs;                 // pairs: neighbours (2i, 2i + 1) rotate together
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return bits_f2(r);
}
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ uint32_t half2_rn(float2 a) { return h2_as_u32(__floats2half2_rn(a.x, a.y)); }

// mean(x^2) + eps as a double word, over the D values of a row: products and
// sums with their rounding errors carried along.
template <int D, int VEC>
__device__ __forceinline__ DW mean_square_dw(const float2* x, float eps) {
  DW t{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float v = (i & 1) ? x[i >> 1].y : x[i >> 1].x;
    const DW p = two_prod(v, v), u = two_sum(t.h, p.h);
    t = {u.h, t.l + (u.l + p.l)};
  }
#pragma unroll
  for (int o = 1; o < D / VEC; o <<= 1) {
    const DW p{__shfl_xor_sync(kFull, t.h, o), __shfl_xor_sync(kFull, t.l, o)}, u = two_sum(t.h, p.h);
    t = {u.h, (t.l + p.l) + u.l};
  }
  if (!isfinite(t.h)) return {t.h, 0.0f};
  const DW u = two_sum(t.h * (1.0f / D), eps);
  return quick(u.h, u.l + t.l * (1.0f / D));
}

// One value: (a c + b s) rs in double-word arithmetic, rounded to fp32 (to odd
// where an fp16 rounding follows).
template <bool F16>
__device__ __forceinline__ float rotate_dw(DW a, DW b, float c, float s, bool on, DW rs) {
  DW t = a;
  if (on) {
    DW p = two_prod(a.h, c), r = two_prod(b.h, s);
    p.l += a.l * c;
    r.l += b.l * s;
    t = add(p, r);
  }
  const DW m = two_prod(t.h, rs.h);
  return round_dw<F16>(quick(m.h, m.l + (t.h * rs.l + t.l * rs.h)));
}
// The same in plain fp32: what a product with an infinity or a NaN is, which has no low word.
__device__ __forceinline__ float rotate_plain(float a, float b, float c, float s, bool on, float rs) {
  return (on ? a * c + b * s : a) * rs;
}

// The correctly rounded rotated row, as its 16 stored bytes.  x: the lane's
// values; w: its weights (ones without a norm).
template <int D>
__device__ __forceinline__ uint4 rotate_row(const float2* x, const float2* w, bool norm, float eps,
                                            const Rotation<8>& rot, float2 nz) {  // fp16
  constexpr int N = 4, TPR = D / 8;
  float2 a[N], b[N];  // x w (exact) and the pair's other value
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = mul2z(x[i], w[i], nz);
#pragma unroll
  for (int i = 0; i < N; ++i)
    b[i] = rot.pairs ? make_float2(a[i].y, a[i].x)
                     : make_float2(__shfl_sync(kFull, a[i].x, rot.partner), __shfl_sync(kFull, a[i].y, rot.partner));
  float rs = 1.0f;
  if (norm) {
    const float2 q = add2(add2(mul2z(x[0], x[0], nz), mul2z(x[1], x[1], nz)),
                          add2(mul2z(x[2], x[2], nz), mul2z(x[3], x[3], nz)));
    float t = q.x + q.y;
#pragma unroll
    for (int o = 1; o < TPR; o <<= 1) t = t + __shfl_xor_sync(kFull, t, o);
    rs = __frsqrt_rn(t * (1.0f / D) + eps);
  }
  uint32_t lo[N], bad = 0;
  float2 finite = make_float2(0.0f, 0.0f);  // stays so
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 p = mul2(b[i], rot.s[i]), e = fma2(b[i], rot.s[i], neg2(p));
    const float2 z = mul2z(add2(fma2(a[i], rot.c[i], p), e), dup2(rs), nz);  // not rotated: c = 1, s = 0
    lo[i] = half2_rn(mul2(z, dup2(1.0f - 0x1.6p-21f)));
    bad |= lo[i] != half2_rn(mul2(z, dup2(1.0f + 0x1.6p-21f))) ? 1u << i : 0u;
    finite = fma2(z, make_float2(0.0f, 0.0f), finite);
  }
  const bool wild = !(finite.x + finite.y == 0.0f);  // a value is infinite or NaN, by itself or through its neighbour here
  if (wild) bad = (1u << N) - 1;
  if (__any_sync(kFull, bad != 0)) {
    const DW r = norm ? rsqrt_dw(mean_square_dw<D, 8>(x, eps)) : DW{1.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((bad >> i) & 1u)
        lo[i] = half2_rn(make_float2(
            rotate_dw<true>({a[i].x, 0.0f}, {b[i].x, 0.0f}, rot.c[i].x, rot.s[i].x, rot.on, r),
            rotate_dw<true>({a[i].y, 0.0f}, {b[i].y, 0.0f}, rot.c[i].y, rot.s[i].y, rot.on, r)));
    if (wild) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x0 = rotate_plain(a[i].x, b[i].x, rot.c[i].x, rot.s[i].x, rot.on, r.h);
        const float x1 = rotate_plain(a[i].y, b[i].y, rot.c[i].y, rot.s[i].y, rot.on, r.h);
        const uint32_t p = half2_rn(make_float2(x0, x1));
        if (!isfinite(x0)) lo[i] = prmt(lo[i], p, 0x3254u);
        if (!isfinite(x1)) lo[i] = prmt(lo[i], p, 0x7610u);
      }
    }
  }
  return make_uint4(lo[0], lo[1], lo[2], lo[3]);
}
template <int D>
__device__ __forceinline__ uint4 rotate_row(const float2* x, const float2* w, bool norm, float eps,
                                            const Rotation<4>& rot, float2) {  // fp32
  DW r{1.0f, 0.0f};
  float by = 1.0f;
  if (norm) {
    DW ms = mean_square_dw<D, 4>(x, eps);
    if (__any_sync(kFull, !(ms.h >= 0x1p-80f && ms.h <= 0x1p96f))) {
      float top = fmaxf(fmaxf(fabsf(x[0].x), fabsf(x[0].y)), fmaxf(fabsf(x[1].x), fabsf(x[1].y)));
#pragma unroll
      for (int o = 1; o < D / 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      // the larger exponent of the row and of eps's root
      const int e = max((int)(__float_as_uint(top) >> 23) - 127,
                        eps > 0.0f ? ((int)(__float_as_uint(eps) >> 23) - 127) >> 1 : -126);
      if (isfinite(top)) by = __int_as_float((127 - max(-126, min(126, e))) << 23);
      const float2 scaled[2] = {make_float2(x[0].x * by, x[0].y * by), make_float2(x[1].x * by, x[1].y * by)};
      ms = mean_square_dw<D, 4>(scaled, eps * by * by);
    }
    r = rsqrt_dw(ms);
  }
  uint32_t z[4];
  DW a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = (i & 1) ? two_prod(x[i >> 1].y * by, w[i >> 1].y) : two_prod(x[i >> 1].x * by, w[i >> 1].x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const DW b = rot.pairs ? a[i ^ 1]
                           : DW{__shfl_sync(kFull, a[i].h, rot.partner), __shfl_sync(kFull, a[i].l, rot.partner)};
    const float2 c2 = rot.c[i >> 1], s2 = rot.s[i >> 1];
    const float c = (i & 1) ? c2.y : c2.x, s = (i & 1) ? s2.y : s2.x;
    float v = rotate_dw<false>(a[i], b, c, s, rot.on, r);
    if (!isfinite(v)) v = rotate_plain(a[i].h, b.h, c, s, rot.on, r.h);
    z[i] = __float_as_uint(v);
  }
  return make_uint4(z[0], z[1], z[2], z[3]);
}

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
    const int half = a.rot / 2, lane = threadIdx.x & 31;
    rot.on = j * VEC < a.rot;
    rot.pairs = a.interleaved != 0;
    const bool first = j * VEC < half;
    rot.partner = rot.on && !rot.pairs ? (first ? lane + half / VEC : lane - half / VEC) : lane;
    const float* row = a.cos_sin + (long long)(in ? pos : 0) * a.rot;
    const int at = first ? j * VEC : j * VEC - half;  // half-split: this lane's entries
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      rot.c[i] = make_float2(1.0f, 1.0f);
      rot.s[i] = make_float2(0.0f, 0.0f);
    }
    if (rot.on && in) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        if (rot.pairs) {
          const float2 c = __ldg(reinterpret_cast<const float2*>(row + (j * VEC + i) / 2));
          const float2 s = __ldg(reinterpret_cast<const float2*>(row + half + (j * VEC + i) / 2));
          rot.c[i / 2] = dup2(c.x);
          rot.c[i / 2 + 1] = dup2(c.y);
          rot.s[i / 2] = make_float2(-s.x, s.x);
          rot.s[i / 2 + 1] = make_float2(-s.y, s.y);
        } else {
          const float4 c = __ldg(reinterpret_cast<const float4*>(row + at + i));
          const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + at + i));
          const float sg = first ? -1.0f : 1.0f;
          rot.c[i / 2] = make_float2(c.x, c.y);
          rot.c[i / 2 + 1] = make_float2(c.z, c.w);
          rot.s[i / 2] = make_float2(sg * s.x, sg * s.y);
          rot.s[i / 2 + 1] = make_float2(sg * s.z, sg * s.w);
        }
      }
    }
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
