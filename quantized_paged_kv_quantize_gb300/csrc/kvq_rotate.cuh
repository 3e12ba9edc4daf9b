// kvq_rotate.cuh -- norm and rotation of rows held in registers, correctly rounded:
// the double-word fp32 arithmetic and the rotation that kvq_rope.cu (which says how
// the rounding is settled) and kvq_latent_write.cu share.  The files that include it
// are compiled with -fmad=false.
#pragma once

#include "kvq_quant.cuh"

namespace kvq {
namespace {

// ---- double-word arithmetic
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

// A token's cosines and sines (its row of the table) for lane j of the group that holds a
// head row, VEC values a lane; neutral where !in.
template <int VEC>
__device__ __forceinline__ void load_rotation(Rotation<VEC>& rot, const float* row, int dims, bool interleaved, int j, bool in) {
  const int half = dims / 2, lane = threadIdx.x & 31;
  rot.on = j * VEC < dims;
  rot.pairs = interleaved;
  const bool first = j * VEC < half;
  rot.partner = rot.on && !rot.pairs ? (first ? lane + half / VEC : lane - half / VEC) : lane;
  const int at = first ? j * VEC : j * VEC - half;  // half-split: this lane's entries
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    rot.c[i] = make_float2(1.0f, 1.0f);
    rot.s[i] = make_float2(0.0f, 0.0f);
  }
  if (!rot.on || !in) return;
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

}  // namespace
}  // namespace kvq
