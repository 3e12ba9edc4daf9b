// kvq_quant.cuh -- quantization of rows held in registers into the paged pool:
// the arithmetic and the stores that every write kernel of the 16-token-page
// modes shares (kvq_write.cu, kvq_rope.cu).  The files that include it are
// compiled with -fmad=false, and the code uses explicit _rn intrinsics, so
// every fp32 operation is individually rounded: the quantized bytes and scales
// are bit-identical to the specification in kvq.h.
#pragma once

#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

struct WriteArgs {
  uint8_t* pool;
  const void* k;
  const void* v;
  const int32_t* slots;
  long long num_tokens;
  int Hkv, P, log2P, num_pages;
  size_t block_bytes;
  // KVarN open tiles (kvq_kvarn_append): sequence of each token, and the tail
  // buffer, K rows [num_seqs][128][Hkv][D] then V rows, io dtype
  const int32_t* seq_ids;
  uint8_t* tail;
  int num_seqs;
  // the pool's blocks and the tail buffer, as spans (debug-build store checks)
  Span pool_span, tail_span;
  // -0.0f, as a value the compiler cannot see: the addend that turns a packed
  // fused multiply-add into an exactly rounded product (see mul2z)
  float neg_zero = -0.0f;
};

template <typename T>
__device__ __forceinline__ void load16(const T* p, float* f);
template <>
__device__ __forceinline__ void load16<__half>(const __half* p, float* f) {
  uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 t = __half22float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <>
__device__ __forceinline__ void load16<float>(const float* p, float* f) {
  float4 u = __ldg(reinterpret_cast<const float4*>(p));
  f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
}

// 16 loaded bytes -> fp32 values (exact widening of fp16; fp32 as is).
template <typename T>
__device__ __forceinline__ void widen16(const uint4& u, float* f);
template <>
__device__ __forceinline__ void widen16<__half>(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(u32_as_h2(w[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <>
__device__ __forceinline__ void widen16<float>(const uint4& u, float* f) {
  f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
}

template <int N>
__device__ __forceinline__ void store_bytes(uint8_t* dst, const uint32_t* w);
template <int N>
__device__ __forceinline__ void store_bytes_chk(uint8_t* dst, const uint32_t* w, const WriteArgs& a) {
  if (in_span(dst, N, a.pool_span, a.pool)) store_bytes<N>(dst, w);
}
template <>
__device__ __forceinline__ void store_bytes<2>(uint8_t* dst, const uint32_t* w) {
  *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(w[0]);
}
template <>
__device__ __forceinline__ void store_bytes<4>(uint8_t* dst, const uint32_t* w) {
  *reinterpret_cast<uint32_t*>(dst) = w[0];
}
template <>
__device__ __forceinline__ void store_bytes<8>(uint8_t* dst, const uint32_t* w) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

// x / d for a constant divisor d, given rd = RN(1/d): q0 = RN(x rd), the
// remainder r = x - q0 d (exact, one FMA), q = RN(q0 + r rd) -- Markstein's
// correction step ("Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  For the divisors and inputs used here it
// returns the IEEE quotient RN(x/d) for every input, checked exhaustively over
// all fp32 values: d = 127, 448, 7 with x >= 1e-8 (scales of max(amax, 1e-8))
// and d = 15, 3 with any finite x >= 0 (KVarN ranges, zero and subnormals
// included); infinities and NaN take the IEEE division.
__device__ __forceinline__ float div_const(float x, float d, float rd) {
  if (!(x <= 0x1.fffffep127f)) return __fdiv_rn(x, d);  // inf and NaN keep IEEE semantics
  const float q0 = __fmul_rn(x, rd);
  const float r = __fmaf_rn(-q0, d, x);
  return __fmaf_rn(r, rd, q0);
}
constexpr float kRcp127 = 0x1.020408p-7f, kRcp448 = 0x1.24924ap-9f, kRcp7 = 0x1.24924ap-3f;
constexpr float kRcp15 = 0x1.111112p-4f, kRcp3 = 0x1.555556p-2f;

// The reciprocals are RN(1/d): checked here against the compiler's own
// correctly rounded constant division.
static_assert(kRcp127 == 1.0f / 127.0f && kRcp448 == 1.0f / 448.0f && kRcp7 == 1.0f / 7.0f,
              "reciprocal constants of the per-token-head scales");
static_assert(kRcp15 == 1.0f / 15.0f && kRcp3 == 1.0f / 3.0f, "reciprocal constants of the RTN scales");

// Packed fp32 pairs (f32x2): each lane is rounded on its own, exactly as the
// scalar __fadd_rn / __fmul_rn, so a pair op is two of the specification's
// operations in one instruction.  Written as PTX with the explicit .rn
// modifier, which keeps the compiler from contracting a product and a sum
// into one fused multiply-add (the packed intrinsics were contracted).
__device__ __forceinline__ unsigned long long f2_bits(float2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 bits_f2(unsigned long long r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return bits_f2(r);
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  unsigned long long r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return bits_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return bits_f2(r);
}
// The code generator fuses a packed product into a packed sum that consumes it
// (explicit .rn and -fmad=false notwithstanding; measured on GB300: 18% of
// (a b) + c pairs differed from the two rounded steps).  A product that feeds
// a sum is therefore written as fma(a, b, -0): a b + (-0) rounded once is the
// rounded product, for every a b (a zero keeps its sign), and a fused
// multiply-add has nothing left to fuse with.  z = (-0, -0) must come from a
// kernel argument so that the addend is not folded away.
__device__ __forceinline__ float2 mul2z(float2 a, float2 b, float2 z) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(z)));
  return bits_f2(r);
}
__device__ __forceinline__ float2 dup2(float a) { return make_float2(a, a); }

// Encoding of the IEEE quotient RN(x/s) without a division on the common path.
// With r the hardware's approximate reciprocal of s (relative error below
// 2^-21 = 8u, u = 2^-24), rlo = RN(r(1 - 2^-20)) and rhi = RN(r(1 + 2^-20)),
// the products RN(x rlo) and RN(x rhi) enclose RN(x/s): their relative
// distance to x/s is at least 16u - 8u - 2u on each side, while RN(x/s) is
// within u of it.  Every encoder used here (round-to-nearest-even onto a
// grid, with saturation) is monotone, so when both ends encode to the same
// code, that is the code of RN(x/s); when they differ the quotient is computed
// exactly.  Scales whose reciprocal is not a comfortable normal number always
// divide.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
struct QDiv {
  float s, rlo, rhi;
  bool fast;
  __device__ __forceinline__ explicit QDiv(float s_) : s(s_) {
    const float r = rcp_approx(s_);
    fast = r >= 0x1p-100f && r <= 0x1p100f;
    rlo = __fmul_rn(r, 1.0f - 0x1p-20f);
    rhi = __fmul_rn(r, 1.0f + 0x1p-20f);
  }
  // E4M3 codes of x1:x0 (x0 in the low byte)
  __device__ __forceinline__ uint32_t e4m3x2(float x1, float x0) const {
    const uint32_t lo = f32x2_to_e4m3x2(__fmul_rn(x1, rlo), __fmul_rn(x0, rlo));
    const uint32_t hi = f32x2_to_e4m3x2(__fmul_rn(x1, rhi), __fmul_rn(x0, rhi));
    if (fast && lo == hi) return lo;
    return f32x2_to_e4m3x2(__fdiv_rn(x1, s), __fdiv_rn(x0, s));
  }
  // Four int8 codes clamp(rint(x/s), -127, 127), x[0] in the low byte.  rint
  // is done by adding 1.5 * 2^23: round-to-nearest-even leaves the integer in
  // the low mantissa bits, whose low byte is the two's-complement code.  The
  // fast path also requires both ends inside [-127, 127] (bit patterns
  // 0x4B400000 -127 .. +127), so neither the clamp nor a NaN can reach it.
  // (The products and the additions run as packed pairs; z = (-0, -0), see mul2z.)
  __device__ __forceinline__ uint32_t int8x4(const float* x, float2 z) const {
    const float2 magic = dup2(12582912.0f);  // 1.5 * 2^23
    uint32_t lo[4], bad = fast ? 0u : 1u;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float2 x2 = make_float2(x[e], x[e + 1]);
      const float2 l2 = add2(mul2z(x2, dup2(rlo), z), magic), h2 = add2(mul2z(x2, dup2(rhi), z), magic);
      lo[e] = __float_as_uint(l2.x);
      lo[e + 1] = __float_as_uint(l2.y);
      bad |= (lo[e] ^ __float_as_uint(h2.x)) | static_cast<uint32_t>(lo[e] - 0x4B3FFF81u > 254u);
      bad |= (lo[e + 1] ^ __float_as_uint(h2.y)) | static_cast<uint32_t>(lo[e + 1] - 0x4B3FFF81u > 254u);
    }
    if (bad == 0) return prmt(prmt(lo[0], lo[1], 0x0040u), prmt(lo[2], lo[3], 0x0040u), 0x5410u);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float qv = fminf(fmaxf(rintf(__fdiv_rn(x[e], s)), -127.0f), 127.0f);
      w |= (static_cast<uint32_t>(__float2int_rn(qv)) & 0xFFu) << (8 * e);
    }
    return w;
  }
  // N <= 8 signed 4-bit codes clamp(rint(x/s), -7, 7) of x[0..N), two's
  // complement.  Same rint as int8x4; the fast path requires both ends inside
  // [-7, 7] (bit patterns 0x4B400000 -7 .. +7), whose low nibble is then the
  // code.  KEY = false: x[e] in nibble e.  KEY = true, the key-word order of
  // an 8-channel group: x[e] in nibble e/2 for even e, 4 + e/2 for odd e.
  template <int N, bool KEY = false>
  __device__ __forceinline__ uint32_t int4x8(const float* x, float2 z) const {
    static_assert(N % 2 == 0, "pairs");
    const float2 magic = dup2(12582912.0f);  // 1.5 * 2^23
    uint32_t lo[N], bad = fast ? 0u : 1u;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 x2 = make_float2(x[e], x[e + 1]);
      const float2 l2 = add2(mul2z(x2, dup2(rlo), z), magic), h2 = add2(mul2z(x2, dup2(rhi), z), magic);
      lo[e] = __float_as_uint(l2.x);
      lo[e + 1] = __float_as_uint(l2.y);
      bad |= (lo[e] ^ __float_as_uint(h2.x)) | static_cast<uint32_t>(lo[e] - 0x4B3FFFF9u > 14u);
      bad |= (lo[e + 1] ^ __float_as_uint(h2.y)) | static_cast<uint32_t>(lo[e + 1] - 0x4B3FFFF9u > 14u);
    }
    if (bad != 0) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float qv = fminf(fmaxf(rintf(__fdiv_rn(x[e], s)), -7.0f), 7.0f);
        lo[e] = static_cast<uint32_t>(__float2int_rn(qv));
      }
    }
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) w |= (lo[e] & 0xFu) << (4 * (KEY ? ((e & 1) ? 4 + e / 2 : e / 2) : e));
    return w;
  }
  // eight E2M1 codes (pairs packed low nibble first) of x[0..n)
  template <int N>
  __device__ __forceinline__ uint32_t e2m1x8(const float* x) const {
    float ylo[8], yhi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ylo[i] = i < N ? __fmul_rn(x[i], rlo) : 0.0f;
      yhi[i] = i < N ? __fmul_rn(x[i], rhi) : 0.0f;
    }
    const uint32_t lo = f32x8_to_e2m1x8(ylo), hi = f32x8_to_e2m1x8(yhi);
    if (fast && lo == hi) return lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) ylo[i] = i < N ? __fdiv_rn(x[i], s) : 0.0f;
    return f32x8_to_e2m1x8(ylo);
  }
};

// Group max over TPR consecutive lanes (TPR a power of two <= 32).
template <int TPR>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = 1; o < TPR; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Squared reconstruction error of a 16-value block whose codes (w, this
// thread's VEC of them) reconstruct as E2M1(code) * den: fp32, every operation
// rounded alone, summed as a pairwise tree of neighbours -- within the thread
// for its VEC consecutive values, then across the TPB lanes of the block
// (xor 1, 2: each level adds two neighbouring subtrees, and fp32 addition is
// commutative, so every lane holds the same total).
// Packed: values i and i + VEC/2 share a pair, so the neighbour levels of the
// tree are pair additions and the last one adds the pair's two halves.
template <int VEC, int TPB>
__device__ __forceinline__ float block_sse(const float* x, uint32_t w, float den, float2 z) {
  constexpr int H = VEC / 2;
  uint32_t h[4];
  e2m1x8_to_f16x2x4(w, h);
  float val[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const __half2 p = u32_as_h2(h[i / 2]);
    val[i] = (i & 1) ? __high2float(p) : __low2float(p);
  }
  float2 e[H];  // (error^2 of value k, of value k + H)
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const float2 d = sub2(make_float2(x[k], x[k + H]), mul2z(make_float2(val[k], val[k + H]), dup2(den), z));
    e[k] = mul2z(d, d, z);
  }
#pragma unroll
  for (int st = 1; st < H; st <<= 1)
#pragma unroll
    for (int k = 0; k < H; k += 2 * st) e[k] = add2(e[k], e[k + st]);
  float t = __fadd_rn(e[0].x, e[0].y);
#pragma unroll
  for (int o = 1; o < TPB; o <<= 1) t = __fadd_rn(t, __shfl_xor_sync(kFull, t, o));
  return t;
}

// NVFP4 codes of a thread's VEC values (its 16-value block shared with TPB =
// 16 / VEC lanes): the E4M3 block scale byte sb and the E2M1 codes packed two
// per byte, even channel in the low nibble (sb = 0 gives all-zero codes).
// F46 (nvfp4_4over6): the block is also coded with the max/4 scale
// E4M3(amax / (4 s_t)), and that coding is kept when its block_sse is smaller.
// q6, q4: the quotient brackets of RN(6 s_t) and RN(4 s_t).
template <int VEC, int TPB, bool F46>
__device__ __forceinline__ void nvfp4_codes(const float* x, float st, const QDiv& q6, const QDiv& q4, float2 z,
                                            uint32_t& w, uint32_t& sb) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = group_max<TPB>(amax);
  sb = q6.e4m3x2(0.0f, amax) & 0xFFu;  // E4M3(RN(amax / (6 s_t)))
  const float sbf = e4m3_to_f32(sb);
  const float den = __fmul_rn(st, sbf);
  w = sbf != 0.0f ? QDiv(den).e2m1x8<VEC>(x) : 0u;
  if constexpr (F46) {
    const uint32_t sb4 = q4.e4m3x2(0.0f, amax) & 0xFFu;  // E4M3(RN(amax / (4 s_t)))
    const float sbf4 = e4m3_to_f32(sb4);
    const float den4 = __fmul_rn(st, sbf4);
    const uint32_t w4 = sbf4 != 0.0f ? QDiv(den4).e2m1x8<VEC>(x) : 0u;
    if (block_sse<VEC, TPB>(x, w4, den4, z) < block_sse<VEC, TPB>(x, w, den, z)) {
      w = w4;
      sb = sb4;
    }
  }
}

template <int MODE>
constexpr bool kFourBit = MODE == KVQ_NVFP4 || MODE == KVQ_NVFP4_4OVER6 || MODE == KVQ_INT4_PER_TOKEN_HEAD;

// The n = 4 or 8 codes packed in w (two per byte) spread one per byte, in the
// low nibble: bytes c0, c1, c2, c3 (| c4..c7).
__device__ __forceinline__ uint2 spread_codes(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  return make_uint2(prmt(even, odd, 0x5140u), prmt(even, odd, 0x7362u));
}

// The side's per-tensor scale (FP8 per-tensor s, NVFP4 s_t) and the quotient
// brackets built from it, set up once per thread: the pool header does not
// change during a write.
struct TensorScale {
  float st;
  QDiv qs;  // FP8 per-tensor: x / s; NVFP4: amax / (6 s_t)
  QDiv q4;  // NVFP4 4over6: amax / (4 s_t)
  template <int MODE>
  __device__ __forceinline__ static TensorScale make(const WriteArgs& a, int side) {
    const float st = *reinterpret_cast<const float*>(a.pool + (side ? kHdrVScaleOffset : kHdrKScaleOffset));
    return TensorScale{st, QDiv(MODE == KVQ_FP8_PER_TENSOR ? st : __fmul_rn(6.0f, st)), QDiv(__fmul_rn(4.0f, st))};
  }
};

// Quantize one (token, kv head, side) row of D values, held by a group of TPR
// threads with VEC values each (thread j: values j*VEC ..), and store it at
// slot (skipped when slot < 0; flagged and skipped when out of range).
template <int MODE, int D, int VEC, int TPR>
__device__ __forceinline__ void quantize_row(const WriteArgs& a, int h, int side, int slot, int j, const float* x,
                                             const TensorScale& ts) {
  bool active = slot >= 0;
  const int page = slot >> a.log2P;
  const int off = slot & (a.P - 1);
  if (active && page >= a.num_pages) {
    if (j == 0) set_error(a.pool, KVQ_DEVERR_SLOT_RANGE);
    active = false;
  }
  uint8_t* blk = a.pool + kHeaderBytes + ((size_t)page * a.Hkv + h) * a.block_bytes;

  if constexpr (MODE == KVQ_FP8_PER_TENSOR) {
    const QDiv& q = ts.qs;
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC; i += 4) w[i / 4] = q.e4m3x2(x[i + 1], x[i]) | (q.e4m3x2(x[i + 3], x[i + 2]) << 16);
    if (active) store_bytes_chk<VEC>(blk + (size_t)side * a.P * D + (size_t)off * D + j * VEC, w, a);
  } else if constexpr (MODE == KVQ_INT8_PER_TOKEN_HEAD || MODE == KVQ_FP8_PER_TOKEN_HEAD) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = group_max<TPR>(amax);
    const float s = MODE == KVQ_INT8_PER_TOKEN_HEAD ? div_const(fmaxf(amax, 1e-8f), 127.0f, kRcp127)
                                                    : div_const(fmaxf(amax, 1e-8f), 448.0f, kRcp448);
    const QDiv q(s);
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      if constexpr (MODE == KVQ_INT8_PER_TOKEN_HEAD) {
        w[i / 4] = q.int8x4(x + i, dup2(a.neg_zero));
      } else {
        w[i / 4] = q.e4m3x2(x[i + 1], x[i]) | (q.e4m3x2(x[i + 3], x[i + 2]) << 16);
      }
    }
    if (active) {
      store_bytes_chk<VEC>(blk + (size_t)side * a.P * D + (size_t)off * D + j * VEC, w, a);
      if (j == 0) st_chk(reinterpret_cast<float*>(blk + (size_t)2 * a.P * D + (size_t)side * 4 * a.P + 4 * off), s, a.pool_span, a.pool);
    }
  } else if constexpr (MODE == KVQ_NVFP4 || MODE == KVQ_NVFP4_4OVER6) {  // keys; values: pair_values_pass
    constexpr int TPB = 16 / VEC;  // threads per 16-value block
    uint32_t w[1], sb;
    nvfp4_codes<VEC, TPB, MODE == KVQ_NVFP4_4OVER6>(x, ts.st, ts.qs, ts.q4, dup2(a.neg_zero), w[0], sb);
    if (active) {
      store_bytes_chk<VEC / 2>(blk + (size_t)off * D / 2 + j * VEC / 2, w, a);
      if ((j % TPB) == 0)
        st_chk(blk + (size_t)a.P * D + (size_t)off * D / 16 + (j * VEC) / 16, static_cast<uint8_t>(sb), a.pool_span, a.pool);
    }
  } else if constexpr (MODE == KVQ_INT4_PER_TOKEN_HEAD) {  // keys; values: pair_values_pass
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = group_max<TPR>(amax);
    const float s = div_const(fmaxf(amax, 1e-8f), 7.0f, kRcp7);
    // a key word holds an 8-channel group, even channels in its low half-word:
    // with 4 values per thread, two lanes fill one word (the odd lane's
    // channels 4..7 sit one byte higher) and the even lane stores it
    uint32_t w[1] = {QDiv(s).int4x8<VEC, true>(x, dup2(a.neg_zero))};
    if constexpr (VEC == 4) {
      if (j & 1) w[0] <<= 8;
      w[0] |= __shfl_xor_sync(kFull, w[0], 1);
    }
    if (active) {
      if (VEC == 8 || (j & 1) == 0) store_bytes_chk<4>(blk + (size_t)off * D / 2 + (j * VEC / 8) * 4, w, a);
      if (j == 0) st_chk(reinterpret_cast<float*>(blk + (size_t)a.P * D + 4 * off), s, a.pool_span, a.pool);
    }
  }
}


// 4-bit values (NVFP4, NVFP4 4over6, INT4): token-pair rows, byte (k, d) of a
// page holding channel d of tokens 2k (low nibble) and 2k + 1.  A token with
// an even slot whose successor in the batch holds the next slot stores the
// pair's bytes whole and the successor stores nothing; every other token
// writes its own nibbles with 32-bit atomic AND/OR (two tokens never share a
// nibble, so these commute), e.g. the one new token of a decode step.  The
// successor's codes come from the next row group of the same warp (a shuffle)
// when a warp holds two row groups (TPR = 16), else through shared memory
// (whole CTA, one barrier).  Scales (NVFP4 block scales, the INT4 token
// scale) are per token and stored directly.
template <int MODE, int D, int VEC, int TPR, int NTOK, int R, typename T>
__device__ __forceinline__ void pair_values_pass(const WriteArgs& a, int h, const int* slot, const uint4* raw,
                                                 int j, const TensorScale& ts) {
  constexpr int TPB = 16 / VEC;
  constexpr int TOK = NTOK / R;
  constexpr bool kInWarp = TPR == 16;
  __shared__ uint32_t codes[kInWarp ? 1 : NTOK * TPR];
  __shared__ int vslot[kInWarp ? 1 : NTOK];
  const int g = threadIdx.x / TPR;
  uint32_t wr[R];
  int sr[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float x[VEC];
    widen16<T>(raw[r], x);
    const int s = slot[r];
    bool active = s >= 0;
    const int page = s >> a.log2P, off = s & (a.P - 1);
    if (active && page >= a.num_pages) {
      if (j == 0) set_error(a.pool, KVQ_DEVERR_SLOT_RANGE);
      active = false;
    }
    uint8_t* blk = a.pool + kHeaderBytes + ((size_t)page * a.Hkv + h) * a.block_bytes;
    if constexpr (MODE == KVQ_INT4_PER_TOKEN_HEAD) {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) amax = fmaxf(amax, fabsf(x[i]));
      amax = group_max<TPR>(amax);
      const float sc = div_const(fmaxf(amax, 1e-8f), 7.0f, kRcp7);
      wr[r] = QDiv(sc).int4x8<VEC>(x, dup2(a.neg_zero));
      if (active && j == 0)
        st_chk(reinterpret_cast<float*>(blk + (size_t)a.P * D + (size_t)4 * a.P + 4 * off), sc, a.pool_span, a.pool);
    } else {
      uint32_t sb;
      nvfp4_codes<VEC, TPB, MODE == KVQ_NVFP4_4OVER6>(x, ts.st, ts.qs, ts.q4, dup2(a.neg_zero), wr[r], sb);
      if (active && (j % TPB) == 0)
        st_chk(blk + (size_t)a.P * D + (size_t)a.P * D / 16 + (size_t)off * D / 16 + (j * VEC) / 16, static_cast<uint8_t>(sb),
               a.pool_span, a.pool);
    }
    sr[r] = active ? s : -1;
    if constexpr (!kInWarp) {
      const int li = g + TOK * r;
      codes[li * TPR + j] = wr[r];
      if (j == 0) vslot[li] = sr[r];
    }
  }
  if constexpr (!kInWarp) __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int s = sr[r];
    int next, prev;
    uint32_t other;
    if constexpr (kInWarp) {  // lanes 0-15: row group g (even), lanes 16-31: g + 1
      const bool lower = (threadIdx.x & 16) == 0;
      const int up = __shfl_down_sync(0xffffffffu, s, 16), down = __shfl_up_sync(0xffffffffu, s, 16);
      other = __shfl_down_sync(0xffffffffu, wr[r], 16);
      next = lower ? up : -1;
      prev = lower ? -1 : down;
    } else {
      const int li = g + TOK * r;
      next = li + 1 < NTOK ? vslot[li + 1] : -1;
      prev = li > 0 ? vslot[li - 1] : -1;
      other = li + 1 < NTOK ? codes[(li + 1) * TPR + j] : 0u;
    }
    if (s < 0 || ((s & 1) && prev == s - 1)) continue;  // nothing, or written with the pair's first token
    const int page = s >> a.log2P, off = s & (a.P - 1);
    uint8_t* dst = a.pool + kHeaderBytes + ((size_t)page * a.Hkv + h) * a.block_bytes + (size_t)a.P * D / 2 +
                   (size_t)(off >> 1) * D + j * VEC;
    if constexpr (MODE == KVQ_INT4_PER_TOKEN_HEAD) {
      // INT4 pair-row word: 4 channels of the even token in the low half-word,
      // the same channels of the odd token in the high half-word
      if (!(s & 1) && next == s + 1) {
        const uint2 both = make_uint2(prmt(wr[r], other, 0x5410u), prmt(wr[r], other, 0x7632u));
        if constexpr (VEC == 8) st_chk(reinterpret_cast<uint2*>(dst), both, a.pool_span, a.pool);
        else st_chk(reinterpret_cast<uint32_t*>(dst), both.x, a.pool_span, a.pool);
      } else {
        const int sh = 16 * (off & 1);
        const uint32_t m = 0xFFFFu << sh;
        unsigned int* wd = reinterpret_cast<unsigned int*>(dst);
        if (!in_span(wd, VEC == 8 ? 8 : 4, a.pool_span, a.pool)) continue;
        atomicAnd(wd, ~m);
        atomicOr(wd, (wr[r] & 0xFFFFu) << sh);
        if constexpr (VEC == 8) {
          atomicAnd(wd + 1, ~m);
          atomicOr(wd + 1, (wr[r] >> 16) << sh);
        }
      }
      continue;
    }
    if (!(s & 1) && next == s + 1) {
      // even channels: my low nibbles | the successor's low nibbles << 4; odd
      // channels: my high nibbles >> 4 | the successor's high nibbles; then
      // interleave the bytes back into channel order
      const uint32_t ev = bitsel(wr[r], other << 4, 0x0F0F0F0Fu);
      const uint32_t od = bitsel(wr[r] >> 4, other, 0x0F0F0F0Fu);
      const uint2 both = make_uint2(prmt(ev, od, 0x5140u), prmt(ev, od, 0x7362u));
      if constexpr (VEC == 8) st_chk(reinterpret_cast<uint2*>(dst), both, a.pool_span, a.pool);
      else st_chk(reinterpret_cast<uint32_t*>(dst), both.x, a.pool_span, a.pool);
    } else {
      const uint2 mine = spread_codes(wr[r]);
      const int sh = 4 * (off & 1);
      const uint32_t m = 0x0F0F0F0Fu << sh;
      unsigned int* wd = reinterpret_cast<unsigned int*>(dst);
      if (!in_span(wd, VEC == 8 ? 8 : 4, a.pool_span, a.pool)) continue;
      atomicAnd(wd, ~m);
      atomicOr(wd, mine.x << sh);
      if constexpr (VEC == 8) {
        atomicAnd(wd + 1, ~m);
        atomicOr(wd + 1, mine.y << sh);
      }
    }
  }
}

}  // namespace
}  // namespace kvq
