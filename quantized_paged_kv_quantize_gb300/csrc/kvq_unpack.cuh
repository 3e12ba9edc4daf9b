// kvq_unpack.cuh -- eight channels of a stored row (16-token-page modes) from a
// page block in global memory: the payload words with the scale beside them,
// and the codes as exact fp16 (E2M1 codes times their E4M3 block scale).
#pragma once

#include <cuda_fp16.h>

#include "kvq_device.cuh"

namespace kvq {

template <int MODE>
constexpr bool kPerTokenScale =
    MODE == KVQ_INT8_PER_TOKEN_HEAD || MODE == KVQ_FP8_PER_TOKEN_HEAD || MODE == KVQ_INT4_PER_TOKEN_HEAD;

// The payload words of channels 8j .. 8j + 7 of a row and its scale (the
// per-token fp32 scale's bits, or the E4M3 block scale's byte).
struct Packed8 {
  uint2 code;
  uint32_t scale;
};

template <int MODE, int D, int SIDE>
__device__ __forceinline__ Packed8 load_packed8(const uint8_t* blk, int off, int j) {
  constexpr int P = 16;
  Packed8 p{make_uint2(0u, 0u), 0u};
  if constexpr (MODE == KVQ_FP8_PER_TENSOR || MODE == KVQ_INT8_PER_TOKEN_HEAD || MODE == KVQ_FP8_PER_TOKEN_HEAD) {
    p.code = __ldg(reinterpret_cast<const uint2*>(blk + SIDE * P * D + off * D + 8 * j));
    if constexpr (MODE != KVQ_FP8_PER_TENSOR)
      p.scale = __ldg(reinterpret_cast<const uint32_t*>(blk + 2 * P * D + SIDE * 4 * P + 4 * off));
  } else {
    if constexpr (SIDE == 0)
      p.code.x = __ldg(reinterpret_cast<const uint32_t*>(blk + off * (D / 2) + 4 * j));
    else
      p.code = __ldg(reinterpret_cast<const uint2*>(blk + P * D / 2 + (off >> 1) * D + 8 * j));
    if constexpr (MODE == KVQ_INT4_PER_TOKEN_HEAD)
      p.scale = __ldg(reinterpret_cast<const uint32_t*>(blk + P * D + SIDE * 4 * P + 4 * off));
    else
      p.scale = __ldg(blk + P * D + SIDE * (P * D / 16) + off * (D / 16) + j / 2);
  }
  return p;
}

// Signed 4-bit codes in nibbles 0 and 4 of w -> f16x2: the lop3 flips each
// code's top bit (code + 8) under the f16 exponent of 1024; subtracting 1032
// leaves the code.
__device__ __forceinline__ uint32_t s4_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(0x000F000Fu), "r"(0x64086408u));
  return h2_as_u32(__hsub2(u32_as_h2(r), u32_as_h2(0x64086408u)));
}

// The codes of those channels as f16x2 pairs in channel order.
template <int MODE, int SIDE>
__device__ __forceinline__ void codes8(const Packed8& p, int off, uint32_t* h) {
  if constexpr (MODE == KVQ_INT8_PER_TOKEN_HEAD) {  // 1024 + (x + 128) - 1152
    const __half2 bias = u32_as_h2(0x64806480u);
    const uint32_t a = p.code.x ^ 0x80808080u, b = p.code.y ^ 0x80808080u;
    h[0] = h2_as_u32(__hsub2(u32_as_h2(prmt(a, 0x64646464u, 0x4140u)), bias));
    h[1] = h2_as_u32(__hsub2(u32_as_h2(prmt(a, 0x64646464u, 0x4342u)), bias));
    h[2] = h2_as_u32(__hsub2(u32_as_h2(prmt(b, 0x64646464u, 0x4140u)), bias));
    h[3] = h2_as_u32(__hsub2(u32_as_h2(prmt(b, 0x64646464u, 0x4342u)), bias));
  } else if constexpr (MODE == KVQ_FP8_PER_TENSOR || MODE == KVQ_FP8_PER_TOKEN_HEAD) {
    h[0] = e4m3x2_to_f16x2(p.code.x & 0xFFFFu);
    h[1] = e4m3x2_to_f16x2(p.code.x >> 16);
    h[2] = e4m3x2_to_f16x2(p.code.y & 0xFFFFu);
    h[3] = e4m3x2_to_f16x2(p.code.y >> 16);
  } else if constexpr (MODE == KVQ_INT4_PER_TOKEN_HEAD) {
    if constexpr (SIDE == 0) {  // key word: channels 2k in nibble k, 2k + 1 in nibble k + 4
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = s4_pair(p.code.x >> (4 * k));
    } else {  // value words of four channels, the odd token's in the high half-word
      const uint32_t a = p.code.x >> (16 * (off & 1)), b = p.code.y >> (16 * (off & 1));
      // nibbles k, k + 1 of the half-word -> nibbles 0 and 4
      const uint32_t a2 = (a & 0xFFu) | ((a & 0xFF00u) << 8), b2 = (b & 0xFFu) | ((b & 0xFF00u) << 8);
      const uint32_t a01 = (a2 & 0xFu) | ((a2 & 0xF0u) << 12), a23 = ((a2 >> 16) & 0xFu) | ((a2 & 0xF00000u) >> 4);
      const uint32_t b01 = (b2 & 0xFu) | ((b2 & 0xF0u) << 12), b23 = ((b2 >> 16) & 0xFu) | ((b2 & 0xF00000u) >> 4);
      h[0] = s4_pair(a01);
      h[1] = s4_pair(a23);
      h[2] = s4_pair(b01);
      h[3] = s4_pair(b23);
    }
  } else {
    uint32_t w = p.code.x;
    if constexpr (SIDE == 1) {  // this token's nibble of eight pair bytes -> four bytes of channel pairs
      const int sh = 4 * (off & 1);
      const uint32_t a = (p.code.x >> sh) & 0x0F0F0F0Fu, b = (p.code.y >> sh) & 0x0F0F0F0Fu;
      w = prmt(a, b, 0x6420u) | (prmt(a, b, 0x7531u) << 4);
    }
    e2m1x8_to_f16x2x4(w, h);
    const __half2 s = __half2half2(__low2half(u32_as_h2(e4m3x2_to_f16x2(p.scale))));
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = h2_as_u32(__hmul2(u32_as_h2(h[i]), s));
  }
}

}  // namespace kvq
