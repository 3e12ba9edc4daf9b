// kvq_chunk_umma.cu -- chunk attention on the 5th-generation tensor cores
// (tcgen05, scores, weights and accumulators in tensor memory) for fp16 queries
// and outputs at head_dim 128, all 16-token-page modes.
//
// Mathematics (kvq_chunk.cu has the operator's definition).  With codes K, V
// (exact in fp16) and scales apart, one 128 x 128 block of (row, token) pairs is
//   S = Q K^T,  y = S ks_t (log2 units),  P = 2^(y - R) vs_t,  O += P V,  l += 2^(y - R)
// in fp32 but for P, which enters its product as an fp16 pair, P rounded and the
// remainder rounded: 2^-22 of a weight.  (One fp16 weight instead is an error of the
// size of the output's own rounding: 2.9e-4 in the 2-norm where an exact result
// rounded to fp16 is 2.1e-4 off.)  R is a row's reference, a whole number: the largest
// y + floor(log2 vs) of the tokens met that the row sees, less kTop, moved (O and l
// rescaled, exactly) only when one passes it by more than 2^(kTop + kSlack).  So a
// row's largest P lies between 2^(kTop - 1 - kEven) and 2^15 whatever the scores, the
// values and the tokens it does not see, and a P below fp16's range is off by 2^-27 of
// the largest at most.  Tiles are taken from the nearest tokens to the farthest: a bias
// by distance then never moves the reference again.  The products cut their fp32 sums off,
// up to 2^-23 of O at each: over 16384 tokens 3e-5 of a result as a rule, 1.2e-4 where all
// values have one sign, below the fp16 output's own rounding.  (Adding O to a sum in memory
// every 16 tiles leaves 4e-6 and takes 25% more time; not kept.)
//
// Roles (16 warps, one CTA per SM; registers are shared out between the warpgroups):
//  warps 0-3, 4-7  softmax of block 0 and block 1: thread = row, 64 of its 128
//                  scores at a time in registers from the load to the weights
//                  (tensor memory is read once, and P can go over S);
//  warps 8-11      dequantization: a warp takes two pages of a 128-token tile, their
//                  packed words in registers one tile ahead, and writes the
//                  codes as fp16 core matrices (8 tokens x 16 bytes), which
//                  serve as the K-major B operand of Q K^T and, for V, as the
//                  MN-major B operand of P V;
//  warp 12         issues the tcgen05.mma (13-15 only fill its warpgroup).
// Two blocks are in work at a time, so that the tensor cores run one block's
// products during the other's softmax.  A CTA with more than 128 rows has two
// blocks of rows that use the same tile of keys and values; one with fewer takes
// even and odd tiles as two streams, with a reference, sum and accumulator each,
// merged at the end.
// Tensor memory: S_0 S_1 O_0 O_1, 128 columns each; over the 64 columns of each half of
// S, the 32 of its P rounded and the 32 of the remainders.
//
// Bound by the softmax warps' latency and the dequantization beside the tensor cores:
// 2048 queries of 64 heads over 32768 nvfp4 tokens take 2.15 ms (1.0 PFLOP/s of the formula;
// the second product runs twice, and the tensor cores are busy for 63%), three int8
// prompts of 700 to 2048 tokens, where a CTA's start and end are half of its time, 138 us.
// With one fp16 weight they took 1.72 ms and 123 us.  Per-token scales cost their loads and
// products: int8 on the long chunk 3.83 ms.
#include <cuda_fp16.h>

#include <algorithm>

#include "kvq_chunk.cuh"
#include "kvq_unpack.cuh"

namespace kvq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kD = 128;
constexpr int kTok = 128;       // tokens of a tile
constexpr int kThreads = 512;
constexpr int kDequantWarp = 8, kIssueWarp = 12;
// Registers a thread (the launch gives 128): 256 x 176 + 128 x 104 + 128 x 48 <= 512 x 128.
constexpr int kRegsSoftmax = 176, kRegsDequant = 104, kRegsIssue = 48;
constexpr int kPages = 2;       // pages of a tile that one warp dequantizes
constexpr int kOpBytes = kTok * kD * 2;  // one fp16 operand tile
constexpr int kLbo = 128, kSbo = 2048;   // core matrices: along channels, along rows / tokens
constexpr int kStageRow = 256 + 16;           // an output row in shared memory; the pad spreads the banks
constexpr int kStageBytes = 32 * kStageRow;   // of one warp
constexpr int kSlots = 4;       // tiles whose scales are kept
// Log2 of the largest weight times value scale when a reference is set, and how far later
// ones may pass it: both below fp16's 2^16.
constexpr float kTop = 6.0f, kSlack = 8.0f;
constexpr uint32_t kIdescQK = umma_idesc_f16(128, 128), kIdescPV = umma_idesc_f16_bmn(128, 128);

struct Smem {
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * kOpBytes;  // two stages each
  static constexpr int V = K + 2 * kOpBytes;
  static constexpr int KS = V + 2 * kOpBytes;                      // [slot][128] key scales times kfac
  static constexpr int VS = KS + kSlots * kTok * 4;                // [slot][128] value scales
  static constexpr int ES = VS + kSlots * kTok * 4;                // [slot][128] their exponents, as floats
  static constexpr int PAGE = ES + kSlots * kTok * 4;              // [slot][8] the pages' exponents, in short
  static constexpr int START = PAGE + kSlots * 8 * 4;              // [slot] first token of the tile
  static constexpr int BYTES = START + kSlots * 4;
  static constexpr size_t dynamic() { return BYTES + 128; }
};
// A page of a tile, as two 16-bit numbers: its largest exponent of a value scale above, its
// smallest, negated, below (0 and 0 in the modes without such scales).  kMissing: not there.
constexpr int kMissing = (int)0x80008000u;
__device__ __forceinline__ int exponents(int top, int neg_low) { return (top << 16) | (neg_low & 0xFFFF); }
__device__ __forceinline__ int both_max(int a, int b) { return (int)__vmaxs2((unsigned)a, (unsigned)b); }
// Where a tile's exponents lie at most this far apart, a row's reference goes by the
// largest instead of each token's own: that raises it by as many bits of P at most.
// Three int8 prompts: 138 us so, 145 us token by token.
constexpr int kEven = 3;

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, 1u << 20); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// 32 columns of this warp's lanes, a lane's row to a thread; the registers hold
// them after the next tm_wait.
#define KVQ_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define KVQ_P8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tm_ld(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KVQ_R8(r, 0), KVQ_R8(r, 8), KVQ_R8(r, 16), KVQ_R8(r, 24)
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tm_wait(uint32_t* r) {  // the registers pass through, so that no use precedes the wait
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KVQ_P8(r, 0), KVQ_P8(r, 8), KVQ_P8(r, 16)::"memory");
  asm volatile("" : KVQ_P8(r, 24)::"memory");
}
#undef KVQ_R8
#undef KVQ_P8
__device__ __forceinline__ float2 get(const uint32_t* r, int i) {  // registers i, i + 1
  return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
}
__device__ __forceinline__ void put(uint32_t* r, int i, float2 x) {
  r[i] = __float_as_uint(x.x);
  r[i + 1] = __float_as_uint(x.y);
}
// The larger magnitude of three, NaN if one is.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  asm("max.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(b), "f"(c));
  return a;
}
// x = hi + lo, both in fp16
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  const float2 f = __half22float2(h), r = __fadd2_rn(x, make_float2(-f.x, -f.y));
  hi = h2_as_u32(h);
  lo = h2_as_u32(__floats2half2_rn(r.x, r.y));
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }  // warps 0-7

// ---------------------------------------------------------------- dequantization of one page by one warp
// A lane's packed words of a page: K and V.
template <int MODE>
struct Words {
  static constexpr bool FOUR = MODE == KVQ_NVFP4 || MODE == KVQ_INT4_PER_TOKEN_HEAD;
  static constexpr int N = FOUR ? 2 : 4;  // 16-byte loads per side
  uint4 w[N];
  uint32_t s[MODE == KVQ_NVFP4 ? 2 : 1];  // NVFP4: the two block scales of each load, as bytes 0 and 1
};

// 16-byte load r of this lane.  One-byte codes: token (lane & 7) + 8 (r & 1),
// channels 16 c .. with c = (lane >> 3) + 4 (r >> 1).  Four-bit keys: token
// (lane & 7) + 8 r, channels 32 (lane >> 3) ..; four-bit values: token pair
// lane & 7, channels 16 c .. with c = (lane >> 3) + 4 r.
template <int MODE, int SIDE>
__device__ __forceinline__ void load_words(const uint8_t* blk, int lane, Words<MODE>& x) {
  using W = Words<MODE>;
  const int a = lane & 7, b = lane >> 3;
#pragma unroll
  for (int r = 0; r < W::N; ++r) {
    int off;
    if constexpr (!W::FOUR) off = SIDE * 16 * kD + (a + 8 * (r & 1)) * kD + 16 * (b + 4 * (r >> 1));
    else if constexpr (SIDE == 0) off = (a + 8 * r) * (kD / 2) + 16 * b;
    else off = 16 * kD / 2 + a * kD + 16 * (b + 4 * r);
    x.w[r] = __ldg(reinterpret_cast<const uint4*>(blk + off));
    if constexpr (MODE == KVQ_NVFP4) {
      const uint8_t* s = blk + 16 * kD + SIDE * 16 * kD / 16;
      if constexpr (SIDE == 0) x.s[r] = __ldg(reinterpret_cast<const uint16_t*>(s + (a + 8 * r) * 8 + 2 * b));
      else x.s[r] = (uint32_t)__ldg(s + 16 * a + b + 4 * r) | ((uint32_t)__ldg(s + 16 * a + 8 + b + 4 * r) << 8);
    }
  }
}
template <int MODE>
__device__ __forceinline__ void zero_words(Words<MODE>& x) {
#pragma unroll
  for (int r = 0; r < Words<MODE>::N; ++r) {
    x.w[r] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (MODE == KVQ_NVFP4) x.s[r] = 0u;
  }
}
// Values of tokens >= valid of the page must not reach a product: E4M3 codes
// and block scales can be NaN there.
template <int MODE>
__device__ __forceinline__ void drop_tokens(Words<MODE>& x, int lane, int valid) {
  const int a = lane & 7;
#pragma unroll
  for (int r = 0; r < Words<MODE>::N; ++r) {
    if constexpr (!Words<MODE>::FOUR) {
      if (a + 8 * (r & 1) >= valid) x.w[r] = make_uint4(0u, 0u, 0u, 0u);
    } else if constexpr (MODE == KVQ_NVFP4) {
      if (2 * a >= valid) x.s[r] &= 0xFF00u;
      if (2 * a + 1 >= valid) x.s[r] &= 0x00FFu;
    }
  }
}

// One-byte codes: four words -> two 16-byte chunks of fp16.
template <int MODE>
__device__ __forceinline__ void codes16(const uint4& w, uint4* out) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (MODE == KVQ_INT8_PER_TOKEN_HEAD) {
      const __half2 bias = u32_as_h2(0x64806480u);  // 1024 + (x + 128) - 1152
      const uint32_t v = in[i] ^ 0x80808080u;
      h[2 * i] = h2_as_u32(__hsub2(u32_as_h2(prmt(v, 0x64646464u, 0x4140u)), bias));
      h[2 * i + 1] = h2_as_u32(__hsub2(u32_as_h2(prmt(v, 0x64646464u, 0x4342u)), bias));
    } else {
      h[2 * i] = e4m3x2_to_f16x2(in[i] & 0xFFFFu);
      h[2 * i + 1] = e4m3x2_to_f16x2(in[i] >> 16);
    }
  }
  out[0] = make_uint4(h[0], h[1], h[2], h[3]);
  out[1] = make_uint4(h[4], h[5], h[6], h[7]);
}

// Write page `w` (tokens 16 w ..) of a tile into the operand at `op`: channel
// group c of token t at (t % 8) 16 + c kLbo + (t / 8) kSbo.  Eight neighbouring
// lanes always fill one core matrix row set, so the stores have no conflicts.
template <int MODE, int SIDE>
__device__ __forceinline__ void store_page(const Words<MODE>& x, uint8_t* op, int w, int lane) {
  const int a = lane & 7, b = lane >> 3;
  uint8_t* base = op + 2 * w * kSbo;
#pragma unroll
  for (int r = 0; r < Words<MODE>::N; ++r) {
    if constexpr (!Words<MODE>::FOUR) {
      uint4 c[2];
      codes16<MODE>(x.w[r], c);
      uint8_t* p = base + (r & 1) * kSbo + a * 16 + 2 * (b + 4 * (r >> 1)) * kLbo;
      *reinterpret_cast<uint4*>(p) = c[0];
      *reinterpret_cast<uint4*>(p + kLbo) = c[1];
    } else if constexpr (SIDE == 0) {
      const uint32_t in[4] = {x.w[r].x, x.w[r].y, x.w[r].z, x.w[r].w};
      uint8_t* p = base + r * kSbo + a * 16 + 4 * b * kLbo;
      __half2 s2[2];
      if constexpr (MODE == KVQ_NVFP4) {
        const __half2 s = u32_as_h2(e4m3x2_to_f16x2(x.s[r]));
        s2[0] = __low2half2(s);
        s2[1] = __high2half2(s);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h[4];
        if constexpr (MODE == KVQ_NVFP4) {
          e2m1x8_to_f16x2x4(in[i], h);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = h2_as_u32(__hmul2(u32_as_h2(h[e]), s2[i >> 1]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = s4_pair(in[i] >> (4 * e));
        }
        *reinterpret_cast<uint4*>(p + i * kLbo) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    } else {
      const uint32_t in[4] = {x.w[r].x, x.w[r].y, x.w[r].z, x.w[r].w};
      // tokens 2a and 2a + 1; lanes 4..7 of each eight take the odd one first, so
      // that the eight rows stored together differ modulo 8
      const uint32_t first = (a & 4) ? 0x7632u : 0x5410u, second = first ^ 0x2222u;
      uint32_t t0[8], t1[8];  // 16 channels of the first and of the second token
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h[4];  // (even token, odd token) of channels 4 i ..
        if constexpr (MODE == KVQ_NVFP4) {
          e2m1x8_to_f16x2x4(in[i], h);
          const __half2 s = u32_as_h2(e4m3x2_to_f16x2(x.s[r]));
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = h2_as_u32(__hmul2(u32_as_h2(h[e]), s));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = s4_pair(in[i] >> (4 * e));
        }
        t0[2 * i] = prmt(h[0], h[1], first);
        t0[2 * i + 1] = prmt(h[2], h[3], first);
        t1[2 * i] = prmt(h[0], h[1], second);
        t1[2 * i + 1] = prmt(h[2], h[3], second);
      }
      uint8_t* p = base + (a >> 2) * kSbo + 2 * (b + 4 * r) * kLbo + ((2 * a) & 7) * 16;
      uint8_t* p0 = p + ((a & 4) ? 16 : 0);
      uint8_t* p1 = p + ((a & 4) ? 0 : 16);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        *reinterpret_cast<uint4*>(p0 + c * kLbo) = make_uint4(t0[4 * c], t0[4 * c + 1], t0[4 * c + 2], t0[4 * c + 3]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        *reinterpret_cast<uint4*>(p1 + c * kLbo) = make_uint4(t1[4 * c], t1[4 * c + 1], t1[4 * c + 2], t1[4 * c + 3]);
    }
  }
}

// ---------------------------------------------------------------- kernel
struct Bars {
  uint64_t q_full, k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full;
};

template <int MODE, bool OPT>
__global__ void __launch_bounds__(kThreads, 1) chunk_umma_kernel(const __grid_constant__ ChunkArgs a) {
  using L = Smem;
  constexpr bool PT = kPerTokenScale<MODE>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  __shared__ Bars bar;
  __shared__ uint32_t tmem_s;
  __shared__ RowTile tile_s;
  __shared__ int failed_s;
  float* ksm = reinterpret_cast<float*>(sm + L::KS);
  float* vsm = reinterpret_cast<float*>(sm + L::VS);
  float* esm = reinterpret_cast<float*>(sm + L::ES);
  int* start_s = reinterpret_cast<int*>(sm + L::START);
  int* page_s = reinterpret_cast<int*>(sm + L::PAGE);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kvh = blockIdx.x % a.Hkv, tile_index = blockIdx.x / a.Hkv, split = blockIdx.y;
  uint8_t* pool = const_cast<uint8_t*>(a.pool);
  if (warp == 0) {
    const RowTile t = find_tile(a, tile_index, kUmmaRows, tile_index == 0 && kvh == 0 && split == 0);
    if (lane == 0) tile_s = t;
  } else if (warp == 1) {
    if (elect_one()) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar.k_full[i], 4);
        mbar_init(&bar.v_full[i], 4);
        mbar_init(&bar.k_free[i], 1);
        mbar_init(&bar.v_free[i], 1);
        mbar_init(&bar.s_full[i], 2);
        mbar_init(&bar.p_full[i], 4);
      }
      mbar_init(&bar.q_full, 8);
      mbar_init(&bar.o_full, 1);
      failed_s = 0;
      mbar_fence_init();
    }
    __syncwarp();
  } else if (warp == kIssueWarp) {
    tmem_alloc(&tmem_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const RowTile t = tile_s;
  if (t.seq < 0) {  // no such tile
    if (warp == kIssueWarp) tmem_dealloc(tmem_s, 512);
    return;
  }
  const TokenRange tr = token_range(a, t, kTok);
  const int i0 = (int)((long long)tr.tiles * split / a.num_splits);
  const int n = (int)((long long)tr.tiles * (split + 1) / a.num_splits) - i0;  // this CTA's tiles,
  const int last = i0 + n - 1;  // taken from the last (the nearest tokens) to the first
  const bool two = t.count <= 128;      // one block of rows, two streams of tiles
  const int items = two ? n : 2 * n;  // (tile, block) pairs; item k belongs to block k & 1
  const uint32_t tb = tmem_s;
  bool ok = true;

  // score factor in log2 units (of the cap where there is one), output factor
  float kfac = OPT && a.cap > 0.0f ? a.scale / a.cap : a.scale * kLog2e, vfac = 1.0f;
  if constexpr (!PT) {
    kfac *= *reinterpret_cast<const float*>(a.pool + kHdrKScaleOffset);
    if (kfac == 0.0f) kfac = 0x1p-126f;  // (a masked score times it stays -inf)
    vfac = *reinterpret_cast<const float*>(a.pool + kHdrVScaleOffset);
  }

  if (warp >= kDequantWarp && warp < kIssueWarp) {
    // ------------------------------------------------------------ dequantization
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDequant));
    Words<MODE> kw[kPages], vw[kPages];
    float sc[kPages];
    int pid[kPages], ahead[kPages];  // page ids of tile i, and (unchecked) of tile i + 1
    auto page = [&](int i, int u) { return tr.tile(last - i) * 8 + (warp - kDequantWarp) + 4 * u; };
    auto wanted = [&](int i, int u) { return i < n && page(i, u) * 16 < t.n && !tr.unseen(page(i, u)); };
    auto page_id = [&](int i, int u) -> int {
      return wanted(i, u)
                 ? __ldg(a.block_table + (long long)t.seq * a.max_pages + page(i, u)) : -1;
    };
    auto checked = [&](int id, int i, int u) -> int {
      if (wanted(i, u) && (id < 0 || id >= a.num_pages)) {
        if (lane == 0) set_error(pool, KVQ_DEVERR_PAGE_RANGE);
        return -1;
      }
      return id;
    };
    auto block = [&](int id) { return a.pool + kHeaderBytes + ((size_t)id * a.Hkv + kvh) * a.block_bytes; };
    auto load_k = [&]() {
#pragma unroll
      for (int u = 0; u < kPages; ++u) {
        sc[u] = 0.0f;
        if (pid[u] >= 0) {
          load_words<MODE, 0>(block(pid[u]), lane, kw[u]);
          if constexpr (PT)
            sc[u] = __ldg(reinterpret_cast<const float*>(block(pid[u]) + (Words<MODE>::FOUR ? 16 * kD : 32 * kD)) + lane);
        } else {
          zero_words<MODE>(kw[u]);
        }
      }
    };
    auto load_v = [&]() {
#pragma unroll
      for (int u = 0; u < kPages; ++u) {
        if (pid[u] >= 0) load_words<MODE, 1>(block(pid[u]), lane, vw[u]);
        else zero_words<MODE>(vw[u]);
      }
    };
#pragma unroll
    for (int u = 0; u < kPages; ++u) {
      pid[u] = checked(page_id(0, u), 0, u);
      ahead[u] = page_id(1, u);
    }
    load_k();
    load_v();
    for (int i = 0; i < n; ++i) {
      const int st = i & 1, slot = i & (kSlots - 1);
      if (i >= 2) ok = wait(&bar.k_free[st], ((i >> 1) - 1) & 1) && ok;
      if (!ok) break;
      if (warp == kDequantWarp && lane == 0) start_s[slot] = tr.tile(last - i) * kTok;
      // Scales of the pages: keys in lanes 0-15, values in 16-31.  The slot's last
      // readers are done: the wait for v_free of tile i - 3 lies behind.
      int valid[kPages];
#pragma unroll
      for (int u = 0; u < kPages; ++u) {
        const int w = (warp - kDequantWarp) + 4 * u;  // page of the tile
        valid[u] = pid[u] >= 0 ? min(16, t.n - page(i, u) * 16) : 0;
        if constexpr (PT) {
          if ((lane & 15) >= valid[u]) sc[u] = 0.0f;
          const int at = slot * kTok + 16 * w + (lane & 15);
          (lane < 16 ? ksm : vsm)[at] = lane < 16 ? sc[u] * kfac : sc[u];
          const float e = scale_exponent(sc[u]);
          if (lane >= 16) esm[at] = e;
          const bool counts = lane >= 16 && (lane & 15) < valid[u];
          const int top = __reduce_max_sync(kFull, counts ? (int)e : -32768);
          const int neg_low = __reduce_max_sync(kFull, counts ? -(int)e : -32768);
          if (lane == 0) page_s[slot * 8 + w] = exponents(top, neg_low);
        } else {
          if (lane == 0) page_s[slot * 8 + w] = pid[u] < 0 ? kMissing : 0;
        }
        store_page<MODE, 0>(kw[u], sm + L::K + st * kOpBytes, w, lane);
        if (valid[u] < 16) drop_tokens<MODE>(vw[u], lane, valid[u]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.k_full[st]);
#pragma unroll
      for (int u = 0; u < kPages; ++u) {
        pid[u] = checked(ahead[u], i + 1, u);
        ahead[u] = page_id(i + 2, u);
      }
      load_k();  // of tile i + 1
      if (i >= 2) ok = wait(&bar.v_free[st], ((i >> 1) - 1) & 1) && ok;
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < kPages; ++u) store_page<MODE, 1>(vw[u], sm + L::V + st * kOpBytes, (warp - kDequantWarp) + 4 * u, lane);
      load_v();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.v_full[st]);
    }
  } else if (warp >= kIssueWarp) {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == kIssueWarp) {
      const uint64_t dq = umma_sdesc(smem_u32(sm + L::Q), kLbo, kSbo);
      const uint64_t dk = umma_sdesc(smem_u32(sm + L::K), kLbo, kSbo);
      const uint64_t dv = umma_sdesc(smem_u32(sm + L::V), kSbo, kLbo);  // MN-major: tokens along K, channels along N
      constexpr uint64_t kStepK = (2 * kLbo) >> 4, kStepV = (2 * kSbo) >> 4, kOp = kOpBytes >> 4;
      // The blocks take turns: O += P V of one item, then S of the same block's next
      // (after the products that read P from the same columns).  A second issuing
      // warp, one for each block, mixes the blocks' products and was slower
      // (2048 queries over 32768 nvfp4 tokens, one fp16 weight: 2.10 against 1.74 ms).
      ok = wait(&bar.q_full, 0);
      for (int k = -2; k < items && ok; ++k) {
        const int b = k & 1;
        if (k >= 0) {
          const int i = two ? k : k >> 1, st = i & 1;
          ok = wait(&bar.v_full[st], (i >> 1) & 1) && ok;
          ok = wait(&bar.p_full[b], (k >> 1) & 1) && ok;
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t B = dv + st * kOp;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t P = tb + 128 * b + 64 * (e >> 2) + 8 * (e & 3);
              umma_f16_ts(tb + 256 + 128 * b, P, B + e * kStepV, kIdescPV, (k > 1 || e > 0) ? 1u : 0u);
              umma_f16_ts(tb + 256 + 128 * b, P + 32, B + e * kStepV, kIdescPV, 1u);
            }
            if (two || b == 1) tc_commit(&bar.v_free[st]);
            if (k + 1 == items) tc_commit(&bar.o_full);
          }
          __syncwarp();
        }
        if (k + 2 < items) {
          const int i = two ? k + 2 : (k + 2) >> 1, st = i & 1;
          ok = wait(&bar.k_full[st], (i >> 1) & 1) && ok;
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t A = dq + (two ? 0 : b * kOp), B = dk + st * kOp;
#pragma unroll
            for (int e = 0; e < 8; ++e) umma_f16_ss(tb + 128 * b, A + e * kStepK, B + e * kStepK, kIdescQK, e > 0 ? 1u : 0u);
            tc_commit(&bar.s_full[b]);
            mbar_arrive(&bar.s_full[b]);  // passes on the scales that came with the keys
            if (two || b == 1) tc_commit(&bar.k_free[st]);
          }
          __syncwarp();
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int blk = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    // Q: row r's channel group c at (r % 8) 16 + c kLbo + (r / 8) kSbo; zero past the tile's rows
    for (int it = tid; it < (two ? 128 : 256) * 16; it += 256) {
      const int r = it >> 4, c = it & 15;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (r < t.count) {
        const int rr = t.r0 + r;
        const long long row = (long long)(t.q0 + rr / a.G) * a.Hq + kvh * a.G + rr % a.G;
        x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __half*>(a.q) + row * kD) + c);
      }
      *reinterpret_cast<uint4*>(sm + L::Q + (r & 7) * 16 + c * kLbo + (r >> 3) * kSbo) = x;
    }
    fence_proxy_async_smem();  // Q is read by the tensor core
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.q_full);
    const int row = two ? (tid & 127) : tid;
    const bool real = row < t.count;
    const int rr = t.r0 + (real ? row : 0);
    const int pos = t.n - t.m + rr / a.G;
    // the block's own positions decide which tiles need a mask
    TokenRange mine = tr;
    if (!two) {
      mine.p_min = t.n - t.m + (t.r0 + 128 * blk) / a.G;
      mine.p_max = t.n - t.m + (t.r0 + min(t.count - 1, 128 * blk + 127)) / a.G;
    }
    const RowSees sees = row_sees(a, tr, pos, real);
    float slope = 0.0f;
    if constexpr (OPT) slope = a.slopes ? -kLog2e * __ldg(a.slopes + kvh * a.G + rr % a.G) : 0.0f;
    const uint32_t tS = tb + 128 * blk + lanes, tO = tb + 256 + 128 * blk + lanes;
    float R = 0.0f, l = 0.0f;
    bool fresh = true;  // the row has met no score yet: its reference is still to be set
    bool any = false;   // the block has accumulated something

    for (int k = blk; k < items; k += 2) {
      const int i = two ? k : k >> 1, slot = i & (kSlots - 1);
      ok = wait(&bar.s_full[blk], (k >> 1) & 1) && ok;
      if (!__all_sync(kFull, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int t0 = start_s[slot];
      const int4 pg0 = *reinterpret_cast<const int4*>(page_s + slot * 8), pg1 = *reinterpret_cast<const int4*>(page_s + slot * 8 + 4);
      const int pmin = min(min(min(pg0.x, pg0.y), min(pg0.z, pg0.w)), min(min(pg1.x, pg1.y), min(pg1.z, pg1.w)));
      const bool masked = pmin == kMissing || !all_see(a, mine, t0, kTok);
      float ve = 0.0f;     // exponent of the tile's largest value scale
      bool apart = false;  // exponents are looked at token by token
      if constexpr (PT) {
        const int es = both_max(both_max(both_max(pg0.x, pg0.y), both_max(pg0.z, pg0.w)),
                                both_max(both_max(pg1.x, pg1.y), both_max(pg1.z, pg1.w)));
        apart = (es >> 16) + (int)(short)es > kEven;
        ve = apart ? 0.0f : (float)(es >> 16);
      }

      // Half a tile's scores at a time: P of a half goes over columns of S that have
      // been read.
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const float* ks = ksm + slot * kTok + 64 * h;
        const float* vs = vsm + slot * kTok + 64 * h;
        const float* es = esm + slot * kTok + 64 * h;
        uint32_t x[64];
        tm_ld(tS + 64 * h, x);
        tm_ld(tS + 64 * h + 32, x + 32);
        tm_wait(x);
        tm_wait(x + 32);

        // Exponents of the weights: scores in log2 units less the reference.  Where
        // one factor serves the whole tile (RAW) the scores stay as they are until the
        // weights are computed: one fused step then does both, in the shadow of the
        // exponentials.
        constexpr bool RAW = !PT && !OPT;
        const float2 nR = make_float2(-R, -R), add = OPT && a.cap > 0.0f ? make_float2(0.0f, 0.0f) : nR;
#pragma unroll
        for (int e = 0; e < (RAW ? 0 : 64); e += 4) {
          float4 f = make_float4(kfac, kfac, kfac, kfac);
          if constexpr (PT) f = *reinterpret_cast<const float4*>(ks + e);
          put(x, e, __ffma2_rn(get(x, e), make_float2(f.x, f.y), add));
          put(x, e + 2, __ffma2_rn(get(x, e + 2), make_float2(f.z, f.w), add));
        }
        if constexpr (OPT) {
          if (a.cap > 0.0f) {
            // (the factors hold 1 / cap)  16 short chunks take 147 us with the polynomial,
            // 163 us with the other form alone and 104 us without a cap.
            const SoftCap cap{a.cap * kLog2e};
            float t4[4] = {};
#pragma unroll
            for (int e = 0; e < 64; e += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                t4[u] = max3_abs_nan(t4[u], __uint_as_float(x[e + 2 * u]), __uint_as_float(x[e + 2 * u + 1]));
            if (__all_sync(kFull, cap.near(max3_abs_nan(max3_abs_nan(t4[0], t4[1], t4[2]), t4[3], 0.0f)))) {
#pragma unroll
              for (int e = 0; e < 64; e += 2) put(x, e, __ffma2_rn(cap.slope(get(x, e)), get(x, e), nR));
            } else {
#pragma unroll
              for (int e = 0; e < 64; ++e) x[e] = __float_as_uint(cap.any(__uint_as_float(x[e])) - R);
            }
          }
          if (a.slopes) {
            const float d = (float)(pos - t0 - 64 * h);  // distances are whole numbers below 2^24: exact
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e] = __float_as_uint(fmaf(slope, fabsf(d - (float)e), __uint_as_float(x[e])));
          }
        }
        if (masked) {
          const int4 pg = h ? pg1 : pg0;
          const int there[4] = {pg.x, pg.y, pg.z, pg.w};
          // tokens of the half that the row sees: [lo, hi) or below pre
          const int lo = sees.lo - t0 - 64 * h, hi = sees.hi - t0 - 64 * h, pre = sees.prefix - t0 - 64 * h;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const bool gone = there[p] == kMissing;
#pragma unroll
            for (int e = 16 * p; e < 16 * p + 16; ++e)
              if (gone || !((e >= lo && e < hi) || e < pre)) x[e] = 0xff800000u;  // -inf
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (PT && apart) {
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(es + e);
            const float2 y0 = __fadd2_rn(get(x, e), make_float2(f.x, f.y)), y1 = __fadd2_rn(get(x, e + 2), make_float2(f.z, f.w));
            m4[(e >> 1) & 2] = max3(m4[(e >> 1) & 2], y0.x, y0.y);
            m4[((e >> 1) & 2) + 1] = max3(m4[((e >> 1) & 2) + 1], y1.x, y1.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 64; e += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) m4[u] = max3(m4[u], __uint_as_float(x[e + 2 * u]), __uint_as_float(x[e + 2 * u + 1]));
        }
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) + ve;
        if constexpr (RAW) mx = fmaf(mx, kfac, -R);  // kfac > 0; ve = 0

        // The reference moves (and exponents, sum, accumulator and the first half's
        // weights with it, all by a power of two) only when a row meets its first score
        // or one passes it by more than the slack.
        if (__any_sync(kFull, mx > (fresh ? -INFINITY : kTop + kSlack))) {
          const bool first = fresh && mx > -INFINITY;
          const float to = ceilf(mx) - kTop, up = first ? to : fmaxf(to, 0.0f);
          // (a first score: nothing accumulated yet)
          const float al = first ? 1.0f : up < 127.0f ? __int_as_float((127 - (int)up) << 23) : 0.0f;
          fresh = fresh && !first;
          R += up;
          l *= al;
#pragma unroll
          for (int e = 0; e < (RAW ? 0 : 64); e += 2) put(x, e, __fadd2_rn(get(x, e), make_float2(-up, -up)));
          tmem_wait_st();  // (the first half may have just rescaled O, and has stored its P: both are read below)
          if (any) {       // every product issued before this S has completed
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t v[16];
              tmem_ld<16>(tO + 16 * c, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
              tmem_st<16>(tO + 16 * c, v);
            }
          }
          if (h) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t v[16];
              tmem_ld<16>(tS + 16 * c, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 w = __half22float2(u32_as_h2(v[e]));
                v[e] = h2_as_u32(__floats2half2_rn(w.x * al, w.y * al));
              }
              tmem_st<16>(tS + 16 * c, v);
            }
          }
        }

        // weights, their sum, and P as fp16 pairs
        const float2 nR2 = make_float2(-R, -R), kf2 = make_float2(kfac, kfac);
        float2 l2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[16], rest[16];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float2 y0 = get(x, 32 * c + 2 * e), y1 = get(x, 32 * c + 2 * e + 2);
            if constexpr (RAW) {
              y0 = __ffma2_rn(y0, kf2, nR2);
              y1 = __ffma2_rn(y1, kf2, nR2);
            }
            float2 p0 = make_float2(ex2(y0.x), ex2(y0.y)), p1 = make_float2(ex2(y1.x), ex2(y1.y));
            l2[0] = __fadd2_rn(l2[0], p0);
            l2[1] = __fadd2_rn(l2[1], p1);
            if constexpr (PT) {
              const float4 f = *reinterpret_cast<const float4*>(vs + 32 * c + 2 * e);
              if (masked) {  // a weight of zero stays zero whatever the scale of a token that is not seen
                p0.x = y0.x == -INFINITY ? 0.0f : p0.x * f.x;
                p0.y = y0.y == -INFINITY ? 0.0f : p0.y * f.y;
                p1.x = y1.x == -INFINITY ? 0.0f : p1.x * f.z;
                p1.y = y1.y == -INFINITY ? 0.0f : p1.y * f.w;
              } else {
                p0 = __fmul2_rn(p0, make_float2(f.x, f.y));
                p1 = __fmul2_rn(p1, make_float2(f.z, f.w));
              }
            }
            split2(p0, p[e], rest[e]);
            split2(p1, p[e + 1], rest[e + 1]);
          }
          tmem_st<16>(tS + 64 * h + 16 * c, p);
          tmem_st<16>(tS + 64 * h + 32 + 16 * c, rest);
        }
        const float2 ls = __fadd2_rn(l2[0], l2[1]);
        l += ls.x + ls.y;
      }
      any = true;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[blk]);
    }

    // ------------------------------------------------------------ outputs
    if (n > 0) ok = wait(&bar.o_full, 0) && ok;
    tc_fence_after();
    if (!ok) failed_s = 1;
    softmax_sync();
    float f0 = 1.0f, f1 = 0.0f;                          // two streams: factors of their accumulators
    float* other = reinterpret_cast<float*>(sm + L::K);  // the second stream's rows: [128][132], then R and l
    constexpr int kStride = 132;
    if (failed_s) {
      if (tid == 0) set_error(pool, KVQ_DEVERR_TIMEOUT);
    } else {
      if (fresh) R = -1e30f;
      if (two) {
        if (blk == 1) {
          float* o = other + row * kStride;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            if (any) {
              tm_ld(tO + 32 * c, v);
              tm_wait(v);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(o + 32 * c + e) = any ? make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3])
                                                              : make_uint4(0u, 0u, 0u, 0u);
          }
          other[128 * kStride + row] = R;
          other[128 * kStride + 128 + row] = l;
        }
        softmax_sync();
        if (blk == 0) {
          const float R1 = other[128 * kStride + row], l1 = other[128 * kStride + 128 + row];
          const float top = fmaxf(R, R1);
          f0 = exp2f(R - top);
          f1 = exp2f(R1 - top);
          l = l * f0 + l1 * f1;
          R = top;
        }
      }
      if ((!two || blk == 0) && row < ((t.count + 31) & ~31)) {  // whole warps
        // Rows leave through shared memory (Q's place, free now), so that each store
        // of a warp writes two whole rows of 256 bytes: 128 halves, or 64 of a partial
        // result's floats.  Thread by row, 16 bytes each, a store touches 32 half sectors.
        const int rel = (rr / a.G - t.r0 / a.G) * a.Hq + kvh * a.G + rr % a.G;
        const long long q_base = (long long)(t.q0 + t.r0 / a.G) * a.Hq;
        const float g = a.num_splits > 1 ? vfac : vfac / l;
        const int rows = min(32, t.count - (row - lane));
        uint8_t* stage = sm + L::Q + warp * kStageBytes;
        auto flush = [&](auto store) {
          __syncwarp();
#pragma unroll 4
          for (int r = lane >> 4; r < 32; r += 2) {
            const long long qrow = q_base + __shfl_sync(kFull, rel, r);
            if (r < rows) store(qrow, lane & 15, *reinterpret_cast<const uint4*>(stage + r * kStageRow + 16 * (lane & 15)));
          }
          __syncwarp();
        };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          if (any) {
            tm_ld(tO + 32 * c, v);
            tm_wait(v);
          }
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = any ? __uint_as_float(v[e]) * f0 : 0.0f;
          if (two) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 u = *reinterpret_cast<const float4*>(other + row * kStride + 32 * c + e);
              o[e] += u.x * f1;
              o[e + 1] += u.y * f1;
              o[e + 2] += u.z * f1;
              o[e + 3] += u.w * f1;
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = l == 0.0f ? 0.0f : o[e] * g;  // (a NaN score makes its row NaN)
          if (a.num_splits == 1) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(stage + lane * kStageRow + 64 * c + 2 * e) =
                  make_uint4(h2_as_u32(__floats2half2_rn(o[e], o[e + 1])), h2_as_u32(__floats2half2_rn(o[e + 2], o[e + 3])),
                             h2_as_u32(__floats2half2_rn(o[e + 4], o[e + 5])), h2_as_u32(__floats2half2_rn(o[e + 6], o[e + 7])));
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(stage + lane * kStageRow + 128 * (c & 1) + 4 * e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            if (c & 1)
              flush([&](long long qrow, int j, uint4 x) {
                st_chk(reinterpret_cast<uint4*>(a.ws_o + (qrow * a.num_splits + split) * kD + 64 * (c >> 1)) + j, x, a.ws_span, a.pool);
              });
          }
        }
        if (a.num_splits == 1)
          flush([&](long long qrow, int j, uint4 x) {
            st_chk(reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + qrow * kD) + j, x, a.out_span, a.pool);
          });
        const long long pi = (q_base + rel) * a.num_splits + split;
        if (real && a.num_splits > 1)
          st_chk(reinterpret_cast<float2*>(a.ws_ml + 2 * pi), make_float2(l == 0.0f ? -INFINITY : R, l), a.ws_span, a.pool);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) tmem_dealloc(tb, 512);
}

template <int MODE, bool OPT>
cudaError_t launch(const ChunkArgs& a, cudaStream_t s) {
  auto kern = chunk_umma_kernel<MODE, OPT>;
  constexpr size_t smem = Smem::dynamic();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long tiles = chunk_tile_bound(a.total_q, a.B, a.G, kUmmaRows);
  kern<<<dim3((unsigned)(tiles * a.Hkv), a.num_splits), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <bool OPT>
cudaError_t launch_mode(int mode, const ChunkArgs& a, cudaStream_t s) {
  switch (mode) {
    case KVQ_FP8_PER_TENSOR: return launch<KVQ_FP8_PER_TENSOR, OPT>(a, s);
    case KVQ_INT8_PER_TOKEN_HEAD: return launch<KVQ_INT8_PER_TOKEN_HEAD, OPT>(a, s);
    case KVQ_FP8_PER_TOKEN_HEAD: return launch<KVQ_FP8_PER_TOKEN_HEAD, OPT>(a, s);
    case KVQ_NVFP4:
    case KVQ_NVFP4_4OVER6: return launch<KVQ_NVFP4, OPT>(a, s);
    case KVQ_INT4_PER_TOKEN_HEAD: return launch<KVQ_INT4_PER_TOKEN_HEAD, OPT>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_chunk_umma(const kvq_cache* c, const ChunkArgs& a, cudaStream_t s) {
  return a.cap > 0.0f || a.slopes ? launch_mode<true>(c->cfg.mode, a, s) : launch_mode<false>(c->cfg.mode, a, s);
}

}  // namespace kvq
