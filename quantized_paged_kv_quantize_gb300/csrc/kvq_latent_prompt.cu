// kvq_latent_prompt.cu -- expanded latent attention on the 5th-generation tensor cores
// (tcgen05): fp16 queries, keys, values and outputs.
//
// Mathematics.  For one head, 128 x 128 blocks of (row, token) pairs:
//   S = Q K^T (192 channels: 128 of the head's key, 64 of the shared rotary part),
//   y = S scale log2(e),  P = 2^(y - M),  O += P V,  l += 2^(y - M)
// in fp32 but for P, one fp16 number to a weight: 2^-11 of it at most, an error of the size
// of the output's own rounding.  M is a row's reference, a whole number: its largest y met
// so far less kTop, moved (O and l with it, exactly) only when a score passes it by more
// than 2^(kTop + kSlack).
//
// Roles (24 warps, one CTA per SM; registers are shared out between the warpgroups):
//  warps 0-7, 8-15  softmax of two blocks of 128 rows; the tensor cores run one block's
//                   products during the other's softmax.  Two threads share a row, 64 tokens
//                   of a tile each, all of them in registers at once (in two halves, with
//                   two exchanges between the threads: 2000 instead of 1400 cycles a tile);
//  warps 16-19      copy queries, keys, rotary parts and values into shared memory, 16 bytes a
//                   copy, rows past the sequence's end as zeros;
//  warps 20, 21     issue the products of a block each (22-23 only fill their warpgroup).  They
//                   take turns: the tensor core takes no product ahead of the one it works on,
//                   so one's waits and fences pass during the other's products (one warp for
//                   both blocks: 1.03 instead of 0.89 ms for the first case below; without
//                   turns the blocks fall into step, 0.99 ms).
// Both blocks use the same keys and values.  These go through a ring of eight units of 16 KB
// (128 tokens x 64 channels in the 128-byte swizzle): a tile is three units of keys and two
// of values, so that the copies run 0.6 tiles ahead beside the 96 KB of queries.  A tile's
// values are one operand of 128 columns (issuing a product takes 75 cycles, twice what one
// of 64 columns is worth).
// Tensor memory: S_0 S_1 O_0 O_1, 128 columns each; P of 64 tokens goes over the first 32 of
// their scores' 64 columns.
//
// Bound by a block's turn: its products (20 of 75 cycles and the wait for the weights) and the
// softmax between them.  Measured: 2048 queries of 128 heads over 8192 keys, causal, 0.83 ms
// (1450 TFLOP/s; 0.88 between other kernels); 4096 queries and keys of 32 heads 0.16 ms (1040); three prompts of 1024, 32
// heads, 78 us (a CTA's start and end beside 8 tiles).
#include <cuda_fp16.h>

#include <algorithm>

#include "kvq_latent.cuh"

namespace kvq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kTok = 128, kRows = 256;
constexpr int kThreads = 768;
constexpr int kCopyWarp = 16, kIssueWarp = 20;
// Registers a thread (the launch gives 80): 512 x 96 + 128 x 40 + 128 x 56 <= 768 x 80.
constexpr int kRegsSoftmax = 96, kRegsCopy = 40, kRegsIssue = 56;
static_assert(512 * kRegsSoftmax + 128 * (kRegsCopy + kRegsIssue) <= kThreads * 80, "registers");
constexpr int kUnit = 128 * 128;       // 128 rows of 64 channels
constexpr int kUnits = 8, kKeyUnits = 3, kTileUnits = 5;
constexpr int kStageRow = 256 + 16;    // an output row in shared memory; the pad spreads the banks
// CTAs run by groups of heads, a group's row tiles longest first: the row tiles of a head read
// its keys and values together, of heads whose keys and values are 32 MB at most (a fraction of
// the L2 cache).  Heads side by side, whatever their lengths: 0.89 instead of 0.83 ms for 2048
// queries of 128 heads over 8192 keys (4 TB/s of rereads); a head after the other: 0.20 instead
// of 0.17 ms for 32 heads of 4096 queries and keys (a long tile begins late).
constexpr long long kGroupBytes = 32ll << 20;
constexpr float kTop = 6.0f, kSlack = 8.0f;
constexpr uint32_t kIdescQK = umma_idesc_f16(128, 128), kIdescPV = umma_idesc_f16_bmn(128, 128);
constexpr uint64_t kSwizzle128 = 2ull << 61;  // of a shared-memory matrix descriptor

struct Smem {
  static constexpr int Q = 0;  // [block][3] units
  static constexpr int RING = Q + 2 * kKeyUnits * kUnit;
  static constexpr int BYTES = RING + kUnits * kUnit;
  static constexpr size_t dynamic() { return BYTES + 1024; }
};
struct Bars {
  uint64_t q_full, k_full[2], v_full[2], k_free[2], v_free[2], s_full[2], p_full[2], o_full[2];  // (k, v: by tile % 2)
};

__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, 1u << 20); }
// For the issuing warp: a wait whose result, and a number, that the compiler knows to be the
// same in all lanes, so that a product's operands are in uniform registers.
__device__ __forceinline__ bool wait_uniform(uint64_t* bar, uint32_t parity) { return __all_sync(kFull, wait(bar, parity)); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(kFull, x, 0); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Whether the phase is over, without a wait.
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return r != 0;
}
// 16 bytes global -> shared; zeros where !there (the source is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// One arrival of this thread once its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void load32(uint32_t t, uint32_t* x) {  // 32 columns of this thread's lane
  tmem_ld<32>(t, x);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 32; ++e) asm volatile("" : "+r"(x[e]));  // (no use before the wait)
}
__device__ __forceinline__ float2 get(const uint32_t* r, int i) {  // registers i, i + 1
  return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  asm("max.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(b), "f"(c));
  return a;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }  // warps 0-15
// The issuing warps' turns: block b's warp waits for the other's products to be issued, and lets it go on.
__device__ __forceinline__ void turn_wait(int b) { asm volatile("bar.sync %0, 64;" ::"r"(10 + b) : "memory"); }
__device__ __forceinline__ void turn_over(int b) { asm volatile("bar.arrive %0, 64;" ::"r"(11 - b) : "memory"); }
// The two warps that share rows (one of eight pairs): whether x holds in either.
__device__ __forceinline__ bool pair_any(int pair, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(2 + pair)
      : "memory");
  return r != 0;
}

__global__ void __launch_bounds__(kThreads, 1) latent_prompt_kernel(const __grid_constant__ LatentArgs a) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bar;
  __shared__ uint32_t tmem_s;
  __shared__ RowTile tile_s;
  __shared__ int failed_s;
  __shared__ float red_s[kRows];  // what a row's two threads exchange
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = a.group * (gridDim.x / a.Hq);
  const int head0 = blockIdx.x / group * a.group, heads = min(a.group, a.Hq - head0);
  const int head = head0 + blockIdx.x % group % heads, index = blockIdx.x % group / heads;
  if (warp == 0) {
    const RowTile t = latent_tile<true>(a, index, kRows, index == 0 && head == 0);
    if (lane == 0) tile_s = t;
  } else if (warp == 1) {
    if (elect_one()) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar.k_full[i], 128);
        mbar_init(&bar.v_full[i], 128);
        mbar_init(&bar.k_free[i], 2);
        mbar_init(&bar.v_free[i], 2);
        mbar_init(&bar.s_full[i], 1);
        mbar_init(&bar.p_full[i], 8);
        mbar_init(&bar.o_full[i], 1);
      }
      mbar_init(&bar.q_full, 128);
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
  const uint32_t tb = tmem_s;
  bool ok = true;
  // tiles of tokens that block b's rows see: the second block's at least the first's
  auto tiles = [&](int b) {
    return t.count <= 128 * b ? 0 : (latent_sees(a, t, t.r0 + min(t.count, 128 * b + 128) - 1) + kTok - 1) / kTok;
  };
  const int n0 = tiles(0), n1 = tiles(1), n = max(n0, n1), last = t.count > 128 ? 1 : 0;
  const int most = latent_sees(a, t, t.r0 + t.count - 1);

  if (warp >= kCopyWarp && warp < kIssueWarp) {
    // ------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCopy));
    // thread: chunk (tid % 8) of rows (tid / 8) + 16 e; row r's chunk c lies at r 128 + (c ^ (r % 8)) 16
    const int r0 = (tid & 127) >> 3, c = tid & 7;
    const uint32_t base = smem_u32(sm) + r0 * 128 + ((c ^ (r0 & 7)) << 4);
    const __half* q = static_cast<const __half*>(a.q) + ((long long)(t.q0 + t.r0) * a.Hq + head) * (kLatentHead + kLatentRope) + 8 * c;
#pragma unroll 1
    for (int u = 0; u < (n > 0 ? kKeyUnits * (last + 1) : 0); ++u) {  // (rows that see nothing: no one waits for these)
      const int b = u / kKeyUnits, part = u % kKeyUnits;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = 128 * b + r0 + 16 * e;
        const bool there = r < t.count;
        copy16(base + Smem::Q + u * kUnit + e * 2048, q + (there ? (long long)r * a.Hq * (kLatentHead + kLatentRope) : 0) + 64 * part, there);
      }
    }
    copy_arrive(&bar.q_full);
    const long long k0 = __ldg(a.cu_k + t.seq);
    const __half* k = static_cast<const __half*>(a.k) + k0 * a.k_stride + head * a.k_head_stride + 8 * c;
    const __half* v = static_cast<const __half*>(a.v) + k0 * a.v_stride + head * a.v_head_stride + 8 * c;
    const __half* kr = static_cast<const __half*>(a.k_rope) + k0 * a.k_rope_stride + 8 * c;
    // Tile i's keys take the places of the last key unit and the values of tile i - 2, its values
    // those of the first key units of tile i - 1.
    int slot = 0;
    for (int i = 0; i < n && ok; ++i) {
#pragma unroll 1
      for (int u = 0; u < kTileUnits; ++u) {
        const bool wraps = slot == (u == kKeyUnits ? kUnits - 1 : 0);  // (of a tile's values: in the ring's last unit and its first)
        const __half* src = u < 2 ? k + 64 * u : u == 2 ? kr : v + 64 * ((u - kKeyUnits) ^ (wraps ? 1 : 0));
        const long long stride = u < 2 ? a.k_stride : u == 2 ? a.k_rope_stride : a.v_stride;
        if (u == 1 && i >= 2 && ok) ok = wait(&bar.v_free[i & 1], ((i - 2) >> 1) & 1);
        if (u == kKeyUnits && i >= 1 && ok) ok = wait(&bar.k_free[(i - 1) & 1], ((i - 1) >> 1) & 1);
        if (!__all_sync(kFull, ok)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int tok = i * kTok + r0 + 16 * e;
          const bool there = tok < most;
          copy16(base + Smem::RING + slot * kUnit + e * 2048, src + (there ? tok : 0) * stride, there);
        }
        if (u == kKeyUnits - 1) copy_arrive(&bar.k_full[i & 1]);
        if (u == kTileUnits - 1) copy_arrive(&bar.v_full[i & 1]);
        slot = (slot + 1) & (kUnits - 1);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= kIssueWarp) {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    const int b = warp - kIssueWarp, nb = b == 0 ? n0 : b == 1 ? n1 : 0;
    if (nb > 0) {
      const int other = b ? n0 : n1;  // tiles from here on are this block's alone
      const uint64_t Q = umma_sdesc(smem_u32(sm + Smem::Q + b * kKeyUnits * kUnit), 16, 1024) | kSwizzle128;
      const uint64_t dk = umma_sdesc(smem_u32(sm + Smem::RING), 16, 1024) | kSwizzle128;  // keys: K-major
      // values: MN-major, 64 channels a unit; in the ring's last unit and its first: those of the first come first
      const uint64_t dv = umma_sdesc(smem_u32(sm + Smem::RING), kUnit, 1024) | kSwizzle128;
      const uint64_t dw = umma_sdesc(smem_u32(sm + Smem::RING), (kUnits - 1) * kUnit, 1024) | kSwizzle128;
      const uint32_t S = uniform(tb + 128 * b), O = uniform(tb + 256 + 128 * b);
      ok = wait_uniform(&bar.q_full, 0);
      fence_proxy_async_smem();
      // A step: O += P V of the last tile, then S of the next (over that P).  The two warps take
      // turns, so that one's waits and fences pass during the other's products.  The
      // fences between the copies and the tensor core's reads stand after the waits.  (A warp
      // whose wait ran out still takes its turns: the other one waits for them.)
      const int turns = min(n0, n1) > 0 ? min(n0, n1) + 1 : 0;
      for (int i = 0; i <= nb; ++i) {
        const int j = i - 1, vu = kTileUnits * j + kKeyUnits, ku = kTileUnits * i;
        const int s0 = vu & (kUnits - 1), s1 = (vu + 1) & (kUnits - 1);
        const uint64_t V = s1 ? dv + uniform(s0 * (kUnit >> 4)) : dw;
        const uint32_t after = uniform(j);
        if (i > 0 && ok) ok = wait_uniform(&bar.v_full[j & 1], (j >> 1) & 1) && wait_uniform(&bar.p_full[b], j & 1);
        const bool there = i < nb && ok && __all_sync(kFull, mbar_done(&bar.k_full[i & 1], (i >> 1) & 1));
        fence_proxy_async_smem();
        tc_fence_after();
        if (i < turns && i + b > 0) turn_wait(b);
        if (i > 0) {
          if (ok && elect_one()) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              umma_f16_ts(O, S + 64 * (e >> 2) + 8 * (e & 3), V + e * (2048 >> 4), kIdescPV, e > 0 ? 1u : after);
            for (int u = 0; u <= (j >= other); ++u) tc_commit(&bar.v_free[j & 1]);
            if (i == nb) tc_commit(&bar.o_full[b]);
          }
          __syncwarp();
        }
        if (i < nb) {
          if (ok && !there) {
            ok = wait_uniform(&bar.k_full[i & 1], (i >> 1) & 1);
            fence_proxy_async_smem();
          }
          uint64_t K[kKeyUnits];
#pragma unroll
          for (int p = 0; p < kKeyUnits; ++p) K[p] = dk + uniform(((ku + p) & (kUnits - 1)) * (kUnit >> 4));
          if (ok && elect_one()) {
#pragma unroll
            for (int e = 0; e < 4 * kKeyUnits; ++e)
              umma_f16_ss(S, Q + (e >> 2) * (kUnit >> 4) + (e & 3) * (32 >> 4), K[e >> 2] + (e & 3) * (32 >> 4), kIdescQK, e > 0 ? 1u : 0u);
            tc_commit(&bar.s_full[b]);
          }
          __syncwarp();
        }
        if (i + b < turns) turn_over(b);
        if (i < nb) {
          if (ok && elect_one()) {
            for (int u = 0; u <= (i >= other); ++u) tc_commit(&bar.k_free[i & 1]);
          }
          __syncwarp();
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int blk = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3, pair = 4 * blk + quad, nb = blk ? n1 : n0;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int row = 128 * blk + 32 * quad + lane;
    const bool real = row < t.count;
    const int sees = real ? latent_sees(a, t, t.r0 + row) : 0;
    const int fewest = latent_sees(a, t, t.r0 + min(128 * blk, t.count - 1));  // of the block's rows
    const float kfac = a.scale * kLog2e;
    const uint32_t tS = tb + 128 * blk + 64 * half + lanes, tO = tb + 256 + 128 * blk + 64 * half + lanes;
    float R = 0.0f, l = 0.0f;
    bool fresh = true;  // the row has met no score yet: its reference is still to be set
    for (int i = 0; i < nb; ++i) {
      if (ok) ok = wait(&bar.s_full[blk], i & 1);
      ok = __all_sync(kFull, ok);  // (the pair's barriers are passed all the same)
      tc_fence_after();
      const bool masked = (i + 1) * kTok > fewest;
      uint32_t x[64];
      tmem_ld<32>(tS, x);
      tmem_ld<32>(tS + 32, x + 32);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 64; ++e) asm volatile("" : "+r"(x[e]));  // (no use before the wait)
      if (masked) {
        const int hi = sees - i * kTok - 64 * half;  // tokens of these that the row sees
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= hi) x[e] = 0xff800000u;  // -inf
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 64; e += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) m4[u] = max3(m4[u], __uint_as_float(x[e + 2 * u]), __uint_as_float(x[e + 2 * u + 1]));
      float mx = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), kfac, -R);
      // The reference moves (and l and O with it, by a power of two) only when a row meets its
      // first score or one passes it by more than the slack.
      if (pair_any(pair, mx > (fresh ? -INFINITY : kTop + kSlack))) {
        if (half == 0) red_s[row] = mx;
        pair_any(pair, false);
        if (half == 1) red_s[row] = mx = fmaxf(mx, red_s[row]);
        pair_any(pair, false);
        mx = red_s[row];
        const bool first = fresh && mx > -INFINITY;
        const float to = ceilf(mx) - kTop, up = first ? to : fmaxf(to, 0.0f);
        const float al = first ? 1.0f : up < 127.0f ? __int_as_float((127 - (int)up) << 23) : 0.0f;
        fresh = fresh && !first;
        R += up;
        l *= al;
        if (i > 0) {  // every product issued before this S has completed
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t v[8];
            tmem_ld<8>(tO + 8 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              asm volatile("" : "+r"(v[e]));
              v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
            }
            tmem_st<8>(tO + 8 * c, v);
          }
        }
        pair_any(pair, false);  // (red_s has been read)
      }
      const float2 nR2 = make_float2(-R, -R), kf2 = make_float2(kfac, kfac);
      float2 l2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 y = __ffma2_rn(get(x, 32 * h + 2 * e), kf2, nR2);
          const float2 w = make_float2(ex2(y.x), ex2(y.y));
          l2[e & 1] = __fadd2_rn(l2[e & 1], w);
          p[e] = h2_as_u32(__floats2half2_rn(w.x, w.y));
        }
        tmem_st<16>(tS + 16 * h, p);
      }
      const float2 ls = __fadd2_rn(l2[0], l2[1]);
      l += ls.x + ls.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[blk]);
    }

    // ------------------------------------------------------------ outputs
    if (nb > 0 && ok) ok = wait(&bar.o_full[blk], 0);
    tc_fence_after();
    if (!ok) failed_s = 1;
    if (half == 0) red_s[row] = l;
    softmax_sync();
    if (half == 1) red_s[row] = l = l + red_s[row];
    softmax_sync();  // (the other block's products have read their queries too, whose place the rows take)
    if (failed_s) {
      if (tid == 0) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_TIMEOUT);
    } else if (128 * blk < t.count) {
      l = red_s[row];
      const float g = 1.0f / l;
      uint8_t* stage = sm + Smem::Q + pair * 32 * kStageRow;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        if (nb > 0) load32(tO + 32 * c, v);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t o[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 x = get(v, e + 2 * u);
            o[u] = nb == 0 || l == 0.0f ? 0u : h2_as_u32(__floats2half2_rn(x.x * g, x.y * g));  // (a NaN score makes its row NaN)
          }
          *reinterpret_cast<uint4*>(stage + lane * kStageRow + 128 * half + 64 * c + 2 * e) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      pair_any(pair, false);
      const int first_row = 128 * blk + 32 * quad;
      const long long row0 = (long long)(t.q0 + t.r0 + first_row) * a.Hq + head;
      const int rows = min(32, t.count - first_row);
#pragma unroll 4
      for (int r = 2 * half + (lane >> 4); r < rows; r += 4)
        st_chk(reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + (row0 + (long long)r * a.Hq) * kLatentHead) + (lane & 15),
               *reinterpret_cast<const uint4*>(stage + r * kStageRow + 16 * (lane & 15)), a.out_span, a.pool);
      if (real && half == 0 && a.lse)
        st_chk(a.lse + row0 + (long long)lane * a.Hq, l == 0.0f ? -INFINITY : (R + log2f(l)) * (1.0f / kLog2e), a.lse_span, a.pool);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) tmem_dealloc(tb, 512);
}

}  // namespace

cudaError_t launch_latent_prompt_umma(const kvq_latent*, const LatentArgs& a, cudaStream_t s) {
  constexpr size_t smem = Smem::dynamic();
  cudaError_t e = cudaFuncSetAttribute(latent_prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long grid = chunk_tile_bound(a.total_q, a.B, 1, kRows) * a.Hq;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  LatentArgs args = a;
  args.group = (int)std::min((long long)a.Hq, std::max(1ll, kGroupBytes / (std::max(1ll, (long long)a.max_seq_len) * 2 * kLatentHead * 2)));
  latent_prompt_kernel<<<(unsigned)grid, kThreads, smem, s>>>(args);
  return cudaGetLastError();
}

}  // namespace kvq
