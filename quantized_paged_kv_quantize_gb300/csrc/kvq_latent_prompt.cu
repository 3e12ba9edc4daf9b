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
// Roles (16 warps, one CTA per SM; registers are shared out between the warpgroups):
//  warps 0-3, 4-7  softmax of two blocks of 128 rows, thread = row; the tensor cores run one
//                  block's products during the other's softmax;
//  warps 8-11      copy queries, keys, rotary parts and values into shared memory, 16 bytes a
//                  copy, rows past the sequence's end as zeros;
//  warp 12         issues the products (13-15 only fill its warpgroup).
// Both blocks use the same keys and values.  These go through a ring of eight units of 16 KB
// (128 tokens x 64 channels in the 128-byte swizzle): a tile is three units of keys and two
// of values, so that the copies run 0.6 tiles ahead beside the 96 KB of queries.
// Tensor memory: S_0 S_1 O_0 O_1, 128 columns each; P goes over the first half of its S.
#include <cuda_fp16.h>

#include <algorithm>

#include "kvq_latent.cuh"

namespace kvq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kTok = 128, kRows = 256;
constexpr int kThreads = 512;
constexpr int kCopyWarp = 8, kIssueWarp = 12;
// Registers a thread (the launch gives 128): 256 x 184 + 128 x 80 + 128 x 56 <= 512 x 128.
constexpr int kRegsSoftmax = 184, kRegsCopy = 80, kRegsIssue = 56;
constexpr int kUnit = 128 * 128;       // 128 rows of 64 channels
constexpr int kUnits = 8, kKeyUnits = 3, kTileUnits = 5;
constexpr int kStageRow = 256 + 16;    // an output row in shared memory; the pad spreads the banks
constexpr float kTop = 6.0f, kSlack = 8.0f;
constexpr uint32_t kIdescQK = umma_idesc_f16(128, 128), kIdescPV = umma_idesc_f16_bmn(128, 64);
constexpr uint64_t kSwizzle128 = 2ull << 61;  // of a shared-memory matrix descriptor

struct Smem {
  static constexpr int Q = 0;  // [block][3] units
  static constexpr int RING = Q + 2 * kKeyUnits * kUnit;
  static constexpr int BYTES = RING + kUnits * kUnit;
  static constexpr size_t dynamic() { return BYTES + 1024; }
};
struct Bars {
  uint64_t q_full, full[kUnits], free[kUnits], s_full[2], p_full[2], o_full[2];
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
// 16 bytes global -> shared; zeros where !there (the source is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// One arrival of this thread once its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void load64(uint32_t t, uint32_t* x) {  // 64 columns of this thread's lane
  tmem_ld<32>(t, x);
  tmem_ld<32>(t + 32, x + 32);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 64; ++e) asm volatile("" : "+r"(x[e]));  // (no use before the wait)
}
__device__ __forceinline__ float2 get(const uint32_t* r, int i) {  // registers i, i + 1
  return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  asm("max.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(b), "f"(c));
  return a;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }  // warps 0-7

__global__ void __launch_bounds__(kThreads, 1) latent_prompt_kernel(const __grid_constant__ LatentArgs a) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bar;
  __shared__ uint32_t tmem_s;
  __shared__ RowTile tile_s;
  __shared__ int failed_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, head = blockIdx.x % a.Hq, index = blockIdx.x / a.Hq;
  if (warp == 0) {
    const RowTile t = latent_tile<true>(a, index, kRows, index == 0 && head == 0);
    if (lane == 0) tile_s = t;
  } else if (warp == 1) {
    if (elect_one()) {
      for (int i = 0; i < kUnits; ++i) {
        mbar_init(&bar.full[i], 128);
        mbar_init(&bar.free[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar.s_full[i], 1);
        mbar_init(&bar.p_full[i], 4);
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
    int slot = 0, round = 0;
    for (int i = 0; i < n && ok; ++i) {
#pragma unroll 1
      for (int u = 0; u < kTileUnits; ++u) {
        const __half* src = u < 2 ? k + 64 * u : u == 2 ? kr : v + 64 * (u - kKeyUnits);
        const long long stride = u < 2 ? a.k_stride : u == 2 ? a.k_rope_stride : a.v_stride;
        if (round > 0 && ok) ok = wait(&bar.free[slot], (round - 1) & 1);
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
        copy_arrive(&bar.full[slot]);
        if (++slot == kUnits) {
          slot = 0;
          ++round;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= kIssueWarp) {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == kIssueWarp && n > 0) {
      const uint64_t dq = umma_sdesc(smem_u32(sm + Smem::Q), 16, 1024) | kSwizzle128;
      const uint64_t dr = umma_sdesc(smem_u32(sm + Smem::RING), 16, 1024) | kSwizzle128;  // keys: K-major; values: MN-major, 64 channels
      const uint32_t tm = uniform(tb);
      ok = wait_uniform(&bar.q_full, 0);
      fence_proxy_async_smem();
      // O += P V of a block's last tile, then S of its next (over that P), the blocks in turn.
      // The fences between the copies and the tensor core's reads stand after the waits.
      for (int i = 0; i <= n && ok; ++i) {
#pragma unroll 1
        for (int b = 0; b <= last && ok; ++b) {
          const int nb = b ? n1 : n0;
          const uint32_t s = uniform(tm + 128 * b);
          if (i > 0 && i <= nb) {
            ok = wait_uniform(&bar.p_full[b], (i - 1) & 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int unit = kTileUnits * (i - 1) + kKeyUnits + h, slot = unit & (kUnits - 1);
              if (ok) ok = wait_uniform(&bar.full[slot], (unit / kUnits) & 1);
              if (!ok) break;
              fence_proxy_async_smem();
              tc_fence_after();
              const uint64_t B = dr + uniform(slot * (kUnit >> 4));
              const uint32_t after = uniform(i - 1);
              if (elect_one()) {
#pragma unroll
                for (int e = 0; e < 8; ++e) umma_f16_ts(s + 256 + 64 * h, s + 8 * e, B + e * (2048 >> 4), kIdescPV, e > 0 ? 1u : after);
                if (b == last) tc_commit(&bar.free[slot]);
                if (h == 1 && i == nb) tc_commit(&bar.o_full[b]);
              }
              __syncwarp();
            }
          }
          if (i < nb && ok) {
#pragma unroll
            for (int p = 0; p < kKeyUnits; ++p) {
              const int unit = kTileUnits * i + p, slot = unit & (kUnits - 1);
              if (ok) ok = wait_uniform(&bar.full[slot], (unit / kUnits) & 1);
              if (!ok) break;
              fence_proxy_async_smem();
              tc_fence_after();
              const uint64_t A = dq + uniform((kKeyUnits * b + p) * (kUnit >> 4)), B = dr + uniform(slot * (kUnit >> 4));
              if (elect_one()) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  umma_f16_ss(s, A + e * (32 >> 4), B + e * (32 >> 4), kIdescQK, (p > 0 || e > 0) ? 1u : 0u);
                if (b == last) tc_commit(&bar.free[slot]);
                if (p == kKeyUnits - 1) tc_commit(&bar.s_full[b]);
              }
              __syncwarp();
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int blk = warp >> 2, nb = blk ? n1 : n0;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const bool real = tid < t.count;
    const int sees = real ? latent_sees(a, t, t.r0 + tid) : 0;
    const int fewest = latent_sees(a, t, t.r0 + min(128 * blk, t.count - 1));  // of the block's rows
    const float kfac = a.scale * kLog2e;
    const uint32_t tS = tb + 128 * blk + lanes, tO = tb + 256 + 128 * blk + lanes;
    float R = 0.0f, l = 0.0f;
    bool fresh = true;  // the row has met no score yet: its reference is still to be set
    for (int i = 0; i < nb; ++i) {
      if (ok) ok = wait(&bar.s_full[blk], i & 1);
      if (!__all_sync(kFull, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool masked = (i + 1) * kTok > fewest;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t x[64];
        load64(tS + 64 * h, x);
        if (masked) {
          const int hi = sees - i * kTok - 64 * h;  // tokens of the half that the row sees
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= hi) x[e] = 0xff800000u;  // -inf
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; e += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u) m4[u] = max3(m4[u], __uint_as_float(x[e + 2 * u]), __uint_as_float(x[e + 2 * u + 1]));
        const float mx = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), kfac, -R);
        // The reference moves (and l, O and the first half's weights with it, all by a power of
        // two) only when a row meets its first score or one passes it by more than the slack.
        if (__any_sync(kFull, mx > (fresh ? -INFINITY : kTop + kSlack))) {
          const bool first = fresh && mx > -INFINITY;
          const float to = ceilf(mx) - kTop, up = first ? to : fmaxf(to, 0.0f);
          const float al = first ? 1.0f : up < 127.0f ? __int_as_float((127 - (int)up) << 23) : 0.0f;
          fresh = fresh && !first;
          R += up;
          l *= al;
          tmem_wait_st();  // (the first half may have just rescaled O, and has stored its P: both are read below)
          if (i > 0) {     // every product issued before this S has completed
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t v[16];
              tmem_ld<16>(tO + 16 * c, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                asm volatile("" : "+r"(v[e]));
                v[e] = __float_as_uint(__uint_as_float(v[e]) * al);
              }
              tmem_st<16>(tO + 16 * c, v);
            }
          }
          if (h) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t v[16];
              tmem_ld<16>(tS + 16 * c, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                asm volatile("" : "+r"(v[e]));
                const float2 w = __half22float2(u32_as_h2(v[e]));
                v[e] = h2_as_u32(__floats2half2_rn(w.x * al, w.y * al));
              }
              tmem_st<16>(tS + 16 * c, v);
            }
          }
        }
        const float2 nR2 = make_float2(-R, -R), kf2 = make_float2(kfac, kfac);
        float2 l2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = __ffma2_rn(get(x, 32 * c + 2 * e), kf2, nR2);
            const float2 w = make_float2(ex2(y.x), ex2(y.y));
            l2[e & 1] = __fadd2_rn(l2[e & 1], w);
            p[e] = h2_as_u32(__floats2half2_rn(w.x, w.y));
          }
          tmem_st<16>(tS + 32 * h + 16 * c, p);
        }
        const float2 ls = __fadd2_rn(l2[0], l2[1]);
        l += ls.x + ls.y;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[blk]);
    }

    // ------------------------------------------------------------ outputs
    if (nb > 0 && ok) ok = wait(&bar.o_full[blk], 0);
    tc_fence_after();
    if (!ok) failed_s = 1;
    softmax_sync();  // (the other block's products have read their queries too, whose place the rows take)
    if (failed_s) {
      if (tid == 0) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_TIMEOUT);
    } else if (128 * blk < t.count) {
      const float g = 1.0f / l;
      uint8_t* stage = sm + Smem::Q + warp * 32 * kStageRow;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[64];
        if (nb > 0) load64(tO + 64 * c, v);
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
          uint32_t o[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 x = get(v, e + 2 * u);
            o[u] = nb == 0 || l == 0.0f ? 0u : h2_as_u32(__floats2half2_rn(x.x * g, x.y * g));  // (a NaN score makes its row NaN)
          }
          *reinterpret_cast<uint4*>(stage + lane * kStageRow + 128 * c + 2 * e) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      __syncwarp();
      const long long row0 = (long long)(t.q0 + t.r0 + 32 * warp) * a.Hq + head;
      const int rows = min(32, t.count - 32 * warp);
#pragma unroll 4
      for (int r = lane >> 4; r < rows; r += 2)
        st_chk(reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + (row0 + (long long)r * a.Hq) * kLatentHead) + (lane & 15),
               *reinterpret_cast<const uint4*>(stage + r * kStageRow + 16 * (lane & 15)), a.out_span, a.pool);
      if (real && a.lse)
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
  latent_prompt_kernel<<<(unsigned)grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
