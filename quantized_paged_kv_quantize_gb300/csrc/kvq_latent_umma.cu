// kvq_latent_umma.cu -- absorbed latent attention on the 5th-generation tensor cores
// (tcgen05): fp16 queries and outputs.
//
// Mathematics.  All rows (query x head) of a sequence read the same tokens, so a CTA takes
// N = 16, 32 or 64 of them against tiles of 128 tokens, transposed: with codes C (exact in
// fp16; NVFP4 codes times their block scales) and rotary parts R of the tile's tokens,
//   Sc = C Qc^T,  Sr = R Qr^T            [128 tokens][N rows], fp32
//   y  = (Sc ks_t + Sr) scale log2(e)    (ks_t: the token's scale)
//   P  = 2^(y - M) ks_t,  l += 2^(y - M),  O^T += C^T P   [L channels][N rows], fp32
// The tile of codes in shared memory is the key operand and, read with tokens along K, the
// value operand: it is dequantized once.  P is one fp16 number to a weight: 2^-11 of it at
// most, an error of the size of the output's own rounding (the pair of numbers that
// kvq_chunk_umma.cu takes would need twice the value products).  M is a row's reference, a
// whole number: the largest y + floor(log2 ks) met so far less kTop, moved (O and l with it,
// exactly) only when a token passes it by more than 2^(kTop + kSlack); so P stays between
// fp16's limits whatever the scores and scales, and what falls below their steps of 2^-24 is at
// most 2^-29 of the row's largest.  Sums are fp32 in tensor memory, cut off (not rounded) by the
// products: up to 2^-23 of O at each 16 tokens.
//
// Shared memory bounds the products: an operand pair of 128 x 16 and N x 16 halves takes
// 32 + N / 4 cycles at 128 bytes a cycle (measured 48.3 for N = 64, 39.3 for 16) where the
// multiplications take N / 2, and the dequantized tile is written once through the same
// port.  The rotary part goes through tensor memory instead (32 cycles at N = 64), which
// also leaves room for P.
//
// Roles (28 warps, one CTA per SM):
//  warps 0-15   softmax: thread = token of the tile and a quarter of the rows;
//  warps 16-23  dequantization: 256 channels of the tile are one entry of a ring; with few
//               rows two teams of four warps take the entries in turn.  A warp's loads in
//               flight are those of its next entry alone: a wait for some of a warp's loads
//               would wait for later ones too.  With a tile's first entry a warp stores the
//               rotary parts of 16 tokens (into tensor memory) and their scales;
//  warp 24      issues the products (25-27 only fill its warpgroup).
// The ring's entries are released by the value products, 256 channels at a time, so the
// next tile is dequantized and its scores begin while these run.  The tensor core takes no
// product ahead of the one it works on: what the issuing warp does between two (a wait takes
// 110 cycles, a fence 30, a release 35) is lost, so an entry is sixteen products each way
// (with eight, measured alone: 76 instead of 49 cycles a product).  Warps that poll a barrier
// slow it further (104 cycles): of the softmax warps one polls, the others wait for it.  Where
// the ring holds two tiles (L = 256) the next tile's scores go before the value products.
//
// Measured: a 1K chunk of 128 heads over 8K int8 tokens 3.39 ms (647 TFLOP/s; 71% of the
// cycles are the port's), 32 single tokens of 128 heads over 1K to 16K fp8 tokens 203 us
// (450 TFLOP/s), 64 of 20 heads over as many nvfp4 tokens 133 us (1.7 TB/s), two of 20 heads
// over 100 to 400 tokens 15 us.
#include <cuda_fp16.h>

#include <algorithm>

#include "kvq_latent.cuh"

namespace kvq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kTok = 128;
constexpr int kThreads = 896, kSoftmax = 512;
constexpr int kDequantWarp = 16, kIssueWarp = 24;
constexpr int kEntry = kTok * 256 * 2;     // one ring entry: 128 tokens x 256 channels of fp16
// An entry holds 64 channels after 64, each part as 128-byte rows of tokens
// with the 16-byte chunks of row t at chunk ^ (t % 8): the 128-byte swizzle of both a
// K-major (tokens x channels) and an MN-major (channels x tokens) operand.
constexpr int kPart = kEntry / 4, kGroup = 1024;  // bytes of a part; of 8 tokens in it
constexpr int kLbo = 128;                  // Q, unswizzled core matrices (8 rows x 16 bytes): along channels
constexpr int kScaleTiles = 4;             // tiles whose scales are kept
constexpr float kTop = 6.0f, kSlack = 8.0f;

template <int L, int N>
struct Shape {
  // Teams of dequantizing warps take the entries in turn, so that a whole tile's loads are in
  // flight.  With 64 rows registers do not allow it: there a warp takes every entry, and the
  // codes of a tile's second one wait in tensor memory (E2M1: in registers).
  static constexpr int TEAMS = N == 64 ? 1 : L / 256;
  static constexpr int WARPS = 8 / TEAMS, PAGES = TEAMS;  // of a team; of a warp
  // Registers a thread (the launch gives 72).
  static constexpr int RS = N == 64 ? 72 : 56, RD = N == 64 ? 80 : 112, RI = 56;
  static_assert(512 * RS + 256 * RD + 128 * RI <= 896 * 72, "registers");
  static constexpr int NB = L / 256;                   // ring entries of a tile
  static constexpr int C = N / 4;                      // rows of a softmax thread
  static constexpr int QCH = (L + kLatentRope) / 8;    // 16-byte chunks of a query row
  static constexpr int QSBO = QCH * 128;               // Q: 8 rows of a chunk together, chunks 128 bytes apart
  static constexpr int Q = 0;
  static constexpr int P = Q + N / 8 * QSBO;
  static constexpr int SC = P + kTok * N * 2;          // [tile % 4][128] scales
  static constexpr int M = SC + kScaleTiles * kTok * 4;  // [N] references
  static constexpr int SEES = M + N * 4;               // [N] tokens a row sees
  static constexpr int RED = SEES + N * 4;             // [4][N]
  static constexpr int UP = RED + 4 * N * 4;           // [N] what a reference moves by
  static constexpr int F = UP + N * 4;                 // [N] the factor that goes with it; at the end, the output's
  static constexpr int REST = (F + N * 4 + 1023) / 1024 * 1024;
  static constexpr int FIT = (227 * 1024 - 1024 - 1024 - REST) / kEntry;
  static constexpr int SLOTS = 2;  // (three fit with few rows and gain nothing: 307 instead of 236 us for 152 rows of 16 heads)
  static constexpr int RING = REST;
  static constexpr int BYTES = RING + SLOTS * kEntry;
  static constexpr size_t dynamic() { return BYTES + 1024; }
  // tensor memory: score buffers (latent, rotary), O^T by 128 channels, rotary operands of two tiles
  static constexpr int SB = L / 128 * N + 64 + 4 * N <= 512 ? 2 : 1;
  static constexpr int TO = SB * 2 * N, TR = TO + L / 128 * N, TP = TR + 64;  // TP: parked codes, 64 columns
  // entries of the next tile whose scores go before this tile's value products
  static constexpr int PRE = SB == 2 ? (SLOTS - NB < NB ? SLOTS - NB : NB) : 0;
  static_assert(FIT >= SLOTS && SLOTS >= NB && TR + 64 <= 512, "fits");
  static_assert(kLatentSeqs * 8 <= SLOTS * kEntry, "fits");
};

constexpr uint64_t kSwizzle128 = 2ull << 61;  // of a shared-memory matrix descriptor
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, 1u << 20); }
// For the issuing warp: a wait whose result, and a number, that the compiler knows to be the
// same in all lanes.  Operands of a product in uniform registers cost nothing to issue;
// moved there from others they cost some 80 cycles a product.
__device__ __forceinline__ bool wait_uniform(uint64_t* bar, uint32_t parity) { return __all_sync(kFull, wait(bar, parity)); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(kFull, x, 0); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }  // warps 0-15
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 512, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
// A warp-wide maximum of floats through whole numbers in the same order (NaN: largest or
// smallest, by its sign; its row is NaN by its weights).
__device__ __forceinline__ float warp_max(float x) {
  const int b = __float_as_int(x), r = __reduce_max_sync(kFull, b ^ ((b >> 31) & 0x7fffffff));
  return __int_as_float(r ^ ((r >> 31) & 0x7fffffff));
}

// Bytes that no other warp of the SM reads.  What a load costs the SM's data port goes by
// the lines that eight neighbouring lanes touch: 128 bytes at a time where the eight read
// one line, 16 where they read eight.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}
__device__ __forceinline__ void load32_once(const void* p, uint32_t* r) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
template <int R>
__device__ __forceinline__ void set_registers() {  // (the launch gives 72)
  if constexpr (R > 72) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// A lane's packed words of half a ring entry (a page's 16 tokens x 128 channels): one-byte
// codes in four loads, token (lane >> 3) + 4 r, channels 16 (lane & 7) ..; E2M1 codes in
// two, token (lane >> 2) + 8 r, channels 32 (lane & 3) .., with the two block scales as
// bytes 0 and 1.
template <int MODE>
struct Words {
  static constexpr int N = kLatentFour<MODE> ? 2 : 4;
  uint4 w[N];
  uint32_t s[kLatentFour<MODE> ? N : 1];
};
// Tokens from `valid` on are zero: their codes must not reach a product.
template <int MODE, int L>
__device__ __forceinline__ void load_words(const uint8_t* page, int j, int lane, int valid, Words<MODE>& x) {
  using PG = LatentPage<MODE, L>;
#pragma unroll
  for (int r = 0; r < Words<MODE>::N; ++r) {
    const int tok = kLatentFour<MODE> ? (lane >> 2) + 8 * r : (lane >> 3) + 4 * r;
    x.w[r] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (kLatentFour<MODE>) x.s[r] = 0u;
    if (tok < valid) {
      if constexpr (kLatentFour<MODE>) {
        x.w[r] = load_once(page + tok * PG::CODES + 64 * j + 16 * (lane & 3));
        x.s[r] = __ldg(reinterpret_cast<const uint16_t*>(page + PG::SCALES + tok * (L / 16) + 8 * j + 2 * (lane & 3)));
      } else {
        x.w[r] = load_once(page + tok * PG::CODES + 128 * j + 16 * (lane & 7));
      }
    }
  }
}
// As fp16: eight chunks of 16 bytes, in the order of store_chunks.  The eight lanes of a
// store's phase have one token (E2M1: two) and every second chunk of both halves (one in
// four); the second half's lanes take their chunks in another order, so that the eight differ.
template <int MODE>
__device__ __forceinline__ int second_half(int lane) { return kLatentFour<MODE> ? (lane >> 1) & 1 : (lane >> 2) & 1; }
template <int MODE>
__device__ __forceinline__ void convert(const Words<MODE>& x, int lane, uint4* out) {
  const int half = second_half<MODE>(lane);
#pragma unroll
  for (int r = 0; r < Words<MODE>::N; ++r) {
    const uint32_t in[4] = {x.w[r].x, x.w[r].y, x.w[r].z, x.w[r].w};
    uint32_t h[8];
    if constexpr (kLatentFour<MODE>) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // the second half's lanes begin with their last sixteen codes
        const uint32_t from[2] = {half ? in[2 * (u ^ 1)] : in[2 * u], half ? in[2 * (u ^ 1) + 1] : in[2 * u + 1]};
        latent_codes16<MODE>(from, x.s[r] >> (8 * (half ? u ^ 1 : u)), h);
        out[4 * r + 2 * u] = make_uint4(h[0], h[1], h[2], h[3]);
        out[4 * r + 2 * u + 1] = make_uint4(h[4], h[5], h[6], h[7]);
      }
    } else {  // with their last eight
      const uint32_t from[4] = {half ? in[2] : in[0], half ? in[3] : in[1], half ? in[0] : in[2], half ? in[1] : in[3]};
      latent_codes16<MODE>(from, 0u, h);
      out[2 * r] = make_uint4(h[0], h[1], h[2], h[3]);
      out[2 * r + 1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
  }
}
// Into the ring entry at `op`, page `pg` of the tile.
template <int MODE>
__device__ __forceinline__ void store_chunks(const uint4* x, uint8_t* op, int pg, int lane) {
  constexpr bool FOUR = kLatentFour<MODE>;
  const int half = second_half<MODE>(lane);
  const int chunk = FOUR ? (4 * (lane & 1)) ^ (2 * half) : (2 * (lane & 3)) ^ half;  // the lane's first
  const int row = FOUR ? lane >> 2 : lane >> 3;                                      // its first token
  uint8_t* p = op + half * kPart + 2 * pg * kGroup + row * 128;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (FOUR)  // tokens row + 8 r: the same place in the group
      *reinterpret_cast<uint4*>(p + (i >> 2) * kGroup + ((chunk ^ row ^ (i & 3)) << 4)) = x[i];
    else  // tokens row + 4 r: the row's bit 2 changes with r
      *reinterpret_cast<uint4*>(p + (i >> 2) * kGroup + ((i >> 1) & 1) * 512 + ((chunk ^ row ^ (i & 1) ^ (4 * ((i >> 1) & 1))) << 4)) = x[i];
  }
}
// 16 rows of tensor memory x 32 columns: lane's row lane / 4, r[4 k] and r[4 k + 1] columns
// 8 k + 2 (lane % 4) and the next; r[4 k + 2] and r[4 k + 3] the row eight further on.
__device__ __forceinline__ void tmem_st_16x256b(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

struct Bars {
  uint64_t q_full, full[2], free[2], rope_full[2], rope_free[2], s_full[2], p_full, p_free;
};

template <int MODE, int L, int N>
__global__ void __launch_bounds__(kThreads, 1) latent_umma_kernel(const __grid_constant__ LatentArgs a) {
  using S = Shape<L, N>;
  using PG = LatentPage<MODE, L>;
  constexpr int NB = S::NB, C = S::C;
  constexpr bool PT = kLatentTokenScale<MODE>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bar;
  __shared__ uint32_t tmem_s;
  __shared__ LatentPart part_s;
  __shared__ int failed_s;
  __shared__ uint32_t fresh_s[2];  // rows 0-31, 32-63: no score met yet
  float* sc_s = reinterpret_cast<float*>(sm + S::SC);
  float* m_s = reinterpret_cast<float*>(sm + S::M);
  int* sees_s = reinterpret_cast<int*>(sm + S::SEES);
  float* red_s = reinterpret_cast<float*>(sm + S::RED);
  float* up_s = reinterpret_cast<float*>(sm + S::UP);
  float* f_s = reinterpret_cast<float*>(sm + S::F);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {
    LatentPart p{{-1, 0, 0, 0, 0, 0, 0}, 0, 0, 1, 0};
    if (a.ctas) p = latent_part(a, blockIdx.x, N, blockIdx.x == 0, reinterpret_cast<int2*>(sm + S::RING));
    else p.t = find_tile(a, blockIdx.x, N, blockIdx.x == 0);
    if (lane == 0) {
      part_s = p;
      if (a.ctas && p.t.seq >= 0 && p.part == 0) st_chk(a.map + p.tile, make_int2(p.first, p.parts), a.ws_span, a.pool);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      static_assert(S::SLOTS == 2, "barriers");
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar.full[i], S::WARPS);
        mbar_init(&bar.free[i], 1);
        mbar_init(&bar.rope_full[i], 8);
        mbar_init(&bar.rope_free[i], 1);
        mbar_init(&bar.s_full[i], 2);
      }
      mbar_init(&bar.q_full, 16);
      mbar_init(&bar.p_full, 16);
      mbar_init(&bar.p_free, 1);
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
  const RowTile t = part_s.t;
  const int part = part_s.part, parts = part_s.parts;
  if (t.seq < 0) {  // no such tile
    if (warp == kIssueWarp) tmem_dealloc(tmem_s, 512);
    return;
  }
  const int fewest = latent_sees(a, t, t.r0), most = latent_sees(a, t, t.r0 + t.count - 1);
  const int tiles = (most + kTok - 1) / kTok;
  const int i0 = (int)((long long)tiles * part / parts);
  const int n = (int)((long long)tiles * (part + 1) / parts) - i0;  // this CTA's tiles
  const uint32_t tb = tmem_s;
  bool ok = true;

  if (warp >= kDequantWarp && warp < kIssueWarp) {
    // ------------------------------------------------------------ dequantization
    set_registers<S::RD>();
    const int w = warp - kDequantWarp, team = w / S::WARPS, first = w % S::WARPS;
    // rotary parts and scales: of the page whose tokens' lanes of tensor memory the warp reaches
    const int mine = 2 * (warp & 3) + (w >> 2);
    constexpr bool TWO = S::TEAMS == 1 && NB == 2;                      // entries of a tile held at once,
    constexpr bool PARK = TWO && !kLatentFour<MODE>;                  // the second in tensor memory
    constexpr int HELD = TWO && !PARK ? 2 : 1;
    static_assert(!PARK || S::TP + 64 <= 512, "fits");
    Words<MODE> words[HELD][S::PAGES][2];  // of pages first, first + WARPS, ..
    const uint32_t parked = tb + S::TP + 32 * (w >> 2) + ((uint32_t)(32 * (warp & 3)) << 16);
    uint32_t rope[16];
    float sc;  // of token lane of page `mine` (lanes 0-15); -1 where it is not there
    // the tile's eight page ids, lane by lane; -1 past the last token
    auto page_ids = [&](int i) -> int {
      const int page = (i0 + i) * 8 + (lane & 7);
      return i < n && page * 16 < most ? __ldg(a.block_table + (long long)t.seq * a.max_pages + page) : -1;
    };
    auto page_at = [&](int ids, int i, int pg, int& valid) -> const uint8_t* {
      const int id = __shfl_sync(kFull, ids, pg);
      const bool in = id >= 0 && id < a.num_pages;
      valid = in ? min(16, most - ((i0 + i) * 8 + pg) * 16) : 0;
      return a.pool + kHeaderBytes + (size_t)(in ? id : 0) * a.block_bytes;
    };
    auto load = [&](int ids, int i, int j, int held) {
#pragma unroll
      for (int u = 0; u < S::PAGES; ++u) {
        int valid;
        const uint8_t* page = page_at(ids, i, first + S::WARPS * u, valid);
#pragma unroll
        for (int e = 0; e < 2; ++e) load_words<MODE, L>(page, 2 * j + e, lane, valid, words[held][u][e]);
      }
    };
    // Four lanes have a row: its 32 bytes from 32 (lane % 4) in the columns 8 k + 2 (lane % 4),
    // + 1 of the four steps k; the queries' rotary channels are in the same order.
    auto load_rope = [&](int ids, int i) {
      int valid;
      const uint8_t* page = page_at(ids, i, mine, valid);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t x[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        const int tok = (lane >> 2) + 8 * g;
        if (tok < valid) load32_once(page + PG::ROPE + tok * kLatentRope * 2 + 32 * (lane & 3), x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          rope[4 * k + 2 * g] = x[2 * k];
          rope[4 * k + 2 * g + 1] = x[2 * k + 1];
        }
      }
      sc = -1.0f;
      if (lane < valid) sc = PT ? __ldg(reinterpret_cast<const float*>(page + PG::SCALES) + lane) : 1.0f;
      if (i < n && valid == 0 && ((i0 + i) * 8 + mine) * 16 < most && lane == 0)
        set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_PAGE_RANGE);
    };
    int ahead = page_ids(1);
    auto load_tile = [&](int ids, int i) {  // the first entry, or both
      if constexpr (PARK) {
        load(ids, i, 1, 0);
        uint32_t r[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 x = words[0][0][e >> 2].w[e & 3];
          r[4 * e] = x.x;
          r[4 * e + 1] = x.y;
          r[4 * e + 2] = x.z;
          r[4 * e + 3] = x.w;
        }
        tmem_st<32>(parked, r);
        tmem_wait_st();
      }
      load(ids, i, team, 0);
      if constexpr (HELD == 2) load(ids, i, 1, HELD - 1);
      load_rope(ids, i);
    };
    auto unpark = [&]() {
      if constexpr (PARK) {
        uint32_t r[32];
        tmem_ld<32>(parked, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          asm volatile("" : "+r"(r[4 * e]), "+r"(r[4 * e + 1]), "+r"(r[4 * e + 2]), "+r"(r[4 * e + 3]));
          words[0][0][e >> 2].w[e & 3] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
        }
      }
    };
    load_tile(page_ids(0), 0);
    int slot = team, round = 0;
    for (int i = 0; i < n; ++i) {
      const int buf = i & 1;
      if (i >= 2 && ok) ok = wait(&bar.rope_free[buf], ((i >> 1) - 1) & 1);
      if (!__all_sync(kFull, ok)) break;
      tc_fence_after();
      tmem_st_16x256b(tb + S::TR + 32 * buf + ((uint32_t)(16 * mine) << 16), rope);
      // The scales' last readers, the softmax of tile i - 4, are done: the scores of tile i - 2
      // that have released this buffer were issued after it.
      if (lane < 16) sc_s[(i & (kScaleTiles - 1)) * kTok + 16 * mine + lane] = sc;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.rope_full[buf]);
#pragma unroll
      for (int j0 = 0; j0 < NB; j0 += S::TEAMS) {
        const int held = HELD == 2 ? j0 : 0;
        if (j0 > 0) unpark();
        if (round > 0 && ok) ok = wait(&bar.free[slot], (round - 1) & 1);
        if (!__all_sync(kFull, ok)) break;
        uint8_t* op = sm + S::RING + slot * kEntry;
#pragma unroll
        for (int u = 0; u < 2 * S::PAGES; ++u) {
          uint4 h[8];
          convert<MODE>(words[held][u >> 1][u & 1], lane, h);
          store_chunks<MODE>(h, op + (u & 1) * 2 * kPart, first + S::WARPS * (u >> 1), lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.full[slot]);
        if (j0 + S::TEAMS == NB) {
          load_tile(ahead, i + 1);
          ahead = page_ids(i + 2);
        }
        slot += S::TEAMS;
        if (slot >= S::SLOTS) {
          slot -= S::SLOTS;
          ++round;
        }
      }
    }
  } else if (warp >= kIssueWarp) {
    // ------------------------------------------------------------ products
    set_registers<S::RI>();
    if (warp == kIssueWarp && n > 0) {
      constexpr uint32_t kIdescS = umma_idesc_f16(128, N), kIdescO = umma_idesc_f16(128, N) | (1u << 15) | (1u << 16);
      const uint64_t dq = umma_sdesc(smem_u32(sm + S::Q), kLbo, S::QSBO);
      const uint64_t dk = umma_sdesc(smem_u32(sm + S::RING), 16, kGroup) | kSwizzle128;     // tokens x channels
      const uint64_t dv = umma_sdesc(smem_u32(sm + S::RING), kPart, kGroup) | kSwizzle128;  // channels x tokens: the same bytes
      const uint64_t dp = umma_sdesc(smem_u32(sm + S::P), N * 16, 128);        // rows x tokens, MN-major
      // The fence between the warps' stores and the tensor core's reads stands here, after the
      // wait for them: once for all of the warps that have arrived.
      const uint32_t tm = uniform(tb);
      int kslot = 0, kround = 0, vslot = 0;
      auto scores = [&](int i, int j) {  // of 256 channels
        if (ok) ok = wait_uniform(&bar.full[kslot], kround & 1);
        if (!ok) return;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t D = uniform(tm + (S::SB == 2 ? (i & 1) * 2 * N : 0)), more = uniform(j);
        const uint64_t A = dk + uniform(kslot * (kEntry >> 4)), B = dq + uniform(j * ((32 * kLbo) >> 4));
        if (elect_one()) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            umma_f16_ss(D, A + (e >> 2) * (kPart >> 4) + (e & 3) * (32 >> 4), B + e * ((2 * kLbo) >> 4), kIdescS, e > 0 ? 1u : more);
          if (j == NB - 1) tc_commit(&bar.s_full[S::SB == 2 ? i & 1 : 0]);
        }
        __syncwarp();
        if (++kslot == S::SLOTS) {
          kslot = 0;
          ++kround;
        }
      };
      auto rotary = [&](int i) {
        const int buf = i & 1, sb = S::SB == 2 ? i & 1 : 0;
        if (ok) ok = wait_uniform(&bar.rope_full[buf], (i >> 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t D = uniform(tm + sb * 2 * N + N), A = uniform(tm + S::TR + 32 * buf);
        if (elect_one()) {
          const uint64_t B = dq + (uint64_t)NB * ((32 * kLbo) >> 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) umma_f16_ts(D, A + 8 * e, B + e * ((2 * kLbo) >> 4), kIdescS, e > 0 ? 1u : 0u);
          tc_commit(&bar.rope_free[buf]);
          mbar_arrive(&bar.s_full[sb]);  // passes on the scales that came with the rotary rows
        }
        __syncwarp();
      };
      ok = wait_uniform(&bar.q_full, 0);
      rotary(0);
      for (int j = 0; j < NB; ++j) scores(0, j);
      for (int i = 0; i < n && ok; ++i) {
        const bool more = i + 1 < n;
        if (more && S::PRE > 0) {
          rotary(i + 1);
#pragma unroll 1
          for (int j = 0; j < S::PRE; ++j) scores(i + 1, j);
        }
        if (ok) ok = wait_uniform(&bar.p_full, i & 1);
        if (!ok) break;
        fence_proxy_async_smem();
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const uint64_t A = dv + uniform(vslot * (kEntry >> 4));
          const uint32_t after = uniform(i);
          uint64_t* done = &bar.free[uniform(vslot)];
          if (elect_one()) {
#pragma unroll
            for (int e = 0; e < 16; ++e)  // 128 channels after 128
              umma_f16_ss(tm + S::TO + (2 * j + (e >> 3)) * N, A + (e >> 3) * (2 * kPart >> 4) + (e & 7) * (2 * kGroup >> 4),
                          dp + (e & 7) * ((2 * N * 16) >> 4), kIdescO, (e & 7) > 0 ? 1u : after);
            tc_commit(done);
            if (j == NB - 1) tc_commit(&bar.p_free);
          }
          __syncwarp();
          if (++vslot == S::SLOTS) vslot = 0;
        }
        if (more) {
          if (S::PRE == 0) rotary(i + 1);
#pragma unroll 1
          for (int j = S::PRE; j < NB; ++j) scores(i + 1, j);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    set_registers<S::RS>();
    const long long row0 = latent_row(a, t, 0, t.r0);  // rows of a tile lie one after the other
    // Q: chunk c of row r at (r % 8) 16 + c kLbo + (r / 8) QSBO; zero past the tile's rows.
    // Rotary channels in the order of the keys' tensor memory: channels 16 m + 4 k .. + 3 are
    // the m-th eight bytes of step k's 32.
    constexpr int QN = (N * S::QCH + kSoftmax - 1) / kSoftmax, QF = QN < 3 ? QN : 3;
#pragma unroll 1
    for (int u0 = 0; u0 < QN; u0 += QF) {
      uint4 x[QF];  // (in flight at once)
#pragma unroll
      for (int u = 0; u < QF; ++u) {
        const int it = tid + (u0 + u) * kSoftmax, r = (it & 7) + it / (8 * S::QCH) * 8, c = (it >> 3) % S::QCH;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < t.count) x[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __half*>(a.q) + (row0 + r) * (L + kLatentRope)) + c);
      }
#pragma unroll
      for (int u = 0; u < QF; ++u) {
        const int it = tid + (u0 + u) * kSoftmax, r = (it & 7) + it / (8 * S::QCH) * 8, c = (it >> 3) % S::QCH;
        uint8_t* row = sm + S::Q + (r & 7) * 16 + (r >> 3) * S::QSBO;
        if (r >= N) continue;
        if (c < L / 8) {
          *reinterpret_cast<uint4*>(row + c * kLbo) = x[u];
        } else {
          const int d = 2 * (c - L / 8), m = d >> 2, k = d & 3;  // eight bytes each: d and d + 1 (of the same m)
          *reinterpret_cast<uint2*>(row + (L / 8 + 2 * k + (m >> 1)) * kLbo + 8 * (m & 1)) = make_uint2(x[u].x, x[u].y);
          *reinterpret_cast<uint2*>(row + (L / 8 + 2 * (k + 1) + (m >> 1)) * kLbo + 8 * (m & 1)) = make_uint2(x[u].z, x[u].w);
        }
      }
    }
    if (tid < N) {
      m_s[tid] = 0.0f;
      sees_s[tid] = tid < t.count ? latent_sees(a, t, t.r0 + tid) : 0;
    }
    if (tid < 2) fresh_s[tid] = kFull;
    fence_proxy_async_smem();  // Q is read by the tensor core
    softmax_sync();
    if (lane == 0) mbar_arrive(&bar.q_full);

    const int quad = warp & 3, tok = 32 * quad + lane, col = (warp >> 2) * C;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const float one = a.scale * kLog2e;
    const float tensor = PT ? 1.0f : *reinterpret_cast<const float*>(a.pool + kHdrKScaleOffset);
    float2 l[C / 2];
#pragma unroll
    for (int c = 0; c < C / 2; ++c) l[c] = make_float2(0.0f, 0.0f);
    uint32_t fresh = (1u << C) - 1;  // this thread's rows that have met no score yet: their reference is 0
    for (int i = 0; i < n; ++i) {
      const int sb = S::SB == 2 ? i & 1 : 0;
      // Where the scores of tile i come after all value products of tile i - 1, these are done
      // too: P of the last tile, and O, are free.
      if (warp == 0 && ok) {
        ok = wait(&bar.s_full[sb], (S::SB == 2 ? i >> 1 : i) & 1);
        if (S::PRE == NB && i > 0 && ok) ok = wait(&bar.p_free, (i - 1) & 1);
      }
      ok = !softmax_any(!ok);
      tc_fence_after();
      float2 y[C / 2];
      const float sc = sc_s[(i & (kScaleTiles - 1)) * kTok + tok];
      {
        // (eight columns of each at a time: registers)
        const float ks = one * (PT ? sc : tensor);
        constexpr int W = C < 8 ? C : 8;
#pragma unroll
        for (int c0 = 0; c0 < C; c0 += W) {
          uint32_t xc[W], xr[W];
          tmem_ld<W>(tb + sb * 2 * N + col + c0 + lanes, xc);
          tmem_ld<W>(tb + sb * 2 * N + N + col + c0 + lanes, xr);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < W; ++c) asm volatile("" : "+r"(xc[c]), "+r"(xr[c]));  // (no use before the wait)
#pragma unroll
          for (int c = 0; c < W; c += 2) {
            const float2 r = __fmul2_rn(make_float2(__uint_as_float(xr[c]), __uint_as_float(xr[c + 1])), make_float2(one, one));
            y[(c0 + c) / 2] = __ffma2_rn(make_float2(__uint_as_float(xc[c]), __uint_as_float(xc[c + 1])), make_float2(ks, ks), r);
          }
        }
      }
      const int tk = (i0 + i) * kTok + tok;
      const bool masked = (i0 + i + 1) * kTok > fewest;
      if (sc < 0.0f) {
#pragma unroll
        for (int c = 0; c < C / 2; ++c) y[c] = make_float2(-INFINITY, -INFINITY);
      } else if (masked) {
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const int4 s = *reinterpret_cast<const int4*>(sees_s + col + c);
          if (tk >= s.x) y[c / 2].x = -INFINITY;
          if (tk >= s.y) y[c / 2].y = -INFINITY;
          if (tk >= s.z) y[c / 2 + 1].x = -INFINITY;
          if (tk >= s.w) y[c / 2 + 1].y = -INFINITY;
        }
      }
      const float ex = PT ? scale_exponent(sc) : 0.0f;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < C; c += 4) {
        const float4 m = *reinterpret_cast<const float4*>(m_s + col + c);
        y[c / 2] = __fadd2_rn(y[c / 2], make_float2(-m.x, -m.y));
        y[c / 2 + 1] = __fadd2_rn(y[c / 2 + 1], make_float2(-m.z, -m.w));
        mx = fmaxf(mx, fmaxf(fmaxf(y[c / 2].x, y[c / 2].y), fmaxf(y[c / 2 + 1].x, y[c / 2 + 1].y)));
      }
      bool moves = mx + ex > kTop + kSlack;
      if (fresh) {
#pragma unroll
        for (int c = 0; c < C; ++c) moves |= ((fresh >> c) & 1u) && (c & 1 ? y[c / 2].y : y[c / 2].x) > -INFINITY;
      }
      if (softmax_any(moves)) {
        // References move: to each row's largest y + ex of the tile, over its 128 tokens.
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float w = warp_max((c & 1 ? y[c / 2].y : y[c / 2].x) + ex);
          if (lane == 0) red_s[quad * N + col + c] = w;
        }
        softmax_sync();
        if (warp < (N + 31) / 32) {
          bool still = false;
          if (tid < N) {
            const float top = fmaxf(fmaxf(red_s[tid], red_s[N + tid]), fmaxf(red_s[2 * N + tid], red_s[3 * N + tid]));
            const bool was = (fresh_s[warp] >> lane) & 1u, first = was && top > -INFINITY;
            const float to = ceilf(top) - kTop, up = first ? to : fmaxf(to, 0.0f);
            still = was && !first;
            m_s[tid] += up;
            up_s[tid] = up;
            f_s[tid] = first ? 1.0f : exp2f(-up);  // (a first score: nothing accumulated yet)
          }
          const uint32_t left = __ballot_sync(kFull, still);
          if (lane == 0) fresh_s[warp] = left;
        }
        softmax_sync();
        fresh = (fresh_s[col >> 5] >> (col & 31)) & ((1u << C) - 1);
        bool any = false;
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const float4 u = *reinterpret_cast<const float4*>(up_s + col + c), g = *reinterpret_cast<const float4*>(f_s + col + c);
          y[c / 2] = __fadd2_rn(y[c / 2], make_float2(-u.x, -u.y));
          y[c / 2 + 1] = __fadd2_rn(y[c / 2 + 1], make_float2(-u.z, -u.w));
          l[c / 2] = __fmul2_rn(l[c / 2], make_float2(g.x, g.y));
          l[c / 2 + 1] = __fmul2_rn(l[c / 2 + 1], make_float2(g.z, g.w));
          any |= g.x != 1.0f || g.y != 1.0f || g.z != 1.0f || g.w != 1.0f;
        }
        if (i > 0 && any) {  // (the same for all tokens)
#pragma unroll 1
          for (int j = 0; j < L / 128; ++j) {
#pragma unroll
            for (int c0 = 0; c0 < C; c0 += 4) {
              const float4 g = *reinterpret_cast<const float4*>(f_s + col + c0);
              uint32_t v[4];
              tmem_ld<4>(tb + S::TO + j * N + col + c0 + lanes, v);
              tmem_wait_ld();
              asm volatile("" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]));
              v[0] = __float_as_uint(__uint_as_float(v[0]) * g.x);
              v[1] = __float_as_uint(__uint_as_float(v[1]) * g.y);
              v[2] = __float_as_uint(__uint_as_float(v[2]) * g.z);
              v[3] = __float_as_uint(__uint_as_float(v[3]) * g.w);
              tmem_st<4>(tb + S::TO + j * N + col + c0 + lanes, v);
            }
          }
          tmem_wait_st();
        }
      }
      uint32_t p[C / 2];
#pragma unroll
      for (int c = 0; c < C / 2; ++c) {
        float2 w = make_float2(ex2(y[c].x), ex2(y[c].y));
        l[c] = __fadd2_rn(l[c], w);
        if (PT) {
          w = __fmul2_rn(w, make_float2(sc, sc));
          if (masked) {  // a weight of zero stays zero whatever the scale of a token that is not seen
            if (y[c].x == -INFINITY) w.x = 0.0f;
            if (y[c].y == -INFINITY) w.y = 0.0f;
          }
        }
        p[c] = h2_as_u32(__floats2half2_rn(w.x, w.y));
      }
      uint8_t* prow = sm + S::P + (tok >> 3) * (N * 16) + (tok & 7) * 16 + (col >> 3) * 128 + (col & 7) * 2;
      if constexpr (C >= 8) {
#pragma unroll
        for (int c = 0; c < C / 2; c += 4) *reinterpret_cast<uint4*>(prow + (c >> 2) * 128) = make_uint4(p[c], p[c + 1], p[c + 2], p[c + 3]);
      } else {
        *reinterpret_cast<uint2*>(prow) = make_uint2(p[0], p[1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full);
    }

    // ------------------------------------------------------------ outputs
    if (n > 0 && ok) ok = wait(&bar.p_free, (n - 1) & 1);
    tc_fence_after();
    if (!ok) failed_s = 1;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float x = c & 1 ? l[c / 2].y : l[c / 2].x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
      if (lane == 0) red_s[quad * N + col + c] = x;
    }
    softmax_sync();
    const bool failed = failed_s != 0;
    if (failed && tid == 0) set_error(const_cast<uint8_t*>(a.pool), KVQ_DEVERR_TIMEOUT);
    if (tid < N) {
      const float sum = red_s[tid] + red_s[N + tid] + red_s[2 * N + tid] + red_s[3 * N + tid];
      f_s[tid] = sum == 0.0f ? 0.0f : parts > 1 ? tensor : tensor / sum;  // (a NaN score makes its row NaN)
      if (tid < t.count && !failed) {
        const long long row = row0 + tid;
        if (parts > 1)
          st_chk(reinterpret_cast<float2*>(a.ws_ml) + (long long)blockIdx.x * N + tid, make_float2(sum == 0.0f ? -INFINITY : m_s[tid], sum),
                 a.ws_span, a.pool);
        else if (a.lse)
          st_chk(a.lse + row, sum == 0.0f ? -INFINITY : (m_s[tid] + log2f(sum)) * (1.0f / kLog2e), a.lse_span, a.pool);
      }
    }
    softmax_sync();
    if (!failed && (n > 0 || parts == 1)) {
      // O^T: a lane has a channel.  Partials leave as 32 neighbouring floats of a row to a
      // warp's store; fp16 rows go through shared memory (the ring is free) and leave 16
      // bytes a lane.
      constexpr int OROW = L * 2 + 16;
      uint8_t* stage = sm + S::RING;
      float f[C];
#pragma unroll
      for (int c = 0; c < C; c += 4) {
        const float4 g = *reinterpret_cast<const float4*>(f_s + col + c);
        f[c] = g.x;
        f[c + 1] = g.y;
        f[c + 2] = g.z;
        f[c + 3] = g.w;
      }
#pragma unroll 1
      for (int j = 0; j < L / 128; ++j) {
        uint32_t v[C];
        if (n > 0) {
          tmem_ld<C>(tb + S::TO + j * N + col + lanes, v);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < C; ++c) asm volatile("" : "+r"(v[c]));
        }
        const int ch = 128 * j + tok;
        float* po = a.ws_o + ((long long)blockIdx.x * N + col) * L + ch;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float x = n > 0 && f[c] != 0.0f ? __uint_as_float(v[c]) * f[c] : 0.0f;
          if (parts == 1) {
            *reinterpret_cast<__half*>(stage + (col + c) * OROW + 2 * ch) = __float2half_rn(x);
          } else if (col + c < t.count) {
            st_chk(po + c * L, x, a.ws_span, a.pool);
          }
        }
      }
      if (parts == 1) {
        softmax_sync();
        __half* out = static_cast<__half*>(a.out) + row0 * L;
#pragma unroll 4
        for (int it = tid; it < t.count * (L / 8); it += kSoftmax)
          st_chk(reinterpret_cast<uint4*>(out) + it, *reinterpret_cast<const uint4*>(stage + it / (L / 8) * OROW + it % (L / 8) * 16),
                 a.out_span, a.pool);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) tmem_dealloc(tb, 512);
}

template <int MODE, int L, int N>
cudaError_t launch(const LatentArgs& a, cudaStream_t s) {
  auto kern = latent_umma_kernel<MODE, L, N>;
  constexpr size_t smem = Shape<L, N>::dynamic();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)(a.ctas ? a.ctas : chunk_tile_bound(a.total_q, a.B, a.G, N)), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}
template <int L, int N>
cudaError_t launch_mode(int mode, const LatentArgs& a, cudaStream_t s) {
  switch (mode) {
    case KVQ_FP8_PER_TENSOR: return launch<KVQ_FP8_PER_TENSOR, L, N>(a, s);
    case KVQ_INT8_PER_TOKEN_HEAD: return launch<KVQ_INT8_PER_TOKEN_HEAD, L, N>(a, s);
    case KVQ_FP8_PER_TOKEN_HEAD: return launch<KVQ_FP8_PER_TOKEN_HEAD, L, N>(a, s);
    case KVQ_NVFP4:
    case KVQ_NVFP4_4OVER6: return launch<KVQ_NVFP4, L, N>(a, s);
    default: return cudaErrorInvalidValue;
  }
}
template <int L>
cudaError_t launch_rows(int mode, const LatentArgs& a, cudaStream_t s) {
  const int rows = latent_umma_rows(a.max_q_len, a.Hq);
  return rows == 16 ? launch_mode<L, 16>(mode, a, s) : rows == 32 ? launch_mode<L, 32>(mode, a, s) : launch_mode<L, 64>(mode, a, s);
}

}  // namespace

cudaError_t launch_latent_umma(const kvq_latent* c, const LatentArgs& a, cudaStream_t s) {
  return c->cfg.latent_dim == 512 ? launch_rows<512>(c->cfg.mode, a, s) : launch_rows<256>(c->cfg.mode, a, s);
}

}  // namespace kvq
