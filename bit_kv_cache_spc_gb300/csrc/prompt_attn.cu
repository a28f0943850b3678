// The causal attention of prompts (SpeCache page, section 3 "Prefilling": the
// attention that Algorithm 1's Quant and Offload follow), over 16-bit keys and
// values, with grouped heads, packed or batched sequences of different
// lengths, and queries that follow a history:
//   o_i = sum_{j <= i + lk - lq} p_ij v_j,  p_ij = exp(scale q_i.k_j - lse_i).
//
// One CTA takes two tiles of 128 query rows (a row is a token and one of the
// G query heads that share the KV head, so K and V are read once per group)
// and walks its keys in blocks of 64 with a running maximum and sum:
//   S = Q K^T (128 x 64 x 128) and O += P V (128 x 128 x 64) go to the tensor
//   cores (tcgen05.mma, bf16 in, fp32 accumulators in TMEM: two S blocks of
//   each tile in columns 0-255, O in 256-511); P replaces its S in TMEM as
//   bf16 and is read from there; K and V arrive by TMA, 128 keys at a time, in
//   a ring of five 32 KB stages.
// Warps 0-3 and 4-7 do the softmax of one tile each, a thread per row, and the
// output; warp 8 issues the copies, warps 9 and 10 the products of one tile
// each, warps 12-15 look after values in masked places (below).
// Why two S blocks per tile: with one block of 128 keys the softmax of a tile
// and its products alternate, and each turn pays the barriers' and the
// loads' latencies (3860 cycles for 2 x 128 keys, of which the tensor cores
// work 2048); with two, the next block's S is there when the softmax ends.
// Why a product warp per tile: a product's issue lasts nearly as long as its
// execution, so what one warp spends on waiting and committing between the
// tiles' products leaves the tensor cores idle.
//
// Bounds: 4*128 operations per visible (query head, key) pair for a prompt;
// for a few queries over a long history the bytes of K and V.
//
// P in bf16: the product's operand type.  Each weight is rounded once (2^-8
// relative at most); the sum of weights uses the fp32 values.
//
// Masked places: a masked score is replaced by -inf, so what K holds there
// does not matter, but 0 * V would still turn an infinity or a NaN of a masked
// value row into NaN.  Only tiles that some row of the pair does not see in
// full can hold such rows: warps 12-15 replace the non-finite elements of
// their value tiles by zeros before the product, and when there were any, the
// epilogue adds the non-finite elements of the visible keys back (their
// weights are positive, so an infinity keeps its sign).
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"

namespace spc {
namespace {

constexpr int kTile = 128;                   // query rows per tile, and keys per copy
constexpr int kBlock = 64;                   // keys per S block
constexpr int kStageBytes = kTile * kD * 2;  // one K or V tile, or one Q tile
constexpr int kStages = 5;
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum is only moved when it grows by more than this (in powers
// of two): weights then stay below 2^8, and O is rescaled a few times per row
// instead of at every tile.
constexpr float kSlack = 8.0f;

struct PromptArgs {
  const uint16_t* v;
  uint16_t* o;
  float* lse;
  const int32_t* q_begin;
  const int32_t* q_len;
  const int32_t* k_begin;
  const int32_t* k_len;
  float* part_o;    // [item][split][tile rows][D]
  float2* part_ml;  // [item][split][tile rows]
  uint32_t* fault;
  int64_t v_b, v_t, v_h, o_b, o_t, o_h, lse_b;
  int32_t S, Hq, Hkv, G, tile_tokens, pairs, splits;
  int32_t q_tokens, k_tokens, q_max, k_max;
  int32_t q_batched, k_batched;  // sequence s lies at s * stride (else on one token axis)
  float scale;
};

struct __align__(8) PromptBars {
  uint64_t q_full[2];
  uint64_t kv_full[kStages];
  uint64_t kv_free[kStages];
  uint64_t v_scan;   // the next value tile that may hold masked places has arrived
  uint64_t v_clean;  // and holds only finite elements
  // per query tile and S buffer: block i's scores are there, and so is the product of block i - 2's weights
  uint64_t s_full[2][2];
  uint64_t p_full[2][2];  // its weights are
  uint32_t tmem;
  uint32_t bad;            // a masked tile held a non-finite value
  volatile uint32_t stop;  // a wait ran out
};

constexpr int kSmemBytes = (2 + kStages) * kStageBytes + 1024 + 512;
static_assert(sizeof(PromptBars) <= 512, "barriers outgrow their place");
static_assert(kSmemBytes <= 232448, "more shared memory than an SM has");

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_addr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_addr(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase; false once this or another wait of the CTA has run out
// (two seconds; the longest regular wait is far below a millisecond).
// The timer is read only after many tries: reading it takes longer than a
// regular wait.
__device__ __forceinline__ bool mbar_wait(PromptBars& bars, uint64_t* b, uint32_t parity) {
  for (int i = 0; i < 64; ++i)
    if (mbar_try(b, parity)) return true;
  uint64_t start, now;
  asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(start));
  for (;;) {
    for (int i = 0; i < 16; ++i)
      if (mbar_try(b, parity)) return true;
    if (bars.stop) return false;
    asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(now));
    if (now - start > 2000000000ull) {
      bars.stop = 1u;
      return false;
    }
  }
}

// For a whole warp: one outcome for all lanes.
__device__ __forceinline__ bool mbar_wait_warp(PromptBars& bars, uint64_t* b, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bars, b, parity));
}

__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                          int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];\n" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_addr(bar))
               : "memory");
}

// 32 consecutive TMEM columns of the thread's lane; the caller waits.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(addr));
}
// Ends the loads in flight; r (32 loaded values) is named so that no use of it moves before the wait.
__device__ __forceinline__ void tmem_wait_ld(float* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), 
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), 
                 "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), 
                 "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
               :
               : "memory");
}
// max(a, b, c), NaN only when all are
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};\n" ::"r"(addr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Instruction word of a bf16 product with fp32 sums, M = 128; B either with
// the contraction contiguous (keys of S) or with N contiguous (values).
__host__ __device__ constexpr uint32_t mma_word(uint32_t n, bool b_n_contiguous) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_n_contiguous ? 1u : 0u) << 16) | ((n / 8) << 17) |
         ((128u / 16) << 24);
}
// Shared-memory operand with 128-byte swizzle; offsets in bytes.  A step of x
// bytes is an addition of x / 16 (addresses stay below 2^18).
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t word, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(word), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t word, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          d),
      "r"(a), "l"(b), "r"(word), "r"((uint32_t)add)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(yes));
  return yes != 0;
}
// S = Q K^T of 64 keys: operands are two halves of 64 columns, rows of 128
// bytes in groups of eight 1024 bytes apart; 16 columns (32 bytes) a step.
__device__ __forceinline__ void product_s(uint32_t d, uint64_t q, uint64_t k) {
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const uint32_t off = ((uint32_t)(s >> 2) * 16384u + (uint32_t)(s & 3) * 32u) / 16;
    mma_ss(d, q + off, k + off, mma_word(kBlock, false), s > 0);
  }
}
// O += P V of 64 keys: V's halves hold channels 0-63 and 64-127 of each key (N
// contiguous, the halves 16384 bytes apart, groups of eight keys 1024 bytes
// apart); 16 keys (2048 bytes, and eight TMEM columns of P) a step.
__device__ __forceinline__ void product_o(uint32_t d, uint32_t p, uint64_t v, bool add) {
#pragma unroll
  for (int s = 0; s < 4; ++s) mma_ts(d, p + 8 * s, v + 2048u / 16 * s, mma_word(kD, true), add || s > 0);
}

// What a CTA works on.
struct PromptItem {
  int s, hkv, pair, split;
  int lq, lk, qb, kb;  // lengths and first tokens of the sequence
  int tok0;            // first query token of the pair
  int lo, hi;          // key tiles [lo, hi)
  int blocks;          // 64-key blocks of them that some row sees
  int edge;            // first key tile that some row does not see in full
  bool two;            // the second query tile has rows
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// Lengths and first tokens as the device arrays give them, held to the
// tensors: no row outside them is read or written whatever the arrays hold.
__device__ __forceinline__ void sequence(const PromptArgs& a, int s, int& lq, int& lk, int& qb, int& kb) {
  qb = a.q_begin ? clampi(a.q_begin[s], 0, a.q_tokens) : 0;
  kb = a.k_begin ? clampi(a.k_begin[s], 0, a.k_tokens) : 0;
  lq = clampi(a.q_len ? a.q_len[s] : a.q_max, 0, min(a.q_max, a.q_tokens - qb));
  lk = clampi(a.k_len ? a.k_len[s] : a.k_max, 0, min(a.k_max, a.k_tokens - kb));
}

// Item `i` of the grid: later pairs (more keys) first, KV heads and sequences
// fastest, so that CTAs that run together read different heads' keys at the
// same depth and several pairs of a head share them in L2.
__device__ __forceinline__ PromptItem prompt_item(const PromptArgs& a, int64_t i) {
  PromptItem w;
  w.split = (int)(i % a.splits);
  i /= a.splits;
  w.hkv = (int)(i % a.Hkv);
  i /= a.Hkv;
  w.s = (int)(i % a.S);
  w.pair = a.pairs - 1 - (int)(i / a.S);
  sequence(a, w.s, w.lq, w.lk, w.qb, w.kb);
  w.tok0 = w.pair * 2 * a.tile_tokens;
  w.two = w.tok0 + a.tile_tokens < w.lq;
  const int last = min(w.tok0 + 2 * a.tile_tokens, w.lq) - 1;  // last query token
  const int most = w.tok0 < w.lq ? clampi(last + w.lk - w.lq + 1, 0, w.lk) : 0;
  const int least = clampi(w.tok0 + w.lk - w.lq + 1, 0, w.lk);
  const int n = (most + kTile - 1) / kTile;
  const int per = (n + a.splits - 1) / a.splits;
  w.lo = min(w.split * per, n);
  w.hi = min(w.lo + per, n);
  w.blocks = max(0, min(2 * (w.hi - w.lo), (most - w.lo * kTile + kBlock - 1) / kBlock));
  w.edge = least / kTile;
  return w;
}

// exp2(x c - m c) of a row's 64 scores, as bf16 pairs into P, and their sum.
__device__ __forceinline__ float row_weights(float* x, float c, float mc, uint32_t p_addr) {
  float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
  const float2 c2 = {c, c}, m2 = {-mc, -mc};
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 y = f2_fma({x[32 * b + 2 * i], x[32 * b + 2 * i + 1]}, c2, m2);
      const float2 e = {fast_exp2(y.x), fast_exp2(y.y)};
      sum[i & 1] = f2_add(sum[i & 1], e);
      u[i] = pack_bf16x2(e.x, e.y);
    }
    tmem_st16(p_addr + 16 * b, u);
  }
  const float2 all = f2_add(sum[0], sum[1]);
  return all.x + all.y;
}

__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PromptArgs a) {
  extern __shared__ uint8_t prompt_smem[];
  const PromptItem w = prompt_item(a, blockIdx.x);
  if (w.tok0 >= w.lq) return;  // uniform: no query rows
  uint8_t* base = prompt_smem + ((1024u - (smem_addr(prompt_smem) & 1023u)) & 1023u);
  PromptBars& bars = *reinterpret_cast<PromptBars*>(base + (2 + kStages) * kStageBytes);
  uint8_t* ring = base + 2 * kStageBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = w.hi - w.lo;

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(&bars.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars.s_full[i][b], 1);
        mbar_init(&bars.p_full[i][b], 4);
      }
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.kv_full[i], 1);
      mbar_init(&bars.kv_free[i], w.two ? 2 : 1);
    }
    mbar_init(&bars.v_scan, w.two ? 2 : 1);
    mbar_init(&bars.v_clean, 4);
    bars.bad = 0;
    bars.stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp >= 8) {
    if (warp == 8) {
      // ---- copies: Q tiles, then K_lo, V_lo, K_lo+1, V_lo+1, ... through the ring ----
      if (lane == 0 && n > 0) {
        const int tile_bytes = a.tile_tokens * a.G * kD * 2;
        auto load_q = [&](int t) {
          mbar_expect(&bars.q_full[t], tile_bytes);
          const int tok = w.qb + w.tok0 + t * a.tile_tokens;
          for (int h = 0; h < 2; ++h)
            tma_load4(base + t * kStageBytes + h * 16384, &qmap, &bars.q_full[t], 64 * h, w.hkv * a.G, tok,
                      a.q_batched ? w.s : 0);
        };
        bool ok = true;
        auto load_kv = [&](int it, const CUtensorMap* map, int j) {
          const int st = it % kStages;
          ok = ok && mbar_wait(bars, &bars.kv_free[st], ((it / kStages) & 1) ^ 1);
          if (!ok) return;
          mbar_expect(&bars.kv_full[st], kStageBytes);
          for (int h = 0; h < 2; ++h)
            tma_load4(ring + st * kStageBytes + h * 16384, map, &bars.kv_full[st], 64 * h, w.hkv, w.kb + j * kTile,
                      a.k_batched ? w.s : 0);
        };
        load_q(0);
        load_kv(0, &kmap, w.lo);
        if (w.two) load_q(1);
        for (int j = 0; j < n && ok; ++j) {
          load_kv(2 * j + 1, &vmap, w.lo + j);
          if (j + 1 < n) load_kv(2 * j + 2, &kmap, w.lo + j + 1);
        }
      }
    } else if (warp == 9 || (warp == 10 && w.two)) {
      // ---- products of a tile: the whole warp walks the blocks, converged, so that operands are formed in uniform
      // registers (a lane alone issued a product every 55 cycles), and one lane issues ----
      const bool lead = elect_lane();
      const int t = __shfl_sync(0xFFFFFFFFu, warp - 9, 0);
      const int blocks = __shfl_sync(0xFFFFFFFFu, w.blocks, 0);
      const int edge = __shfl_sync(0xFFFFFFFFu, w.edge - w.lo, 0);  // the first tile to be scanned
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t base_addr = __shfl_sync(0xFFFFFFFFu, smem_addr(base), 0);
      const uint64_t qd = smem_operand(base_addr + kStageBytes * t, 16, 1024);
      const uint64_t kd = smem_operand(base_addr + 2 * kStageBytes, 16, 1024);
      const uint64_t vd = smem_operand(base_addr + 2 * kStageBytes, 16384, 1024);
      const uint32_t sp = tm + 128 * t, op = tm + 256 + 128 * t;
      constexpr uint32_t kStep = kStageBytes / 16, kHalf = kBlock * 128 / 16;  // a stage, 64 of its rows
      uint32_t scans = 0;
      bool ok = blocks > 0 && mbar_wait_warp(bars, &bars.kv_full[0], 0) && mbar_wait_warp(bars, &bars.q_full[t], 0);
      if (ok && lead) {
        product_s(sp, qd, kd);
        tc_commit(&bars.s_full[t][0]);
        if (blocks > 1) product_s(sp + kBlock, qd, kd + kHalf);
        tc_commit(&bars.s_full[t][1]);
        tc_commit(&bars.kv_free[0]);
      }
      __syncwarp();
      int sv = 1, sk = 2;       // stages of V_j and K_j+1
      uint32_t pv = 0, pk = 0;  // and the phases of their barriers
      for (int j = 0; 2 * j < blocks && ok; ++j) {
        ok = mbar_wait_warp(bars, &bars.kv_full[sv], pv);
        if (ok && j >= edge) {
          if (lead) mbar_arrive(&bars.v_scan);
          __syncwarp();
          ok = mbar_wait_warp(bars, &bars.v_clean, scans++ & 1u);
        }
        if (ok && 2 * j + 2 < blocks) ok = mbar_wait_warp(bars, &bars.kv_full[sk], pk);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (2 * j + b >= blocks || !ok) break;
          ok = mbar_wait_warp(bars, &bars.p_full[t][b], j & 1);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
            product_o(op, sp + kBlock * b, vd + kStep * sv + kHalf * b, j + b > 0);
            if (2 * j + b + 2 < blocks) product_s(sp + kBlock * b, qd, kd + kStep * sk + kHalf * b);
            tc_commit(&bars.s_full[t][b]);
          }
          __syncwarp();
        }
        if (ok && lead) {
          tc_commit(&bars.kv_free[sv]);
          if (2 * j + 2 < blocks) tc_commit(&bars.kv_free[sk]);
        }
        __syncwarp();
        sv += 2;
        if (sv >= kStages) { sv -= kStages; pv ^= 1; }
        sk += 2;
        if (sk >= kStages) { sk -= kStages; pk ^= 1; }
      }
    } else if (warp >= 12) {
      // ---- values in masked places: tile by tile as the product warp asks (a wait on the stage alone could
      // take an earlier phase of its barrier for the awaited one) ----
      uint32_t scans = 0;
      for (int j = max(w.edge - w.lo, 0); j < n; ++j) {
        const int iv = 2 * j + 1, sv = iv % kStages;
        if (!mbar_wait_warp(bars, &bars.v_scan, scans++ & 1u)) break;
        if (!mbar_wait_warp(bars, &bars.kv_full[sv], (iv / kStages) & 1)) break;
        uint4* tile = reinterpret_cast<uint4*>(ring + sv * kStageBytes);
        bool touched = false;
#pragma unroll 4
        for (int i = tid - 384; i < kStageBytes / 16; i += 128) {
          const uint4 x = tile[i];
          // 16-bit halves with an exponent of all ones
          const uint32_t m0 = __vcmpeq2(x.x & 0x7F807F80u, 0x7F807F80u), m1 = __vcmpeq2(x.y & 0x7F807F80u, 0x7F807F80u);
          const uint32_t m2 = __vcmpeq2(x.z & 0x7F807F80u, 0x7F807F80u), m3 = __vcmpeq2(x.w & 0x7F807F80u, 0x7F807F80u);
          if (m0 | m1 | m2 | m3) {
            tile[i] = make_uint4(x.x & ~m0, x.y & ~m1, x.z & ~m2, x.w & ~m3);
            touched = true;
          }
        }
        if (touched) bars.bad = 1u;
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.v_clean);
      }
    }
  } else {
    // ---- softmax of one tile, a thread per row ----
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    const uint32_t s_addr = tmem + lanes + 128 * t, o_addr = tmem + lanes + 256 + 128 * t;
    const int tok = w.tok0 + t * a.tile_tokens + r / a.G;
    const int head = w.hkv * a.G + r % a.G;
    const bool row = r < a.tile_tokens * a.G && tok < w.lq;
    const int seen = row ? clampi(tok + w.lk - w.lq + 1, 0, w.lk) : w.lk;  // keys of this row
    const float c = a.scale * kLog2e;
    const bool active = t == 0 || w.two;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (active) {
      for (int i = 0; i < w.blocks; ++i) {
        const int b = i & 1;
        const uint32_t sp = s_addr + kBlock * b;
        ok = mbar_wait_warp(bars, &bars.s_full[t][b], (i >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        float x[kBlock];
        tmem_ld32(sp, x);
        tmem_ld32(sp + 32, x + 32);
        tmem_wait_ld(x);
        tmem_wait_ld(x + 32);
        if (w.lo + (i >> 1) >= w.edge) {
          const int vis = seen - w.lo * kTile - i * kBlock;
#pragma unroll
          for (int e = 0; e < kBlock; ++e) x[e] = e < vis ? x[e] : -INFINITY;
        }
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int e = 4; e < kBlock; e += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            top[u] = e + 4 + u < kBlock ? max3(top[u], x[e + u], x[e + 4 + u]) : fmaxf(top[u], x[e + u]);
        const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]);
        const bool grow = mx > m && !((mx - m) * c <= kSlack);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float f = grow ? fast_exp2((m - mx) * c) : 1.f;  // m = -inf: 0
          if (grow) m = mx;
          l *= f;
          if (i > 0) {
            // the product of the block before has to be complete: the next use of the other buffer says so
            ok = mbar_wait_warp(bars, &bars.s_full[t][b ^ 1], ((i + 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float y[32];
              tmem_ld32(o_addr + 32 * q, y);
              tmem_wait_ld(y);
              uint32_t u[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(y[e] * f);
              tmem_st16(o_addr + 32 * q, u);
              tmem_st16(o_addr + 32 * q + 16, u + 16);
            }
          }
        }
        l += row_weights(x, c, m == -INFINITY ? 0.f : m * c, sp);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[t][b]);
      }
      // ---- output ----
      const int64_t part = ((int64_t)blockIdx.x * 2 + t) * kTile + r;  // splits are fastest in the grid
      if (n > 0 && ok) ok = mbar_wait_warp(bars, &bars.s_full[t][(w.blocks + 1) & 1], ((w.blocks + 1) >> 1) & 1);
      if (ok) {
        tc_fence_after();
        const bool bad = *(volatile uint32_t*)&bars.bad != 0u;
        const int first = max(w.edge, w.lo) * kTile, end = min(seen, w.hi * kTile);
        // no visible key: 0; otherwise the sum is positive, or not a number when the scores are not
        const bool any = seen > w.lo * kTile;
        const float inv = a.splits > 1 ? 1.f : (any ? 1.f / l : 0.f);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float y[32];
          if (n > 0) {
            tmem_ld32(o_addr + 32 * b, y);
            tmem_wait_ld(y);
          }
          if (!any) {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = 0.f;
          }
          if (bad && row) {
            const uint16_t* vr = a.v + w.s * a.v_b + (int64_t)(w.kb + first) * a.v_t + w.hkv * a.v_h + 32 * b;
            for (int key = first; key < end; ++key, vr += a.v_t) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const uint32_t e = vr[i];
                if ((e & 0x7F80u) == 0x7F80u) y[i] += bf16_to_f32(e);
              }
            }
          }
          if (!row) continue;
          if (a.splits > 1) {
            float4* po = reinterpret_cast<float4*>(a.part_o + part * kD + 32 * b);
#pragma unroll
            for (int i = 0; i < 8; ++i) po[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          } else {
            uint4* po = reinterpret_cast<uint4*>(a.o + w.s * a.o_b + (int64_t)(w.qb + tok) * a.o_t + head * a.o_h + 32 * b);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              po[i] = make_uint4(pack_bf16x2(y[8 * i] * inv, y[8 * i + 1] * inv),
                                 pack_bf16x2(y[8 * i + 2] * inv, y[8 * i + 3] * inv),
                                 pack_bf16x2(y[8 * i + 4] * inv, y[8 * i + 5] * inv),
                                 pack_bf16x2(y[8 * i + 6] * inv, y[8 * i + 7] * inv));
          }
        }
        if (row) {
          if (a.splits > 1)
            a.part_ml[part] = make_float2(any ? m * c : -INFINITY, any ? l : 0.f);
          else if (a.lse)
            a.lse[w.s * a.lse_b + (int64_t)(w.qb + tok) * a.Hq + head] = any ? m * a.scale + logf(l) : -INFINITY;
        }
      }
    }
  }
  if (bars.stop) {  // a wait ran out: report it, and let copies in flight land
    if (tid == 0 && a.fault != nullptr) *a.fault = 1u;
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the splits of a row: o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s,
// in the order of the splits.  One warp per row, four channels a lane.
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ PromptArgs a) {
  const int64_t rows_per_pair = 2 * (int64_t)a.tile_tokens * a.G;
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t item = i / rows_per_pair;  // as the grid numbers them, without the split
  if (item >= (int64_t)a.S * a.Hkv * a.pairs) return;
  const int in_pair = (int)(i % rows_per_pair);
  const int per_tile = a.tile_tokens * a.G;
  const int t = in_pair / per_tile, r = in_pair % per_tile;
  const int lane = threadIdx.x & 31;
  const int hkv = (int)(item % a.Hkv), s = (int)(item / a.Hkv % a.S);
  const int pair = a.pairs - 1 - (int)(item / a.Hkv / a.S);
  int lq, lk, qb, kb;
  sequence(a, s, lq, lk, qb, kb);
  const int tok = (pair * 2 + t) * a.tile_tokens + r / a.G, head = hkv * a.G + r % a.G;
  if (tok >= lq) return;
  float m = -INFINITY;
  for (int z = 0; z < a.splits; ++z) m = fmaxf(m, a.part_ml[((item * a.splits + z) * 2 + t) * kTile + r].x);
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool any = tok + lk - lq + 1 > 0 && lk > 0;
  if (any) {
    for (int z = 0; z < a.splits; ++z) {
      const int64_t part = ((item * a.splits + z) * 2 + t) * kTile + r;
      const float2 ml = a.part_ml[part];
      if (ml.y == 0.f) continue;  // nothing visible in this split
      const float f = exp2f(ml.x - m);
      const float4 x = reinterpret_cast<const float4*>(a.part_o + part * kD)[lane];
      l += f * ml.y;
      o = make_float4(o.x + f * x.x, o.y + f * x.y, o.z + f * x.z, o.w + f * x.w);
    }
  }
  const float inv = any ? 1.f / l : 0.f;
  uint2* po = reinterpret_cast<uint2*>(a.o + s * a.o_b + (int64_t)(qb + tok) * a.o_t + head * a.o_h) + lane;
  *po = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (lane == 0 && a.lse) a.lse[s * a.lse_b + (int64_t)(qb + tok) * a.Hq + head] = any ? m * kLn2 + logf(l) : -INFINITY;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::mutex mu;
  static EncodeTiled fn = nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  }
  return fn;
}

// Map of [batch][token][head][128] with the given strides: boxes of `heads`
// heads and `tokens` tokens of half a row (64 channels, 128 bytes, swizzled).
bool encode_map(CUtensorMap* map, const uint16_t* p, int64_t batch, int64_t tokens, int64_t heads,
                const spc_layout& st, uint32_t box_heads, uint32_t box_tokens) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  // an axis of one element is never stepped along: any valid stride does
  const auto stride = [](int64_t n, int64_t s) { return (cuuint64_t)(n > 1 ? s * 2 : kD * 2); };
  const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {stride(heads, st.h), stride(tokens, st.t), stride(batch, st.b)};
  const cuuint32_t box[4] = {64, box_heads, box_tokens, 1}, step[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(p), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Grid of a call: pairs of query tiles per (sequence, KV head), and splits of
// the keys where the pairs alone do not fill the GPU.
void prompt_grid(const spc_prompt_dims* d, int& tile_tokens, int& pairs, int& splits) {
  const int G = d->Hq / d->Hkv;
  tile_tokens = kTile / G;
  pairs = (int)(((int64_t)d->q_max + 2 * tile_tokens - 1) / (2 * tile_tokens));
  const int64_t items = (int64_t)d->S * d->Hkv * pairs;
  const int64_t sms = spc_host::sm_count();
  const int64_t ktiles = ((int64_t)d->k_max + kTile - 1) / kTile;
  splits = 1;
  if (items > 0 && items < sms) splits = (int)std::max<int64_t>(1, std::min<int64_t>(ktiles / 4, 4 * sms / items));
}

constexpr size_t kPromptHead = 256;  // the fault word

}  // namespace

size_t prompt_workspace_bytes(const spc_prompt_dims* d) {
  int tile_tokens, pairs, splits;
  prompt_grid(d, tile_tokens, pairs, splits);
  if (splits == 1) return kPromptHead;
  const size_t rows = (size_t)d->S * d->Hkv * pairs * splits * 2 * kTile;
  return kPromptHead + rows * (kD * sizeof(float) + sizeof(float2));
}

spc_status launch_prompt_attn(const spc_prompt_dims* d, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                              const int32_t* q_begin, const int32_t* q_len, const int32_t* k_begin,
                              const int32_t* k_len, uint16_t* o, float* lse, void* ws, cudaStream_t stream) {
  PromptArgs a = {};
  a.v = v;
  a.o = o;
  a.lse = lse;
  a.q_begin = q_begin;
  a.q_len = q_len;
  a.k_begin = k_begin;
  a.k_len = k_len;
  a.v_b = d->v.b;
  a.v_t = d->v.t;
  a.v_h = d->v.h;
  a.o_b = d->o.b;
  a.o_t = d->o.t;
  a.o_h = d->o.h;
  a.q_batched = d->q.b != 0;
  a.k_batched = d->k.b != 0;
  a.lse_b = a.q_batched ? (int64_t)d->q_tokens * d->Hq : 0;
  a.S = d->S;
  a.Hq = d->Hq;
  a.Hkv = d->Hkv;
  a.G = d->Hq / d->Hkv;
  a.q_tokens = d->q_tokens;
  a.k_tokens = d->k_tokens;
  a.q_max = d->q_max;
  a.k_max = d->k_max;
  a.scale = d->scale;
  prompt_grid(d, a.tile_tokens, a.pairs, a.splits);
  a.fault = static_cast<uint32_t*>(ws);
  const int64_t items = (int64_t)d->S * d->Hkv * a.pairs;
  const size_t rows = (size_t)items * a.splits * 2 * kTile;
  a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kPromptHead);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * kD);
  CUtensorMap qm, km, vm;
  const int64_t kt = std::max(d->k_tokens, 1);  // no keys at all: the maps are never read through
  if (!encode_map(&qm, q, a.q_batched ? d->S : 1, d->q_tokens, d->Hq, d->q, a.G, a.tile_tokens) ||
      !encode_map(&km, k ? k : q, a.k_batched ? d->S : 1, kt, d->Hkv, d->k, 1, kTile) ||
      !encode_map(&vm, v ? v : q, a.k_batched ? d->S : 1, kt, d->Hkv, d->v, 1, kTile)) {
    spc_host::set_cuda_error(cudaErrorInvalidValue);
    return SPC_ERR_CUDA;
  }
  static unsigned long long configured = 0ull;
  cudaError_t e = spc_host::ensure_smem_limit(configured, prompt_attn_kernel, kSmemBytes);
  if (e == cudaSuccess) {
    prompt_attn_kernel<<<(unsigned)(items * a.splits), kThreads, kSmemBytes, stream>>>(qm, km, vm, a);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && a.splits > 1) {
    const int64_t warps = items * 2 * a.tile_tokens * a.G;
    prompt_join_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace spc
