// The causal attention of prompts (SpeCache page, section 3 "Prefilling": the
// attention that Algorithm 1's Quant and Offload follow), over 16-bit keys and
// values, with grouped heads, packed or batched sequences of different
// lengths, and queries that follow a history:
//   o_i = sum_{j <= i + lk - lq} p_ij v_j,  p_ij = exp(scale q_i.k_j - lse_i).
//
// A CTA takes one or two tiles of 128 query rows (a row is a token and one of
// the G query heads that share the KV head, so K and V are read once per
// group) and walks its keys in blocks of 64 with a running maximum and sum:
//   S = Q K^T (128 x 64 x 128) and O += P V (128 x 128 x 64) go to the tensor
//   cores (tcgen05.mma, bf16 in, fp32 accumulators in TMEM: two S blocks and O
//   of each tile); P replaces its S in TMEM as bf16 and is read from there; K
//   and V arrive by TMA in a ring of stages.
// Four warps per tile do its softmax, a thread per row, and the output; one
// warp issues the copies, one per tile the products, and some look after
// values in masked places (below).
// Two tiles (256 rows) share every K and V stage, 128 keys each: prompts,
// bound by the tensor cores.  One tile, where a sequence's rows fit into it
// (single tokens, short turns: bound by the bytes of K and V) and for short
// prompts: half the TMEM and shared memory, 64 keys a stage, so that two CTAs
// share an SM and one's start and output overlap the other's copies.
// Why two S blocks per tile: with one block of 128 keys the softmax of a tile
// and its products alternate, and each turn pays the barriers' and the
// loads' latencies (3860 cycles for 2 x 128 keys, of which the tensor cores
// work 2048); with two, the next block's S is there when the softmax ends
// (2620 cycles; S of 64 keys is bound by shared memory, 384 cycles where its
// operations would take 256, so 2480 is the least).
// Why a product warp per tile: a product's issue lasts nearly as long as its
// execution, so what one warp spends on waiting and committing between the
// tiles' products leaves the tensor cores idle (3980 cycles).
// Items are numbered densely over the sequences' actual lengths, longer rows
// of keys first.  CTAs that stay and take item after item measured slower
// (a 32768-token prompt 5.68 ms against 5.43, eight single tokens over up to
// 32768 keys 140 us against 103): the next item's copies wait for Q's place,
// and its softmax for the last one's output, all the same.
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
// full can hold such rows: the scan warps replace the non-finite elements of
// their value tiles by zeros before the product, and when there were any, the
// epilogue adds the non-finite elements of the visible keys back (their
// weights are positive, so an infinity keeps its sign).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "common.cuh"

namespace spc {
namespace {

constexpr int kTile = 128;                  // query rows per tile
constexpr int kBlock = 64;                  // keys per S block
constexpr int kTileBytes = kTile * kD * 2;  // of a Q tile

// What depends on the number of query tiles of a CTA.
template <int TILES>
struct Shape {
  static constexpr int kKeys = TILES == 2 ? 128 : 64;  // keys per stage
  static constexpr int kPerStage = kKeys / kBlock;     // S blocks of a stage
  static constexpr int kAhead = 2 / kPerStage;         // K stages before the first V
  static constexpr int kStages = TILES == 2 ? 5 : 4;
  static constexpr int kStageBytes = kKeys * kD * 2;
  static constexpr int kSoftmaxWarps = 4 * TILES;
  static constexpr int kCopyWarp = kSoftmaxWarps;
  static constexpr int kProductWarp = kCopyWarp + 1;              // and the next one
  static constexpr int kScanWarp = TILES == 2 ? 12 : 6;           // from here on
  static constexpr int kThreads = TILES == 2 ? 512 : 256;
  static constexpr uint32_t kTmemCols = 256 * TILES;              // S of all tiles, then O
  static constexpr int kSmemBytes = TILES * kTileBytes + kStages * kStageBytes + 1024 + 512;
};
static_assert(Shape<2>::kSmemBytes <= 232448 && 2 * (Shape<1>::kSmemBytes + 1024) <= 233472,
              "more shared memory than an SM has");

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum is only moved when it grows by more than this (in powers
// of two): weights then stay below 2^8, and O is rescaled a few times per row
// instead of at every tile.
constexpr float kSlack = 8.0f;
constexpr int kDense = 256;  // sequences whose actual lengths number the items

__device__ uint32_t prompt_device_fault;  // a wait of some call on the device ran out

struct PromptArgs {
  const uint16_t* v;
  uint16_t* o;
  float* lse;
  const int32_t* q_begin;
  const int32_t* q_len;
  const int32_t* k_begin;
  const int32_t* k_len;
  float* part_o;    // [split][sequence][q_max][query head][D]
  float2* part_ml;  // and their (maximum, sum)
  int64_t part_rows;
  uint32_t* fault;
  uint64_t limit;   // of a wait, in ns
  int64_t v_b, v_t, v_h, o_b, o_t, o_h;
  int32_t S, Hq, Hkv, G, tile_tokens, pair_tokens, pairs, splits;
  int32_t q_tokens, k_tokens, q_max, k_max;
  int32_t rounds, gap;           // of the last split's CTAs, and the stages that these cost more
  uint32_t items;                // without splits
  int32_t dense;                 // items are numbered over the pairs that exist
  int32_t q_batched, k_batched;  // sequence s lies at s * stride (else on one token axis)
  float scale;
};

// What a CTA works on.
struct PromptItem {
  int s, hkv, pair, split;  // s < 0: nothing
  int lq, lk, qb, kb;       // lengths and first tokens of the sequence
  int tok0;                 // first query token
  int lo, hi;               // stages of keys [lo, hi)
  int blocks[2];            // 64-key blocks of them that some row of each tile sees
  int edge;                 // first stage that some row does not see in full
  int two;                  // the second query tile has rows
};

struct __align__(16) PromptBars {
  PromptItem item;
  uint64_t q_full[2];
  uint64_t kv_full[5];
  uint64_t kv_free[5];
  uint64_t v_scan[2];   // a value stage that may hold masked places is on its way (requests by turns)
  uint64_t v_clean[5];  // the stage has arrived and holds only finite elements
  // per query tile and S buffer: block i's scores are there, and so is the product of block i - 2's weights
  uint64_t s_full[2][2];
  uint64_t p_full[2][2];  // its weights are
  uint64_t drained[2];    // after a wait that ran out: the tile's products have ended
  uint64_t limit;         // of a wait, in ns
  uint32_t* fault;        // the workspace's word, or null
  int filled;             // stages copied in all
  uint32_t tmem;
  uint32_t bad;            // a masked stage held a non-finite value
  volatile uint32_t stop;  // a wait ran out
};
static_assert(sizeof(PromptBars) <= 512, "barriers outgrow their place");

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
// (two seconds unless the caller sets another limit).  The thread whose wait
// runs out reports it: no other has to be there still to see it.  The timer is
// read only after many tries: reading it takes longer than a regular wait.
// A wait for something that regularly comes after `stages` stages of keys has a
// 65536th of the limit more for each (30 us at two seconds; a stage takes 1.4).
__device__ __forceinline__ bool mbar_wait(PromptBars& bars, uint64_t* b, uint32_t parity, uint32_t stages = 0) {
  for (int i = 0; i < 64; ++i)
    if (mbar_try(b, parity)) return true;
  uint64_t start, now;
  asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(start));
  for (;;) {
    for (int i = 0; i < 16; ++i)
      if (mbar_try(b, parity)) return true;
    if (bars.stop) return false;
    asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(now));
    if (now - start > bars.limit + (bars.limit >> 16) * stages) {
      *(volatile uint32_t*)&prompt_device_fault = 1u;
      if (bars.fault != nullptr) *(volatile uint32_t*)bars.fault = 1u;
      bars.stop = 1u;
      return false;
    }
  }
}

// After a wait that ran out: waits, for a second at most, for a phase that work in flight completes by itself.
__device__ __forceinline__ void mbar_drain(uint64_t* b, uint32_t parity) {
  uint64_t start, now;
  asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(start));
  do {
    if (mbar_try(b, parity)) return;
    asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(now));
  } while (now - start < 1000000000ull);
}

// For a whole warp: one outcome for all lanes.
__device__ __forceinline__ bool mbar_wait_warp(PromptBars& bars, uint64_t* b, uint32_t parity, uint32_t stages = 0) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bars, b, parity, stages));
}

__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                          int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];\n" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
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
// S = Q K^T of 64 keys: operands are two halves of 64 columns (k_half bytes
// apart), rows of 128 bytes in groups of eight 1024 bytes apart; 16 columns
// (32 bytes) a step.
__device__ __forceinline__ void product_s(uint32_t d, uint64_t q, uint64_t k, uint32_t k_half) {
#pragma unroll
  for (int s = 0; s < 8; ++s)
    mma_ss(d, q + ((s >> 2) * (kTileBytes / 2) + (s & 3) * 32) / 16, k + ((s >> 2) * k_half + (s & 3) * 32) / 16,
           mma_word(kBlock, false), s > 0);
}
// O += P V of 64 keys: V's halves hold channels 0-63 and 64-127 of each key (N
// contiguous, groups of eight keys 1024 bytes apart); 16 keys (2048 bytes, and
// eight TMEM columns of P) a step.
__device__ __forceinline__ void product_o(uint32_t d, uint32_t p, uint64_t v, bool add) {
#pragma unroll
  for (int s = 0; s < 4; ++s) mma_ts(d, p + 8 * s, v + 2048u / 16 * s, mma_word(kD, true), add || s > 0);
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// Lengths and first tokens as the device arrays give them, held to the
// tensors: no row outside them is read or written whatever the arrays hold.
__device__ __forceinline__ void sequence(const PromptArgs& a, int s, int& lq, int& lk, int& qb, int& kb) {
  qb = a.q_begin ? clampi(a.q_begin[s], 0, a.q_tokens) : 0;
  kb = a.k_begin ? clampi(a.k_begin[s], 0, a.k_tokens) : 0;
  lq = clampi(a.q_len ? a.q_len[s] : a.q_max, 0, min(a.q_max, a.q_tokens - qb));
  lk = clampi(a.k_len ? a.k_len[s] : a.k_max, 0, min(a.k_max, a.k_tokens - kb));
}

// Item k of those that exist, numbered over the pairs of up to 32 * N
// sequences (a whole warp; lane l looks after sequences l, l + 32, ...): later
// pairs first, then the sequences that have the pair.  False for none.
template <int N>
__device__ __forceinline__ bool dense_item(const PromptArgs& a, int k, PromptItem& w) {
  const int lane = threadIdx.x & 31;
  int lq, lk, qb, kb, mine[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    lq = 0;
    if (32 * u + lane < a.S) sequence(a, 32 * u + lane, lq, lk, qb, kb);
    mine[u] = (lq + a.pair_tokens - 1) / a.pair_tokens;
  }
  const auto pairs_from = [&](int p) {  // sum over the sequences of the pairs from pair p on
    int n = 0;
#pragma unroll
    for (int u = 0; u < N; ++u) n += max(0, mine[u] - p);
    return __reduce_add_sync(0xFFFFFFFFu, n);
  };
  if (pairs_from(0) <= k) return false;
  int lo = 0, hi = a.pairs, behind = 0;  // pairs_from(lo) > k >= pairs_from(hi) = behind
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2, n = pairs_from(mid);
    if (n > k) {
      lo = mid;
    } else {
      hi = mid;
      behind = n;
    }
  }
  w.pair = lo;
  w.s = 0;
  k -= behind;  // the k-th sequence that has this pair
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const bool has = mine[u] > lo;
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, has);
    const uint32_t it = __ballot_sync(0xFFFFFFFFu, has && __popc(who & ((1u << lane) - 1u)) == k);
    if (it != 0u) w.s = 32 * u + __ffs((int)it) - 1;
    k -= __popc(who);  // negative once found
  }
  if (N == 1) {  // the lane has them
    w.lq = __shfl_sync(0xFFFFFFFFu, lq, w.s);
    w.lk = __shfl_sync(0xFFFFFFFFu, lk, w.s);
    w.qb = __shfl_sync(0xFFFFFFFFu, qb, w.s);
    w.kb = __shfl_sync(0xFFFFFFFFu, kb, w.s);
  } else {
    sequence(a, w.s, w.lq, w.lk, w.qb, w.kb);
  }
  return true;
}

// Item i of all (a whole warp): split fastest (slowest where the last one is
// shorter than the others, and so taken last), then KV head, then sequence,
// then pair, later pairs (more keys) first.  CTAs that run together then read
// different heads' keys at the same depth, and several pairs of a head share
// them in L2.  Up to kDense sequences of different lengths are numbered over
// the pairs that exist, so that long and short prompts packed together leave
// no empty CTAs; more, or equal ones, over all pairs.  False for none.
template <int TILES>
__device__ __forceinline__ bool prompt_item(const PromptArgs& a, uint32_t i, PromptItem& w) {
  constexpr int kKeys = Shape<TILES>::kKeys;
  w.split = 0;
  if (a.rounds > 1) {
    w.split = (int)(i / a.items);
    i -= w.split * a.items;
  } else if (a.splits > 1) {
    w.split = (int)(i % a.splits);
    i /= a.splits;
  }
  w.hkv = (int)(i % a.Hkv);
  i /= a.Hkv;
  if (!a.dense) {
    w.s = (int)(i % a.S);
    w.pair = a.pairs - 1 - (int)(i / a.S);
    if (w.pair < 0) return false;
    sequence(a, w.s, w.lq, w.lk, w.qb, w.kb);
  } else if (!(a.S <= 32 ? dense_item<1>(a, (int)i, w) : dense_item<kDense / 32>(a, (int)i, w))) {
    return false;
  }
  if (w.pair * a.pair_tokens >= w.lq) return false;
  w.tok0 = w.pair * a.pair_tokens;
  w.two = TILES == 2 && w.tok0 + a.tile_tokens < w.lq;
  const int last = min(w.tok0 + a.pair_tokens, w.lq) - 1;  // last query token
  const int most = w.tok0 < w.lq ? clampi(last + w.lk - w.lq + 1, 0, w.lk) : 0;
  const int least = clampi(w.tok0 + w.lk - w.lq + 1, 0, w.lk);
  const int n = (most + kKeys - 1) / kKeys;
  int per = n;
  if (a.splits > 1) per = (n + a.splits - 1) / a.splits;
  if (a.rounds > 1) {  // `rounds` of the last split take the time of one of the others
    const int large = a.splits - 1, small = max(0, n - large * a.gap) / (large * a.rounds + 1);
    per = (n - small + large - 1) / large;
  }
  w.lo = min(w.split * per, n);
  w.hi = min(w.lo + per, n);
  const int last0 = min(w.tok0 + a.tile_tokens, w.lq) - 1, most0 = min(most, clampi(last0 + w.lk - w.lq + 1, 0, w.lk));
  const auto blocks = [&](int keys) {
    return max(0, min(Shape<TILES>::kPerStage * (w.hi - w.lo), (keys - w.lo * kKeys + kBlock - 1) / kBlock));
  };
  w.blocks[0] = blocks(most0);
  w.blocks[1] = blocks(most);
  w.edge = least / kKeys;
  return true;
}

// A query row's place in lse, and among the partial results of a split.
__device__ __forceinline__ int64_t lse_place(const PromptArgs& a, int s, int token, int head) {
  return ((a.q_batched ? (int64_t)s * a.q_tokens : 0) + token) * a.Hq + head;
}
__device__ __forceinline__ int64_t part_place(const PromptArgs& a, int split, int s, int tok, int head) {
  return split * a.part_rows + ((int64_t)s * a.q_max + tok) * a.Hq + head;
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

template <int TILES>
__global__ void __launch_bounds__(Shape<TILES>::kThreads, TILES == 2 ? 1 : 2)
prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PromptArgs a) {
  using H = Shape<TILES>;
  constexpr int kStages = H::kStages;
  extern __shared__ uint8_t prompt_smem[];
  uint8_t* base = prompt_smem + ((1024u - (smem_addr(prompt_smem) & 1023u)) & 1023u);
  uint8_t* ring = base + TILES * kTileBytes;
  PromptBars& bars = *reinterpret_cast<PromptBars*>(ring + kStages * H::kStageBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int x = 0;  // the copy warp: stages filled so far
  const auto load_kv = [&](const PromptItem& w, const CUtensorMap* map, int j) {
    const int st = x % kStages;
    if (!mbar_wait(bars, &bars.kv_free[st], ((x / kStages) & 1) ^ 1)) return false;
    ++x;
    mbar_expect(&bars.kv_full[st], H::kStageBytes);
    for (int h = 0; h < 2; ++h)
      tma_load4(ring + st * H::kStageBytes + h * (H::kStageBytes / 2), map, &bars.kv_full[st], 64 * h, w.hkv,
                w.kb + (w.lo + j) * H::kKeys, a.k_batched ? w.s : 0);
    return true;
  };
  if (warp == H::kScanWarp) {
    if (lane == 0) {
      for (int i = 0; i < TILES; ++i) {
        mbar_init(&bars.q_full[i], 1);
        for (int b = 0; b < 2; ++b) {
          mbar_init(&bars.s_full[i][b], 1);
          mbar_init(&bars.p_full[i][b], 4);
        }
      }
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&bars.kv_full[i], 1);
        mbar_init(&bars.kv_free[i], TILES);
        mbar_init(&bars.v_clean[i], H::kThreads / 32 - H::kScanWarp);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.v_scan[i], 1);
        mbar_init(&bars.drained[i], 1);
      }
      bars.bad = 0;
      bars.stop = 0;
      bars.limit = a.limit;
      bars.fault = a.fault;
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    }
    __syncwarp();
    asm volatile("bar.sync 1, 64;\n" ::: "memory");
  } else if (warp == H::kCopyWarp) {
    // looks the item up while the barriers are set up, and starts the first copies before all others are ready
    if (lane == 0) {
      prefetch_map(&kmap);
      prefetch_map(&qmap);
      prefetch_map(&vmap);
    }
    __syncwarp();
    PromptItem w;
    if (!prompt_item<TILES>(a, blockIdx.x, w)) {
      w.s = -1;
      w.lo = w.hi = 0;
    }
    asm volatile("bar.sync 1, 64;\n" ::: "memory");
    if (lane == 0) {
      bars.item = w;
      if (w.hi > w.lo) {
        load_kv(w, &kmap, 0);
        for (int t = 0; t < (w.two ? 2 : 1); ++t) {
          mbar_expect(&bars.q_full[t], a.tile_tokens * a.G * kD * 2);
          for (int h = 0; h < 2; ++h)
            tma_load4(base + t * kTileBytes + h * (kTileBytes / 2), &qmap, &bars.q_full[t], 64 * h, w.hkv * a.G,
                      w.qb + w.tok0 + t * a.tile_tokens, a.q_batched ? w.s : 0);
        }
        for (int j = 1; j < H::kAhead && w.lo + j < w.hi; ++j) load_kv(w, &kmap, j);
      }
    }
    __syncwarp();
  } else if (warp == H::kProductWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(&bars.tmem)),
                 "r"(H::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  const PromptItem& w = bars.item;
  const int n = w.s < 0 ? 0 : w.hi - w.lo;  // stages of keys

  // Registers: a thread starts with 128, half of the threads do the softmax (168 + 88 = 2 * 128).
  if (warp >= H::kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    if (warp == H::kCopyWarp) {
      // ---- copies: V_j and K_j+kAhead by turns, through the ring ----
      if (lane == 0) {
        bool ok = true;
        for (int j = 0; j < n && ok; ++j) {
          ok = load_kv(w, &vmap, j);
          if (ok && j + H::kAhead < n) ok = load_kv(w, &kmap, j + H::kAhead);
        }
        bars.filled = x;
      }
    } else if (warp >= H::kProductWarp && warp < H::kProductWarp + TILES) {
      // ---- products of a tile: the whole warp walks the blocks, converged, so that operands are formed in uniform
      // registers (a lane alone issued a product every 55 cycles), and one lane issues ----
      const bool lead = elect_lane();
      const int t = __shfl_sync(0xFFFFFFFFu, warp - H::kProductWarp, 0);
      const int stages = __shfl_sync(0xFFFFFFFFu, n, 0);
      const int blocks = stages > 0 ? __shfl_sync(0xFFFFFFFFu, w.blocks[t], 0) : 0;
      const int edge = __shfl_sync(0xFFFFFFFFu, w.edge - w.lo, 0);  // the first stage to be scanned
      const bool here = __shfl_sync(0xFFFFFFFFu, t == 0 || w.two, 0);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t base_addr = __shfl_sync(0xFFFFFFFFu, smem_addr(base), 0);
      const uint64_t qd = smem_operand(base_addr + kTileBytes * t, 16, 1024);
      const uint64_t kd = smem_operand(base_addr + TILES * kTileBytes, 16, 1024);
      const uint64_t vd = smem_operand(base_addr + TILES * kTileBytes, H::kStageBytes / 2, 1024);
      const uint32_t sp = tm + 2 * kBlock * t, op = tm + 2 * kBlock * TILES + kD * t;
      constexpr uint32_t kStep = H::kStageBytes / 16, kNext = kBlock * 128 / 16;  // a stage, 64 of its rows
      uint32_t requests = 0, clean = 0;  // scans asked for; phases of v_clean
      const auto request = [&]() {
        if (t == 0 && lead) mbar_arrive(&bars.v_scan[requests & 1u]);
        ++requests;
        __syncwarp();
      };
      bool ok = true;
      int first = min(H::kAhead, stages);  // K stages of the first two blocks
      for (int k = 0; k < first && ok; ++k) ok = mbar_wait_warp(bars, &bars.kv_full[k], 0);
      if (here && blocks > 0) {  // a tile may see less than the other, or nothing
        ok = ok && mbar_wait_warp(bars, &bars.q_full[t], 0);
        if (ok && lead) {
          product_s(sp, qd, kd, H::kStageBytes / 2);
          tc_commit(&bars.s_full[t][0]);
          if (blocks > 1) product_s(sp + kBlock, qd, kd + (H::kPerStage == 2 ? kNext : kStep), H::kStageBytes / 2);
          tc_commit(&bars.s_full[t][1]);
        }
        __syncwarp();
      }
      for (int k = 0; k < first && ok; ++k)
        if (lead) {
          if (here)
            tc_commit(&bars.kv_free[k]);
          else
            mbar_arrive(&bars.kv_free[k]);  // a tile without rows only keeps step
        }
      __syncwarp();
      int x = first;
      if (edge <= 0 && stages > 0) request();
      for (int j = 0; j < stages && ok; ++j) {
        const int xv = x++, sv = xv % kStages;
        const bool more = j + H::kAhead < stages;
        const int xk = more ? x++ : xv, sk = xk % kStages;
        ok = mbar_wait_warp(bars, &bars.kv_full[sv], (xv / kStages) & 1);
        // the scan of the next stage may begin: the copy before in its place has been waited for above
        if (ok && j + 1 >= edge && j + 1 > 0 && j + 1 < stages) request();
        if (ok && j >= edge) {
          ok = mbar_wait_warp(bars, &bars.v_clean[sv], (clean >> sv) & 1u);
          clean ^= 1u << sv;
        }
        if (ok && more) ok = mbar_wait_warp(bars, &bars.kv_full[sk], (xk / kStages) & 1);
        if (!here) {
          if (ok && lead) {
            mbar_arrive(&bars.kv_free[sv]);
            if (more) mbar_arrive(&bars.kv_free[sk]);
          }
          __syncwarp();
          continue;
        }
  #pragma unroll
        for (int h = 0; h < H::kPerStage; ++h) {
          const int i = H::kPerStage * j + h, b = i & 1;
          if (i >= blocks || !ok) break;
          ok = mbar_wait_warp(bars, &bars.p_full[t][b], (i >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
            product_o(op, sp + kBlock * b, vd + kStep * sv + kNext * h, i > 0);
            if (i + 2 < blocks) product_s(sp + kBlock * b, qd, kd + kStep * sk + kNext * h, H::kStageBytes / 2);
            tc_commit(&bars.s_full[t][b]);
          }
          __syncwarp();
        }
        if (ok && lead) {
          tc_commit(&bars.kv_free[sv]);
          if (more) tc_commit(&bars.kv_free[sk]);
        }
        __syncwarp();
      }
    } else if (warp >= H::kScanWarp) {
      // ---- values in masked places: stage by stage as the first product warp asks, one ahead of its own (a wait
      // on the stage alone could take an earlier phase of its barrier for the awaited one) ----
      uint32_t scans = 0;
      const int first = min(H::kAhead, n);
      for (int j = max(w.edge - w.lo, 0); j < n; ++j, ++scans) {
        const int xv = first + j + min(j, n - first), sv = xv % kStages;
        // (the first one comes after all stages that need no scan)
        if (!mbar_wait_warp(bars, &bars.v_scan[scans & 1u], (scans >> 1) & 1u, n)) break;
        if (!mbar_wait_warp(bars, &bars.kv_full[sv], (xv / kStages) & 1)) break;
        uint4* tile = reinterpret_cast<uint4*>(ring + sv * H::kStageBytes);
        bool touched = false;
  #pragma unroll 4
        for (int i = tid - 32 * H::kScanWarp; i < H::kStageBytes / 16; i += H::kThreads - 32 * H::kScanWarp) {
          const uint4 v = tile[i];
          // 16-bit halves with an exponent of all ones
          const uint32_t m0 = __vcmpeq2(v.x & 0x7F807F80u, 0x7F807F80u), m1 = __vcmpeq2(v.y & 0x7F807F80u, 0x7F807F80u);
          const uint32_t m2 = __vcmpeq2(v.z & 0x7F807F80u, 0x7F807F80u), m3 = __vcmpeq2(v.w & 0x7F807F80u, 0x7F807F80u);
          if (m0 | m1 | m2 | m3) {
            tile[i] = make_uint4(v.x & ~m0, v.y & ~m1, v.z & ~m2, v.w & ~m3);
            touched = true;
          }
        }
        if (touched) bars.bad = 1u;
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.v_clean[sv]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n");
    if (w.s >= 0) {
      // ---- softmax and output of one tile, a thread per row ----
      const int t = warp >> 2, r = tid & 127;
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
      const uint32_t s_addr = tmem + lanes + 2 * kBlock * t, o_addr = tmem + lanes + 2 * kBlock * TILES + kD * t;
      const int tok = w.tok0 + t * a.tile_tokens + r / a.G;
      const int head = w.hkv * a.G + r % a.G;
      const bool row = r < a.tile_tokens * a.G && tok < w.lq;
      const int seen = row ? clampi(tok + w.lk - w.lq + 1, 0, w.lk) : w.lk;  // keys of this row
      const int from = w.lo * H::kKeys, blocks = w.blocks[t];
      const int masked = H::kPerStage * (w.edge - w.lo);  // the first block that some row does not see in full
      const float c = a.scale * kLog2e;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      if (t == 0 || w.two) {
        for (int i = 0; i < blocks; ++i) {
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
          if (i >= masked) {
            const int vis = seen - from - i * kBlock;
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
        if (blocks > 0 && ok) ok = mbar_wait_warp(bars, &bars.s_full[t][(blocks + 1) & 1], ((blocks + 1) >> 1) & 1);
        if (blocks == 0 && n > 0) ok = mbar_wait_warp(bars, &bars.q_full[t], 0);  // Q's place is used below
        if (ok) {
          tc_fence_after();
          const bool bad = *(volatile uint32_t*)&bars.bad != 0u;
          const int first = max(w.edge, w.lo) * H::kKeys, end = min(seen, w.hi * H::kKeys);
          // no visible key: 0; otherwise the sum is positive, or not a number when the scores are not
          const bool any = seen > from;
          const float inv = a.splits > 1 ? 1.f : (any ? 1.f / l : 0.f);
          const int64_t part = part_place(a, w.split, w.s, tok, head);
          // Through shared memory (the tile's Q has been used up), 256 bytes of every row at a time, so that a warp
          // stores whole rows: chunk c of row i of the warp lies at chunk c ^ (i % 8).
          uint4* stage = reinterpret_cast<uint4*>(base + t * kTileBytes) + (warp & 3) * 512;
          uint4* mine = stage + lane * 16;
          uint64_t out = 0;  // where the row goes
          if (row)
            out = a.splits > 1 ? (uint64_t)(a.part_o + part * kD)
                               : (uint64_t)(a.o + w.s * a.o_b + (int64_t)(w.qb + tok) * a.o_t + head * a.o_h);
          // Rolled loops: this runs once per item, and unrolled it is bound by fetching its instructions.
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float y[32];
            if (blocks > 0) {
              tmem_ld32(o_addr + 32 * q, y);
              tmem_wait_ld(y);
            }
            if (!any) {
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = 0.f;
            }
            if (bad && row) {
              const uint16_t* vr = a.v + w.s * a.v_b + (int64_t)(w.kb + first) * a.v_t + w.hkv * a.v_h + 32 * q;
              for (int key = first; key < end; ++key, vr += a.v_t) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const uint32_t e = vr[i];
                  if ((e & 0x7F80u) == 0x7F80u) y[i] += bf16_to_f32(e);
                }
              }
            }
            bool full;  // 256 bytes of every row are staged
            if (a.splits > 1) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                mine[(8 * (q & 1) + i) ^ (lane & 7)] =
                    make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), __float_as_uint(y[4 * i + 2]),
                               __float_as_uint(y[4 * i + 3]));
              full = q & 1;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mine[(4 * q + i) ^ (lane & 7)] = make_uint4(pack_bf16x2(y[8 * i] * inv, y[8 * i + 1] * inv),
                                                            pack_bf16x2(y[8 * i + 2] * inv, y[8 * i + 3] * inv),
                                                            pack_bf16x2(y[8 * i + 4] * inv, y[8 * i + 5] * inv),
                                                            pack_bf16x2(y[8 * i + 6] * inv, y[8 * i + 7] * inv));
              full = q == 3;
            }
            if (!full) continue;
            __syncwarp();
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {  // two rows at a time
              const int rr = 2 * i + (lane >> 4), cc = lane & 15;
              const uint64_t to = __shfl_sync(0xFFFFFFFFu, out, rr);
              const uint4 v = stage[rr * 16 + (cc ^ (rr & 7))];
              if (to != 0) reinterpret_cast<uint4*>(to)[(a.splits > 1 ? 16 * (q >> 1) : 0) + cc] = v;
            }
            __syncwarp();
          }
          if (row) {
            if (a.splits > 1)
              a.part_ml[part] = make_float2(any ? m * c : -INFINITY, any ? l : 0.f);
            else if (a.lse)
              a.lse[lse_place(a, w.s, w.qb + tok, head)] = any ? m * a.scale + logf(l) : -INFINITY;
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (bars.stop) {  // a wait ran out (none is left): what is in flight ends before its memory goes
    tc_fence_after();
    if (warp == H::kCopyWarp && lane == 0) {
      for (int f = max(bars.filled - kStages, 0); f < bars.filled; ++f) mbar_drain(&bars.kv_full[f % kStages], (f / kStages) & 1);
      for (int t = 0; t < (n == 0 ? 0 : w.two ? 2 : 1); ++t) mbar_drain(&bars.q_full[t], 0);
    } else if (warp >= H::kProductWarp && warp < H::kProductWarp + TILES && elect_lane()) {
      tc_commit(&bars.drained[warp - H::kProductWarp]);  // of the products that this lane issued
      mbar_drain(&bars.drained[warp - H::kProductWarp], 0);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
  }
  if (warp == H::kProductWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(H::kTmemCols) : "memory");
  }
}

// Joins the splits of a row: o = sum_z 2^(m_z - m) o_z / sum_z 2^(m_z - m) l_z,
// in a fixed order.  WARPS warps per row (sequence in blockIdx.y), each with
// eight splits at a time, four channels a lane; lane z holds split z's maximum
// and sum (two each past 32).  Four warps where there are more than eight
// splits, whose loads then take one or two turns, and the rows' CTAs fit on
// the SMs (7 each) at once: one token over 32768 keys 33.4 us against 34.9,
// over 8000 14.0 and 16.2, 16 over 4000 12.3 and 12.8; but 64 over 32768 40.4
// and 38.4.
template <int WARPS>
__global__ void __launch_bounds__(128) prompt_join_kernel(const __grid_constant__ PromptArgs a) {
  __shared__ float4 parts[WARPS][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, s = blockIdx.y;
  const int row = WARPS == 1 ? blockIdx.x * 4 + warp : blockIdx.x, part = WARPS == 1 ? 0 : warp;
  const int tok = row / a.Hq, head = row - tok * a.Hq;
  int lq, lk, qb, kb;
  sequence(a, s, lq, lk, qb, kb);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the partial results are there
  if (tok >= lq) return;
  const bool any = tok + lk - lq + 1 > 0 && lk > 0;
  float2 ml[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int z = lane + 32 * u;
    ml[u] = z < a.splits ? a.part_ml[part_place(a, z, s, tok, head)] : make_float2(-INFINITY, 0.f);
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f), x[8];
  const auto load = [&](int z0) {  // eight splits' loads in flight
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (z0 + u < a.splits)
        x[u] = reinterpret_cast<const float4*>(a.part_o + part_place(a, z0 + u, s, tok, head) * kD)[lane];
  };
  load(8 * part);
  float m = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  float f[2], l = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    f[u] = ml[u].y == 0.f ? 0.f : exp2f(ml[u].x - m);  // a sum of 0: nothing visible there
    l += f[u] * ml[u].y;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
  for (int z0 = 8 * part; z0 < a.splits; z0 += 8 * WARPS) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int z = z0 + u;
      const float g = __shfl_sync(0xFFFFFFFFu, z < 32 ? f[0] : f[1], z & 31);
      const float sum = __shfl_sync(0xFFFFFFFFu, z < 32 ? ml[0].y : ml[1].y, z & 31);
      if (z >= a.splits || sum == 0.f) continue;
      o = make_float4(o.x + g * x[u].x, o.y + g * x[u].y, o.z + g * x[u].z, o.w + g * x[u].w);
    }
    load(z0 + 8 * WARPS);
  }
  if (WARPS > 1) {
    parts[warp][lane] = o;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int u = 1; u < WARPS; ++u) {
      const float4 p = parts[u][lane];
      o = make_float4(o.x + p.x, o.y + p.y, o.z + p.z, o.w + p.w);
    }
  }
  const float inv = any ? 1.f / l : 0.f;
  uint2* po = reinterpret_cast<uint2*>(a.o + s * a.o_b + (int64_t)(qb + tok) * a.o_t + head * a.o_h) + lane;
  *po = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (lane == 0 && a.lse) a.lse[lse_place(a, s, qb + tok, head)] = any ? m * kLn2 + logf(l) : -INFINITY;
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

// Grid of a call.  One query tile per CTA where every sequence's rows fit into
// it, or where the keys are few and the tiles not more than the SMs (a 50-token
// prompt of 32 and 8 heads 6.8 us, two tiles 7.8; 300 tokens 10.0 and 10.4, 600
// the same; 300 after a history of 1700 27.9 and 23.0), else two; the items
// without splits that there can be (packed sequences share the tokens of one
// axis); and splits of the keys where these do not fill the GPU.
//
// The number of splits is the one for which this estimate is least (in ns, of
// measurements): an item costs its start and output and its 64-key blocks; a
// block takes what its products take, or its 32 KB at the rate of HBM where
// one tile streams them.  Items of one sequence within the CTAs' places end
// together; where one split more would not fit, it is made so short that the
// places left over take all items' in a few rounds by the time the others end.
// Items of several sequences are taken as they come (these are taken to be a
// little more than half as long as k_max, so rounds are not counted on), and
// the last one ends alone.  A split's partial results are written and read
// back, and joined in a launch of their own.  Measured against it: one token
// over 32768 keys 391 us in one piece, 106 in 4, 43 in 14, 38 in 28 and 41 in
// 38, over 500 keys 11.7 in one, 9.3 in 4 and 8.7 in 8; eight over up to 32768
// keys 206 in 2, 135 in 4, 108 in 7 and in 14, 120 in 28; 64 over up to 8000
// 209 in one, 184 in 3 and 200 in 8; 500 tokens over 32768 keys 373 in one, 202 in 2, 277 in 3 equal ones, 181
// in 3 of which the last takes a third of the others' time, 213 in 7 and 267
// in 14; 800 over 16384 191 in one and 163 in 2 so; a 1024-token prompt 23 in
// one and 43 in 2.
constexpr int kMaxSplits = 64;

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

struct PromptGrid {
  int tiles, tile_tokens, pair_tokens, pairs, splits, rounds, gap;
  int64_t items;
};

PromptGrid prompt_grid(const spc_prompt_dims* d) {
  PromptGrid g;
  const int G = d->Hq / d->Hkv;
  g.tile_tokens = kTile / G;
  const auto count = [&](int tiles) {
    g.tiles = tiles;
    g.pair_tokens = tiles * g.tile_tokens;
    g.pairs = (d->q_max + g.pair_tokens - 1) / g.pair_tokens;
    int64_t all = (int64_t)d->S * g.pairs;
    if (d->q.b == 0 && d->S <= kDense) all = std::min(all, d->S + (int64_t)d->q_tokens / g.pair_tokens);
    g.items = all * d->Hkv;
  };
  count(1);
  if (g.pairs > 1 && (d->k_max > 512 || g.items > spc_host::sm_count())) count(2);
  g.splits = g.rounds = 1;
  g.gap = 0;
  const int64_t places = spc_host::sm_count() * (g.tiles == 1 ? 2 : 1);
  const int64_t blocks = ((int64_t)d->k_max + kBlock - 1) / kBlock;
  const int64_t rows = (int64_t)d->S * d->q_max * d->Hq;
  // (the join numbers sequences in the grid's second dimension)
  if (g.items >= places && (g.tiles == 2 || d->S == 1 || d->S > 65535)) return g;
  double best = 0.0;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(blocks / g.tiles, kMaxSplits));
  for (int64_t z = 1; z <= most; ++z) {
    const int64_t busy = std::min(g.items * z, places), share = (blocks + z - 1) / z, start = 4000;
    const int64_t alone = g.tiles == 2 ? 690 : 760, block = g.tiles == 2 ? 690 : std::max<int64_t>(760, busy * 5);
    const int64_t whole = d->S == 1 ? blocks * block : blocks * block * 11 / 20;
    double cost = (double)g.items * (double)(whole + z * start) / (double)places + (double)(share * alone);
    int64_t rounds = 1;
    if (d->S == 1 && g.items * z <= places) {
      cost = (double)(share * block + start);
    } else if (d->S == 1 && g.items * (z - 1) < places) {
      const int64_t r = ceil_div(g.items, places - g.items * (z - 1));
      const int64_t small = (blocks - (z - 1) * (r - 1) * (start / block)) / ((z - 1) * r + 1);
      if (small >= 4) {
        cost = (double)(ceil_div(blocks - small, z - 1) * block + start);
        rounds = r;
      }
    }
    if (z > 1) cost += 3000.0 + (double)(z * rows) / 5.0;
    if (z == 1 || cost < best) {
      best = cost;
      g.splits = (int)z;
      g.rounds = (int)rounds;
      g.gap = (int)((rounds - 1) * (start / block) * kBlock / (g.tiles == 2 ? Shape<2>::kKeys : Shape<1>::kKeys));
    }
  }
  return g;
}

constexpr size_t kPromptHead = 256;  // the fault word

std::atomic<int64_t> prompt_limit{2000000000};  // of a wait in the kernels launched from now on, in ns

template <int TILES>
cudaError_t launch_prompt_k(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const PromptArgs& a,
                            int64_t grid, cudaStream_t stream) {
  static unsigned long long configured = 0ull;
  const cudaError_t e =
      spc_host::ensure_smem_limit(configured, prompt_attn_kernel<TILES>, Shape<TILES>::kSmemBytes);
  if (e != cudaSuccess) return e;
  prompt_attn_kernel<TILES><<<(unsigned)grid, Shape<TILES>::kThreads, Shape<TILES>::kSmemBytes, stream>>>(qm, km, vm, a);
  return cudaGetLastError();
}

}  // namespace

// (held to 1000 s, so that no sum of times overflows: mbar_wait)
int64_t prompt_wait_limit(int64_t ns) {
  return ns > 0 ? prompt_limit.exchange(std::min<int64_t>(ns, 1000000000000)) : prompt_limit.load();
}

cudaError_t prompt_fault_word(void** word) { return cudaGetSymbolAddress(word, prompt_device_fault); }

size_t prompt_workspace_bytes(const spc_prompt_dims* d) {
  const PromptGrid g = prompt_grid(d);
  if (g.splits == 1) return kPromptHead;
  const size_t rows = (size_t)d->S * d->q_max * d->Hq * g.splits;
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
  a.S = d->S;
  a.Hq = d->Hq;
  a.Hkv = d->Hkv;
  a.G = d->Hq / d->Hkv;
  a.q_tokens = d->q_tokens;
  a.k_tokens = d->k_tokens;
  a.q_max = d->q_max;
  a.k_max = d->k_max;
  a.scale = d->scale;
  const PromptGrid g = prompt_grid(d);
  a.tile_tokens = g.tile_tokens;
  a.pair_tokens = g.pair_tokens;
  a.pairs = g.pairs;
  // one pair each is numbered as it is: an empty sequence costs no more than looking for the others would
  a.dense = (q_len != nullptr || q_begin != nullptr) && d->S > 1 && d->S <= kDense && g.pairs > 1;
  a.splits = g.splits;
  a.rounds = g.rounds;
  a.items = (uint32_t)g.items;
  a.gap = g.gap;
  a.fault = static_cast<uint32_t*>(ws);
  a.limit = (uint64_t)prompt_limit.load(std::memory_order_relaxed);
  a.part_rows = (int64_t)d->S * d->q_max * d->Hq;
  if (a.splits > 1) {
    a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kPromptHead);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + a.part_rows * a.splits * kD);
  }
  CUtensorMap qm, km, vm;
  const int64_t kt = std::max(d->k_tokens, 1);  // no keys at all: the maps are never read through
  const uint32_t keys = g.tiles == 2 ? Shape<2>::kKeys : Shape<1>::kKeys;
  if (!encode_map(&qm, q, a.q_batched ? d->S : 1, d->q_tokens, d->Hq, d->q, a.G, a.tile_tokens) ||
      !encode_map(&km, k ? k : q, a.k_batched ? d->S : 1, kt, d->Hkv, d->k, 1, keys) ||
      !encode_map(&vm, v ? v : q, a.k_batched ? d->S : 1, kt, d->Hkv, d->v, 1, keys)) {
    spc_host::set_cuda_error(cudaErrorInvalidValue);
    return SPC_ERR_CUDA;
  }
  const int64_t grid = g.items * a.splits;
  cudaError_t e = g.tiles == 2 ? launch_prompt_k<2>(qm, km, vm, a, grid, stream)
                               : launch_prompt_k<1>(qm, km, vm, a, grid, stream);
  if (e == cudaSuccess && a.splits > 1) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int64_t rows = (int64_t)d->q_max * d->Hq;
    const bool wide = a.splits > 8 && rows * d->S <= (int64_t)spc_host::sm_count() * 7;
    cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + 3) / 4), (unsigned)d->S);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, wide ? prompt_join_kernel<4> : prompt_join_kernel<1>, a);
  }
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace spc
