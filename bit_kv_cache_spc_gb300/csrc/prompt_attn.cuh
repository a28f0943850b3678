// The attention of prompts' queries, for prompt_attn.cu (causal), window_attn.cu
// (a sliding window) and prefix_attn.cu (a shared prefix): one kernel, whose
// walk over the keys the kind of call decides.  For the last two the walk's
// 64-key blocks are two runs (PromptItem), rows and partial results leave by
// bulk copies, and the splits of an item may join in a cluster.
//
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
// of keys first.  For long walks CTAs that stay and take item after item (as
// prompt_stay.cuh's do for short ones) measured slower (a 32768-token prompt 5.68 ms against 5.43, eight single tokens over up to
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
#pragma once

#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"

namespace spc {

int64_t prompt_wait_limit(int64_t ns);  // of a wait in the kernels launched from now on; ns > 0 sets it

namespace {

// What a query sees of the keys, and so which of them a CTA walks over.
enum PromptKind {
  kPlain = 0,   // all that are not behind it
  kWindow = 1,  // of those the last `window`, and the first `sinks` of the sequence
  kPrefix = 2   // all of a prefix that the sequences share, then those of its sequence that are not behind it
};

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
  int32_t window, sinks;  // kWindow
  const uint16_t* pv;     // kPrefix: the shared rows of values, their length and most tokens
  const int32_t* p_len;
  int64_t pv_t, pv_h;
  int32_t p_tokens;
  // kPrefix with rows of all sequences together in the prefix's tiles:
  int32_t together;
  int32_t p_items, p_tiles, p_pieces;  // items of the prefix (0 in the launch of the sequences' own); CTAs' rows; splits
  int32_t p_splits;                    // of these, what is left to be joined behind the clusters
  int32_t p_bt, p_bs;                  // a tile of batched queries: p_bt tokens of p_bs sequences each (packed: 0)
  int32_t row_tiles;                   // tiles of rows in all
  int32_t p_rounds, p_gap;             // as rounds and gap, of the prefix's splits
  int32_t mixed;                       // the prefix's items walk over their sequences' own keys too
  int32_t parts;                       // not kPlain: partial results are written, to be joined
  int32_t cluster;                     // CTAs that share an item's keys and join their results (1, 2 or 4)
  int32_t o_boxes;                     // not kPlain: a warp's 32 rows are whole tokens, so that the map of o has them
  int64_t p_rows;                      // rows of the prefix's partial results; the sequences' own come behind
  // few_attn.cuh's:
  const uint16_t *q, *k;
  int64_t q_b, q_t, q_h, k_b, k_t, k_h;
  int32_t few_ctas;  // that share a sequence's keys
};

template <int KIND>
struct PromptMaps {
  CUtensorMap q, k, v, o;  // o: of a warp's 32 rows
};
template <>
struct PromptMaps<kPlain> {
  CUtensorMap q, k, v;
};
template <>
struct PromptMaps<kPrefix> {
  CUtensorMap q, k, v, o, pk, pv, qs;  // qs: of tiles with several sequences' rows
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
  // Not kPlain: the walk's 64-key blocks are two runs, the first nb0 from key 0 on (of the prefix, or of the sequence's
  // first tokens), the others from key1 of the sequence on; stages are numbered over both.
  int nb0, key1, nb;  // nb: blocks in all
  int ma, mb, mc;  // blocks that some row does not see in full: [ma, mb) and from mc on
  int prefix;      // tokens of the shared prefix
  int shared;      // rows of several sequences, the prefix's keys alone (tok0: the first token on the axis of packed
                   // queries; s: the first sequence of batched ones)
  int mixed;       // of those, the sequences whose own keys are walked as well
};

__device__ __forceinline__ int block_key(const PromptItem& w, int g) {
  return kBlock * (g < w.nb0 ? g : g - w.nb0) + (g < w.nb0 ? 0 : w.key1);
}
// Whether partial results are written, to be joined.
template <int KIND>
__device__ __forceinline__ bool in_parts(const PromptArgs& a) {
  return KIND == kPlain ? a.splits > 1 : a.parts != 0;
}

// The sequences of a mixed item, in shared memory behind the barriers: sequence s has rows in its tiles, and its keys'
// blocks are those from number g0 of the walk on.
struct MixedSeq {
  int s, qb, lq, kb, lk, g0;
};
constexpr int kMixed = 64;
template <int TILES, int KIND>
constexpr int smem_bytes() {
  return Shape<TILES>::kSmemBytes + (KIND == kPrefix ? kMixed * (int)sizeof(MixedSeq) : 0);
}
static_assert(smem_bytes<2, kPrefix>() <= 232448 && 2 * (smem_bytes<1, kPrefix>() + 1024) <= 233472,
              "more shared memory than an SM has");
// Of block g, from entry e on.
__device__ __forceinline__ int mixed_entry(const MixedSeq* table, int n, int g, int e = 0) {
  while (e + 1 < n && table[e + 1].g0 <= g) ++e;
  return e;
}

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
// The softmax warps take UNROLL = 1: with 64 tries written out at each of their
// waits, their code and the other warps' come late from the instruction cache
// (prefix attention of 8192 queries 676 to 665 us, of 17 turns 109.4 to
// 106.6; 17216 packed tokens, window 128, 160 to 147).  For the warps of the
// products they are written out: rolled, a 32768-token prompt takes 5.73 ms
// instead of 5.59.
template <int UNROLL = 64, class Bars>
__device__ __forceinline__ bool mbar_wait(Bars& bars, uint64_t* b, uint32_t parity, uint32_t stages = 0) {
#pragma unroll UNROLL
  for (int i = 0; i < 64; ++i)
    if (mbar_try(b, parity)) return true;
  uint64_t start, now;
  asm volatile("mov.u64 %0, %%globaltimer;\n" : "=l"(start));
  for (;;) {
#pragma unroll(UNROLL < 16 ? UNROLL : 16)
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
template <int UNROLL = 64, class Bars>
__device__ __forceinline__ bool mbar_wait_warp(Bars& bars, uint64_t* b, uint32_t parity, uint32_t stages = 0) {
  return __all_sync(0xFFFFFFFFu, mbar_wait<UNROLL>(bars, b, parity, stages));
}

__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                          int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];\n" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// The same with a word on how long the lines stay in L2.
__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                          int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, "
      "%5, %6}], [%2], %7;\n" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}
// Lines that are read once leave L2 first: what is read again, kernels' instructions among it, stays (64 tokens behind
// 32768 keys 76 us without, 67 with).
__device__ __forceinline__ uint64_t l2_policy(bool once) {
  uint64_t p, q;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(p));
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(q));
  return once ? p : q;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// The address of another CTA's shared memory in the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_st2(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};\n" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void cluster_st4(uint32_t addr, const float* v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
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

// Replaces the non-finite bf16 elements of the 16-byte words first, first + step, ... of n by zeros; says whether there
// was one.
__device__ __forceinline__ bool clear_non_finite(uint4* tile, int first, int n, int step) {
  bool touched = false;
#pragma unroll 4
  for (int i = first; i < n; i += step) {
    const uint4 v = tile[i];
    // an exponent of all ones carries into the sign's place
    const auto carry = [](uint32_t x) { return (x & 0x7F807F80u) + 0x00800080u; };
    if (((carry(v.x) | carry(v.y) | carry(v.z) | carry(v.w)) & 0x80008000u) == 0u) continue;
    // 16-bit halves with an exponent of all ones
    const uint32_t m0 = __vcmpeq2(v.x & 0x7F807F80u, 0x7F807F80u), m1 = __vcmpeq2(v.y & 0x7F807F80u, 0x7F807F80u);
    const uint32_t m2 = __vcmpeq2(v.z & 0x7F807F80u, 0x7F807F80u), m3 = __vcmpeq2(v.w & 0x7F807F80u, 0x7F807F80u);
    tile[i] = make_uint4(v.x & ~m0, v.y & ~m1, v.z & ~m2, v.w & ~m3);
    touched = true;
  }
  return touched;
}

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

// Item i of the prefix's, rows of all sequences together: the cluster's split fastest, then tile of rows, so that CTAs that
// run together share keys, then KV head, then the other splits.  False where no sequence has a row in the tile.
template <int TILES>
__device__ __forceinline__ bool shared_item(const PromptArgs& a, uint32_t i, PromptItem& w, MixedSeq* table) {
  constexpr int kPerStage = Shape<TILES>::kPerStage;
  const int rank = (int)(i % a.cluster);
  i /= a.cluster;
  const int lane = threadIdx.x & 31, tile = (int)(i % a.p_tiles);
  i /= a.p_tiles;
  w = PromptItem();
  w.shared = 1;
  w.hkv = (int)(i % a.Hkv);
  w.split = (int)(i / a.Hkv) * a.cluster + rank;
  const int per_tile = a.p_bt > 0 ? a.p_bs : a.tile_tokens;  // sequences or tokens
  const int first = tile * TILES * per_tile, end = first + TILES * per_tile;
  w.s = a.p_bt > 0 ? first : 0;
  w.tok0 = a.p_bt > 0 ? 0 : first;
  w.two = TILES == 2 && first + per_tile < (a.p_bt > 0 ? a.S : a.q_tokens);
  w.prefix = a.p_len ? clampi(a.p_len[0], 0, a.p_tokens) : a.p_tokens;
  w.nb = w.nb0 = w.mc = (w.prefix + kBlock - 1) / kBlock;
  bool live = false;
  if (a.mixed) {  // 64 sequences at most, two a lane: those with rows here, one behind the other
#pragma unroll
    for (int u = 0; u < kMixed / 32; ++u) {
      const int s = 32 * u + lane;
      int lq = 0, lk = 0, qb = 0, kb = 0;
      if (s < a.S) sequence(a, s, lq, lk, qb, kb);
      const bool here = lq > 0 && (a.p_bt > 0 ? s >= first && s < end : qb < end && qb + lq > first);
      // keys that its last row here sees
      const int rows = a.p_bt > 0 ? lq : min(end - qb, lq);
      int blocks = here ? (clampi(rows + lk - lq, 0, lk) + kBlock - 1) / kBlock : 0;
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, here);
      const int own = blocks;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int other = __shfl_up_sync(0xFFFFFFFFu, blocks, off);
        if (lane >= off) blocks += other;
      }
      if (here) table[w.mixed + __popc(who & ((1u << lane) - 1u))] = {s, qb, lq, kb, lk, w.nb + blocks - own};
      w.mixed += __popc(who);
      w.nb += __shfl_sync(0xFFFFFFFFu, blocks, 31);
    }
    __syncwarp();
    live = w.mixed > 0;
  } else if (a.p_bt > 0) {
    for (int s = first + lane; s < min(end, a.S); s += 32) live |= (a.q_len ? a.q_len[s] : a.q_max) > 0;
    live = __any_sync(0xFFFFFFFFu, live);
  } else {  // from where the sequence is likely to stand on, 256 sequences at a time
    const int chunks = (a.S + 255) / 256, start = (int)((int64_t)first * a.S / a.q_tokens) / 256;
    for (int c = 0; c < chunks && !live; ++c) {
      const int base = (start + c) % chunks * 256 + lane;
      bool here = false;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        int lq = 0, lk, qb = 0, kb;
        if (base + 32 * u < a.S) sequence(a, base + 32 * u, lq, lk, qb, kb);
        here |= lq > 0 && qb < end && qb + lq > first;
      }
      live = __any_sync(0xFFFFFFFFu, here);
    }
  }
  if (!live) return false;
  w.mb = w.prefix % kBlock != 0 ? w.nb0 : 0;
  w.ma = max(w.mb - 1, 0);
  const int n = (w.nb + kPerStage - 1) / kPerStage;
  int per = (n + a.p_pieces - 1) / a.p_pieces;
  if (a.p_rounds > 1) {  // the last split is shorter, as in prompt_item
    const int large = a.p_pieces - 1, small = max(0, n - large * a.p_gap) / (large * a.p_rounds + 1);
    per = (n - small + large - 1) / large;
  }
  w.lo = min(w.split * per, n);
  w.hi = min(w.lo + per, n);
  w.blocks[0] = w.blocks[1] = max(0, min(kPerStage * (w.hi - w.lo), w.nb - w.lo * kPerStage));
  return true;
}

// Item i of all (a whole warp): split fastest (slowest where the last one is
// shorter than the others, and so taken last), then KV head, then sequence,
// then pair, later pairs (more keys) first.  CTAs that run together then read
// different heads' keys at the same depth, and several pairs of a head share
// them in L2.  Up to kDense sequences of different lengths are numbered over
// the pairs that exist, so that long and short prompts packed together leave
// no empty CTAs; more, or equal ones, over all pairs.  False for none.
template <int TILES, int KIND>
__device__ __forceinline__ bool prompt_item(const PromptArgs& a, uint32_t i, PromptItem& w, MixedSeq* table) {
  constexpr int kKeys = Shape<TILES>::kKeys;
  constexpr int kPerStage = Shape<TILES>::kPerStage;
  if constexpr (KIND == kPrefix) {
    if (i < (uint32_t)a.p_items) return shared_item<TILES>(a, i, w, table);
    i -= a.p_items;
    w.shared = w.mixed = 0;
  }
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
  const int last0 = min(w.tok0 + a.tile_tokens, w.lq) - 1, most0 = min(most, clampi(last0 + w.lk - w.lq + 1, 0, w.lk));
  int n = (most + kKeys - 1) / kKeys;
  if constexpr (KIND == kWindow) {
    const int low = max(0, w.tok0 + w.lk - w.lq + 1 - a.window);  // where the first row's window begins, and the last's
    const int low_last = max(0, last + w.lk - w.lq + 1 - a.window);
    w.nb0 = (min(a.sinks, w.lk) + kBlock - 1) / kBlock;
    w.key1 = low;
    if (low <= w.nb0 * kBlock) w.nb0 = w.key1 = 0;  // the first tokens' blocks reach the windows: one run
    w.ma = 0;
    w.mb = w.nb0 + max(0, low_last - w.key1 + kBlock - 1) / kBlock;
    w.mc = w.nb0 + (least - w.key1) / kBlock;
    w.nb = most == 0 ? 0 : w.nb0 + (most - w.key1 + kBlock - 1) / kBlock;
    n = (w.nb + kPerStage - 1) / kPerStage;
  } else if constexpr (KIND == kPrefix) {
    w.prefix = a.together ? 0 : a.p_len ? clampi(a.p_len[0], 0, a.p_tokens) : a.p_tokens;
    w.nb0 = (w.prefix + kBlock - 1) / kBlock;
    w.key1 = 0;
    w.mb = w.prefix % kBlock != 0 ? w.nb0 : 0;
    w.ma = max(w.mb - 1, 0);
    w.mc = w.nb0 + least / kBlock;
    w.nb = w.nb0 + (most + kBlock - 1) / kBlock;
    n = (w.nb + kPerStage - 1) / kPerStage;
  }
  int per = n;
  if (a.splits > 1) per = (n + a.splits - 1) / a.splits;
  if (a.rounds > 1) {  // `rounds` of the last split take the time of one of the others
    const int large = a.splits - 1, small = max(0, n - large * a.gap) / (large * a.rounds + 1);
    per = (n - small + large - 1) / large;
  }
  w.lo = min(w.split * per, n);
  w.hi = min(w.lo + per, n);
  const auto blocks = [&](int keys) {
    if constexpr (KIND != kPlain) {
      const int all = KIND == kWindow && keys == 0 ? 0 : w.nb0 + max(0, keys - w.key1 + kBlock - 1) / kBlock;
      return max(0, min(kPerStage * (w.hi - w.lo), all - w.lo * kPerStage));
    }
    return max(0, min(kPerStage * (w.hi - w.lo), (keys - w.lo * kKeys + kBlock - 1) / kBlock));
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
// Partial results of the prefix's items lie before the sequences' own, tile by tile, as the CTAs' shared memory holds
// them (so that a warp's 32 rows leave in four copies): 32 rows of 32 floats after 32 rows of the next 32, each 16-byte
// chunk i of a row at i ^ (row % 8).  Number of row r of a tile, and of a token's and head's row:
__device__ __forceinline__ int64_t shared_row(const PromptArgs& a, int split, int hkv, int tile, int r) {
  return ((int64_t)(split * a.Hkv + hkv) * a.row_tiles + tile) * kTile + r;
}
__device__ __forceinline__ int64_t shared_row(const PromptArgs& a, int split, int s, int qb, int tok, int head) {
  const int unit = a.p_bt > 0 ? a.p_bs : a.tile_tokens, at = a.p_bt > 0 ? s : qb + tok, tile = at / unit;
  const int token = a.p_bt > 0 ? (at - tile * unit) * a.p_bt + tok : at - tile * unit;
  return shared_row(a, split, head / a.G, tile, token * a.G + head % a.G);
}
// Lane `lane`'s four channels of such a row.
__device__ __forceinline__ float4 shared_part(const PromptArgs& a, int64_t row, int lane) {
  const int r = (int)(row & 31);
  return reinterpret_cast<const float4*>(a.part_o)[(row - r) * (kD / 4) + (lane >> 3) * 256 + r * 8 + ((lane & 7) ^ (r & 7))];
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

template <int TILES, int KIND>
__global__ void __launch_bounds__(Shape<TILES>::kThreads, TILES == 2 ? 1 : 2)
prompt_attn_kernel(const __grid_constant__ PromptMaps<KIND> maps, const __grid_constant__ PromptArgs a) {
  using H = Shape<TILES>;
  constexpr int kStages = H::kStages;
  extern __shared__ uint8_t prompt_smem[];
  uint8_t* base = prompt_smem + ((1024u - (smem_addr(prompt_smem) & 1023u)) & 1023u);
  uint8_t* ring = base + TILES * kTileBytes;
  PromptBars& bars = *reinterpret_cast<PromptBars*>(ring + kStages * H::kStageBytes);
  MixedSeq* table = reinterpret_cast<MixedSeq*>(ring + kStages * H::kStageBytes + 512);  // kPrefix
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if constexpr (KIND == kPrefix) {  // the launch behind the prefix's waits for its results itself
    if (a.p_items > 0) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  }
  int x = 0;  // the copy warp: stages filled so far
  int at_k = 0, at_v = 0;  // and the sequence of a mixed item whose keys and values it copies
  // values: of the values' rows (else of the keys')
  const auto load_kv = [&](const PromptItem& w, bool values, int j) {
    const int st = x % kStages;
    if (!mbar_wait(bars, &bars.kv_free[st], ((x / kStages) & 1) ^ 1)) return false;
    ++x;
    mbar_expect(&bars.kv_full[st], H::kStageBytes);
    const CUtensorMap* map = values ? &maps.v : &maps.k;
    if constexpr (KIND != kPlain) {  // each block from its own place
      const uint64_t policy = KIND == kPrefix ? l2_policy(w.shared) : 0;
#pragma unroll
      for (int b = 0; b < H::kPerStage; ++b) {
        const int g = min((w.lo + j) * H::kPerStage + b, w.nb - 1);  // behind the last one it is not used: any will do
        int key = w.kb + block_key(w, g), batch = a.k_batched ? w.s : 0;
        if constexpr (KIND == kPrefix) {
          map = values ? &maps.v : &maps.k;
          if (g < w.nb0) {
            map = values ? &maps.pv : &maps.pk;
            key = g * kBlock;
            batch = 0;
          } else if (w.mixed > 0) {
            int& at = values ? at_v : at_k;
            at = mixed_entry(table, w.mixed, g, at);
            const MixedSeq& e = table[at];
            key = e.kb + (g - e.g0) * kBlock;
            batch = a.k_batched ? e.s : 0;
          }
        }
        for (int h = 0; h < 2; ++h) {
          uint8_t* to = ring + st * H::kStageBytes + h * (H::kStageBytes / 2) + b * kBlock * 128;
          if (KIND == kPrefix)
            tma_load4(to, map, &bars.kv_full[st], 64 * h, w.hkv, key, batch, policy);
          else
            tma_load4(to, map, &bars.kv_full[st], 64 * h, w.hkv, key, batch);
        }
      }
    } else {
      for (int h = 0; h < 2; ++h)
        tma_load4(ring + st * H::kStageBytes + h * (H::kStageBytes / 2), map, &bars.kv_full[st], 64 * h, w.hkv,
                  w.kb + (w.lo + j) * H::kKeys, a.k_batched ? w.s : 0);
    }
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
      prefetch_map(&maps.k);
      prefetch_map(&maps.q);
      prefetch_map(&maps.v);
      if constexpr (KIND == kPrefix) {
        prefetch_map(&maps.pk);
        prefetch_map(&maps.pv);
      }
    }
    __syncwarp();
    PromptItem w;
    if (!prompt_item<TILES, KIND>(a, blockIdx.x, w, table)) {
      w.s = -1;
      w.lo = w.hi = 0;
    }
    asm volatile("bar.sync 1, 64;\n" ::: "memory");
    if (lane == 0) {
      bars.item = w;
      if (w.hi > w.lo) {
        load_kv(w, false, 0);
        for (int t = 0; t < (w.two ? 2 : 1); ++t) {
          if constexpr (KIND == kPrefix) {
            if (w.shared && a.p_bt > 0) {
              mbar_expect(&bars.q_full[t], a.p_bt * a.p_bs * a.G * kD * 2);
              for (int h = 0; h < 2; ++h)
                tma_load4(base + t * kTileBytes + h * (kTileBytes / 2), &maps.qs, &bars.q_full[t], 64 * h, w.hkv * a.G, 0,
                          w.s + t * a.p_bs);
              continue;
            }
          }
          mbar_expect(&bars.q_full[t], a.tile_tokens * a.G * kD * 2);
          for (int h = 0; h < 2; ++h)
            tma_load4(base + t * kTileBytes + h * (kTileBytes / 2), &maps.q, &bars.q_full[t], 64 * h, w.hkv * a.G,
                      w.qb + w.tok0 + t * a.tile_tokens, a.q_batched ? w.s : 0);
        }
        for (int j = 1; j < H::kAhead && w.lo + j < w.hi; ++j) load_kv(w, false, j);
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
  // Whether some row does not see stage j of them in full.
  const auto partly = [&](int j) {
    if constexpr (KIND != kPlain) {
      const int g = (w.lo + j) * H::kPerStage, end = g + H::kPerStage;
      return (end > w.ma && g < w.mb) || end > w.mc;
    }
    return w.lo + j >= w.edge;
  };

  // Registers: a thread starts with 128, half of the threads do the softmax (168 + 88 = 2 * 128).
  if (warp >= H::kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    if (warp == H::kCopyWarp) {
      // ---- copies: V_j and K_j+kAhead by turns, through the ring ----
      if (lane == 0) {
        bool ok = true;
        if constexpr (KIND != kPlain) {
          const PromptItem here = w;  // in registers
          for (int j = 0; j < n && ok; ++j) {
            ok = load_kv(here, true, j);
            if (ok && j + H::kAhead < n) ok = load_kv(here, false, j + H::kAhead);
          }
        } else {
          for (int j = 0; j < n && ok; ++j) {
            ok = load_kv(w, true, j);
            if (ok && j + H::kAhead < n) ok = load_kv(w, false, j + H::kAhead);
          }
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
      // stages with a block of [ma, mb) or from mc on, in uniform registers
      const int from_a = KIND == kPlain ? 0 : __shfl_sync(0xFFFFFFFFu, w.ma / H::kPerStage - w.lo, 0);
      const int to_a = KIND == kPlain ? 0 : __shfl_sync(0xFFFFFFFFu, (w.mb + H::kPerStage - 1) / H::kPerStage - w.lo, 0);
      const int from_c = KIND == kPlain ? 0 : __shfl_sync(0xFFFFFFFFu, w.mc / H::kPerStage - w.lo, 0);
      const auto scanned = [&](int j) {
        if constexpr (KIND != kPlain) return (j >= from_a && j < to_a) || j >= from_c;
        return j >= edge;
      };
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
      if (stages > 0 && scanned(0)) request();
      for (int j = 0; j < stages && ok; ++j) {
        const int xv = x++, sv = xv % kStages;
        const bool more = j + H::kAhead < stages;
        const int xk = more ? x++ : xv, sk = xk % kStages;
        ok = mbar_wait_warp(bars, &bars.kv_full[sv], (xv / kStages) & 1);
        // the scan of the next stage may begin: the copy before in its place has been waited for above
        if (ok && j + 1 < stages && scanned(j + 1)) request();
        if (ok && scanned(j)) {
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
      for (int j = KIND == kPlain ? max(w.edge - w.lo, 0) : 0; j < n; ++j) {
        if (KIND != kPlain && !partly(j)) continue;
        const int xv = first + j + min(j, n - first), sv = xv % kStages;
        // (one may come after all stages that need no scan)
        if (!mbar_wait_warp(bars, &bars.v_scan[scans & 1u], (scans >> 1) & 1u, n)) break;
        ++scans;
        if (!mbar_wait_warp(bars, &bars.kv_full[sv], (xv / kStages) & 1)) break;
        uint4* tile = reinterpret_cast<uint4*>(ring + sv * H::kStageBytes);
        const bool touched = clear_non_finite(tile, tid - 32 * H::kScanWarp, H::kStageBytes / 16, H::kThreads - 32 * H::kScanWarp);
        if (touched) bars.bad = 1u;
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.v_clean[sv]);
      }
    }
    if constexpr (KIND != kPlain) {
      if (a.cluster > 1) {  // the softmax warps' (below)
        __syncwarp();
        cluster_sync();
        cluster_sync();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n");
    bool synced = KIND == kPlain || a.cluster == 1;
    if (w.s >= 0) {
      // ---- softmax and output of one tile, a thread per row ----
      const int t = warp >> 2, r = tid & 127;
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
      const uint32_t s_addr = tmem + lanes + 2 * kBlock * t, o_addr = tmem + lanes + 2 * kBlock * TILES + kD * t;
      int tok = w.tok0 + t * a.tile_tokens + r / a.G, seq = w.s;
      const int head = w.hkv * a.G + r % a.G;
      bool row = r < a.tile_tokens * a.G && tok < w.lq;
      int entry = -1, own_seen = 0;  // the row's sequence of a mixed item, and how many of its keys it sees
      if constexpr (KIND == kPrefix) {
        if (w.shared && a.p_bt > 0) {
          const int u = r / a.G;
          seq = w.s + t * a.p_bs + u / a.p_bt;
          tok = u % a.p_bt;
          row = u < a.p_bt * a.p_bs && seq < a.S;
        } else if (w.shared) {
          row = r < a.tile_tokens * a.G && tok < a.q_tokens;
        }
        if (w.mixed > 0) {
          for (int e = 0; e < w.mixed && row && entry < 0; ++e) {
            const int at = a.p_bt > 0 ? tok : tok - table[e].qb;
            if (at < 0 || at >= table[e].lq || (a.p_bt > 0 && table[e].s != seq)) continue;
            entry = e;
            own_seen = clampi(at + table[e].lk - table[e].lq + 1, 0, table[e].lk);
          }
          row = entry >= 0;
        }
      }
      const int seen = row ? clampi(tok + w.lk - w.lq + 1, 0, w.lk) : w.lk;  // keys of this row
      const int from = w.lo * H::kKeys, blocks = w.blocks[t];
      const int masked = H::kPerStage * (w.edge - w.lo);  // the first block that some row does not see in full
      const int g0 = H::kPerStage * w.lo;
      const int from_a = w.ma - g0, to_a = w.mb - g0, from_c = w.mc - g0;  // the same, for the two runs of not kPlain
      const int low = KIND == kWindow ? max(0, seen - a.window) : 0;  // where the row's window begins
      // the keys of block g that the row sees, as bits
      const auto visible = [&](int g, int& at) {  // at: the block's sequence of a mixed item, or one before it
        const auto first = [](int k) { return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1ull; };
        const int key = block_key(w, g);
        if (KIND == kPrefix && g < w.nb0) return first(w.prefix - key);
        if (KIND == kPrefix && w.mixed > 0) {
          at = mixed_entry(table, w.mixed, g, at);
          return at == entry ? first(own_seen - (g - table[at].g0) * kBlock) : 0ull;
        }
        const uint64_t m = first(seen - key);
        return KIND == kWindow ? m & (~first(low - key) | first(a.sinks - key)) : m;
      };
      const float c = a.scale * kLog2e;
      float m = -INFINITY, l = 0.f;
      int at = 0;
      bool ok = true;
      if (t == 0 || w.two) {
        for (int i = 0; i < blocks; ++i) {
          const int b = i & 1;
          const uint32_t sp = s_addr + kBlock * b;
          ok = mbar_wait_warp<1>(bars, &bars.s_full[t][b], (i >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          float x[kBlock];
          tmem_ld32(sp, x);
          tmem_ld32(sp + 32, x + 32);
          tmem_wait_ld(x);
          tmem_wait_ld(x + 32);
          if constexpr (KIND != kPlain) {
            if ((i >= from_a && i < to_a) || i >= from_c) {
              const uint64_t vis = visible(g0 + i, at);
              const uint32_t half[2] = {(uint32_t)vis, (uint32_t)(vis >> 32)};
#pragma unroll
              for (int e = 0; e < kBlock; ++e) x[e] = (half[e / 32] >> (e % 32)) & 1u ? x[e] : -INFINITY;
            }
          } else if (i >= masked) {
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
              ok = mbar_wait_warp<1>(bars, &bars.s_full[t][b ^ 1], ((i + 1) >> 1) & 1);
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
        if (blocks > 0 && ok) ok = mbar_wait_warp<1>(bars, &bars.s_full[t][(blocks + 1) & 1], ((blocks + 1) >> 1) & 1);
        if (blocks == 0 && n > 0) ok = mbar_wait_warp<1>(bars, &bars.q_full[t], 0);  // Q's place is used below
        if (ok || !synced) {
          tc_fence_after();
          const bool bad = *(volatile uint32_t*)&bars.bad != 0u;
          const int first = max(w.edge, w.lo) * H::kKeys, end = min(seen, w.hi * H::kKeys);
          // no visible key: 0; otherwise the sum is positive, or not a number when the scores are not
          const bool parts = in_parts<KIND>(a);
          const bool some_key = seen + own_seen > 0 || (KIND == kPrefix && w.prefix > 0);
          const bool any = KIND == kPlain                    ? seen > from
                           : parts || !synced || blocks == 0 ? blocks > 0 && l != 0.f
                                                             : some_key;
          const float inv = parts ? 1.f : (any ? 1.f / l : 0.f);
          int64_t part = part_place(a, w.split, w.s, tok, head);
          if constexpr (KIND == kPrefix) {
            if (w.shared) {
              const int first = a.p_bt > 0 ? w.s / a.p_bs : w.tok0 / a.tile_tokens;
              part = shared_row(a, w.split / a.cluster, w.hkv, first + t, r);
            } else if (parts) {
              part += a.p_rows;
            }
          }
          // Through shared memory (the tile's Q has been used up), 256 bytes of every row at a time, so that a warp
          // stores whole rows: chunk c of row i of the warp lies at chunk c ^ (i % 8).
          uint4* stage = reinterpret_cast<uint4*>(base + t * kTileBytes) + (warp & 3) * 512;
          uint4* mine = stage + lane * 16;
          uint64_t out = 0;  // where the row goes
          if (row)
            out = parts ? (uint64_t)(a.part_o + part * kD)
                               : (uint64_t)(a.o + (KIND == kPrefix ? seq : w.s) * a.o_b + (int64_t)(w.qb + tok) * a.o_t + head * a.o_h);
          // 32 channels of the row's sum
          const auto sums = [&](int q, float* y) {
            if (blocks > 0) {
              tmem_ld32(o_addr + 32 * q, y);
              tmem_wait_ld(y);
            }
            if (!any) {
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = 0.f;
            }
            if (KIND != kPlain && bad && row) {
              for (int j = 0; j < n; ++j) {
                if (!partly(j)) continue;
                for (int g = g0 + j * H::kPerStage; g < g0 + (j + 1) * H::kPerStage && g < g0 + blocks; ++g) {
                  int any_at = 0;
                  const uint64_t vis = visible(g, any_at);
                  const uint16_t* vr = a.v + w.s * a.v_b + (int64_t)(w.kb + block_key(w, g)) * a.v_t + w.hkv * a.v_h;
                  int64_t step = a.v_t;
                  if (KIND == kPrefix && g < w.nb0) {
                    vr = a.pv + (int64_t)(g * kBlock) * a.pv_t + w.hkv * a.pv_h;
                    step = a.pv_t;
                  } else if (KIND == kPrefix && w.mixed > 0) {
                    const MixedSeq& e = table[mixed_entry(table, w.mixed, g)];
                    vr = a.v + (a.k_batched ? e.s : 0) * a.v_b + (int64_t)(e.kb + (g - e.g0) * kBlock) * a.v_t + w.hkv * a.v_h;
                  }
                  for (int e = 0; e < kBlock; ++e) {
                    if (((vis >> e) & 1u) == 0) continue;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                      const uint32_t x = vr[e * step + 32 * q + i];
                      if ((x & 0x7F80u) == 0x7F80u) y[i] += bf16_to_f32(x);
                    }
                  }
                }
              }
            } else if (bad && row) {
              const uint16_t* vr = a.v + w.s * a.v_b + (int64_t)(w.kb + first) * a.v_t + w.hkv * a.v_h + 32 * q;
              for (int key = first; key < end; ++key, vr += a.v_t) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const uint32_t e = vr[i];
                  if ((e & 0x7F80u) == 0x7F80u) y[i] += bf16_to_f32(e);
                }
              }
            }
          };
          bool stored = false;
          if constexpr (KIND != kPlain) {
            if (!synced) {
              // ---- splits of a cluster: each CTA takes its share of the channels (64 or 32) of all rows ----
              // Once all walks have ended, the ring takes the other CTAs' (maximum, sum) of each row and their sums of these
              // channels, chunk by chunk of all rows, so that a warp writes 512 bytes in a row.
              synced = stored = true;
              constexpr int kRows = TILES * kTile;
              const int C = a.cluster, me = w.split % C, per = 4 / C, R = t * kTile + r;  // per: quarters of the channels
              const uint32_t ml_at = smem_addr(ring), o_at = ml_at + C * kRows * 8;
              const float2 own = make_float2(any ? m * c : -INFINITY, any ? l : 0.f);
              __syncwarp();
              cluster_sync();
              if (ok) {
                for (int p = 0; p < C; ++p)
                  if (p != me) cluster_st2(cluster_addr(ml_at + (me * kRows + R) * 8, p), own);
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                  const int p = q / per;
                  if (p == me) continue;
                  float y[32];
                  sums(q, y);
                  const int slot = (me < p ? me : me - 1) * per + q % per;
                  const uint32_t to = cluster_addr(o_at + (slot * 8 * kRows + R) * 16, p);
#pragma unroll
                  for (int i = 0; i < 8; ++i) cluster_st4(to + i * kRows * 16, y + 4 * i);
                }
              }
              __syncwarp();
              cluster_sync();
              if (ok) {
                const float2* ml = reinterpret_cast<const float2*>(ring) + R;
                float2 other[3];
                float top = own.x;
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                  other[u] = u < C - 1 ? ml[(u < me ? u : u + 1) * kRows] : make_float2(-INFINITY, 0.f);
                  top = fmaxf(top, other[u].x);
                }
                const auto weight = [&](float2 x) { return x.y == 0.f ? 0.f : fast_exp2(x.x - top); };  // 0: nothing visible there
                const float f0 = weight(own);
                float total = f0 * own.y;
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                  const float f = weight(other[u]);
                  total += f * other[u].y;
                  other[u].x = f;
                }
                const bool seen_any = parts ? total != 0.f : some_key;
                const float inv_all = parts ? 1.f : (seen_any ? 1.f / total : 0.f);
                const bool whole = !parts && C == 2 && a.o_boxes && !(KIND == kPrefix && w.shared && a.p_bt > 0) &&
                                   __all_sync(0xFFFFFFFFu, row);
                const bool tile_rows = parts && __any_sync(0xFFFFFFFFu, row);
#pragma unroll 1
                for (int k = 0; k < per; ++k) {
                  const int q = me * per + k;
                  float y[32];
                  sums(q, y);
#pragma unroll
                  for (int i = 0; i < 32; ++i) y[i] *= f0;
#pragma unroll
                  for (int u = 0; u < 3; ++u) {
                    if (u >= C - 1 || other[u].y == 0.f) continue;
                    const float4* from = reinterpret_cast<const float4*>(ring + C * kRows * 8) + (u * per + k) * 8 * kRows + R;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                      const float4 v = from[i * kRows];
                      y[4 * i] = fmaf(other[u].x, v.x, y[4 * i]);
                      y[4 * i + 1] = fmaf(other[u].x, v.y, y[4 * i + 1]);
                      y[4 * i + 2] = fmaf(other[u].x, v.z, y[4 * i + 2]);
                      y[4 * i + 3] = fmaf(other[u].x, v.w, y[4 * i + 3]);
                    }
                  }
                  if (parts) {  // a quarter of the tile's partial results, as below
                    if (!tile_rows) continue;
                    uint4* here = stage + k * 256;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                      here[lane * 8 + (i ^ (lane & 7))] = make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]),
                                                                     __float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3]));
                    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], 4096;\n" ::"l"(
                                       a.part_o + (part - lane) * kD + q * 1024),
                                   "r"(smem_addr(here))
                                   : "memory");
                      asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
                    }
                    continue;
                  }
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint4 v = make_uint4(pack_bf16x2(y[8 * i] * inv_all, y[8 * i + 1] * inv_all),
                                               pack_bf16x2(y[8 * i + 2] * inv_all, y[8 * i + 3] * inv_all),
                                               pack_bf16x2(y[8 * i + 4] * inv_all, y[8 * i + 5] * inv_all),
                                               pack_bf16x2(y[8 * i + 6] * inv_all, y[8 * i + 7] * inv_all));
                    if (whole)
                      stage[lane * 8 + ((4 * k + i) ^ (lane & 7))] = v;
                    else if (row)
                      reinterpret_cast<uint4*>(out)[4 * q + i] = v;
                  }
                }
                if (whole) {
                  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                  __syncwarp();
                  if (lane == 0) {
                    asm volatile(
                        "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n" ::"l"(&maps.o),
                        "r"(smem_addr(stage)), "r"(64 * me), "r"(w.hkv * a.G), "r"(w.qb + tok), "r"(a.q_batched ? w.s : 0)
                        : "memory");
                    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
                  }
                }
                if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
                if (row && me == 0) {
                  if (parts)
                    a.part_ml[part] = make_float2(top, total);
                  else if (a.lse)
                    a.lse[lse_place(a, KIND == kPrefix ? seq : w.s, w.qb + tok, head)] =
                        seen_any ? top * kLn2 + logf(total) : -INFINITY;
                }
                __syncwarp();
              }
            }
          }
          if constexpr (KIND == kPrefix) {
            // A whole tile, whatever rows it has: each warp's 8 KB hold its rows' 32 channels twice.
            if (w.shared && parts && !stored) {
              stored = true;
              float* to = a.part_o + (part - lane) * kD;
              const bool some = __any_sync(0xFFFFFFFFu, row);
#pragma unroll 1
              for (int q = 0; q < 4 && some; ++q) {
                float y[32];
                sums(q, y);
                if (q >= 2) {
                  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;\n" ::: "memory");
                  __syncwarp();
                }
                uint4* here = stage + (q & 1) * 256;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  here[lane * 8 + (i ^ (lane & 7))] = make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]),
                                                                 __float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3]));
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], 4096;\n" ::"l"(to + q * 1024),
                               "r"(smem_addr(here))
                               : "memory");
                  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
                }
              }
              if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
              __syncwarp();
            }
          }
          if constexpr (KIND != kPlain) {
            // Rows of the sequence to the warp's last one: as two boxes of 64 channels, swizzled like Q's.
            if (!stored && !parts && a.o_boxes && !(KIND == kPrefix && w.shared && a.p_bt > 0) && __all_sync(0xFFFFFFFFu, row)) {
              stored = true;
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                float y[32];
                sums(q, y);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  stage[(q >> 1) * 256 + lane * 8 + ((4 * (q & 1) + i) ^ (lane & 7))] =
                      make_uint4(pack_bf16x2(y[8 * i] * inv, y[8 * i + 1] * inv), pack_bf16x2(y[8 * i + 2] * inv, y[8 * i + 3] * inv),
                                 pack_bf16x2(y[8 * i + 4] * inv, y[8 * i + 5] * inv),
                                 pack_bf16x2(y[8 * i + 6] * inv, y[8 * i + 7] * inv));
              }
              asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
              __syncwarp();
              if (lane == 0) {
                for (int h = 0; h < 2; ++h)
                  asm volatile(
                      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n" ::"l"(&maps.o),
                      "r"(smem_addr(stage + 256 * h)), "r"(64 * h), "r"(w.hkv * a.G), "r"(w.qb + tok), "r"(a.q_batched ? w.s : 0)
                      : "memory");
                asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
              }
              __syncwarp();
            }
          }
          // Rolled loops: this runs once per item, and unrolled it is bound by fetching its instructions.
#pragma unroll 1
          for (int q = 0; q < 4 && !stored; ++q) {
            float y[32];
            sums(q, y);
            bool full;  // 256 bytes of every row are staged
            if (parts) {
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
              if (to != 0) reinterpret_cast<uint4*>(to)[(parts ? 16 * (q >> 1) : 0) + cc] = v;
            }
            __syncwarp();
          }
          if (row && !(KIND != kPlain && a.cluster > 1)) {
            if (parts)
              a.part_ml[part] = make_float2(any ? m * c : -INFINITY, any ? l : 0.f);
            else if (a.lse)
              a.lse[lse_place(a, KIND == kPrefix ? seq : w.s, w.qb + tok, head)] = any ? m * a.scale + logf(l) : -INFINITY;
          }
        }
      }
    }
    if constexpr (KIND != kPlain) {
      if (!synced) {  // a tile without rows, an item without work: the others' walks and results
        __syncwarp();
        cluster_sync();
        cluster_sync();
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
  if constexpr (KIND == kPrefix) {  // the join comes when this launch has ended, and needs both
    if (a.together && a.p_items == 0) asm volatile("griddepcontrol.wait;\n" ::: "memory");
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
template <int WARPS, int KIND>
__global__ void __launch_bounds__(128) prompt_join_kernel(const __grid_constant__ PromptArgs a) {
  __shared__ float4 parts[WARPS][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, s = blockIdx.y;
  const int row = WARPS == 1 ? blockIdx.x * 4 + warp : blockIdx.x, part = WARPS == 1 ? 0 : warp;
  const int tok = row / a.Hq, head = row - tok * a.Hq;
  int lq, lk, qb, kb;
  sequence(a, s, lq, lk, qb, kb);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the partial results are there
  if (tok >= lq) return;
  bool any = tok + lk - lq + 1 > 0 && lk > 0;
  if (KIND == kPrefix) any = any || (a.p_len ? clampi(a.p_len[0], 0, a.p_tokens) : a.p_tokens) > 0;
  const int splits = a.splits + (KIND == kPrefix ? a.p_splits : 0);
  const int shared = KIND == kPrefix ? a.p_splits : 0;  // they come first
  const auto place = [&](int z) {
    if (z < shared) return shared_row(a, z, s, qb, tok, head);
    return (KIND == kPrefix ? a.p_rows : 0) + part_place(a, z - shared, s, tok, head);
  };
  float2 ml[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int z = lane + 32 * u;
    ml[u] = z < splits ? a.part_ml[place(z)] : make_float2(-INFINITY, 0.f);
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f), x[8];
  const auto load = [&](int z0) {  // eight splits' loads in flight
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (z0 + u < shared)
        x[u] = shared_part(a, place(z0 + u), lane);
      else if (z0 + u < splits)
        x[u] = reinterpret_cast<const float4*>(a.part_o + place(z0 + u) * kD)[lane];
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
  for (int z0 = 8 * part; z0 < splits; z0 += 8 * WARPS) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int z = z0 + u;
      const float g = __shfl_sync(0xFFFFFFFFu, z < 32 ? f[0] : f[1], z & 31);
      const float sum = __shfl_sync(0xFFFFFFFFu, z < 32 ? ml[0].y : ml[1].y, z & 31);
      if (z >= splits || sum == 0.f) continue;
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

// Map of [batch][token][head][128] with the given strides: boxes of so many
// heads, tokens and sequences of half a row (64 channels, 128 bytes, swizzled).
bool encode_map(CUtensorMap* map, const uint16_t* p, int64_t batch, int64_t tokens, int64_t heads,
                const spc_layout& st, uint32_t box_heads, uint32_t box_tokens, uint32_t box_batch = 1) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  // an axis of one element is never stepped along: any valid stride does
  const auto stride = [](int64_t n, int64_t s) { return (cuuint64_t)(n > 1 ? s * 2 : kD * 2); };
  const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {stride(heads, st.h), stride(tokens, st.t), stride(batch, st.b)};
  const cuuint32_t box[4] = {64, box_heads, box_tokens, box_batch}, step[4] = {1, 1, 1, 1};
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

// What a call's sequences see, for the grid.
struct PromptRule {
  int32_t window = 0, sinks = 0;  // kWindow
  int32_t prefix = 0;             // kPrefix: most tokens of it
  // most keys that an item of so many query tokens walks over
  int64_t keys(const spc_prompt_dims* d, int pair_tokens) const {
    const int64_t sink_keys = ceil_div(std::min(sinks, d->k_max), kBlock) * kBlock;
    return window > 0 ? std::min<int64_t>(d->k_max, (int64_t)window + pair_tokens - 1 + sink_keys) : (int64_t)prefix + d->k_max;
  }
  // time of the blocks of an item on average, where the longest has `blocks` of `block` ns
  int64_t average(const spc_prompt_dims* d, int64_t blocks, int64_t block) const {
    if (window > 0 && 2 * (int64_t)window < d->k_max) return blocks * block * 9 / 10;  // most windows are full
    const int64_t all = prefix / kBlock;
    return all * block + (blocks - all) * block * 11 / 20;
  }
};

struct PromptGrid {
  int tiles, tile_tokens, pair_tokens, pairs, splits, rounds, gap;
  int cluster = 1;  // CTAs that join an item's splits on the chip
  int64_t items;
  // kPrefix with all sequences' rows together:
  int p_tiles = 0, p_pieces = 0, p_splits = 0, p_bt = 0, p_bs = 0, p_rounds = 1, p_gap = 0;
  bool p_two = false;  // two-tile CTAs
  bool mixed = false;  // these walk over the own keys too
  int64_t p_rows = 0, p_items = 0;
};

PromptGrid prompt_grid(const spc_prompt_dims* d, const PromptRule& rule) {
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
  if (g.pairs > 1 && (rule.keys(d, 2 * g.tile_tokens) > 512 || g.items > spc_host::sm_count())) count(2);
  g.splits = g.rounds = 1;
  g.gap = 0;
  const int64_t places = spc_host::sm_count() * (g.tiles == 1 ? 2 : 1);
  const int64_t blocks = ceil_div(rule.keys(d, g.pair_tokens), kBlock);
  const int64_t rows = (int64_t)d->S * d->q_max * d->Hq;
  // (the join numbers sequences in the grid's second dimension)
  if (g.items >= places && (g.tiles == 2 || d->S == 1 || d->S > 65535)) return g;
  double best = 0.0;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(blocks / g.tiles, kMaxSplits));
  for (int64_t z = 1; z <= most; ++z) {
    const int64_t busy = std::min(g.items * z, places), share = (blocks + z - 1) / z, start = 4000;
    const int64_t alone = g.tiles == 2 ? 690 : 760, block = g.tiles == 2 ? 690 : std::max<int64_t>(760, busy * 5);
    const int64_t whole = d->S == 1 ? blocks * block : rule.average(d, blocks, block);
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
    const bool cluster = (rule.window > 0 || rule.prefix > 0) && rounds == 1 && (z == 2 || z == 4);
    if (z > 1) cost += cluster ? 1500.0 : 3000.0 + (double)(z * rows) / 5.0;
    if (z == 1 || cost < best) {
      best = cost;
      g.cluster = cluster ? (int)z : 1;
      g.splits = (int)z;
      g.rounds = (int)rounds;
      g.gap = (int)((rounds - 1) * (start / block) * kBlock / (g.tiles == 2 ? Shape<2>::kKeys : Shape<1>::kKeys));
    }
  }
  return g;
}

// Whether a call's queries are single tokens of few heads: few_attn.cuh's.
constexpr int kFewRows = 16;  // of its products
bool few_rows(const spc_prompt_dims* d) { return d->q_max == 1 && d->Hq / d->Hkv <= kFewRows; }

// Grid of a call behind a prefix whose tiles hold the rows of all sequences
// together, so that the prefix's keys are walked once for them and not once for
// each (two-tile CTAs where the rows fill more than one tile).  The sequences'
// own keys come in the same walk, masked for the rows of the others (`mixed`,
// up to 64 sequences: 17 prompts of up to 77 tokens behind 8011 keys 104 us, in
// a launch of their own and joined 118; 40 of 20 tokens 88 and 102), or for
// more sequences, and for single tokens, in a launch of their own.
// p_items = 0 where that does not pay: the sequences' own tiles are as few, or
// the partial results cost more than what is saved.
//
// Of the splits of the walk, the number with the least estimate (in ns): the
// items taken in turns by the CTAs' places, or the last split shorter as in
// prompt_grid, and the partial results.  Own keys in a launch of their own are
// split where their items would take longer than one of the prefix's.  Measured
// against it: the 17 prompts 104 us in 2 (129 in equal ones), 106 in 3, 121 in
// 4; the 40 127 in one piece, 88 in 2, 111 and 98; 64 single tokens behind 32768
// keys 126 in 4, 76 in 9, 62 in 18.
PromptGrid together_grid(const spc_prompt_dims* d, const PromptRule& rule) {
  PromptGrid g = {};
  const int G = d->Hq / d->Hkv, sms = spc_host::sm_count();
  const bool batched = d->q.b != 0 && d->S > 1, few = few_rows(d);
  g.tiles = 1;
  g.tile_tokens = g.pair_tokens = kTile / G;
  if ((d->S < 2 && !few) || d->S > 65535 || d->q_max == 0 || rule.prefix == 0) return g;
  if (batched ? 2 * d->q_max > g.tile_tokens : d->q_tokens > 4 * (int64_t)d->S * d->q_max) return g;  // tiles with few rows
  g.pairs = (int)ceil_div(d->q_max, g.tile_tokens);
  int64_t tokens = (int64_t)d->S * d->q_max, own_tiles = (int64_t)d->S * g.pairs, tiles;
  if (batched) {
    g.p_bt = d->q_max;
    g.p_bs = g.tile_tokens / d->q_max;
    tiles = ceil_div(d->S, g.p_bs);
  } else {
    tokens = std::min<int64_t>(tokens, d->q_tokens);
    tiles = ceil_div(d->q_tokens, g.tile_tokens);
    if (d->S <= kDense) own_tiles = std::min(own_tiles, d->S + (int64_t)d->q_tokens / g.tile_tokens);
  }
  g.items = few ? 0 : own_tiles * d->Hkv;
  g.rounds = 1;
  // (a long prefix also with one: the larger ring hides more of HBM's latency; 32 tokens behind 32768 keys 47.9 to 45.0 us)
  g.p_two = tiles > 1 || ceil_div(rule.prefix, kBlock) * d->Hkv > 8 * sms;
  const int two = g.p_two ? 2 : 1;
  g.p_tiles = (int)ceil_div(tiles, two);
  const int64_t shared = (int64_t)d->Hkv * g.p_tiles * two * kTile;  // rows of partial results per split
  const int64_t items = (int64_t)g.p_tiles * d->Hkv, start = 8000, places = sms * (g.p_two ? 1 : 2);
  if (items > (1 << 24)) return g;
  const int64_t blocks = ceil_div(rule.prefix, kBlock), own = ceil_div(d->k_max, kBlock);
  // sequences with rows in a CTA's tiles, and their blocks (lengths are taken to be a little more than half of k_max)
  const int64_t here = batched ? std::min<int64_t>(d->S, (int64_t)g.p_bs * two)
                               : std::min<int64_t>(d->S, (int64_t)two * g.tile_tokens * d->S / d->q_tokens + 1);
  const int64_t inside = here * ceil_div(own * 11, 20);
  // In the walk the own keys' blocks take nearly twice the others' time: masked in every row, their values looked through.
  // (64 sequences of 4 tokens behind 32768 keys, 16 a CTA with up to 1024 keys each: 188 us so, 149 in a launch of their own.)
  const double within = (double)(items * inside * 2 * 690) / sms;
  const double behind = (double)(g.items * (4000 + own * 760 * 11 / 20)) / (2 * sms) + (double)(tokens * d->Hq) / 5.0 + 8000.0;
  g.mixed = d->S <= kMixed && !few && within <= behind;
  const int64_t walk = blocks + (g.mixed ? inside : 0);
  double best = 0.0;
  for (int64_t z = 1; z <= std::min<int64_t>(walk, few || g.mixed ? kMaxSplits : kMaxSplits / 2); ++z) {
    const int64_t share = ceil_div(walk, z);
    const int64_t oz = few || g.mixed ? 0 : std::min<int64_t>(std::max<int64_t>(1, ceil_div(own, share)), kMaxSplits / 2);
    const int64_t block = std::max<int64_t>(g.p_two ? 690 : 760, std::min(items * z, places) * 5 / std::min(g.p_tiles, 2));
    double cost = (double)(ceil_div(items * z, places) * (start + share * block));
    int64_t rounds = 1;
    int64_t gap = 0;
    if (z > 1 && items * z > places && items * (z - 1) < places) {  // the last split shorter, in a few rounds on what is left
      const int64_t r = ceil_div(items, places - items * (z - 1)), behind = g.mixed ? inside : 0;
      const int64_t less = (r - 1) * (start / block) + r * behind;  // what its starts and own keys take besides
      const int64_t small = (walk - (z - 1) * less) / ((z - 1) * r + 1);
      const int64_t last = r * (start + (small + std::min(behind, small)) * block);
      const double one = (double)std::max(start + ceil_div(walk - small, z - 1) * block, last);
      if (small >= 4 && one < cost) {
        cost = one;
        rounds = r;
        gap = less;
      }
    }
    if (oz > 0) cost += (double)(g.items * (oz * 4000 + own * 760 * 11 / 20)) / (2 * sms);
    // Splits that join on the chip, in whole clusters of a GPC's SMs (not single tokens', whose next launch joins what there
    // is in any case: five behind 2003 keys 12.8 us, 18.0 so).
    for (int64_t cluster = 1; cluster <= 4; cluster *= 2) {
      if (z % cluster != 0 || (cluster > 1 && (few || rounds > 1 || items * z > places * (20 - cluster) / 19))) break;
      const int64_t left = z / cluster;
      double all = cost + (cluster > 1 ? 1500.0 : 0.0);
      if (!g.mixed || left > 1) all += 6000.0 + ((double)(left * shared) + (double)(oz * tokens * d->Hq)) / 5.0;
      if (best == 0.0 || all < best) {
        best = all;
        g.cluster = (int)cluster;
        g.p_pieces = (int)z;
        g.p_splits = (int)left;
        g.splits = (int)oz;
        g.p_rounds = (int)rounds;
        g.p_gap = (int)(gap / two);  // stages have two blocks where CTAs have two tiles
      }
    }
  }
  if (g.mixed) g.items = 0;
  g.p_rows = g.mixed && g.p_splits == 1 ? 0 : shared * g.p_splits;
  // against the sequences one by one, whose tiles walk over the prefix each
  const bool pairs = g.pairs > 1;
  int64_t own_pairs = (int64_t)d->S * ceil_div(d->q_max, 2 * g.tile_tokens);
  if (!batched && d->S <= kDense) own_pairs = std::min(own_pairs, d->S + (int64_t)d->q_tokens / (2 * g.tile_tokens));
  const int64_t each = blocks + own * 11 / 20, alone = (pairs ? own_pairs : own_tiles) * d->Hkv;
  const int64_t one = pairs ? 690 : 760, room = pairs ? sms : 2 * sms;
  double apart = (double)(ceil_div(alone, room) * (start + each * one));
  if (alone < room / 2) apart = (double)(alone * each * one) / (double)room + 12000.0;  // its keys split
  // (pairs of tiles that are nearly as many: four prompts of up to 2048 tokens behind 16384 keys 709 us together, 668 apart)
  const bool as_many = pairs && 10 * (int64_t)g.p_tiles > 9 * own_pairs;
  // Single tokens: always (one to 16 behind 2003 keys 12.4 to 13.3 us together, 15 to 27 apart).
  if (few || (1.1 * best < apart && !as_many)) g.p_items = items * g.p_pieces;
  return g;
}

// Whether a call takes that grid (placed: with a q_begin).
bool taken_together(const spc_prompt_dims* d, const PromptGrid& g, bool placed) {
  return g.p_items > 0 && !(d->q.b != 0 && placed);
}

constexpr size_t kPromptHead = 256;  // the fault word

int64_t part_rows(const spc_prompt_dims* d, const PromptGrid& g) {
  return g.p_rows + (int64_t)d->S * d->q_max * d->Hq * g.splits;
}

size_t prompt_bytes(const spc_prompt_dims* d, const PromptRule& rule) {
  PromptGrid g = prompt_grid(d, rule);
  int64_t rows = g.splits > 1 && g.cluster == 1 ? part_rows(d, g) : 0;
  if (rule.prefix > 0) {  // (batched queries with first tokens of their own are not taken together)
    g = together_grid(d, rule);
    if (g.p_items > 0) rows = d->q.b != 0 ? std::max(rows, part_rows(d, g)) : part_rows(d, g);
  }
  return kPromptHead + (size_t)rows * (kD * sizeof(float) + sizeof(float2));
}

// early: may start while the launch before it runs (which says when, and is waited for in the kernel).
template <int TILES, int KIND>
cudaError_t launch_prompt_k(const PromptMaps<KIND>& maps, const PromptArgs& a, int64_t grid, cudaStream_t stream,
                            bool early = false) {
  static unsigned long long configured = 0ull;
  const cudaError_t e =
      spc_host::ensure_smem_limit(configured, prompt_attn_kernel<TILES, KIND>, smem_bytes<TILES, KIND>());
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2] = {};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(Shape<TILES>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<TILES, KIND>();
  cfg.stream = stream;
  cfg.attrs = attr;
  if (early) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
  }
  if (a.cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)a.cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, prompt_attn_kernel<TILES, KIND>, maps, a);
}

// Whether two-tile CTAs stay and take item after item (prompt_stay.cuh), or
// leave and the next one starts wherever there is a place.  Staying saves a part
// of each item's start and output, but fixes which CTA takes which items: what
// one CTA has more of than the others counts the less the more items it takes
// and the shorter they are.  32 and 8 heads, us leaving and staying, by items a
// CTA: 1.7 (2048 tokens), window 128 24.6 and 21.6, 1024 36.6 and 39.5; 3.4,
// window 512 58 and 53, 1024 71 and 72; 6.7, window 1024 141 and 133, 2048 203
// and 204; 13.5, window 1024 278 and 259, 2048 423 and 421; 27, window 128 277
// and 196, 2048 865 and 847, 4096 1490 and 1515.
bool stays(const spc_prompt_dims* d, const PromptRule& rule, const PromptGrid& g) {
  const int64_t sms = spc_host::sm_count(), keys = rule.keys(d, g.pair_tokens);
  return g.tiles == 2 && g.splits == 1 && g.items > sms && keys <= 2560 && keys * sms <= 256 * g.items;
}

// What the caller gives besides the shape; pk, pv, p: kPrefix.
struct PromptTensors {
  const uint16_t *q, *k, *v;
  const int32_t *q_begin, *q_len, *k_begin, *k_len;
  uint16_t* o;
  float* lse;
  void* ws;
  const uint16_t *pk = nullptr, *pv = nullptr;
  const int32_t* p_len = nullptr;
  const spc_prefix* p = nullptr;
};

PromptArgs prompt_args(const spc_prompt_dims* d, const PromptRule& rule, const PromptTensors& x) {
  PromptArgs a = {};
  a.q = x.q;
  a.k = x.k;
  a.q_b = d->q.b;
  a.q_t = d->q.t;
  a.q_h = d->q.h;
  a.k_b = d->k.b;
  a.k_t = d->k.t;
  a.k_h = d->k.h;
  a.v = x.v;
  a.o = x.o;
  a.lse = x.lse;
  a.q_begin = x.q_begin;
  a.q_len = x.q_len;
  a.k_begin = x.k_begin;
  a.k_len = x.k_len;
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
  a.window = rule.window;
  a.sinks = rule.sinks;
  if (x.p != nullptr) {
    a.pv = x.pv;
    a.pv_t = x.p->v.t;
    a.pv_h = x.p->v.h;
    a.p_tokens = x.p->tokens;
    a.p_len = x.p_len;
  }
  a.fault = static_cast<uint32_t*>(x.ws);
  a.limit = (uint64_t)prompt_wait_limit(0);
  a.part_rows = (int64_t)d->S * d->q_max * d->Hq;
  a.splits = a.rounds = 1;
  return a;
}

// few: the launch of single tokens' own keys, with what joins them with the prefix; stay: of CTAs that take item after item.
template <int KIND>
spc_status launch_prompt(const spc_prompt_dims* d, const PromptRule& rule, const PromptTensors& x, cudaStream_t stream,
                         spc_status (*few)(PromptArgs&, const spc_prompt_dims*, cudaStream_t) = nullptr,
                         cudaError_t (*stay)(const PromptMaps<KIND>&, const PromptArgs&, cudaStream_t) = nullptr) {
  PromptArgs a = prompt_args(d, rule, x);
  PromptGrid g = prompt_grid(d, rule);
  if constexpr (KIND == kPrefix) {
    const PromptGrid all = together_grid(d, rule);
    a.together = taken_together(d, all, x.q_begin != nullptr);
    if (a.together) g = all;
    a.p_items = (int32_t)g.p_items;
    a.p_tiles = g.p_tiles;
    a.p_pieces = g.p_pieces;
    a.p_splits = g.p_splits;
    a.p_rounds = g.p_rounds;
    a.p_gap = g.p_gap;
    a.p_bt = g.p_bt;
    a.p_bs = g.p_bs;
    a.p_rows = g.p_rows;
    a.mixed = a.together && g.mixed;
    a.row_tiles = g.p_tiles * (g.p_two ? 2 : 1);
  }
  a.tile_tokens = g.tile_tokens;
  a.pair_tokens = g.pair_tokens;
  a.pairs = g.pairs;
  // one pair each is numbered as it is: an empty sequence costs no more than looking for the others would
  a.dense = (x.q_len != nullptr || x.q_begin != nullptr) && d->S > 1 && d->S <= kDense && g.pairs > 1;
  a.splits = g.splits;
  a.rounds = g.rounds;
  a.items = (uint32_t)g.items;
  a.gap = g.gap;
  a.cluster = KIND == kPlain ? 1 : g.cluster;
  const bool parts = a.together ? !(a.mixed && a.p_splits == 1) : a.splits > 1 && a.cluster == 1;
  a.parts = parts;
  if (parts) {
    a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(x.ws) + kPromptHead);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + part_rows(d, g) * kD);
  }
  PromptMaps<KIND> maps;
  const int64_t kt = std::max(d->k_tokens, 1);  // no keys at all: the maps are never read through
  const uint32_t keys = KIND == kPlain && g.tiles == 2 ? Shape<2>::kKeys : kBlock;
  bool ok = encode_map(&maps.q, x.q, a.q_batched ? d->S : 1, d->q_tokens, d->Hq, d->q, a.G, a.tile_tokens) &&
            encode_map(&maps.k, x.k ? x.k : x.q, a.k_batched ? d->S : 1, kt, d->Hkv, d->k, 1, keys) &&
            encode_map(&maps.v, x.v ? x.v : x.q, a.k_batched ? d->S : 1, kt, d->Hkv, d->v, 1, keys);
  if constexpr (KIND != kPlain) {
    a.o_boxes = a.G <= 32 && 32 % a.G == 0;
    ok = ok && encode_map(&maps.o, x.o, a.q_batched ? d->S : 1, d->q_tokens, d->Hq, d->o, a.o_boxes ? a.G : 1,
                          a.o_boxes ? 32 / a.G : 1);
  }
  if constexpr (KIND == kPrefix) {
    ok = ok && encode_map(&maps.pk, x.pk, 1, x.p->tokens, d->Hkv, x.p->k, 1, keys) &&
         encode_map(&maps.pv, x.pv, 1, x.p->tokens, d->Hkv, x.p->v, 1, keys) &&
         encode_map(&maps.qs, x.q, a.q_batched ? d->S : 1, d->q_tokens, d->Hq, d->q, a.G, std::max(a.p_bt, 1),
                    std::max(a.p_bs, 1));
  }
  if (!ok) {
    spc_host::set_cuda_error(cudaErrorInvalidValue);
    return SPC_ERR_CUDA;
  }
  cudaError_t e = cudaSuccess;
  if (a.together) {
    e = g.p_two ? launch_prompt_k<2, KIND>(maps, a, g.p_items, stream) : launch_prompt_k<1, KIND>(maps, a, g.p_items, stream);
    if (e == cudaSuccess && g.items == 0 && !a.mixed) return few(a, d, stream);
    a.p_items = 0;
    a.cluster = 1;
  }
  const int64_t grid = g.items * a.splits;
  if (e == cudaSuccess && stay != nullptr && stays(d, rule, g))
    e = stay(maps, a, stream);
  else if (e == cudaSuccess && grid > 0)
    e = g.tiles == 2 ? launch_prompt_k<2, KIND>(maps, a, grid, stream)
                     : launch_prompt_k<1, KIND>(maps, a, grid, stream, a.together);
  if (e == cudaSuccess && parts) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int64_t rows = (int64_t)d->q_max * d->Hq;
    const bool wide = a.splits + a.p_splits > 8 && rows * d->S <= (int64_t)spc_host::sm_count() * 7;
    cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + 3) / 4), (unsigned)d->S);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, wide ? prompt_join_kernel<4, KIND> : prompt_join_kernel<1, KIND>, a);
  }
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace
}  // namespace spc
