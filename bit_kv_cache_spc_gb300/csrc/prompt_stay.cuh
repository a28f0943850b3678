// The kernel of prompt_attn.cuh for many items of short walks (sliding
// windows): two-tile CTAs that stay, one on each SM, and take item after item
// (item i, i + CTAs, ...), so that an item's lookup and first copies lie under
// the softmax and output of the one before.
//
// What it takes beside that kernel: items handed over in two places; Q copied
// again once the tile's last scores have been formed; output staged apart from
// Q (32 KB, 64 channels at a time), for which the ring has four stages instead
// of five; barriers that count on through all items.
// The order of the products on the tensor cores keeps buffers apart: the next
// item's first scores come behind the last product of this one's weights, its
// first sum of values behind the softmax warps' reads of O, as they form the
// weights that it takes.
//
// 17216 packed tokens of 32 ungrouped heads, window 128: 180 us by CTAs that
// leave, 142 so (564 MB: 59% of the copy rate); of 8 KV heads 146 and 93; 32768
// tokens of 32 and 8 heads 274 and 196.  Bound by the chain of an item: where
// heads are grouped 6 us for four blocks, 3.4 of them the softmax, 1.9 from the
// last product until the rows are stored, 0.6 until the next item's scores.
// Measured against it: the next item looked up by a warp of its own 160 us where
// this took 160.5, and a window of 4096 1.50 ms instead of 1.47; looked up
// before the last copies of this one 170; the output's 64 channels held in
// registers until what was staged before has left 159, and the long window
// 1.50.
#pragma once

#include "prompt_attn.cuh"

namespace spc {
namespace {

constexpr int kStayStages = 4;
constexpr int kStayStaging = 8 * 4096;  // 32 rows of 128 bytes for each softmax warp
constexpr int kStaySmemBytes = 2 * kTileBytes + kStayStages * Shape<2>::kStageBytes + kStayStaging + 1024 + 1024;
static_assert(kStaySmemBytes <= 232448, "more shared memory than an SM has");

struct __align__(16) StayBars {
  PromptItem item[2];
  uint64_t item_full[2], item_free[2];
  uint64_t q_full[2], q_free[2];  // q_free: a copied tile's last scores have been formed (once for each copy)
  uint64_t kv_full[kStayStages], kv_free[kStayStages];
  uint64_t v_scan[2], v_clean[kStayStages];
  uint64_t s_full[2][2], p_full[2][2];
  uint64_t s_seen[2];  // the tile's softmax warps have seen an item's last product end: the next item's scores may say so too
  uint64_t drained[2];
  uint64_t limit;
  uint32_t* fault;
  int filled, q_filled[2];  // stages and Q tiles copied in all
  uint32_t tmem;
  uint32_t bad[2];          // a masked stage of the item held a non-finite value
  volatile uint32_t stop;
  int first1[2];            // AHEAD: the item's first stage with keys that the second tile sees
};
static_assert(sizeof(StayBars) <= 1024, "barriers outgrow their place");

// 16 consecutive TMEM columns of the thread's lane, loaded.
__device__ __forceinline__ void tmem_get16(uint32_t addr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]),
                 "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
               :
               : "memory");
}

// AHEAD: the second tile may have stages in front that none of its rows sees; it
// leaves them out (17216 packed tokens of 32 ungrouped heads, window 128, whose
// items have six blocks for tiles that see four: 147 to 142 us, window 1024 279
// to 273; in the kernel of all calls grouped heads lose 2 to 4%).
template <bool AHEAD>
__global__ void __launch_bounds__(Shape<2>::kThreads, 1)
stay_attn_kernel(const __grid_constant__ PromptMaps<kWindow> maps, const __grid_constant__ PromptArgs a) {
  using H = Shape<2>;
  constexpr int kStages = kStayStages;
  constexpr int kScanWarps = H::kThreads / 32 - H::kScanWarp;
  extern __shared__ uint8_t prompt_smem[];
  uint8_t* base = prompt_smem + ((1024u - (smem_addr(prompt_smem) & 1023u)) & 1023u);
  uint8_t* ring = base + 2 * kTileBytes;
  uint8_t* staging = ring + kStages * H::kStageBytes;
  StayBars& bars = *reinterpret_cast<StayBars*>(staging + kStayStaging);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == H::kScanWarp) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.item_full[i], 1);
        mbar_init(&bars.item_free[i], H::kSoftmaxWarps + 2 + kScanWarps);
        mbar_init(&bars.q_full[i], 1);
        mbar_init(&bars.q_free[i], 1);
        mbar_init(&bars.v_scan[i], 1);
        mbar_init(&bars.s_seen[i], 4);
        mbar_init(&bars.drained[i], 1);
        for (int b = 0; b < 2; ++b) {
          mbar_init(&bars.s_full[i][b], 1);
          mbar_init(&bars.p_full[i][b], 4);
        }
        bars.q_filled[i] = 0;
        bars.bad[i] = 0;
      }
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&bars.kv_full[i], 1);
        mbar_init(&bars.kv_free[i], 2);
        mbar_init(&bars.v_clean[i], kScanWarps);
      }
      bars.filled = 0;
      bars.stop = 0;
      bars.limit = a.limit;
      bars.fault = a.fault;
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    }
    __syncwarp();
  } else if (warp == H::kCopyWarp) {
    if (lane == 0) {
      prefetch_map(&maps.k);
      prefetch_map(&maps.q);
      prefetch_map(&maps.v);
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
  const uint32_t skip = a.items / gridDim.x;  // items without rows that may be looked up on the way to the next one
  // Whether some row does not see stage j of an item in full.
  const auto partly = [](const PromptItem& w, int j) {
    const int g = (w.lo + j) * H::kPerStage, end = g + H::kPerStage;
    return (end > w.ma && g < w.mb) || end > w.mc;
  };
  // A role is done with item `it`.
  const auto leave = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.item_free[it & 1]);
  };

  if (warp >= H::kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    if (warp == H::kCopyWarp) {
      // ---- items and copies ----
      int x = 0, q_copied[2] = {0, 0};
      bool ok = true;
      uint32_t next = blockIdx.x;
      for (int it = 0, walk = 0; ok; ++it) {
        PromptItem w;
        bool have = false;
        while (!have && next < a.items) {  // items without rows are left out
          have = prompt_item<2, kWindow>(a, next, w, nullptr);
          next += gridDim.x;
        }
        if (!have) w.s = -1;
        if (it >= 2) ok = mbar_wait_warp(bars, &bars.item_free[it & 1], ((it >> 1) - 1) & 1, walk);
        if (!ok) break;
        const int n = have ? w.hi - w.lo : 0;
        if (lane == 0) {
          bars.item[it & 1] = w;
          if constexpr (AHEAD) {
            const int low = w.tok0 + a.tile_tokens + w.lk - w.lq + 1 - a.window;  // where its first row's window begins
            bars.first1[it & 1] = n > 1 && w.two ? clampi((low - w.key1) / H::kKeys, 0, n - 1) : 0;
          }
          bars.bad[it & 1] = 0;
          mbar_arrive(&bars.item_full[it & 1]);
          const auto load_kv = [&](bool values, int j) {
            const int st = x % kStages;
            if (!mbar_wait(bars, &bars.kv_free[st], ((x / kStages) & 1) ^ 1)) return false;
            ++x;
            mbar_expect(&bars.kv_full[st], H::kStageBytes);
#pragma unroll
            for (int b = 0; b < H::kPerStage; ++b) {
              const int g = min((w.lo + j) * H::kPerStage + b, w.nb - 1);  // behind the last one it is not used: any will do
              for (int h = 0; h < 2; ++h)
                tma_load4(ring + st * H::kStageBytes + h * (H::kStageBytes / 2) + b * kBlock * 128, values ? &maps.v : &maps.k,
                          &bars.kv_full[st], 64 * h, w.hkv, w.kb + block_key(w, g), a.k_batched ? w.s : 0);
            }
            return true;
          };
          if (n > 0) {
            ok = load_kv(false, 0);
            for (int t = 0; t < 2 && ok; ++t) {
              if (t == 1 && !w.two) continue;
              if (q_copied[t] > 0) ok = mbar_wait(bars, &bars.q_free[t], (q_copied[t] - 1) & 1, walk);
              if (!ok) break;
              ++q_copied[t];
              mbar_expect(&bars.q_full[t], a.tile_tokens * a.G * kD * 2);
              for (int h = 0; h < 2; ++h)
                tma_load4(base + t * kTileBytes + h * (kTileBytes / 2), &maps.q, &bars.q_full[t], 64 * h, w.hkv * a.G,
                          w.qb + w.tok0 + t * a.tile_tokens, a.q_batched ? w.s : 0);
            }
            for (int j = 0; j < n && ok; ++j) {
              ok = load_kv(true, j);
              if (ok && j + 1 < n) ok = load_kv(false, j + 1);
            }
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
        walk = n;
        if (!have) break;
      }
      if (lane == 0) {
        bars.filled = x;
        bars.q_filled[0] = q_copied[0];
        bars.q_filled[1] = q_copied[1];
      }
    } else if (warp >= H::kProductWarp && warp < H::kProductWarp + 2) {
      // ---- products of a tile, as in prompt_attn_kernel; u: scores formed so far (and two commits an item more) ----
      const bool lead = elect_lane();
      const int t = __shfl_sync(0xFFFFFFFFu, warp - H::kProductWarp, 0);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t base_addr = __shfl_sync(0xFFFFFFFFu, smem_addr(base), 0);
      const uint64_t qd = smem_operand(base_addr + kTileBytes * t, 16, 1024);
      const uint64_t kd = smem_operand(base_addr + 2 * kTileBytes, 16, 1024);
      const uint64_t vd = smem_operand(base_addr + 2 * kTileBytes, H::kStageBytes / 2, 1024);
      const uint32_t sp = tm + 2 * kBlock * t, op = tm + 4 * kBlock + kD * t;
      constexpr uint32_t kStep = H::kStageBytes / 16, kNext = kBlock * 128 / 16;
      uint32_t requests = 0, clean = 0, weights = 0;  // scans asked for; phases of v_clean and of p_full
      int x = 0, u = 0, q_here = 0, walked = 0, walk = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        ok = mbar_wait_warp(bars, &bars.item_full[it & 1], (it >> 1) & 1, walk + skip);
        if (!ok) break;
        const PromptItem& w = bars.item[it & 1];
        if (__shfl_sync(0xFFFFFFFFu, w.s, 0) < 0) break;
        int stages = __shfl_sync(0xFFFFFFFFu, w.hi - w.lo, 0);
        const bool here = __shfl_sync(0xFFFFFFFFu, (int)(t == 0 || w.two), 0) != 0;
        int blocks = here && stages > 0 ? __shfl_sync(0xFFFFFFFFu, w.blocks[t], 0) : 0;
        int from_a = __shfl_sync(0xFFFFFFFFu, w.ma / H::kPerStage - w.lo, 0);
        int to_a = __shfl_sync(0xFFFFFFFFu, (w.mb + H::kPerStage - 1) / H::kPerStage - w.lo, 0);
        int from_c = __shfl_sync(0xFFFFFFFFu, w.mc / H::kPerStage - w.lo, 0);
        const auto scanned = [&](int j) { return (j >= from_a && j < to_a) || j >= from_c; };
        const auto request = [&]() {
          if (t == 0 && lead) mbar_arrive(&bars.v_scan[requests & 1u]);
          ++requests;
          __syncwarp();
        };
        walk = stages;
        if (stages == 0) {
          leave(it);
          continue;
        }
        if constexpr (AHEAD) {
          const int first = t == 1 && here ? __shfl_sync(0xFFFFFFFFu, bars.first1[it & 1], 0) : 0;
          for (int j = 0; j < 2 * first && ok; ++j, ++x) {  // (the other tile frees what it uses, and what is looked through)
            ok = mbar_wait_warp(bars, &bars.kv_full[x % kStages], (x / kStages) & 1);
            if (ok && lead) mbar_arrive(&bars.kv_free[x % kStages]);
            if (j % 2 == 1 && scanned(j / 2)) clean ^= 1u << (x % kStages);
          }
          stages -= first;
          from_a -= first;
          to_a -= first;
          from_c -= first;
          blocks -= H::kPerStage * first;
        }
        const int xk0 = x++, s0 = xk0 % kStages;
        ok = mbar_wait_warp(bars, &bars.kv_full[s0], (xk0 / kStages) & 1);
        if (ok && here) ok = mbar_wait_warp(bars, &bars.q_full[t], q_here++ & 1);
        if (blocks > 0) {
          if (ok && walked > 0) ok = mbar_wait_warp(bars, &bars.s_seen[t], (walked - 1) & 1);
          ++walked;
        }
        if (ok && lead) {
          if (blocks > 0) {
            product_s(sp + kBlock * (u & 1), qd, kd + kStep * s0, H::kStageBytes / 2);
            tc_commit(&bars.s_full[t][u & 1]);
            if (blocks > 1) product_s(sp + kBlock * ((u + 1) & 1), qd, kd + kStep * s0 + kNext, H::kStageBytes / 2);
            tc_commit(&bars.s_full[t][(u + 1) & 1]);
          }
          if (blocks > 0 && blocks <= 2) tc_commit(&bars.q_free[t]);
          if (here && blocks == 0) mbar_arrive(&bars.q_free[t]);  // (its copy has been waited for)
          if (here)
            tc_commit(&bars.kv_free[s0]);
          else
            mbar_arrive(&bars.kv_free[s0]);
        }
        __syncwarp();
        if (ok && scanned(0)) request();
        for (int j = 0; j < stages && ok; ++j) {
          const int xv = x++, sv = xv % kStages;
          const bool more = j + 1 < stages;
          const int xk = more ? x++ : xv, sk = xk % kStages;
          ok = mbar_wait_warp(bars, &bars.kv_full[sv], (xv / kStages) & 1);
          if (ok && more && scanned(j + 1)) request();
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
            const int i = H::kPerStage * j + h, b = (u + i) & 1;
            if (i >= blocks || !ok) break;
            ok = mbar_wait_warp(bars, &bars.p_full[t][b], (weights >> b) & 1u);
            weights ^= 1u << b;
            if (!ok) break;
            tc_fence_after();
            if (lead) {
              product_o(op, sp + kBlock * b, vd + kStep * sv + kNext * h, i > 0);
              if (i + 2 < blocks) product_s(sp + kBlock * b, qd, kd + kStep * sk + kNext * h, H::kStageBytes / 2);
              tc_commit(&bars.s_full[t][b]);
              if (i + 3 == blocks) tc_commit(&bars.q_free[t]);
            }
            __syncwarp();
          }
          if (ok && lead) {
            tc_commit(&bars.kv_free[sv]);
            if (more) tc_commit(&bars.kv_free[sk]);
          }
          __syncwarp();
        }
        if (blocks > 0) u += blocks + 2;
        leave(it);
      }
    } else if (warp >= H::kScanWarp) {
      // ---- values in masked places ----
      uint32_t scans = 0;
      int x = 0, walk = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        ok = mbar_wait_warp(bars, &bars.item_full[it & 1], (it >> 1) & 1, walk + skip);
        if (!ok) break;
        const PromptItem& w = bars.item[it & 1];
        if (__shfl_sync(0xFFFFFFFFu, w.s, 0) < 0) break;
        const int n = w.hi - w.lo;
        for (int j = 0; j < n && ok; ++j) {
          if (!partly(w, j)) continue;
          const int xv = x + 1 + 2 * j, sv = xv % kStages;
          ok = mbar_wait_warp(bars, &bars.v_scan[scans & 1u], (scans >> 1) & 1u, n);
          ++scans;
          if (ok) ok = mbar_wait_warp(bars, &bars.kv_full[sv], (xv / kStages) & 1);
          if (!ok) break;
          uint4* tile = reinterpret_cast<uint4*>(ring + sv * H::kStageBytes);
          if (clear_non_finite(tile, tid - 32 * H::kScanWarp, H::kStageBytes / 16, 32 * kScanWarps)) bars.bad[it & 1] = 1u;
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.v_clean[sv]);
        }
        x += 2 * n;
        walk = n;
        leave(it);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n");
    // ---- softmax and output of one tile, a thread per row ----
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    const uint32_t s_addr = tmem + lanes + 2 * kBlock * t, o_addr = tmem + lanes + 4 * kBlock + kD * t;
    const float c = a.scale * kLog2e;
    uint4* stage = reinterpret_cast<uint4*>(staging) + warp * 256;
    int u = 0, walk = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      ok = mbar_wait_warp<1>(bars, &bars.item_full[it & 1], (it >> 1) & 1, walk + skip);
      if (!ok) break;
      const PromptItem& w = bars.item[it & 1];
      if (__shfl_sync(0xFFFFFFFFu, w.s, 0) < 0) break;
      walk = w.hi - w.lo;
      if (t == 1 && !w.two) {
        leave(it);
        continue;
      }
      const int tok = w.tok0 + t * a.tile_tokens + r / a.G, head = w.hkv * a.G + r % a.G;
      const bool row = r < a.tile_tokens * a.G && tok < w.lq;
      const int seen = row ? clampi(tok + w.lk - w.lq + 1, 0, w.lk) : w.lk;
      int blocks = w.blocks[t], g0 = H::kPerStage * w.lo, first = 0;
      if constexpr (AHEAD) {
        first = t == 1 ? bars.first1[it & 1] : 0;
        blocks -= H::kPerStage * first;
        g0 += H::kPerStage * first;
      }
      const int from_a = w.ma - g0, to_a = w.mb - g0, from_c = w.mc - g0;
      const int low = max(0, seen - a.window);
      const auto visible = [&](int g) {
        const auto first = [](int k) { return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1ull; };
        const int key = block_key(w, g);
        return first(seen - key) & (~first(low - key) | first(a.sinks - key));
      };
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < blocks; ++i) {
        const int b = (u + i) & 1;
        const uint32_t sp = s_addr + kBlock * b;
        ok = mbar_wait_warp<1>(bars, &bars.s_full[t][b], ((u + i) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        float x[kBlock];
        tmem_ld32(sp, x);
        tmem_ld32(sp + 32, x + 32);
        tmem_wait_ld(x);
        tmem_wait_ld(x + 32);
        if ((i >= from_a && i < to_a) || i >= from_c) {
          const uint64_t vis = visible(g0 + i);
          const uint32_t half[2] = {(uint32_t)vis, (uint32_t)(vis >> 32)};
#pragma unroll
          for (int e = 0; e < kBlock; ++e) x[e] = (half[e / 32] >> (e % 32)) & 1u ? x[e] : -INFINITY;
        }
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int e = 4; e < kBlock; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            top[k] = e + 4 + k < kBlock ? max3(top[k], x[e + k], x[e + 4 + k]) : fmaxf(top[k], x[e + k]);
        const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]);
        const bool grow = mx > m && !((mx - m) * c <= kSlack);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float f = grow ? fast_exp2((m - mx) * c) : 1.f;  // m = -inf: 0
          if (grow) m = mx;
          l *= f;
          if (i > 0) {
            // the product of the block before has to be complete: the next use of the other buffer says so
            ok = mbar_wait_warp<1>(bars, &bars.s_full[t][b ^ 1], ((u + i + 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {  // (32 columns at a time take registers that the scores need)
              float y[16];
              tmem_get16(o_addr + 16 * q, y);
              uint32_t v[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(y[e] * f);
              tmem_st16(o_addr + 16 * q, v);
            }
          }
        }
        l += row_weights(x, c, m == -INFINITY ? 0.f : m * c, sp);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[t][b]);
      }
      // ---- output: 64 channels at a time ----
      if (blocks > 0 && ok) ok = mbar_wait_warp<1>(bars, &bars.s_full[t][(u + blocks + 1) & 1], ((u + blocks + 1) >> 1) & 1);
      if (!ok) break;
      if (blocks > 0) {
        u += blocks + 2;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_seen[t]);
      }
      tc_fence_after();
      const bool bad = *(volatile uint32_t*)&bars.bad[it & 1] != 0u;
      const bool any = blocks > 0 && seen > 0;
      const float inv = any ? 1.f / l : 0.f;
      const uint64_t out =
          row ? (uint64_t)(a.o + w.s * a.o_b + (int64_t)(w.qb + tok) * a.o_t + head * a.o_h) : 0;  // where the row goes
      const bool whole = a.o_boxes && __all_sync(0xFFFFFFFFu, row);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");  // what lay there has left
        __syncwarp();
#pragma unroll 1
        for (int q = 2 * h; q < 2 * h + 2; ++q) {
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
            for (int j = 0; j < walk - first; ++j) {
              if (!partly(w, j + first)) continue;
              for (int g = g0 + j * H::kPerStage; g < g0 + (j + 1) * H::kPerStage && g < g0 + blocks; ++g) {
                const uint64_t vis = visible(g);
                const uint16_t* vr = a.v + w.s * a.v_b + (int64_t)(w.kb + block_key(w, g)) * a.v_t + w.hkv * a.v_h;
                for (int e = 0; e < kBlock; ++e) {
                  if (((vis >> e) & 1u) == 0) continue;
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    const uint32_t x = vr[e * a.v_t + 32 * q + i];
                    if ((x & 0x7F80u) == 0x7F80u) y[i] += bf16_to_f32(x);
                  }
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            stage[lane * 8 + ((4 * (q & 1) + i) ^ (lane & 7))] =
                make_uint4(pack_bf16x2(y[8 * i] * inv, y[8 * i + 1] * inv), pack_bf16x2(y[8 * i + 2] * inv, y[8 * i + 3] * inv),
                           pack_bf16x2(y[8 * i + 4] * inv, y[8 * i + 5] * inv),
                           pack_bf16x2(y[8 * i + 6] * inv, y[8 * i + 7] * inv));
        }
        if (whole) {
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            asm volatile(
                "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n" ::"l"(&maps.o),
                "r"(smem_addr(stage)), "r"(64 * h), "r"(w.hkv * a.G), "r"(w.qb + tok), "r"(a.q_batched ? w.s : 0)
                : "memory");
            asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
          }
        } else {
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < 8; ++i) {  // four rows at a time
            const int rr = 4 * i + (lane >> 3), cc = lane & 7;
            const uint64_t to = __shfl_sync(0xFFFFFFFFu, out, rr);
            const uint4 v = stage[rr * 8 + (cc ^ (rr & 7))];
            if (to != 0) reinterpret_cast<uint4*>(to)[8 * h + cc] = v;
          }
          __syncwarp();
        }
      }
      if (row && a.lse) a.lse[lse_place(a, w.s, w.qb + tok, head)] = any ? m * a.scale + logf(l) : -INFINITY;
      tc_fence_before();  // O has been read: the next item's products come behind its first weights
      leave(it);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (bars.stop) {  // a wait ran out (none is left): what is in flight ends before its memory goes
    tc_fence_after();
    if (warp == H::kCopyWarp && lane == 0) {
      for (int f = max(bars.filled - kStages, 0); f < bars.filled; ++f) mbar_drain(&bars.kv_full[f % kStages], (f / kStages) & 1);
      for (int t = 0; t < 2; ++t)
        if (bars.q_filled[t] > 0) mbar_drain(&bars.q_full[t], (bars.q_filled[t] - 1) & 1);
    } else if (warp >= H::kProductWarp && warp < H::kProductWarp + 2 && elect_lane()) {
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

cudaError_t launch_stay(const PromptMaps<kWindow>& maps, const PromptArgs& a, cudaStream_t stream) {
  // tiles of as many tokens as a stage has keys, one head a KV head: such stages there may be (first tokens are seen by all)
  const auto kernel = a.sinks == 0 && a.tile_tokens >= Shape<2>::kKeys ? stay_attn_kernel<true> : stay_attn_kernel<false>;
  static unsigned long long configured[2] = {0ull, 0ull};
  const cudaError_t e = spc_host::ensure_smem_limit(configured[kernel == stay_attn_kernel<true>], kernel, kStaySmemBytes);
  if (e != cudaSuccess) return e;
  kernel<<<std::min<unsigned>(a.items, (unsigned)spc_host::sm_count()), Shape<2>::kThreads, kStaySmemBytes, stream>>>(maps, a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace spc
