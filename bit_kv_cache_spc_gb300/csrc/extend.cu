// A run of n new tokens joins the cache at once (SpeCache page, Algorithm 1
// for a prompt; a follow-up prompt of a conversation), with the result of n
// appends: the groups that complete are coded straight from where their rows
// are (the window's old rows, then the new tokens' views), then the window
// shifts and takes the rows that stay in 16 bits.
//
// A code is a comparison: an element of a group has a code of at least L
// exactly when it is at least the group's threshold of level L, a bf16 value
// (code_threshold).  So a group's thresholds are found once and its elements
// are compared two at a time, as packed bf16 pairs; the masks that result
// (0xFFFF per half) are cut to their bits of the record's words by one AND-OR
// each.  A 128-thread CTA codes one group of tokens at a time:
//   - values: thread (token, 32 channels) holds a whole g = 32 group (half a
//     g = 64 one) in 16 registers: extremes, thresholds and codes without a
//     barrier; four shuffles gather a word's bits from the four threads of a
//     token and from the next token's;
//   - keys: a pass over channel pairs for the extremes, a thread per channel
//     for the thresholds, then thread (token mod 8, channel pair mod 8, four
//     chunks of channels) builds one word.
// The high bit of a 2-bit code is the comparison with the second threshold,
// the low bit one with the third or the first as the high bit says.
// Bound by HBM: 512 bytes read and 48 to 96 written per token and KV head.
#include <algorithm>

#include "quant.cuh"

namespace spc {
namespace {

struct ExtendArgs {
  const uint16_t* k_new;  // views [B][n][Hkv][D]
  const uint16_t* v_new;
  spc_layout lk, lv;
  uint8_t* records;
  uint16_t* resid;
  uint16_t* host;  // device address of [B][Hkv][n_cap][2][D], or null
  int64_t n_cap, total_groups;
  int32_t Hkv, N, n, nq, nq1, resid_cap, units_cap;
  int32_t window_parts;  // CTAs per (b, hkv) that write the window
};

// 16-byte piece `q` (0-15 key, 16-31 value) of token t of (b, hkv).
__device__ __forceinline__ const uint4* extend_source(const ExtendArgs& a, int64_t bh, int t, int q) {
  if (t < a.N) return reinterpret_cast<const uint4*>(a.resid + (bh * a.resid_cap + (t - a.nq)) * 2 * kD) + q;
  const int64_t b = bh / a.Hkv, h = bh % a.Hkv;
  return q < 16 ? reinterpret_cast<const uint4*>(a.k_new + b * a.lk.b + (t - a.N) * a.lk.t + h * a.lk.h) + q
                : reinterpret_cast<const uint4*>(a.v_new + b * a.lv.b + (t - a.N) * a.lv.t + h * a.lv.h) + (q - 16);
}

// A row of 256 bytes takes 272, so that rows' equal chunks lie in different banks.
constexpr int kPitch = 136;  // in elements

template <int BITS, int GROUP>
struct ExtendSmem {
  uint16_t k[GROUP * kPitch];
  uint16_t v[GROUP * kPitch];
  uint32_t lo[2][kD / 2], hi[2][kD / 2];            // key extremes of each half of the tokens, channel pairs
  uint16_t thr[(1 << BITS) - 1][kD];                // key thresholds
  uint32_t rec[GROUP == 32 ? 256 * (BITS + 1) : 512 * BITS + 256];
};

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 0xFFFF in each half where a >= b (false with a NaN).
__device__ __forceinline__ uint32_t ge_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n .reg .b32 t;\n set.ge.u32.bf16x2 t, %1, %2;\n mov.b32 %0, t;\n}\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The thresholds of a group, as bf16 patterns, and its (min, max) word.
template <int BITS>
__device__ __forceinline__ uint32_t group_thresholds(float lo, float hi, uint32_t* thr) {
  float z, s;
  quant_params(BITS, lo, hi, z, s);
  code_thresholds<BITS>(lo, hi, z, s, thr);
  return bf16_bits_canonical(lo) | (bf16_bits_canonical(hi) << 16);
}

// acc[p] |= plane p of the codes of the pair x, in the places `bit`.
template <int BITS>
__device__ __forceinline__ void code_pair(uint32_t x, const uint32_t* thr, uint32_t bit, uint32_t* acc) {
  if (BITS == 1) {
    acc[0] |= ge_bf16x2(x, thr[0]) & bit;
  } else {
    const uint32_t high = ge_bf16x2(x, thr[1]);
    acc[0] |= ge_bf16x2(x, (thr[2] & high) | (thr[0] & ~high)) & bit;
    acc[BITS - 1] |= high & bit;
  }
}

template <int BITS, int GROUP>
__device__ __forceinline__ void code_tokens(ExtendSmem<BITS, GROUP>& sm, uint8_t* dst_rec) {
  constexpr int kHalves = GROUP / 32, kCodes = 128 * BITS, kLevels = (1 << BITS) - 1;
  constexpr int KMETA = kHalves * kCodes, VCODES = KMETA + 128, VMETA = VCODES + kHalves * kCodes;  // in words
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- key extremes: thread (channel pair, half of the tokens) ----
  {
    const int p = tid & 63, part = tid >> 6;
    const uint32_t* col = reinterpret_cast<const uint32_t*>(sm.k + part * (GROUP / 2) * kPitch) + p;
    uint32_t lo = col[0], hi = lo;
#pragma unroll
    for (int n = 1; n < GROUP / 2; ++n) {
      const uint32_t x = col[n * (kPitch / 2)];
      lo = min_bf16x2(lo, x);
      hi = max_bf16x2(hi, x);
    }
    sm.lo[part][p] = lo;
    sm.hi[part][p] = hi;
  }
  // ---- values: thread (token, 32 channels) ----
#pragma unroll
  for (int half = 0; half < kHalves; ++half) {
    const int n = tid >> 2, cg = tid & 3;  // token of the half, channels 32 cg ..
    const uint4* row = reinterpret_cast<const uint4*>(sm.v + (32 * half + n) * kPitch + 32 * cg);
    // the chunks in an order that puts the eight threads of a shared-memory phase in different banks
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = row[(u + (cg & 2)) & 3];
    uint32_t lo2 = x[0].x, hi2 = lo2;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      lo2 = min_bf16x2(min_bf16x2(lo2, min_bf16x2(x[u].x, x[u].y)), min_bf16x2(x[u].z, x[u].w));
      hi2 = max_bf16x2(max_bf16x2(hi2, max_bf16x2(x[u].x, x[u].y)), max_bf16x2(x[u].z, x[u].w));
    }
    if (GROUP == 64) {
      lo2 = min_bf16x2(lo2, __shfl_xor_sync(0xFFFFFFFFu, lo2, 1));
      hi2 = max_bf16x2(hi2, __shfl_xor_sync(0xFFFFFFFFu, hi2, 1));
    }
    const float lo = fminf(bf16_to_f32(lo2 & 0xFFFFu), bf16_to_f32(lo2 >> 16));
    const float hi = fmaxf(bf16_to_f32(hi2 & 0xFFFFu), bf16_to_f32(hi2 >> 16));
    uint32_t thr[kLevels];
    const uint32_t mm = group_thresholds<BITS>(lo, hi, thr);
#pragma unroll
    for (int l = 0; l < kLevels; ++l) thr[l] *= 0x10001u;
    if (GROUP == 32) sm.rec[VMETA + vmeta_word(n, cg)] = mm;
    if (GROUP == 64 && (cg & 1) == 0) sm.rec[VMETA + 64 * half + vmeta64_word(n, cg >> 1)] = mm;
    // acc[p][w]: bits `chunk` of plane p of channels 2w (low half) and 2w + 1 (high half) mod 8
    uint32_t acc[4][BITS];
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int p = 0; p < BITS; ++p) acc[w][p] = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t bit = 0x10001u << (4 * cg + ((u + (cg & 2)) & 3));
      code_pair<BITS>(x[u].x, thr, bit, acc[0]);
      code_pair<BITS>(x[u].y, thr, bit, acc[1]);
      code_pair<BITS>(x[u].z, thr, bit, acc[2]);
      code_pair<BITS>(x[u].w, thr, bit, acc[3]);
    }
#pragma unroll
    for (int p = 0; p < BITS; ++p) {
      // the token's four threads: thread cg collects pair cg
      const bool up = cg & 2, odd = cg & 1, next = n & 1;
      uint32_t a0 = up ? acc[2][p] : acc[0][p], a1 = up ? acc[3][p] : acc[1][p];
      a0 |= __shfl_xor_sync(0xFFFFFFFFu, up ? acc[0][p] : acc[2][p], 2);
      a1 |= __shfl_xor_sync(0xFFFFFFFFu, up ? acc[1][p] : acc[3][p], 2);
      uint32_t w = odd ? a1 : a0;
      w |= __shfl_xor_sync(0xFFFFFFFFu, odd ? a0 : a1, 1);
      // tokens 2t and 2t + 1: the first takes channel 2 cg, the second 2 cg + 1 (mod 8)
      const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, w, 4);
      const uint32_t word = next ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
      const int a = 2 * cg + next, t = (n >> 1) & 3, j = n >> 3;
      sm.rec[VCODES + half * kCodes + 128 * p + 16 * a + 4 * t + j] = word;
    }
  }
  __syncthreads();
  // ---- key thresholds: a thread per channel ----
  {
    const int c = tid, sh = 16 * (c & 1);
    const auto of = [&](uint32_t w) { return __uint_as_float(((w >> sh) & 0xFFFFu) << 16); };
    const float lo = fminf(of(sm.lo[0][c >> 1]), of(sm.lo[1][c >> 1]));
    const float hi = fmaxf(of(sm.hi[0][c >> 1]), of(sm.hi[1][c >> 1]));
    uint32_t thr[kLevels];
    sm.rec[KMETA + 32 * ((c >> 1) & 3) + 2 * (c >> 3) + (c & 1)] = group_thresholds<BITS>(lo, hi, thr);
#pragma unroll
    for (int l = 0; l < kLevels; ++l) sm.thr[l][c] = (uint16_t)thr[l];
  }
  __syncthreads();
  // ---- key codes: warp j, lane (a, t): word 4 (4a + t) + j ----
  {
    const int j = warp, a = lane >> 2, t = lane & 3;
    uint32_t thr[4][kLevels];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int l = 0; l < kLevels; ++l)
        thr[i][l] = *reinterpret_cast<const uint32_t*>(&sm.thr[l][8 * (4 * j + i) + 2 * t]);
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
      uint32_t acc[BITS], wrapped[BITS];  // the word, and the one pair whose bits 31 and 15 are exchanged
#pragma unroll
      for (int p = 0; p < BITS; ++p) acc[p] = wrapped[p] = 0u;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x =
              *reinterpret_cast<const uint32_t*>(sm.k + (32 * half + 8 * n + a) * kPitch + 8 * (4 * j + i) + 2 * t);
          const int at = 11 + n - 4 * i;  // the pair's bits: at and at + 16 (mod 32)
          if (at < 0)
            code_pair<BITS>(x, thr[i], 0x80008000u, wrapped);
          else
            code_pair<BITS>(x, thr[i], 0x10001u << at, acc);
        }
#pragma unroll
      for (int p = 0; p < BITS; ++p)
        sm.rec[half * kCodes + 128 * p + 16 * a + 4 * t + j] = acc[p] | __funnelshift_l(wrapped[p], wrapped[p], 16);
    }
  }
  __syncthreads();
  // ---- the record out ----
  uint4* dst = reinterpret_cast<uint4*>(dst_rec);
  const uint4* src = reinterpret_cast<const uint4*>(sm.rec);
  for (int i = tid; i < (int)sizeof(sm.rec) / 16; i += 128) dst[i] = src[i];
}

// Codes group g of (b, hkv): its rows into shared memory, its record out.
template <int BITS, int GROUP>
__device__ __forceinline__ void extend_group(const ExtendArgs& a, ExtendSmem<BITS, GROUP>& sm, int64_t bh, int g) {
  const int tid = threadIdx.x, q = tid & 31, t0 = a.nq + g * GROUP;
  uint16_t* tile = (q < 16 ? sm.k : sm.v) + 8 * (q & 15);
  if (t0 >= a.N) {  // none of the window's rows
    const int64_t b = bh / a.Hkv, h = bh % a.Hkv, step = q < 16 ? a.lk.t : a.lv.t;
    const uint16_t* src = (q < 16 ? a.k_new + b * a.lk.b + h * a.lk.h : a.v_new + b * a.lv.b + h * a.lv.h) +
                          8 * (q & 15) + (t0 - a.N + (tid >> 5)) * step;
#pragma unroll 8
    for (int row = tid >> 5; row < GROUP; row += 4, src += 4 * step) cp_async16(tile + row * kPitch, src);
  } else {
    for (int row = tid >> 5; row < GROUP; row += 4) cp_async16(tile + row * kPitch, extend_source(a, bh, t0 + row, q));
  }
  cp_async_commit();
  cp_async_wait<0>();
  __syncthreads();
  code_tokens<BITS, GROUP>(sm, a.records + (bh * a.units_cap + a.nq / GROUP + g) * record_bytes(BITS, GROUP));
}

// CTAs that an SM holds: 10 (1 bit) and 9 (2 bits) at g = 32, 5 at g = 64.
template <int BITS, int GROUP>
constexpr int kResident = 232448 / (sizeof(ExtendSmem<BITS, GROUP>) + 1024);

// A group per CTA; the other CTAs of the SM fill its waits.  CTAs that stay
// and take group after group end 10% apart (105 us against 93 below), two
// groups per CTA are slower where groups are few (300 tokens into eight caches
// 8.3 us against 6.9), and neighbours that take the KV heads of the same
// tokens instead of a head's groups in turn are too (98).
// 1 bit, g = 32, four 32768-token prompts over 8 KV heads (606 MB): 93 to 102
// us from process to process, 5.9 to 6.5 TB/s, 87 to 96% of the measured copy
// bandwidth; g = 64 91 us; 2 bits 128 and 113 us, 74% of it at g = 32, bound by
// the thresholds' and comparisons' issue (68% of the cycles issue, and of the
// waiting warps more are ready or wait for the arithmetic pipes than for
// memory; 56 registers, nine CTAs an SM).
template <int BITS, int GROUP>
__global__ void __launch_bounds__(128, kResident<BITS, GROUP>) extend_groups_kernel(const __grid_constant__ ExtendArgs a) {
  extern __shared__ __align__(16) uint8_t extend_smem[];
  ExtendSmem<BITS, GROUP>& sm = *reinterpret_cast<ExtendSmem<BITS, GROUP>*>(extend_smem);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // the window's kernel may be set up meanwhile
  const uint32_t per = (a.nq1 - a.nq) / GROUP, bh = blockIdx.x / per;
  extend_group<BITS, GROUP>(a, sm, bh, (int)(blockIdx.x - bh * per));
}

// The same and the window's rows in one launch, for turns of few groups: a
// cluster of eight CTAs takes a (b, hkv).  They code its groups, a group each,
// and hold the window's next rows in registers; once every CTA has read what
// it needs of the old window (a cluster barrier), they write the new one.
// A 77-token turn of eight conversations (8 KV heads, R = 128): one launch of
// 5.0 us against two of 9.4.
constexpr int kTurnCtas = 8, kTurnPieces = 8;
constexpr int kTurnRows = kTurnCtas * kTurnPieces * 128 / 32;  // of the window

template <int BITS, int GROUP>
__global__ void __launch_bounds__(128) __cluster_dims__(kTurnCtas, 1, 1)
extend_turn_kernel(const __grid_constant__ ExtendArgs a) {
  extern __shared__ __align__(16) uint8_t extend_smem[];
  ExtendSmem<BITS, GROUP>& sm = *reinterpret_cast<ExtendSmem<BITS, GROUP>*>(extend_smem);
  const int rank = blockIdx.x % kTurnCtas, id = rank * 128 + threadIdx.x;
  const int64_t bh = blockIdx.x / kTurnCtas;
  const int pieces = (a.N + a.n - a.nq1) * 32;  // of 16 bytes
  uint4 next[kTurnPieces];
#pragma unroll
  for (int i = 0; i < kTurnPieces; ++i) {
    const int p = id + i * kTurnCtas * 128;
    if (p < pieces) next[i] = *extend_source(a, bh, a.nq1 + (p >> 5), p & 31);
  }
  if (rank < (a.nq1 - a.nq) / GROUP) extend_group<BITS, GROUP>(a, sm, bh, rank);
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  uint4* win = reinterpret_cast<uint4*>(a.resid + bh * a.resid_cap * 2 * kD);
#pragma unroll
  for (int i = 0; i < kTurnPieces; ++i) {
    const int p = id + i * kTurnCtas * 128;
    if (p < pieces) win[p] = next[i];
  }
  if (a.host != nullptr) {
    uint4* host = reinterpret_cast<uint4*>(a.host + (bh * a.n_cap + a.N) * 2 * kD);
    for (int p = id; p < a.n * 32; p += kTurnCtas * 128) host[p] = *extend_source(a, bh, a.N + (p >> 5), p & 31);
  }
}

// The window's rows (tokens nq1 .. N+n-1), and the new rows of the host cache.
// Old rows that stay move down by nq1 - nq; a CTA that moves them owns the
// window of its (b, hkv) (window_parts = 1) and moves 32 at a time, each chunk
// read in full before it is written, before it writes the new rows.
__global__ void __launch_bounds__(256) extend_window_kernel(const __grid_constant__ ExtendArgs a) {
  const int64_t bh = blockIdx.x;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the groups' kernel, which reads the window, has ended
  if ((int)blockIdx.y < a.window_parts) {
    uint4* win = reinterpret_cast<uint4*>(a.resid + bh * a.resid_cap * 2 * kD);  // 32 pieces a row
    const int shift = a.nq1 - a.nq, kept = max(a.N - a.nq1, 0);                   // old rows that stay
    if (shift > 0) {
      for (int c0 = 0; c0 < kept; c0 += 32) {
        const int pieces = 32 * min(32, kept - c0);
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = tid + 256 * u;
          if (i < pieces) v[u] = win[(int64_t)(shift + c0) * 32 + i];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = tid + 256 * u;
          if (i < pieces) win[(int64_t)c0 * 32 + i] = v[u];
        }
        __syncthreads();
      }
    }
    const int first = max(a.N, a.nq1);  // the first new token that stays
    const int64_t pieces = (int64_t)(a.N + a.n - first) * 32;
    for (int64_t i = blockIdx.y * 256 + tid; i < pieces; i += 256 * a.window_parts) {
      const int t = first + (int)(i >> 5);
      win[(int64_t)(t - a.nq1) * 32 + (i & 31)] = *extend_source(a, bh, t, (int)(i & 31));
    }
  } else {
    uint4* host = reinterpret_cast<uint4*>(a.host + (bh * a.n_cap + a.N) * 2 * kD);
    const int64_t pieces = (int64_t)a.n * 32;
    const int parts = gridDim.y - a.window_parts;
    for (int64_t i = (blockIdx.y - a.window_parts) * 256 + tid; i < pieces; i += 256 * parts)
      host[i] = *extend_source(a, bh, a.N + (int)(i >> 5), (int)(i & 31));
  }
}

template <int BITS, int GROUP>
cudaError_t launch_extend_k(const ExtendArgs& a, int64_t BH, bool turn, cudaStream_t stream) {
  const int smem = (int)sizeof(ExtendSmem<BITS, GROUP>);
  if (turn) {
    static unsigned long long turn_configured = 0ull;
    const cudaError_t e = spc_host::ensure_smem_limit(turn_configured, extend_turn_kernel<BITS, GROUP>, smem);
    if (e != cudaSuccess) return e;
    extend_turn_kernel<BITS, GROUP><<<(unsigned)(BH * kTurnCtas), 128, smem, stream>>>(a);
    return cudaGetLastError();
  }
  static unsigned long long configured = 0ull;
  const cudaError_t e = spc_host::ensure_smem_limit(configured, extend_groups_kernel<BITS, GROUP>, smem);
  if (e != cudaSuccess) return e;
  extend_groups_kernel<BITS, GROUP><<<(unsigned)a.total_groups, 128, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

spc_status launch_extend(const spc_dims* d, int32_t n, const uint16_t* k_new, const uint16_t* v_new,
                         const spc_layout* lk, const spc_layout* lv, void* records, uint16_t* resid,
                         uint16_t* host_dev, int64_t n_cap, cudaStream_t stream) {
  ExtendArgs a = {};
  a.k_new = k_new;
  a.v_new = v_new;
  a.lk = *lk;
  a.lv = *lv;
  a.records = static_cast<uint8_t*>(records);
  a.resid = resid;
  a.host = host_dev;
  a.n_cap = n_cap;
  a.Hkv = d->Hkv;
  a.N = d->N;
  a.n = n;
  a.nq = num_quantized(d->N, d->R, d->group);
  a.nq1 = num_quantized(d->N + n, d->R, d->group);
  a.resid_cap = d->resid_cap;
  a.units_cap = records_cap(d->group, d->q_groups_cap);
  const int64_t BH = (int64_t)d->B * d->Hkv;
  a.total_groups = BH * ((a.nq1 - a.nq) / d->group);
  if (a.total_groups > 0x7FFFFFFF) return SPC_ERR_UNSUPPORTED;
  // One launch where a cluster's CTAs have a group each at most and hold the
  // window, and the clusters are on the SMs together (5 CTAs each); else the
  // groups first, over all SMs, then the window.  200 tokens into 8 caches of
  // 8 KV heads: 6.9 us and 6.8, 16: 11.2 and 8.9, 64: 32.8 and 27.0; 77 tokens
  // 5.3 and 8.5, 7.6 and 8.9, 24.2 and 24.5.
  const bool turn = a.total_groups > 0 && a.total_groups <= BH * kTurnCtas && a.N + n - a.nq1 <= kTurnRows &&
                    BH * kTurnCtas <= (int64_t)spc_host::sm_count() * 5;
  cudaError_t e = cudaSuccess;
  if (a.total_groups > 0) {
    if (d->bits == 1)
      e = d->group == 64 ? launch_extend_k<1, 64>(a, BH, turn, stream) : launch_extend_k<1, 32>(a, BH, turn, stream);
    else
      e = d->group == 64 ? launch_extend_k<2, 64>(a, BH, turn, stream) : launch_extend_k<2, 32>(a, BH, turn, stream);
  }
  if (e == cudaSuccess && !turn) {
    const bool moves = a.nq1 > a.nq && a.N > a.nq1;
    const int32_t rows = a.N + n - std::max(a.N, a.nq1);
    a.window_parts = moves ? 1 : (int32_t)std::min<int64_t>(64, (rows + 31) / 32);
    const int host_parts = host_dev != nullptr ? (int)std::min<int64_t>(64, (n + 31) / 32) : 0;
    if (a.window_parts + host_parts > 0) {
      cudaLaunchAttribute attr = {};
      attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr.val.programmaticStreamSerializationAllowed = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)BH, (unsigned)(a.window_parts + host_parts));
      cfg.blockDim = dim3(256);
      cfg.stream = stream;
      cfg.attrs = &attr;
      cfg.numAttrs = a.total_groups > 0 ? 1 : 0;
      e = cudaLaunchKernelEx(&cfg, extend_window_kernel, a);
    }
  }
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace spc
