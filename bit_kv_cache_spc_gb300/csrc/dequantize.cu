// Reading the low-bit cache back: tokens first .. first+n-1 as bf16 rows, for
// the attention of a follow-up prompt over its history.
//
// A CTA takes 32 tokens of one (b, hkv), half a g = 64 record, a g = 32 record
// or 32 rows of the residual window: 128 threads the keys, 128 the values.  An
// element of the record stands for one of 2 or 4 levels of its group,
// fl(z + fl(s code)), so the levels are formed and rounded once per group (in
// shared memory), and an element costs a bit mask and a select of packed
// pairs:
//   - keys: lane (token row, 8 channels) finds its channels' pairs (2t, 2t+1)
//     in four words, the pair's two bits 16 apart (spc.h: rotated left by 4i,
//     bits 11 + n and 27 + n);
//   - values: a word holds two tokens' bits of one channel (mod 8) 16 apart,
//     so a lane takes a token pair and eight channels from eight words.
// Bound by HBM: 512 bytes written per token and KV head against 48 to 96 read.
// Eight 32768-token caches of 8 KV heads at 1 bit (1.21 GB) take 176 us, the
// measured copy rate (g = 64 171); at 2 bits (1.28 GB) 212, 89% of it, bound
// by the selects' issue (74% of the cycles issue; eight CTAs an SM leave 32
// registers, and 32 bytes spill).  The code words come through shared memory, so that a
// thread holds few of them and eight CTAs fit on an SM (words straight into
// registers, five CTAs: 240 us, and 179 at 1 bit with six).  Levels per thread
// instead of per group: 24 us against 18 for two 2-bit caches of 32 heads and
// 2003 tokens, then.  CTAs that walk over tiles, 16 per SM, wait for each
// tile's words with nothing else to do (219 us against 181, then).
#include "common.cuh"

namespace spc {
namespace {

struct ReadArgs {
  const uint8_t* records;
  const uint16_t* resid;
  uint16_t *k, *v;
  spc_layout lk, lv;
  int32_t Hkv, nq, resid_cap, units_cap, first, end, tile0, tiles_per, low_tiles;
};

// The levels of a group, as written (no fused multiply-add).
template <int BITS>
__device__ __forceinline__ void levels(uint32_t mm, float* out) {
  const float lo = bf16_to_f32(mm & 0xFFFFu), hi = __uint_as_float(mm & 0xFFFF0000u);
  float z, s;
  if (BITS == 1) {
    z = __fmul_rn(__fadd_rn(__fmul_rn(3.0f, lo), hi), 0.25f);
    s = __fmul_rn(__fsub_rn(hi, lo), 0.5f);
  } else {
    z = lo;
    s = __fdiv_rn(__fsub_rn(hi, lo), 3.0f);
  }
#pragma unroll
  for (int c = 0; c < (1 << BITS); ++c) out[c] = __fadd_rn(z, __fmul_rn(s, (float)c));
}

__device__ __forceinline__ uint32_t read_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 0xFFFF in a half for each of two picked bytes whose top bit is set: selector
// nibbles 8 + byte of (a, b).
template <uint32_t SEL>
__device__ __forceinline__ uint32_t top_bits(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "n"(SEL));
  return r;
}

__device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t yes, uint32_t no) { return (yes & mask) | (no & ~mask); }

template <int BITS, int GROUP>
__global__ void __launch_bounds__(256, 8) dequantize_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int kWords = GROUP == 32 ? 256 * (BITS + 1) : 512 * BITS + 256;  // of a record
  constexpr int kCodes = 128 * BITS;                                        // words of 32 tokens' codes
  constexpr int L = 1 << BITS;
  const bool keys = threadIdx.x < 128;
  const int tid = threadIdx.x & 127, row = tid >> 4, chunk = tid & 15, e = 8 * chunk;  // channels e .. e+7
  const uint32_t bh = blockIdx.x / (uint32_t)a.tiles_per, tile = a.tile0 + blockIdx.x % (uint32_t)a.tiles_per;
  const uint32_t b = bh / (uint32_t)a.Hkv, h = bh - b * a.Hkv;
  const bool low = tile < (uint32_t)a.low_tiles;
  const int t0 = low ? 32 * (int)tile : a.nq + 32 * (int)(tile - a.low_tiles);  // the tile's first token
  // where the tile's first token would go, and the stride of tokens
  const int64_t step = keys ? a.lk.t : a.lv.t;
  uint16_t* to = (keys ? a.k + b * a.lk.b + h * a.lk.h : a.v + b * a.lv.b + h * a.lv.h) + (t0 - a.first) * step + e;
  const int skip = a.first - t0, count = a.end - a.first;  // token i of the tile is wanted: 0 <= i - skip < count
  const auto store = [&](int i, uint16_t* at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    if ((uint32_t)(i - skip) < (uint32_t)count) *reinterpret_cast<uint4*>(at) = make_uint4(x, y, z, w);
  };
  if (!low) {  // the residual window
    const uint16_t* from = a.resid + (bh * (int64_t)a.resid_cap + (t0 - a.nq)) * 2 * kD + (keys ? 0 : kD) + e;
    for (int i = row; i < 32; i += 8)
      if ((uint32_t)(i - skip) < (uint32_t)count)
        *reinterpret_cast<uint4*>(to + i * step) = *reinterpret_cast<const uint4*>(from + i * 2 * kD);
    return;
  }
  const uint32_t unit = GROUP == 32 ? tile : tile >> 1, half = GROUP == 32 ? 0 : tile & 1;
  const uint32_t* rec = reinterpret_cast<const uint32_t*>(a.records) + (bh * (int64_t)a.units_cap + unit) * kWords;
  constexpr int kKeyMeta = GROUP / 32 * kCodes, kValueCodes = kKeyMeta + 128, kValueMeta = kValueCodes + kKeyMeta;

  // ---- the levels, a group per thread, into shared memory; the code words are copied there meanwhile ----
  __shared__ __align__(16) uint16_t klev[L][kD];  // of a channel
  __shared__ uint32_t vlev[L][128];               // of a token's group, twice in a word
  constexpr int kVGroups = kD / GROUP;            // groups of a token
  __shared__ __align__(16) uint32_t codes[2][kCodes];  // keys', values'
  if (tid < kCodes / 4)
    cp_async16(codes[keys ? 0 : 1] + 4 * tid, rec + (keys ? 0 : kValueCodes) + half * kCodes + 4 * tid);
  cp_async_commit();
  if (keys) {
    const int t = tid >> 5, m = tid & 31;  // word 32 t + m
    float lv[L];
    levels<BITS>(rec[kKeyMeta + tid], lv);
#pragma unroll
    for (int c = 0; c < L; ++c)
      klev[c][16 * (m >> 2) + 2 * t + 8 * ((m >> 1) & 1) + (m & 1)] = (uint16_t)read_pack(lv[c], lv[c]);
  } else {
    if (tid < 32 * kVGroups) {
      int token, group;
      if (GROUP == 32) {
        const int t = tid >> 5, m = tid & 31;
        token = 16 * (m >> 4) + 8 * ((m >> 3) & 1) + 2 * t + ((m >> 2) & 1);
        group = m & 3;
      } else {
        const int m = tid >> 1;
        token = 16 * ((m >> 2) & 1) + 8 * ((m >> 1) & 1) + 2 * (m >> 3) + (m & 1);
        group = tid & 1;
      }
      float lv[L];
      levels<BITS>(rec[kValueMeta + 64 * half + tid], lv);
#pragma unroll
      for (int c = 0; c < L; ++c) vlev[c][kVGroups * token + group] = read_pack(lv[c], lv[c]);
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  if (keys) {
    // ---- rows a, a + 8, a + 16, a + 24 of lane a = tid >> 4: channel pairs e + 2t, e + 2t + 1 ----
    uint32_t lev[L][4];
#pragma unroll
    for (int c = 0; c < L; ++c) {
      const uint4 x = *reinterpret_cast<const uint4*>(&klev[c][e]);
      lev[c][0] = x.x;
      lev[c][1] = x.y;
      lev[c][2] = x.z;
      lev[c][3] = x.w;
    }
    uint32_t w[BITS][4];  // words 4t + j of row a
#pragma unroll
    for (int p = 0; p < BITS; ++p)
#pragma unroll
      for (int t = 0; t < 4; ++t) {  // row 8n + a's two bits to n and 16 + n
        const uint32_t x = codes[0][128 * p + 16 * row + 4 * t + (chunk >> 2)];
        w[p][t] = __funnelshift_l(x, x, 4 * (chunk & 3) + 21);
      }
    to += row * step;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      uint32_t out[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t m0 = top_bits<0xBB99>(w[0][u] << (15 - n), 0u);  // bits 16 + n and n
        if (BITS == 1) {
          out[u] = pick(m0, lev[1][u], lev[0][u]);
        } else {
          const uint32_t m1 = top_bits<0xBB99>(w[BITS - 1][u] << (15 - n), 0u);
          out[u] = pick(m1, pick(m0, lev[L - 1][u], lev[L - 2][u]), pick(m0, lev[1][u], lev[0][u]));
        }
      }
      store(8 * n + row, to, out[0], out[1], out[2], out[3]);
      to += 8 * step;
    }
  } else {
    // ---- token pairs ----
    to += 2 * row * step;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      // tokens 8 j + 2 t + {0, 1} with t = row % 4, j = 2 r + row / 4
      const int first = 2 * (8 * r + row);  // the pair's first token
      const uint32_t* vc = codes[1] + 4 * (row & 3) + (row >> 2) + 2 * r;
      uint32_t lev[2][L];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int c = 0; c < L; ++c) lev[x][c] = vlev[c][kVGroups * (first + x) + e / GROUP];
      uint32_t out[2][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {  // channels e + 2u, e + 2u + 1
        uint32_t m[2][BITS];
#pragma unroll
        for (int q = 0; q < BITS; ++q) {
          const uint32_t x = vc[128 * q + 32 * u] << (15 - chunk), y = vc[128 * q + 32 * u + 16] << (15 - chunk);
          m[0][q] = top_bits<0xDD99>(x, y);  // the first token: bits chunk
          m[1][q] = top_bits<0xFFBB>(x, y);  // the second: bits 16 + chunk
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
          out[x][u] = BITS == 1 ? pick(m[x][0], lev[x][1], lev[x][0])
                                : pick(m[x][BITS - 1], pick(m[x][0], lev[x][L - 1], lev[x][L - 2]),
                                       pick(m[x][0], lev[x][1], lev[x][0]));
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) store(first + x, to + x * step, out[x][0], out[x][1], out[x][2], out[x][3]);
      to += 16 * step;
    }
  }
}

}  // namespace

spc_status launch_dequantize(const spc_dims* d, const void* records, const uint16_t* resid, int32_t first, int32_t n,
                             uint16_t* k, uint16_t* v, const spc_layout* lk, const spc_layout* lv,
                             cudaStream_t stream) {
  ReadArgs a = {};
  a.records = static_cast<const uint8_t*>(records);
  a.resid = resid;
  a.k = k;
  a.v = v;
  a.lk = *lk;
  a.lv = *lv;
  a.Hkv = d->Hkv;
  a.nq = num_quantized(d->N, d->R, d->group);
  a.resid_cap = d->resid_cap;
  a.units_cap = records_cap(d->group, d->q_groups_cap);
  a.first = first;
  a.end = first + n;
  // tiles of 32 tokens: those of the records, then those of the window
  a.low_tiles = a.nq / kGroup;
  const auto tile_of = [&](int32_t t) { return t < a.nq ? t / kGroup : a.low_tiles + (t - a.nq) / kGroup; };
  a.tile0 = tile_of(first);
  a.tiles_per = tile_of(a.end - 1) - a.tile0 + 1;
  const int64_t tiles = (int64_t)d->B * d->Hkv * a.tiles_per;
  if (tiles > 0x7FFFFFFF) return SPC_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)tiles;
  if (d->group == 64) {
    if (d->bits == 1)
      dequantize_kernel<1, 64><<<grid, 256, 0, stream>>>(a);
    else
      dequantize_kernel<2, 64><<<grid, 256, 0, stream>>>(a);
  } else {
    if (d->bits == 1)
      dequantize_kernel<1, 32><<<grid, 256, 0, stream>>>(a);
    else
      dequantize_kernel<2, 32><<<grid, 256, 0, stream>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace spc
