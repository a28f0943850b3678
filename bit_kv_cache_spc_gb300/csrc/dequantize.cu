// Reading the low-bit cache back: tokens first .. first+n-1 as bf16 rows, for
// the attention of a follow-up prompt over its history.
//
// A CTA takes 32 tokens of one (b, hkv), half a g = 64 record, a g = 32 record
// or 32 rows of the residual window: 128 threads the keys, 128 the values.  An element of
// the record stands for one of 2 or 4 levels of its group, fl(z + fl(s code)),
// so the levels are formed and rounded once per group and lane, and an
// element costs a bit mask and a select of packed pairs:
//   - keys: lane (token row, 8 channels) finds its channels' pairs (2t, 2t+1)
//     in four words, the pair's two bits 16 apart (spc.h: rotated left by 4i,
//     bits 11 + n and 27 + n);
//   - values: a word holds two tokens' bits of one channel (mod 8) 16 apart,
//     so a lane takes a token pair and eight channels from eight words.
// Bound by HBM: 512 bytes written per token and KV head against 48 to 96 read.
// A CTA per tile: CTAs that walk over tiles, 16 per SM, wait for each tile's
// words with nothing else to do (219 us against 179 for eight 32768-token
// caches of 8 KV heads at 1 bit, 1.21 GB; 179 us are the measured copy rate).
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

__device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t yes, uint32_t no) { return (yes & mask) | (no & ~mask); }

template <int BITS, int GROUP>
__global__ void __launch_bounds__(256) dequantize_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int kWords = GROUP == 32 ? 256 * (BITS + 1) : 512 * BITS + 256;  // of a record
  constexpr int kCodes = 128 * BITS;                                        // words of 32 tokens' codes
  constexpr int L = 1 << BITS;
  const int tid = threadIdx.x & 127;
  const bool keys = threadIdx.x < 128;
  const int64_t bh = blockIdx.x / a.tiles_per;
  const int tile = a.tile0 + (int)(blockIdx.x % a.tiles_per);
  const int64_t b = bh / a.Hkv, h = bh % a.Hkv;
  uint16_t* kd = a.k + b * a.lk.b + h * a.lk.h;
  uint16_t* vd = a.v + b * a.lv.b + h * a.lv.h;
  const int chunk = tid & 15, e = 8 * chunk;  // this lane's channels e .. e+7
  if (tile >= a.low_tiles) {                  // the residual window
    const int t0 = a.nq + 32 * (tile - a.low_tiles);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + 8 * r + (tid >> 4);
      if (t < a.first || t >= a.end) continue;
      const uint16_t* row = a.resid + (bh * a.resid_cap + (t - a.nq)) * 2 * kD + (keys ? 0 : kD);
      uint16_t* to = keys ? kd + (int64_t)(t - a.first) * a.lk.t : vd + (int64_t)(t - a.first) * a.lv.t;
      *reinterpret_cast<uint4*>(to + e) = *reinterpret_cast<const uint4*>(row + e);
    }
    return;
  }
  const int unit = GROUP == 32 ? tile : tile >> 1, half = GROUP == 32 ? 0 : tile & 1;
  const uint32_t* rec = reinterpret_cast<const uint32_t*>(a.records) + (bh * a.units_cap + unit) * kWords;
  const uint32_t* kc = rec + half * kCodes;
  const uint32_t* km = rec + (GROUP / 32) * kCodes;
  const uint32_t* vc = km + 128 + half * kCodes;
  const uint32_t* vm = km + 128 + (GROUP / 32) * kCodes + 64 * half;  // g = 32: half = 0
  const int t0 = 32 * tile;

  if (keys) {
    // ---- keys: rows a, a + 8, a + 16, a + 24 of lane a = tid >> 4 ----
    const int row = tid >> 4, j = chunk >> 2, rot = 4 * (chunk & 3);
    uint32_t lev[4][L];  // of channel pairs e + 2t, e + 2t + 1
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // channel 16 k + 8 h + 2t + x stands at minmax word 32 t + 4 k + 2 h + x
      const uint2 mm = *reinterpret_cast<const uint2*>(km + 32 * t + 2 * chunk);
      float p[L], q[L];
      levels<BITS>(mm.x, p);
      levels<BITS>(mm.y, q);
#pragma unroll
      for (int c = 0; c < L; ++c) lev[t][c] = read_pack(p[c], q[c]);
    }
    uint32_t w[BITS][4];
#pragma unroll
    for (int p = 0; p < BITS; ++p)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t x = kc[128 * p + 16 * row + 4 * t + j];
        w[p][t] = __funnelshift_l(x, x, rot + 21);  // row 8n + a's two bits at n and 16 + n
      }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int t = t0 + 8 * n + row;
      uint32_t out[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t m0 = ((w[0][u] >> n) & 0x00010001u) * 0xFFFFu;
        if (BITS == 1) {
          out[u] = pick(m0, lev[u][1], lev[u][0]);
        } else {
          const uint32_t m1 = ((w[BITS - 1][u] >> n) & 0x00010001u) * 0xFFFFu;
          out[u] = pick(m1, pick(m0, lev[u][L - 1], lev[u][L - 2]), pick(m0, lev[u][1], lev[u][0]));
        }
      }
      if (t >= a.first && t < a.end)
        *reinterpret_cast<uint4*>(kd + (int64_t)(t - a.first) * a.lk.t + e) = make_uint4(out[0], out[1], out[2], out[3]);
    }
    return;
  }
  // ---- values: token pairs 2p, 2p + 1 for p = tid >> 4 and 8 + (tid >> 4) ----
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int p = 8 * r + (tid >> 4), j = p >> 2, t = p & 3;  // tokens 8 j + 2 t + {0, 1}
    uint32_t lev[2][L];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t mm;
      if (GROUP == 32)
        mm = vm[32 * t + 16 * (j >> 1) + 8 * (j & 1) + 4 * x + (chunk >> 2)];
      else
        mm = vm[2 * (8 * t + 4 * (j >> 1) + 2 * (j & 1) + x) + (chunk >> 3)];
      float lv[L];
      levels<BITS>(mm, lv);
#pragma unroll
      for (int c = 0; c < L; ++c) lev[x][c] = read_pack(lv[c], lv[c]);
    }
    uint32_t out[2][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // channels e + 2u, e + 2u + 1
      uint32_t m[2][BITS];
#pragma unroll
      for (int q = 0; q < BITS; ++q) {
        const uint32_t x = (vc[128 * q + 16 * (2 * u) + 4 * t + j] >> chunk) & 0x00010001u;
        const uint32_t y = (vc[128 * q + 16 * (2 * u + 1) + 4 * t + j] >> chunk) & 0x00010001u;
        m[0][q] = __byte_perm(x, y, 0x5410) * 0xFFFFu;
        m[1][q] = __byte_perm(x, y, 0x7632) * 0xFFFFu;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        out[x][u] = BITS == 1 ? pick(m[x][0], lev[x][1], lev[x][0])
                              : pick(m[x][BITS - 1], pick(m[x][0], lev[x][L - 1], lev[x][L - 2]),
                                     pick(m[x][0], lev[x][1], lev[x][0]));
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int tok = t0 + 2 * p + x;
      if (tok >= a.first && tok < a.end)
        *reinterpret_cast<uint4*>(vd + (int64_t)(tok - a.first) * a.lv.t + e) =
            make_uint4(out[x][0], out[x][1], out[x][2], out[x][3]);
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
