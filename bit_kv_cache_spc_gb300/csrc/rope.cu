// Rotary positions of a run of tokens' query and key rows, and the copy of
// their value rows, from the projection to where they are used.
//
// Pair i at position p is turned by p * turns[i] (mod 2^64, 64-bit fractions
// of a turn): the integer product is exact, its top 32 bits give the angle in
// [-1/2, 1/2) turns to 2^-32, and sincospi needs no range reduction.
//
// Eight lanes hold a head's row, 16 elements each: lane l < rot/16 the eight
// pairs 8l .. 8l+7 (the half layout: elements 8l .. and rot/2 + 8l ..;
// interleaved: 16l .. 16l+15), the other lanes the elements that stay as they
// are.  A CTA forms the angles of its tokens once, in shared memory, and each
// lane walks over a few heads with its eight in registers (a lane that formed
// them itself took most of the time where it had few heads: 4096 tokens 23 us
// against 19).
// Bound by HBM: every row is read and written once.  Two heads' loads are in
// flight before the first store, the first ones before the angles: a
// 32768-token prompt of 32 + 8 + 8 heads (805 MB) takes 122 us, 97% of the
// measured copy rate, against 138 with one head in flight and 123 to 135 with
// four (fewer resident warps).
#include <algorithm>

#include "common.cuh"

namespace spc {
namespace {

struct RopeArgs {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_out, *v_out;
  const int32_t* pos;
  const uint64_t* turns;
  spc_layout lq, lk, lv, oq, ok, ov;
  uint32_t tokens;                      // B * T
  int32_t T, Hq, Hkv, heads, rot, per;  // heads of all three; heads a group of lanes walks over
  int32_t slices;                       // groups of `per` heads
  float mscale;
};

__device__ __forceinline__ uint32_t rope_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight pairs in the 16 bytes of u and w: word by word of both (interleaved:
// pairs 0-3 are u's words, 4-7 w's), element by element of u with those of w
// in the half layout.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_pairs(uint4& u, uint4& w, const float* c, const float* s) {
  uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = __uint_as_float(x[i] << 16), x1 = __uint_as_float(x[i] & 0xFFFF0000u);
    const float y0 = __uint_as_float(y[i] << 16), y1 = __uint_as_float(y[i] & 0xFFFF0000u);
    if (INTERLEAVED) {
      x[i] = rope_pack(x0 * c[i] - x1 * s[i], x0 * s[i] + x1 * c[i]);
      y[i] = rope_pack(y0 * c[4 + i] - y1 * s[4 + i], y0 * s[4 + i] + y1 * c[4 + i]);
    } else {
      x[i] = rope_pack(x0 * c[2 * i] - y0 * s[2 * i], x1 * c[2 * i + 1] - y1 * s[2 * i + 1]);
      y[i] = rope_pack(x0 * s[2 * i] + y0 * c[2 * i], x1 * s[2 * i + 1] + y1 * c[2 * i + 1]);
    }
  }
  u = make_uint4(x[0], x[1], x[2], x[3]);
  w = make_uint4(y[0], y[1], y[2], y[3]);
}

constexpr int kBatch = 2;

template <bool INTERLEAVED>
__global__ void __launch_bounds__(256, 4) rope_kernel(const __grid_constant__ RopeArgs a) {
  // (cos, sin) of the CTA's tokens (32 at most), two pairs a chunk: lane l's chunk i of a token lies at 4l + (i ^ l/2),
  // so that the eight lanes of a token read from different banks.
  __shared__ float4 turned_by[32][kD / 4];
  const uint32_t g0 = blockIdx.x * 32u, token0 = g0 / (uint32_t)a.slices, rest = g0 - token0 * a.slices;
  const uint32_t local = rest + (threadIdx.x >> 3), at = local / (uint32_t)a.slices, token = token0 + at;
  const int l = threadIdx.x & 7;
  const uint32_t b = token / (uint32_t)a.T, t = token - b * a.T;
  const int h0 = (int)(local - at * a.slices) * a.per, h1 = token < a.tokens ? min(h0 + a.per, a.heads) : 0;
  const bool turned = l < a.rot / 16;
  // kBatch heads' loads in flight before the first store (which the compiler cannot move them across)
  uint4 u[kBatch], w[kBatch];
  uint16_t* dst[kBatch];
  const auto load = [&](int hb) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = hb + i;
      if (h >= h1) break;
      const uint16_t* src;
      if (h < a.Hq) {
        src = a.q + b * a.lq.b + t * a.lq.t + h * a.lq.h;
        dst[i] = a.q_out + b * a.oq.b + t * a.oq.t + h * a.oq.h;
      } else if (h < a.Hq + a.Hkv) {
        src = a.k + b * a.lk.b + t * a.lk.t + (h - a.Hq) * a.lk.h;
        dst[i] = a.k_out + b * a.ok.b + t * a.ok.t + (h - a.Hq) * a.ok.h;
      } else {
        src = a.v + b * a.lv.b + t * a.lv.t + (h - a.Hq - a.Hkv) * a.lv.h;
        dst[i] = a.v_out + b * a.ov.b + t * a.ov.t + (h - a.Hq - a.Hkv) * a.ov.h;
      }
      const bool rot = turned && h < a.Hq + a.Hkv;
      u[i] = *reinterpret_cast<const uint4*>(src + (!INTERLEAVED && rot ? 8 * l : 16 * l));
      w[i] = *reinterpret_cast<const uint4*>(src + (!INTERLEAVED && rot ? 8 * l + a.rot / 2 : 16 * l + 8));
    }
  };
  load(h0);  // on its way while the angles are formed
  const uint32_t here = min((rest + 31u) / (uint32_t)a.slices + 1u, a.tokens - token0);  // tokens of the CTA
  for (uint32_t i = threadIdx.x; i < here * (kD / 2); i += 256) {
    const uint32_t n = i / (kD / 2), pair = i % (kD / 2);
    if (pair >= (uint32_t)a.rot / 2) continue;
    const uint64_t p = (uint64_t)(int64_t)a.pos[token0 + n];
    const int32_t turn = (int32_t)((p * a.turns[pair]) >> 32);
    float c, s;
    sincospif((float)turn * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    reinterpret_cast<float2*>(&turned_by[n][(pair >> 1) ^ (pair >> 4)])[pair & 1] = make_float2(c * a.mscale, s * a.mscale);
  }
  __syncthreads();
  float c[8], s[8];
  if (turned && h0 < min(h1, a.Hq + a.Hkv)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = turned_by[at][(4 * l + i) ^ (l >> 1)];
      c[2 * i] = x.x;
      s[2 * i] = x.y;
      c[2 * i + 1] = x.z;
      s[2 * i + 1] = x.w;
    }
  }
  for (int hb = h0; hb < h1;) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = hb + i;
      if (h >= h1) break;
      const bool rot = turned && h < a.Hq + a.Hkv;
      if (rot) turn_pairs<INTERLEAVED>(u[i], w[i], c, s);
      *reinterpret_cast<uint4*>(dst[i] + (!INTERLEAVED && rot ? 8 * l : 16 * l)) = u[i];
      *reinterpret_cast<uint4*>(dst[i] + (!INTERLEAVED && rot ? 8 * l + a.rot / 2 : 16 * l + 8)) = w[i];
    }
    hb += kBatch;
    load(hb);
  }
}

}  // namespace

spc_status launch_rope(const spc_rope_dims* d, const int32_t* pos, const uint64_t* turns, const uint16_t* q,
                       const uint16_t* k, const uint16_t* v, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out,
                       cudaStream_t stream) {
  RopeArgs a = {q, k, v, q_out, k_out, v_out, pos, turns, d->q, d->k, d->v, d->q_out, d->k_out, d->v_out};
  const int64_t tokens = (int64_t)d->B * d->T;
  a.T = d->T;
  a.Hq = d->Hq;
  a.Hkv = d->Hkv;
  a.heads = d->Hq + (v != nullptr ? 2 : 1) * d->Hkv;
  a.rot = d->rot;
  a.mscale = d->mscale;
  // Few tokens: a head per group of lanes, for latency; many: up to four heads
  // once that leaves 128 groups for each SM (1024 tokens of 48 heads 5.5 us,
  // with 256 7.0; 32768 tokens 122 us, 127 with two heads and 124 with eight).
  const int64_t rows = tokens * a.heads, fill = (int64_t)spc_host::sm_count() * 128;
  a.per = (int32_t)std::max<int64_t>(1, std::min<int64_t>(4, rows / fill));
  a.slices = (a.heads + a.per - 1) / a.per;
  if (tokens * a.slices > 0x7FFFFFFF) return SPC_ERR_UNSUPPORTED;
  a.tokens = (uint32_t)tokens;
  const int64_t blocks = (tokens * a.slices + 31) / 32;
  if (d->interleaved)
    rope_kernel<true><<<(unsigned)blocks, 256, 0, stream>>>(a);
  else
    rope_kernel<false><<<(unsigned)blocks, 256, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace spc
