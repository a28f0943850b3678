// Norms of query and key heads with the rotation by their positions in the
// same pass, and the copy of the value rows, from the projection to where they
// are used:
//   y_j = x_j w_j / sqrt(mean(x^2) + eps),  pair i of y turned by
//   pos[axis[i]] * turns[i] (mod 2^64, 64-bit fractions of a turn: exact).
// The rotation and the root are one linear map of x * w, so the root's
// reciprocal multiplies the turned elements, and its latency lies under the
// rotation.  Sums, norm and rotation are binary32; one rounding, at the store.
//
// Eight lanes hold a head's row, two runs of eight elements each, so that the
// lanes' runs lie side by side: in the half layout lane l < rot/16 elements
// 8l .. and rot/2 + 8l .. (the pairs 8l ..), the others rot/2 + 8l .. and
// 64 + 8l .., which are not turned; interleaved, 8l .. and 64 + 8l ...  (With
// 16 elements in a row to a lane, each copy reads half sectors, twice: a
// 32768-token prompt 156 us against 122.)  Three shuffles join the lanes' sums of squares.  A CTA forms the
// angles of its tokens once, in shared memory; a group of eight lanes walks
// over a few heads of one kind (queries, keys or values) of a token, so that
// what depends on the kind is settled before the loop.
// Bound by HBM (every row is read and written once): a 32768-token prompt of 32
// + 8 + 8 heads (805 MB) takes 121 us, 99% of the measured copy rate.  What it
// took: coefficients that join weights and angles, formed once per group of
// lanes, packed binary32 pairs, addresses that only step (177 to 150 us), and
// copies of two heads in flight in shared memory, where they take no registers
// (150 to 122 us; at four CTAs an SM with a few registers spilled 146).
#include <algorithm>
#include <cstring>

#include "common.cuh"

namespace spc {
namespace {

constexpr int kStages = 3;    // of a thread's copies: two heads in flight while one is computed
constexpr int kMostHeads = 8;  // that a group of lanes walks over

// Rows of one kind.
struct NormRows {
  const uint16_t* in;
  uint16_t* out;
  const float* weight;  // null: not normed
  spc_layout li, lo;
  int32_t heads, slices;  // slices of `per` heads
};

struct NormRopeArgs {
  NormRows kind[3];  // queries, keys, values
  const int32_t* pos;
  const uint64_t* turns;
  uint32_t tokens;  // B * T
  int32_t T, rot, per, slices;
  float mscale, eps;
  uint8_t axis[kD / 2];  // of positions, of each pair
};

__device__ __forceinline__ uint32_t norm_pack(float2 x) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(x.y), "f"(x.x));
  return r;
}

// The row's sum of squares (x: the lane's elements; row: the row's lanes).
__device__ __forceinline__ float row_squares(const float2* x, uint32_t row) {
  float2 sum = f2_mul(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) sum = f2_fma(x[i], x[i], sum);
  float all = sum.x + sum.y;
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) all += __shfl_xor_sync(row, all, off);
  return all;
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(256, 3) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  // (cos, sin) of the CTA's tokens (32 at most), two pairs a chunk: chunk i of a token lies at i ^ (i / 8), so that the
  // eight lanes of a token, four chunks each, read from different banks.
  __shared__ float4 turned_by[32][kD / 4];
  __shared__ float4 weights[2][kD / 4];
  __shared__ uint4 rows[kStages][512];
  const uint32_t g0 = blockIdx.x * 32u, token0 = g0 / (uint32_t)a.slices, rest = g0 - token0 * a.slices;
  const uint32_t local = rest + (threadIdx.x >> 3), at = local / (uint32_t)a.slices, token = token0 + at;
  const int l = threadIdx.x & 7;
  int slice = (int)(local - at * a.slices), kind = 0;
  if (slice >= a.kind[0].slices) {
    slice -= a.kind[0].slices;
    kind = 1;
    if (slice >= a.kind[1].slices) {
      slice -= a.kind[1].slices;
      kind = 2;
    }
  }
  const NormRows& r = a.kind[kind];
  const int h0 = slice * a.per;
  const int n = token < a.tokens ? min(a.per, r.heads - h0) : 0;  // heads of the group
  const bool norm = r.weight != nullptr, first = l < a.rot / 16;
  const int at_u = INTERLEAVED || first ? 8 * l : a.rot / 2 + 8 * l;
  const int at_w = INTERLEAVED || !first ? 64 + 8 * l : a.rot / 2 + 8 * l;
  // whether the lane's runs are turned
  const bool turn_u = kind < 2 && (INTERLEAVED ? at_u < a.rot : first), turn_w = kind < 2 && (INTERLEAVED ? at_w < a.rot : first);
  const uint32_t b = token / (uint32_t)a.T, t = token - b * a.T;
  const uint16_t* src = r.in + b * r.li.b + t * r.li.t + h0 * r.li.h + at_u;
  uint16_t* dst = r.out + b * r.lo.b + t * r.lo.t + h0 * r.lo.h + at_u;
  const int64_t step_in = r.li.h, step_out = r.lo.h;
  // Every thread copies its own elements, so it alone waits for them.
  const auto load = [&](int i) {
    if (i < n) {
      uint4* to = rows[i % kStages] + threadIdx.x;
      cp_async16(to, src);
      cp_async16(to + 256, src + (at_w - at_u));
      src += step_in;
    }
    cp_async_commit();
  };
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // launched while the kernel before in the stream ends
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i);  // on their way while the angles are formed
  {
    const float* from = a.kind[threadIdx.x / kD].weight;
    if (from != nullptr) reinterpret_cast<float*>(weights)[threadIdx.x] = from[threadIdx.x % kD];
  }
  const uint32_t here = min((rest + 31u) / (uint32_t)a.slices + 1u, a.tokens - token0);  // tokens of the CTA
  for (uint32_t i = threadIdx.x; i < here * (kD / 2); i += 256) {
    const uint32_t m = i / (kD / 2), pair = i % (kD / 2);
    if (pair >= (uint32_t)a.rot / 2) continue;
    const uint64_t p = (uint64_t)(int64_t)a.pos[(int64_t)a.axis[pair] * a.tokens + token0 + m];
    const int32_t turn = (int32_t)((p * a.turns[pair]) >> 32);
    float c, s;
    sincospif((float)turn * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    reinterpret_cast<float2*>(&turned_by[m][(pair >> 1) ^ (pair >> 4)])[pair & 1] = make_float2(c * a.mscale, s * a.mscale);
  }
  __syncthreads();
  // The lane's coefficients: weights w of its elements and (cos, sin) of its pairs as one map of each pair (half layout:
  // two pairs a float2; interleaved: x's and y's products of one pair), or the weights alone where it does not turn.
  float2 ca[8], cb[8];
  {
    const float4 *wu = weights[kind & 1] + at_u / 4, *ww = weights[kind & 1] + at_w / 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = norm ? (i < 2 ? wu[i] : ww[i - 2]) : make_float4(1.f, 1.f, 1.f, 1.f);
      ca[2 * i] = {x.x, x.y};
      ca[2 * i + 1] = {x.z, x.w};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int chunk = INTERLEAVED ? 2 * l + (i < 2 ? i : 14 + i) : 4 * l + i;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      const bool turn = INTERLEAVED && i >= 2 ? turn_w : turn_u;
      if (turn) x = turned_by[at][chunk ^ (chunk >> 3)];  // (cos, sin) of pairs 2 chunk and 2 chunk + 1
      if (INTERLEAVED) {                                  // x' = x ca.x + y cb.x, y' = x ca.y + y cb.y
#pragma unroll
        for (int j = 2 * i; j < 2 * i + 2; ++j) {
          const float cj = j & 1 ? x.z : x.x, sj = j & 1 ? x.w : x.y;
          cb[j] = f2_mul({ca[j].y, ca[j].y}, {-sj, cj});
          if (turn) ca[j] = f2_mul({ca[j].x, ca[j].x}, {cj, sj});
        }
      } else {  // x' = x ca[i] + y cb[i], y' = x cb[4 + i] + y ca[4 + i]
        cb[i] = f2_mul(ca[4 + i], {-x.y, -x.w});
        cb[4 + i] = f2_mul(ca[i], {x.y, x.w});
        if (turn) {
          ca[i] = f2_mul(ca[i], {x.x, x.z});
          ca[4 + i] = f2_mul(ca[4 + i], {x.x, x.z});
        }
      }
    }
  }
  const uint32_t row = 0xFFu << (threadIdx.x & 24u);
  for (int i = 0; i < n; ++i) {
    cp_async_wait<kStages - 2>();
    const uint4 u = rows[i % kStages][threadIdx.x], w = rows[i % kStages][threadIdx.x + 256];
    load(i + kStages - 1);  // where the head before lay
    uint32_t bits[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
    if (norm || turn_u || turn_w) {
      float2 x[8];  // u's elements, then w's
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = {__uint_as_float(bits[j] << 16), __uint_as_float(bits[j] & 0xFFFF0000u)};
      float root = 1.f;
      if (norm) {  // alike for the row's lanes
        float sum = row_squares(x, row), eps = a.eps;
        if (sum == INFINITY) {  // elements from 2^60 on: their squares overflow, those of 2^-70 of them do not
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = f2_mul(x[j], {8.470329472543003e-22f, 8.470329472543003e-22f});
          sum = row_squares(x, row);
          eps = 0.f;
        }
        root = rsqrtf(fmaf(sum, 1.f / kD, eps));
      }
      if (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j < 4 ? turn_u : turn_w)  // (packed, each element would first be copied into both halves of a pair)
            x[j] = {fmaf(x[j].x, ca[j].x, x[j].y * cb[j].x), fmaf(x[j].x, ca[j].y, x[j].y * cb[j].y)};
          else
            x[j] = f2_mul(x[j], ca[j]);
        }
      } else if (turn_u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = f2_fma(x[j], ca[j], f2_mul(x[4 + j], cb[j]));
          x[4 + j] = f2_fma(x[j], cb[4 + j], f2_mul(x[4 + j], ca[4 + j]));
          x[j] = y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = f2_mul(x[j], ca[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)  // what is neither normed nor turned stays as it is, bit by bit
        if (norm || (j < 4 ? turn_u : turn_w)) bits[j] = norm_pack(f2_mul(x[j], {root, root}));
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(bits[0], bits[1], bits[2], bits[3]);
    *reinterpret_cast<uint4*>(dst + (at_w - at_u)) = make_uint4(bits[4], bits[5], bits[6], bits[7]);
    dst += step_out;
  }
}

}  // namespace

spc_status launch_norm_rope(const spc_norm_rope_dims* dn, const int32_t* pos, const uint64_t* turns,
                            const float* q_weight, const float* k_weight, const uint16_t* q, const uint16_t* k,
                            const uint16_t* v, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out, cudaStream_t stream) {
  const spc_rope_dims* d = &dn->rope;
  NormRopeArgs a = {};
  a.kind[0] = {q, q_out, q_weight, d->q, d->q_out, d->Hq, 0};
  a.kind[1] = {k, k_out, k_weight, d->k, d->k_out, d->Hkv, 0};
  a.kind[2] = {v, v_out, nullptr, d->v, d->v_out, v != nullptr ? d->Hkv : 0, 0};
  a.pos = pos;
  a.turns = turns;
  const int64_t tokens = (int64_t)d->B * d->T;
  a.T = d->T;
  a.rot = d->rot;
  a.mscale = d->mscale;
  a.eps = dn->eps;
  std::memcpy(a.axis, dn->axis, sizeof(a.axis));
  // Few tokens: a head per group of lanes, for latency; many: up to eight heads
  // once that leaves 128 groups for each SM (32768 tokens 121 us, 135 with four
  // and 131 with 16; 4096 tokens 19.3, 20.9 and 21.3).
  const int64_t rows = tokens * (a.kind[0].heads + a.kind[1].heads + a.kind[2].heads);
  const int64_t fill = (int64_t)spc_host::sm_count() * 128;
  a.per = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kMostHeads, rows / fill));
  for (NormRows& r : a.kind) {
    r.slices = (r.heads + a.per - 1) / a.per;
    a.slices += r.slices;
  }
  if (tokens * a.slices > 0x7FFFFFFF) return SPC_ERR_UNSUPPORTED;
  a.tokens = (uint32_t)tokens;
  const int64_t blocks = (tokens * a.slices + 31) / 32;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, d->interleaved ? norm_rope_kernel<true> : norm_rope_kernel<false>, a);
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace spc
