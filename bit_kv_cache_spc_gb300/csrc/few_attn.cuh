// The attention of single tokens: one query token per sequence, G <= 16 query
// heads over each KV head, whose keys are those that the token sees (a window
// and the first tokens, or all), optionally joined with the partial results
// that another launch left of a shared prefix.
//
// Bound by the bytes of K and V.  The tiles of prompt_attn.cuh need 128 rows and
// about 4 us from a CTA's start to its first scores; here the 16 rows of one
// mma.sync product hold the G heads, and what counts is the copies in flight:
// each of four warps walks over its own blocks of 16 keys, with three stages of
// 8 KB that it alone fills (cp.async) and waits for.  Two CTAs an SM keep 128 KB
// on their way.  S = Q K^T is 16 x 16 x 128, O += P V 16 x 128 x 16, both in
// registers; the tensor cores are busy a fifth of the time.
// Every row of a CTA sees the same keys, so keys that are not seen are not
// copied at all: zeros stand in their places, and masked infinities and NaN
// cannot reach a product.
// The keys of one sequence and KV head are shared out to the CTAs of a cluster
// (1 to 8), which join their warps' results through each other's shared memory:
// no partial results in memory and no launch to join them.
// Eight tokens with a window of 4096 over 8 KV heads (126 MB): 23.3 us, 80% of
// the measured copy rate (by prompt_attn.cuh's tiles 34.5); 64 of them over up
// to 4100 keys 146 us (1.07 GB, above that rate).
//
// P in bf16: the product's operand type, as in prompt_attn.cuh.
#pragma once

#include "prompt_attn.cuh"

namespace spc {
namespace {

constexpr int kFewKeys = 16;     // a block
constexpr int kFewWarps = 4;
constexpr int kFewStages = 3;
constexpr int kFewStageBytes = 2 * kFewKeys * kD * 2;  // K, then V
constexpr int kFewWarpBytes = kFewStages * kFewStageBytes;
constexpr int kFewRowFloats = kD + 4;  // of a warp's result in shared memory: rows start in different banks
constexpr int kFewSmemBytes = kFewWarps * kFewWarpBytes + kFewWarps * kFewRows * 8;
constexpr int kFewCluster = 8;   // CTAs at most
constexpr int kFewLoads = 16;    // of the prefix's splits' results in flight
static_assert(kFewRows * kFewRowFloats * 4 <= kFewWarpBytes, "a warp's result outgrows its stages");
static_assert(2 * (kFewSmemBytes + 1024) <= 233472, "more shared memory than two CTAs have");

// Copies 16 bytes, or fills in zeros.
__device__ __forceinline__ void copy_or_zero(uint32_t to, const void* from, bool copy, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n" ::"r"(to), "l"(from), "r"(copy ? 16 : 0),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void load_matrices_turned(uint32_t addr, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c (16 x 8) += a (16 x 16) b (16 x 8), bf16 in, binary32 sums
__device__ __forceinline__ void mma_bf16(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool PREFIX>
__global__ void __launch_bounds__(32 * kFewWarps, 2) few_attn_kernel(const __grid_constant__ PromptArgs a) {
  extern __shared__ __align__(1024) uint8_t few_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % a.few_ctas), hkv = (int)(blockIdx.x / a.few_ctas % a.Hkv);
  const int s = (int)(blockIdx.x / a.few_ctas / a.Hkv);
  // Launched while the kernel before in the stream ends.  (Behind a prefix's launch, which has waited for the ones before
  // it, only that launch's results are waited for, below.)
  if (!PREFIX) asm volatile("griddepcontrol.wait;\n" ::: "memory");
  int lq, lk, qb, kb;
  sequence(a, s, lq, lk, qb, kb);
  if (lq == 0) {  // in all CTAs of the cluster
    if (PREFIX) asm volatile("griddepcontrol.wait;\n" ::: "memory");  // what comes behind this launch comes behind both
    return;
  }
  // Keys that the token sees: the first `ns` and those from `low` on, numbered through.
  const int low = a.window > 0 ? max(0, lk - a.window) : 0, ns = min(a.sinks, low), n = ns + lk - low;
  const int blocks = (n + kFewKeys - 1) / kFewKeys;
  const int b0 = (int)((int64_t)blocks * rank / a.few_ctas) + warp, b1 = (int)((int64_t)blocks * (rank + 1) / a.few_ctas);
  const uint32_t mine = smem_addr(few_smem) + warp * kFewWarpBytes;
  const int seq_q = a.q_batched ? s : 0, seq_k = a.k_batched ? s : 0;

  // ---- copies: a lane takes chunk lane % 16 of every second row ----
  const uint16_t* kp = a.k + seq_k * a.k_b + (int64_t)kb * a.k_t + hkv * a.k_h + (lane & 15) * 8;
  const uint16_t* vp = a.v + seq_k * a.v_b + (int64_t)kb * a.v_t + hkv * a.v_h + (lane & 15) * 8;
  const uint64_t policy = l2_policy(true);
  const auto load = [&](int it) {
    const int b = b0 + it * kFewWarps;
    if (b < b1) {
      const uint32_t to = mine + (it % kFewStages) * kFewStageBytes;
#pragma unroll
      for (int i = 0; i < kFewKeys / 2; ++i) {
        const int row = 2 * i + (lane >> 4), x = kFewKeys * b + row;
        const bool there = x < n;
        const int64_t key = there ? (x < ns ? x : x + (low - ns)) : 0;
        const uint32_t at = to + row * 256 + (((lane & 15) ^ (row & 7)) << 4);  // so that eight rows' chunks lie in all banks
        copy_or_zero(at, kp + key * a.k_t, there, policy);
        copy_or_zero(at + kFewStageBytes / 2, vp + key * a.v_t, there, policy);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kFewStages - 1; ++i) load(i);

  // ---- the query rows as operands: rows lane / 4 and 8 behind it, channels 2 (lane % 4) on ----
  uint32_t q[8][4];
  {
    const uint16_t* qp = a.q + seq_q * a.q_b + (int64_t)qb * a.q_t + (int64_t)hkv * a.G * a.q_h + (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = (lane >> 2) + 8 * (u & 1);
        q[k][u] = row < a.G ? *reinterpret_cast<const uint32_t*>(qp + row * a.q_h + 16 * k + 8 * (u >> 1)) : 0u;
      }
  }
  const float c = a.scale * kLog2e;
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 16; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) o[t][u] = 0.f;

  for (int it = 0; b0 + it * kFewWarps < b1; ++it) {
    cp_async_wait<kFewStages - 2>();
    __syncwarp();  // all lanes' copies are there, and the block before has been read
    load(it + kFewStages - 1);
    const uint32_t ks = mine + (it % kFewStages) * kFewStageBytes, vs = ks + kFewStageBytes / 2;
    float x[2][4] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t r[4];
      const int row = ((lane >> 4) << 3) + (lane & 7);
      load_matrices(ks + row * 256 + (((2 * k + ((lane >> 3) & 1)) ^ (row & 7)) << 4), r);
      mma_bf16(x[0], q[k], r[0], r[1]);
      mma_bf16(x[1], q[k], r[2], r[3]);
    }
    const int left = n - (b0 + it * kFewWarps) * kFewKeys;
    if (left < kFewKeys) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (8 * t + 2 * (lane & 3) + (u & 1) >= left) x[t][u] = -INFINITY;
    }
    float mx[2];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 2));
      if (!(mx[r] > m[r] && !((mx[r] - m[r]) * c <= kSlack))) mx[r] = m[r];
      grow |= mx[r] != m[r];
    }
    if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = mx[r] == m[r] ? 1.f : fast_exp2((m[r] - mx[r]) * c);  // m = -inf: 0
        m[r] = mx[r];
        l[r] *= f;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          o[t][2 * r] *= f;
          o[t][2 * r + 1] *= f;
        }
      }
    }
    uint32_t p[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float mc = m[r] == -INFINITY ? 0.f : m[r] * c;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float e0 = fast_exp2(fmaf(x[t][2 * r], c, -mc)), e1 = fast_exp2(fmaf(x[t][2 * r + 1], c, -mc));
        l[r] += e0 + e1;
        p[2 * t + r] = pack_bf16x2(e0, e1);
      }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      uint32_t r[4];
      const int row = (((lane >> 3) & 1) << 3) + (lane & 7);
      load_matrices_turned(vs + row * 256 + (((2 * t + (lane >> 4)) ^ (row & 7)) << 4), r);
      mma_bf16(o[2 * t], p, r[0], r[1]);
      mma_bf16(o[2 * t + 1], p, r[2], r[3]);
    }
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---- the warp's result: (maximum, sum) and the weighted sum of each row ----
  const uint32_t ml_at = smem_addr(few_smem) + kFewWarps * kFewWarpBytes;
  float* res = reinterpret_cast<float*>(few_smem + warp * kFewWarpBytes);
  float2* ml = reinterpret_cast<float2*>(few_smem + kFewWarps * kFewWarpBytes) + warp * kFewRows;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
    l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
    const int row = (lane >> 2) + 8 * r;
    if ((lane & 3) == 0) ml[row] = make_float2(l[r] == 0.f ? -INFINITY : m[r] * c, l[r]);
    if (row < a.G) {
#pragma unroll
      for (int t = 0; t < 16; ++t)
        *reinterpret_cast<float2*>(res + row * kFewRowFloats + 8 * t + 2 * (lane & 3)) = make_float2(o[t][2 * r], o[t][2 * r + 1]);
    }
  }
  if (a.few_ctas > 1)
    cluster_sync();
  else
    __syncthreads();
  if (PREFIX) asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the prefix's partial results are there

  // ---- joined: a warp per row, four channels a lane; lane j holds warp j's maximum and sum, and the prefix's splits' ----
  const int parts = kFewWarps * a.few_ctas, splits = PREFIX ? a.p_splits : 0;
  for (int row = rank * kFewWarps + warp; row < a.G; row += parts) {
    const int head = hkv * a.G + row;
    float2 in = make_float2(-INFINITY, 0.f), out[2] = {in, in};
    float4 x[kFewLoads];
    int64_t first = 0, step = 0;  // the row among the prefix's partial results, and from one split to the next
    const auto load_parts = [&](int z0) {
#pragma unroll
      for (int u = 0; u < kFewLoads; ++u)
        if (z0 + u < splits) x[u] = shared_part(a, first + (z0 + u) * step, lane);
    };
    if (PREFIX) {
      first = shared_row(a, 0, s, qb, 0, head);
      step = (int64_t)a.Hkv * a.row_tiles * kTile;
      load_parts(0);
    }
    if (lane < parts) in = cluster_ld2(cluster_addr(ml_at + ((lane & 3) * kFewRows + row) * 8, lane >> 2));
    if (PREFIX) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (lane + 32 * u < splits) out[u] = a.part_ml[first + (lane + 32 * u) * step];
    }
    float top = fmaxf(in.x, fmaxf(out[0].x, out[1].x));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    const auto weight = [&](float2 x) { return x.y == 0.f ? 0.f : exp2f(x.x - top); };  // a sum of 0: nothing visible there
    const float f = weight(in), g[2] = {weight(out[0]), weight(out[1])};
    float sum = f * in.y + g[0] * out[0].y + g[1] * out[1].y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](float w, float4 x) { y = make_float4(y.x + w * x.x, y.y + w * x.y, y.z + w * x.z, y.w + w * x.w); };
    if (PREFIX) {
      for (int z0 = 0; z0 < splits; z0 += kFewLoads) {
        if (z0 > 0) load_parts(z0);
#pragma unroll
        for (int u = 0; u < kFewLoads; ++u) {
          const int z = z0 + u;
          const float w = __shfl_sync(0xFFFFFFFFu, z < 32 ? g[0] : g[1], z & 31);
          const float total = __shfl_sync(0xFFFFFFFFu, z < 32 ? out[0].y : out[1].y, z & 31);
          if (z < splits && total != 0.f) add(w, x[u]);
        }
      }
    }
    for (int j = 0; j < parts; ++j) {
      const float w = __shfl_sync(0xFFFFFFFFu, f, j), total = __shfl_sync(0xFFFFFFFFu, in.y, j);
      if (total == 0.f) continue;
      const uint32_t at = smem_addr(few_smem) + (j & 3) * kFewWarpBytes + (row * kFewRowFloats + 4 * lane) * 4;
      add(w, cluster_ld4(cluster_addr(at, j >> 2)));
    }
    bool any = n > 0;
    if (PREFIX) any = any || (a.p_len ? clampi(a.p_len[0], 0, a.p_tokens) : a.p_tokens) > 0;
    const float inv = any ? 1.f / sum : 0.f;
    uint2* po = reinterpret_cast<uint2*>(a.o + s * a.o_b + (int64_t)qb * a.o_t + head * a.o_h) + lane;
    *po = make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
    if (lane == 0 && a.lse) a.lse[lse_place(a, s, qb, head)] = any ? top * kLn2 + logf(sum) : -INFINITY;
  }
  if (a.few_ctas > 1) cluster_sync();  // its shared memory has been read
}

// CTAs that share a sequence's keys: as many as fill the SMs' places in equal turns, while a warp has four blocks or more
// (of the longest sequence).
int few_cluster(const spc_prompt_dims* d, int64_t keys) {
  const int64_t items = (int64_t)d->S * d->Hkv, places = 2 * spc_host::sm_count();
  int best = 1;
  double least = 0.0;
  for (int n = 1; n <= kFewCluster; n *= 2) {
    const int64_t blocks = ceil_div(ceil_div(keys, kFewKeys), kFewWarps * n);
    if (n > 1 && (blocks < 4 || items * n > (1 << 24))) break;
    const double cost = (double)ceil_div(items * n, places) * (double)(blocks + 10);
    if (n == 1 || cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

template <bool PREFIX>
spc_status launch_few(PromptArgs& a, const spc_prompt_dims* d, cudaStream_t stream) {
  const int64_t keys = a.window > 0 ? std::min<int64_t>(d->k_max, (int64_t)a.window + a.sinks) : d->k_max;
  a.few_ctas = few_cluster(d, keys);
  static unsigned long long configured = 0ull;
  cudaError_t e = spc_host::ensure_smem_limit(configured, few_attn_kernel<PREFIX>, kFewSmemBytes);
  if (e == cudaSuccess) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.few_ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)a.S * a.Hkv * a.few_ctas));
    cfg.blockDim = dim3(32 * kFewWarps);
    cfg.dynamicSmemBytes = kFewSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, few_attn_kernel<PREFIX>, a);
  }
  if (e != cudaSuccess) {
    spc_host::set_cuda_error(e);
    return SPC_ERR_CUDA;
  }
  return SPC_OK;
}

}  // namespace
}  // namespace spc
