// The prefix part of tr_prefix_attention in fp32 on the CUDA cores.
//
// As in the tensor-core kernel, a request's query rows of one key head form one matrix against
// its shared keys; a CTA takes 64 (or, of few rows, 16) of them over a chunk of the prefix, 64 keys
// at a time: S = Q K^T, the running maximum and sum, P = 2^(c S - c m) through shared memory,
// O += P V.  Products are pairs of fp32 FMAs (one instruction for two); a thread holds 8 x 4
// scores and 8 x 8 outputs, so that an operand read from shared memory feeds four to eight of
// them.  The K of the next step is copied while P V runs, the V of this one while S is formed.
// FMA throughput (2 d_head x 2 per row and key) bounds it for many rows, the read of K and V for
// few.  3 x 37 sequences of 3 query tokens, 6 heads of 80 on 2, prefixes of up to 1501 tokens: 31 us (38 with
// d_head padded to 128), 216 CTAs of two steps at about one warp per scheduler; the FMA pipes are 23 % busy.
#include <math.h>

#include <algorithm>

#include "prefix_attention.cuh"

namespace tr {
namespace attn {
namespace {

constexpr int kThreads = 128, kN = kStepKeysF32;

__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t r) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int RT, int DP>     // rows per thread (8 threads down), d_head padded to 64, 96 or 128
struct Layout {
  static constexpr int BM = 8 * RT, KP = DP + 4;
  static constexpr int Q = 0, K = Q + BM * DP, V = K + kN * KP, P = V + kN * DP;
  static constexpr int BYTES = (P + kN * BM) * 4;
};
static_assert(2 * (Layout<8, 128>::BYTES + 1024) <= 233472, "two CTAs per SM");

// Keys `first` .. of a step into shared memory, rows at `pitch` floats; rows behind the chunk as zeros.
__device__ __forceinline__ void copy_keys(float* dst, int pitch, const float* src, int64_t stride, int n, int D) {
  const int chunks = D / 4;
  for (int i = threadIdx.x; i < kN * chunks; i += kThreads) {
    const int j = i / chunks, c = i % chunks;
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(dst + j * pitch + c * 4);
    const int bytes = j < n ? 16 : 0;                     // 0: the destination is zeroed
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(src + (j < n ? j : 0) * stride + c * 4), "r"(bytes)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int RT, int DP>
__global__ void __launch_bounds__(kThreads, 2) prefix_f32_kernel(const __grid_constant__ AttnParams p) {
  using L = Layout<RT, DP>;
  // columns of O per thread: CB blocks of VW neighbours, the blocks 16 VW apart
  constexpr int VW = DP % 64 ? 2 : 4, CB = DP / (16 * VW), NP = CB * VW / 2;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm + L::Q, *sk = sm + L::K, *sv = sm + L::V, *sp = sm + L::P;
  const Unit x = unit_at(p, blockIdx.x, L::BM, kN);
  const RequestPlan& rq = p.req[x.r];
  const int D = p.d.d_head, H = p.d.n_head, G = H / p.d.n_kv_head;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t ko = x.tok * p.d.prefix_token + x.hk * p.d.prefix_head;
  const float *kp = static_cast<const float*>(p.k_prefix) + ko, *vp = static_cast<const float*>(p.v_prefix) + ko;
  cudaTriggerProgrammaticLaunchCompletion();
  copy_keys(sk, L::KP, kp, p.d.prefix_token, x.keys, D);
  copy_keys(sv, DP, vp, p.d.prefix_token, x.keys, D);
  // Q, times scale log2(e)
  const float c = p.d.scale * kLog2e;
  for (int i = threadIdx.x; i < L::BM * (D / 4); i += kThreads) {
    const int r = i / (D / 4), e = i % (D / 4), m = x.m0 + r;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < x.rows) {
      const int64_t token = (int64_t)rq.s0 * p.d.L_t + m / G;
      v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + token * p.d.q_token + (int64_t)(x.hk * G + m % G) * D) + e);
    }
    *reinterpret_cast<float4*>(sq + r * DP + 4 * e) = make_float4(v.x * c, v.y * c, v.z * c, v.w * c);
  }
  float mx[RT], l[RT];
  uint64_t o[RT][NP];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    mx[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < NP; ++e) o[i][e] = 0;
  }
  for (int step = 0; step < x.steps; ++step) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // K of this step (V may be on its way)
    __syncthreads();
    // ---- S: rows ty + 8 i, keys tx + 16 j
    uint64_t s[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0;
#pragma unroll 2
    for (int e = 0; e < D; e += 4) {
      ulonglong2 k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 16 * j) * L::KP + e);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(sq + (ty + 8 * i) * DP + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = fma2(q.y, k[j].y, fma2(q.x, k[j].x, s[i][j]));
      }
    }
    const int valid = x.keys - step * kN;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float a[4], top = mx[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = unpair(s[i][j]);
        a[j] = tx + 16 * j < valid ? y.x + y.y : -INFINITY;
        top = fmaxf(top, a[j]);
      }
#pragma unroll
      for (int y = 8; y; y >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
      const float base = top == -INFINITY ? 0.f : top;    // keys of -inf weigh nothing, NaN stays NaN
      const float f = exp2f(mx[i] - base);
      mx[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = exp2f(a[j] - base);
        sum += a[j];
        // row position ty RT + i, its groups of eight turned by the key against bank conflicts
        const int key = tx + 16 * j, pos = ty * RT + i;
        sp[key * L::BM + (pos ^ ((key & (L::BM / 8 - 1)) << 3))] = a[j];
      }
      l[i] = l[i] * f + sum;                              // (this lane's keys only)
      const uint64_t f2 = pair(f, f);
#pragma unroll
      for (int e = 0; e < NP; ++e) o[i][e] = mul2(o[i][e], f2);
    }
    __syncthreads();
    if (step + 1 < x.steps)
      copy_keys(sk, L::KP, kp + (int64_t)(step + 1) * kN * p.d.prefix_token, p.d.prefix_token, valid - kN, D);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // V of this step
    __syncthreads();
    // ---- O += P V: columns VW (tx + 16 b) ..
#pragma unroll 4
    for (int key = 0; key < kN; ++key) {
      uint64_t v[NP];
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const float* src = sv + key * DP + VW * (tx + 16 * b);
        if constexpr (VW == 4)
          *reinterpret_cast<ulonglong2*>(v + 2 * b) = *reinterpret_cast<const ulonglong2*>(src);
        else
          v[b] = *reinterpret_cast<const uint64_t*>(src);
      }
      float w[RT];
      const float* pr = sp + key * L::BM + ((ty * RT) ^ ((key & (L::BM / 8 - 1)) << 3));
      if constexpr (RT == 8) {
        *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(pr);
        *reinterpret_cast<float4*>(w + 4) = *reinterpret_cast<const float4*>(pr + 4);
      } else {
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = pr[i];
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const uint64_t w2 = pair(w[i], w[i]);
#pragma unroll
        for (int e = 0; e < NP; ++e) o[i][e] = fma2(w2, v[e], o[i][e]);
      }
    }
    __syncthreads();
    if (step + 1 < x.steps)
      copy_keys(sv, DP, vp + (int64_t)(step + 1) * kN * p.d.prefix_token, p.d.prefix_token, valid - kN, D);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // ---- this chunk's result
  const int64_t rows = request_rows(p, x.r);
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int y = 8; y; y >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], y);
    const int r = ty + 8 * i, m = x.m0 + r;
    if (r >= x.rows) continue;
    const int64_t part = rq.part + x.split * rows + (int64_t)(m / G) * H + x.hk * G + m % G;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    if (tx == 0) p.part_lse[part] = l[i] == 0.f ? -INFINITY : mx[i] + log2f(l[i]);
#pragma unroll
    for (int b = 0; b < CB; ++b)
      if (VW * (tx + 16 * b) < D) {
#pragma unroll
        for (int e = 0; e < VW / 2; ++e) {
          const float2 y = unpair(o[i][b * VW / 2 + e]);
          *reinterpret_cast<float2*>(p.part_o + part * D + VW * (tx + 16 * b) + 2 * e) = make_float2(y.x * inv, y.y * inv);
        }
      }
  }
}

template <int RT, int DP>
tr_status launch(const AttnParams& p, cudaStream_t st) {
  TR_TRY(ensure_smem_attr((const void*)prefix_f32_kernel<RT, DP>, Layout<RT, DP>::BYTES));
  prefix_f32_kernel<RT, DP><<<p.n_units, kThreads, Layout<RT, DP>::BYTES, st>>>(p);
  TR_LAUNCH_CHECK("prefix_f32_kernel");
  return TR_OK;
}

}  // namespace

tr_status launch_prefix_f32(const AttnParams& p, int unit_rows, cudaStream_t st) {
  const int D = p.d.d_head;
  if (unit_rows == 64) return D <= 64 ? launch<8, 64>(p, st) : D <= 96 ? launch<8, 96>(p, st) : launch<8, 128>(p, st);
  return D <= 64 ? launch<2, 64>(p, st) : D <= 96 ? launch<2, 96>(p, st) : launch<2, 128>(p, st);
}

}  // namespace attn
}  // namespace tr
