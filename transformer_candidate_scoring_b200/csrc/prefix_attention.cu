// Attention of sequences that share their request's prefix (tr_prefix_attention).
//
// For query token (s, t) and head h of request r, over the request's prefix keys and then the
// keys of the sequence's own suffix:
//     a_j = scale q.k_j,   m = max_j a_j,   l = sum_j exp(a_j - m),   o = sum_j exp(a_j - m) v_j / l
// with m, l and o carried from key to key (a new maximum rescales l and o), so that no score is
// ever stored.  Exponentials are powers of two: a_j is kept times log2(e).
#include <math.h>

#include <algorithm>

#include "model.cuh"

namespace tr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRowWarps = 4;
constexpr int kMaxDHead = 128;

struct AttnParams {
  const void *q, *k_prefix, *v_prefix, *k_suffix, *v_suffix;
  const int32_t* suffix_len;
  void* out;
  float* lse;
  int* status;
  tr_attn_desc d;
  int R;
  int64_t n_rows;
  int64_t seq[TR_MAX_REQUESTS + 1];
  int64_t prefix[TR_MAX_REQUESTS + 1];
};

__device__ __forceinline__ int request_of(const int64_t* seq, int R, int64_t s) {
  int lo = 0, hi = R - 1;          // the last request that starts at or before s and is not empty
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq[mid] <= s) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Suffix keys that query token t of sequence s sees; a length outside the buffer is clamped.
__device__ __forceinline__ int visible_suffix(const AttnParams& p, int64_t s, int t) {
  if (p.d.suffix_cap == 0) return 0;
  int len = p.suffix_len[s];
  if (len < 0 || len > p.d.suffix_cap) {
    if ((threadIdx.x & 31) == 0) atomicOr(p.status, STATUS_KEY_RANGE);
    len = min(max(len, 0), p.d.suffix_cap);
  }
  return p.d.causal ? max(0, len - (p.d.L_t - 1 - t)) : len;
}

// One warp per (s, t, head): 32 keys at a time, each lane one key's product with the query, then
// each lane some of the output columns.
template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32) attn_row_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float sq[kRowWarps][kMaxDHead];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t row = (int64_t)blockIdx.x * kRowWarps + warp;
  if (row >= p.n_rows) return;
  const int D = p.d.d_head, H = p.d.n_head;
  const int h = (int)(row % H);
  const int64_t st = row / H, s = st / p.d.L_t;
  const int t = (int)(st % p.d.L_t), hk = h / (H / p.d.n_kv_head);
  const int r = request_of(p.seq, p.R, s);
  const T* q = static_cast<const T*>(p.q) + st * p.d.q_token + (int64_t)h * D;
  for (int i = lane; i < D; i += 32) sq[warp][i] = to_f32(q[i]);
  __syncwarp();
  const float c = p.d.scale * kLog2e;
  float m = -INFINITY, l = 0.f, o[kMaxDHead / 32] = {};
  auto keys = [&](const T* k, const T* v, int64_t stride, int64_t n) {
    for (int64_t j0 = 0; j0 < n; j0 += 32) {
      const int64_t j = j0 + lane;
      float a = -INFINITY;
      if (j < n) {
        const T* kr = k + j * stride;
        constexpr int N = 16 / sizeof(T);
        float acc = 0.f;
        for (int i = 0; i < D; i += N) {
          T kv[N];
          *reinterpret_cast<uint4*>(kv) = *reinterpret_cast<const uint4*>(kr + i);
#pragma unroll
          for (int e = 0; e < N; ++e) acc = fmaf(sq[warp][i + e], to_f32(kv[e]), acc);
        }
        a = acc * c;
      }
      float bm = a;
#pragma unroll
      for (int x = 16; x; x >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, x));
      const float nm = fmaxf(m, bm);
      const float base = nm == -INFINITY ? 0.f : nm;    // keys of -inf weigh nothing, NaN stays NaN
      const float f = exp2f(m - base), w = exp2f(a - base);
      float ws = w;
#pragma unroll
      for (int x = 16; x; x >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, x);
      l = l * f + ws;
      m = nm;
#pragma unroll
      for (int i = 0; i < kMaxDHead / 32; ++i) o[i] *= f;
      const int cnt = (int)min((int64_t)32, n - j0);
      for (int e = 0; e < cnt; ++e) {
        const float we = __shfl_sync(0xffffffffu, w, e);
        const T* vr = v + (j0 + e) * stride;
#pragma unroll
        for (int i = 0; i < kMaxDHead / 32; ++i)
          if (lane + 32 * i < D) o[i] = fmaf(we, to_f32(vr[lane + 32 * i]), o[i]);
      }
    }
  };
  const int64_t po = p.prefix[r] * p.d.prefix_token + hk * p.d.prefix_head;
  keys(static_cast<const T*>(p.k_prefix) + po, static_cast<const T*>(p.v_prefix) + po, p.d.prefix_token,
       p.prefix[r + 1] - p.prefix[r]);
  const int64_t so = s * p.d.suffix_seq + hk * p.d.suffix_head;
  keys(static_cast<const T*>(p.k_suffix) + so, static_cast<const T*>(p.v_suffix) + so, p.d.suffix_token,
       visible_suffix(p, s, t));
  T* out = static_cast<T*>(p.out) + row * D;
  const float inv = l == 0.f ? 0.f : 1.f / l;   // (a NaN score gives a NaN row)
#pragma unroll
  for (int i = 0; i < kMaxDHead / 32; ++i)
    if (lane + 32 * i < D) out[lane + 32 * i] = from_f32<T>(o[i] * inv);
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

tr_status check_offsets(const tr_attn_desc* d, const int64_t* seq, const int64_t* prefix, int R) {
  if (!d) return fail(TR_ERR_INVALID_ARG, "desc is null");
  if (d->dtype != TR_F32 && d->dtype != TR_BF16) return fail(TR_ERR_INVALID_ARG, "dtype=%d", (int)d->dtype);
  if (d->n_kv_head < 1 || d->n_head < 1 || d->n_head > 1024 || d->n_head % d->n_kv_head)
    return fail(TR_ERR_INVALID_ARG, "n_head=%d, n_kv_head=%d: need a multiple of n_kv_head, 1..1024", d->n_head, d->n_kv_head);
  if (d->d_head < 8 || d->d_head % 8 || d->d_head > kMaxDHead)
    return fail(TR_ERR_UNSUPPORTED, "d_head=%d: need a multiple of 8 <= %d", d->d_head, kMaxDHead);
  if (d->L_t < 1 || d->L_t > TR_MAX_LT) return fail(TR_ERR_INVALID_ARG, "L_t=%d (need 1..%d)", d->L_t, TR_MAX_LT);
  if (d->causal != 0 && d->causal != 1) return fail(TR_ERR_INVALID_ARG, "causal=%d", d->causal);
  if (d->suffix_cap < 0) return fail(TR_ERR_INVALID_ARG, "suffix_cap=%d", d->suffix_cap);
  if (!isfinite(d->scale)) return fail(TR_ERR_INVALID_ARG, "scale is not finite");
  const int64_t unit = d->dtype == TR_F32 ? 4 : 8;
  const int64_t strides[6] = {d->q_token, d->prefix_token, d->prefix_head, d->suffix_seq, d->suffix_token, d->suffix_head};
  for (int i = 0; i < 6; ++i)
    if (strides[i] < 0 || strides[i] % unit || strides[i] > (1ll << 38))
      return fail(TR_ERR_INVALID_ARG, "stride %d = %lld elements: need a non-negative multiple of 16 bytes", i, (long long)strides[i]);
  if (R < 1 || R > TR_MAX_REQUESTS) return fail(TR_ERR_INVALID_ARG, "R=%d (need 1..%d)", R, TR_MAX_REQUESTS);
  if (!seq || !prefix) return fail(TR_ERR_INVALID_ARG, "null host array");
  if (seq[0] != 0) return fail(TR_ERR_INVALID_ARG, "seq_offsets must start at 0");
  if (prefix[0] < 0) return fail(TR_ERR_INVALID_ARG, "prefix_offsets must not be negative");
  for (int r = 0; r < R; ++r) {
    if (seq[r + 1] < seq[r]) return fail(TR_ERR_INVALID_ARG, "seq_offsets decrease at %d", r);
    if (prefix[r + 1] < prefix[r]) return fail(TR_ERR_INVALID_ARG, "prefix_offsets decrease at %d", r);
  }
  if (prefix[R] > INT32_MAX) return fail(TR_ERR_UNSUPPORTED, "2^31 or more prefix tokens");
  if (seq[R] > INT32_MAX || seq[R] * d->L_t * d->n_head > (int64_t)INT32_MAX)
    return fail(TR_ERR_UNSUPPORTED, "2^31 or more query rows (n * L_t * n_head)");
  return TR_OK;
}

}  // namespace
}  // namespace tr

using namespace tr;

extern "C" size_t tr_prefix_attention_workspace(const tr_attn_desc* desc, const int64_t* seq_offsets,
                                                const int64_t* prefix_offsets, int R) {
  if (check_offsets(desc, seq_offsets, prefix_offsets, R) != TR_OK) return SIZE_MAX;
  return 0;
}

extern "C" tr_status tr_prefix_attention(const tr_attn_desc* desc, const void* q, const int64_t* seq_offsets,
                                         const void* k_prefix, const void* v_prefix, const int64_t* prefix_offsets,
                                         const void* k_suffix, const void* v_suffix, const int32_t* suffix_len, int R,
                                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                                         tr_stream stream) {
  TR_TRY(check_offsets(desc, seq_offsets, prefix_offsets, R));
  const int64_t n = seq_offsets[R];
  if (n == 0) return TR_OK;
  if (!q || !out) return fail(TR_ERR_INVALID_ARG, "null device pointer");
  if (prefix_offsets[R] > prefix_offsets[0] && (!k_prefix || !v_prefix))
    return fail(TR_ERR_INVALID_ARG, "k_prefix or v_prefix is null");
  if (desc->suffix_cap > 0 && (!k_suffix || !v_suffix || !suffix_len))
    return fail(TR_ERR_INVALID_ARG, "k_suffix, v_suffix or suffix_len is null");
  if (((uintptr_t)q | (uintptr_t)k_prefix | (uintptr_t)v_prefix | (uintptr_t)k_suffix | (uintptr_t)v_suffix |
       (uintptr_t)out) % 16)
    return fail(TR_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  if ((uintptr_t)suffix_len % 4 || (uintptr_t)lse % 4) return fail(TR_ERR_INVALID_ARG, "suffix_len or lse is not aligned to its type");
  DeviceState* ds = nullptr;
  TR_TRY(device_state(&ds));
  const cudaStream_t st = (cudaStream_t)stream;
  AttnParams p{};
  p.q = q;
  p.k_prefix = k_prefix;
  p.v_prefix = v_prefix;
  p.k_suffix = k_suffix;
  p.v_suffix = v_suffix;
  p.suffix_len = suffix_len;
  p.out = out;
  p.lse = lse;
  p.status = ds->status;
  p.d = *desc;
  p.R = R;
  p.n_rows = n * desc->L_t * desc->n_head;
  for (int r = 0; r <= R; ++r) {
    p.seq[r] = seq_offsets[r];
    p.prefix[r] = prefix_offsets[r];
  }
  (void)workspace;
  (void)workspace_bytes;
  const unsigned grid = (unsigned)((p.n_rows + kRowWarps - 1) / kRowWarps);
  if (desc->dtype == TR_F32)
    attn_row_kernel<float><<<grid, kRowWarps * 32, 0, st>>>(p);
  else
    attn_row_kernel<__nv_bfloat16><<<grid, kRowWarps * 32, 0, st>>>(p);
  TR_LAUNCH_CHECK("attn_row_kernel");
  return TR_OK;
}
