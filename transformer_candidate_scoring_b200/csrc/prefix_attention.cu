// Attention of sequences that share their request's prefix (tr_prefix_attention).
//
// For query token (s, t) and head h of request r, over the request's prefix keys and then the
// keys of the sequence's own suffix:
//     a_j = scale q.k_j,   m = max_j a_j,   l = sum_j exp(a_j - m),   o = sum_j exp(a_j - m) v_j / l
// with m, l and o carried from key to key (a new maximum rescales l and o), so that no score is
// ever stored.  Exponentials are powers of two: a_j is kept times log2(e).
#include <math.h>

#include <algorithm>

#include "prefix_attention.cuh"

namespace tr {
namespace attn {
namespace {

constexpr int kRowWarps = 4;

__device__ __forceinline__ int request_of(const AttnParams& p, int64_t s) {
  int lo = 0, hi = p.R - 1;        // the last request that starts at or before s and is not empty
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.req[mid].s0 <= s) lo = mid; else hi = mid - 1;
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
// each lane some of the output columns.  With kPartial the prefix part of the row has been
// computed (launch_prefix_tc): its partial results are merged instead of the prefix being read.
template <typename T, bool kPartial>
__global__ void __launch_bounds__(kRowWarps * 32) attn_row_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float sq[kRowWarps][kMaxDHead];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t row = (int64_t)blockIdx.x * kRowWarps + warp;
  if (row >= p.n_rows) return;
  const int D = p.d.d_head, H = p.d.n_head;
  const int h = (int)(row % H);
  const int64_t st = row / H, s = st / p.d.L_t;
  const int t = (int)(st % p.d.L_t), hk = h / (H / p.d.n_kv_head);
  const int r = request_of(p, s);
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
  const RequestPlan& rq = p.req[r];
  if constexpr (kPartial) {
    const int64_t rows = request_rows(p, r);
    for (int i = 0; i < rq.n_split; ++i) {
      const int64_t at = rq.part + i * rows + (row - (int64_t)rq.s0 * p.d.L_t * H);
      const float z = p.part_lse[at];
      if (z == -INFINITY) continue;
      const float nm = fmaxf(m, z), f = exp2f(m - nm), w = exp2f(z - nm);
      l = l * f + w;
      m = nm;
#pragma unroll
      for (int e = 0; e < kMaxDHead / 32; ++e)
        if (lane + 32 * e < D) o[e] = o[e] * f + w * p.part_o[at * D + lane + 32 * e];
    }
  } else {
    const int64_t po = rq.p0 * p.d.prefix_token + hk * p.d.prefix_head;
    keys(static_cast<const T*>(p.k_prefix) + po, static_cast<const T*>(p.v_prefix) + po, p.d.prefix_token, rq.p1 - rq.p0);
  }
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
  if (!(isfinite(d->scale) && d->scale > 0)) return fail(TR_ERR_INVALID_ARG, "scale=%g: need a positive number", (double)d->scale);
  const int64_t unit = d->dtype == TR_F32 ? 4 : 8;
  const int64_t strides[6] = {d->q_token, d->prefix_token, d->prefix_head, d->suffix_seq, d->suffix_token, d->suffix_head};
  for (int i = 0; i < (d->suffix_cap > 0 ? 6 : 3); ++i)
    if (strides[i] <= 0 || strides[i] % unit || strides[i] > (1ll << 38))
      return fail(TR_ERR_INVALID_ARG, "stride %d = %lld elements: need a positive multiple of 16 bytes", i, (long long)strides[i]);
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

// How many steps of 128 keys a unit takes.  Fewer steps give more units to spread over the SMs,
// but every unit costs about three tile steps (Q, the first scores, the result) and every chunk of
// a prefix a partial result per row.  The candidates are: no split, and the shortest chunks that
// give one, two or four units per SM.
void plan_units(AttnParams& p, int sms) {
  const int G = p.d.n_head / p.d.n_kv_head;
  int steps[TR_MAX_REQUESTS], n_m[TR_MAX_REQUESTS];
  int longest = 0;
  int64_t rows_all = 0;
  bool two = false;
  for (int r = 0; r < p.R; ++r) {
    const int64_t m = (int64_t)(p.req[r].s1 - p.req[r].s0) * p.d.L_t * G;
    steps[r] = m > 0 ? ceil_div(p.req[r].p1 - p.req[r].p0, kStepKeys) : 0;
    n_m[r] = ceil_div(m, kUnitRows);
    two = two || m > kUnitRows / 2;
    longest = std::max(longest, steps[r]);
    rows_all += request_rows(p, r);
  }
  auto units = [&](int c) {
    int64_t n = 0;
    for (int r = 0; r < p.R; ++r) n += (int64_t)p.d.n_kv_head * n_m[r] * ceil_div(steps[r], c);
    return n;
  };
  int best = std::max(longest, 1);
  double best_cost = 1e300;
  for (int w = 0; w <= 4 && longest > 0; w = w ? 2 * w : 1) {
    int c = longest;
    if (w > 0) {
      int lo = 1, hi = longest;               // units(c) falls with c
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (units(mid) <= (int64_t)w * sms) hi = mid; else lo = mid + 1;
      }
      c = lo;
    }
    // tile steps of the busiest SM (about 0.7 us each), and the partial results' traffic
    const double waves = (double)((units(c) + sms - 1) / sms);
    const double split = (double)ceil_div(longest, c);
    const double bytes = split > 1 ? (double)rows_all * split * p.d.d_head * 8.0 : 0.0;
    const double cost = waves * (c * (two ? 2.0 : 1.0) + 3.0) + bytes / 3.5e6;
    if (cost < best_cost) {
      best_cost = cost;
      best = c;
    }
  }
  int unit = 0;
  int64_t part = 0;
  for (int r = 0; r < p.R; ++r) {
    RequestPlan& q = p.req[r];
    q.first_unit = unit;
    q.chunk = best;
    q.n_split = ceil_div(steps[r], best);
    q.part = part;
    unit += p.d.n_kv_head * n_m[r] * q.n_split;
    part += request_rows(p, r) * q.n_split;
  }
  p.req[p.R].first_unit = p.n_units = unit;
  p.req[p.R].part = part;
}

// The plan of a call; p.n_units is 0 where the row kernel reads the prefixes itself.
struct Plan {
  bool direct = false;        // the tensor-core kernel writes the results
  size_t bytes = 0;
};
tr_status make_plan(const tr_attn_desc* d, const int64_t* seq, const int64_t* prefix, int R, AttnParams& p, Plan& plan) {
  TR_TRY(check_offsets(d, seq, prefix, R));
  p.d = *d;
  p.R = R;
  p.n_rows = seq[R] * d->L_t * d->n_head;
  for (int r = 0; r <= R; ++r) {
    RequestPlan& q = p.req[r];
    q.s0 = (int)seq[r];
    q.p0 = (int)prefix[r];
    q.s1 = (int)seq[std::min(r + 1, R)];
    q.p1 = (int)prefix[std::min(r + 1, R)];
  }
  p.n_units = 0;
  if (d->dtype != TR_BF16) return TR_OK;
  int dev = 0, sms = 0;
  TR_CUDA_TRY(cudaGetDevice(&dev));
  TR_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  plan_units(p, sms);
  plan.direct = d->suffix_cap == 0;
  for (int r = 0; r < R; ++r) plan.direct = plan.direct && (p.req[r].n_split == 1 || p.req[r].s0 == p.req[r].s1);
  if (!plan.direct) plan.bytes = (size_t)p.req[R].part * (d->d_head + 1) * sizeof(float);
  return TR_OK;
}

}  // namespace
}  // namespace attn
}  // namespace tr

using namespace tr;
using namespace tr::attn;

extern "C" size_t tr_prefix_attention_workspace(const tr_attn_desc* desc, const int64_t* seq_offsets,
                                                const int64_t* prefix_offsets, int R) {
  AttnParams p{};
  Plan plan;
  return make_plan(desc, seq_offsets, prefix_offsets, R, p, plan) == TR_OK ? plan.bytes : SIZE_MAX;
}

extern "C" tr_status tr_prefix_attention(const tr_attn_desc* desc, const void* q, const int64_t* seq_offsets,
                                         const void* k_prefix, const void* v_prefix, const int64_t* prefix_offsets,
                                         const void* k_suffix, const void* v_suffix, const int32_t* suffix_len, int R,
                                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                                         tr_stream stream) {
  TR_TRY(check_offsets(desc, seq_offsets, prefix_offsets, R));
  if (seq_offsets[R] == 0) return TR_OK;
  if (!q || !out) return fail(TR_ERR_INVALID_ARG, "null device pointer");
  if (prefix_offsets[R] > prefix_offsets[0] && (!k_prefix || !v_prefix))
    return fail(TR_ERR_INVALID_ARG, "k_prefix or v_prefix is null");
  if (desc->suffix_cap > 0 && (!k_suffix || !v_suffix || !suffix_len))
    return fail(TR_ERR_INVALID_ARG, "k_suffix, v_suffix or suffix_len is null");
  if (((uintptr_t)q | (uintptr_t)k_prefix | (uintptr_t)v_prefix | (uintptr_t)k_suffix | (uintptr_t)v_suffix |
       (uintptr_t)out) % 16)
    return fail(TR_ERR_INVALID_ARG, "a device pointer is not 16-byte aligned");
  if ((uintptr_t)suffix_len % 4 || (uintptr_t)lse % 4) return fail(TR_ERR_INVALID_ARG, "suffix_len or lse is not aligned to its type");
  AttnParams p{};
  Plan plan;
  TR_TRY(make_plan(desc, seq_offsets, prefix_offsets, R, p, plan));
  if (plan.bytes > 0 && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < plan.bytes))
    return fail(TR_ERR_INVALID_ARG, "workspace: need %zu bytes, 16-byte aligned", plan.bytes);
  DeviceState* ds = nullptr;
  TR_TRY(device_state(&ds));
  const cudaStream_t st = (cudaStream_t)stream;
  p.q = q;
  p.k_prefix = k_prefix;
  p.v_prefix = v_prefix;
  p.k_suffix = k_suffix;
  p.v_suffix = v_suffix;
  p.suffix_len = suffix_len;
  p.out = out;
  p.lse = lse;
  p.status = ds->status;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + p.req[R].part * desc->d_head;
  if (p.n_units > 0) TR_TRY(launch_prefix_tc(p, plan.direct, st));
  if (plan.direct) return TR_OK;
  const unsigned grid = (unsigned)((p.n_rows + kRowWarps - 1) / kRowWarps);
  if (desc->dtype == TR_F32)
    attn_row_kernel<float, false><<<grid, kRowWarps * 32, 0, st>>>(p);
  else
    attn_row_kernel<__nv_bfloat16, true><<<grid, kRowWarps * 32, 0, st>>>(p);
  TR_LAUNCH_CHECK("attn_row_kernel");
  return TR_OK;
}
