// Shared by the kernels of tr_prefix_attention: the call's parameters, and how the work over a
// request's prefix is cut into units and its partial results are stored.
#pragma once

#include "common.cuh"

namespace tr {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxDHead = 128;
constexpr int kStepKeys = 128;      // keys of one step of the tensor-core kernel
constexpr int kUnitRows = 256;      // query rows of a unit (two tiles of 128)

// The prefix part of one request: rows = sequences x query tokens x heads of a key head.  A unit
// is up to 256 rows of one key head over `chunk` steps of 128 keys; a prefix of several chunks
// gives each row several partial results.
struct RequestPlan {
  int first_unit;      // units of request r: first_unit[r] .. first_unit[r+1]-1
  int n_split;         // chunks of the prefix (0: no prefix or no sequences)
  int chunk;           // steps per chunk
  int p0, p1;          // prefix tokens
  int s0, s1;          // sequences
  int64_t part;        // the request's first partial result
};

struct AttnParams {
  const void *q, *k_suffix, *v_suffix, *k_prefix, *v_prefix;
  const int32_t* suffix_len;
  void* out;
  float* lse;
  int* status;
  tr_attn_desc d;
  int R, n_units;
  int64_t n_rows;      // query rows of all requests: n * L_t * n_head
  // partial result i of row `row` of request r (its rows counted from 0, head fastest) is
  // part_o[(part + i * rows of r + row) * d_head ..] and part_lse[the same] (times log2 e)
  float *part_o, *part_lse;
  RequestPlan req[TR_MAX_REQUESTS + 1];
};

__host__ __device__ inline int64_t request_rows(const AttnParams& p, int r) {
  return (int64_t)(p.req[r].s1 - p.req[r].s0) * p.d.L_t * p.d.n_head;
}

// Launches the tensor-core kernel over every unit of the plan (bf16).  With `direct`, each row
// has one partial result and no suffix: out and lse are written instead of it.
tr_status launch_prefix_tc(const AttnParams& p, bool direct, cudaStream_t st);

}  // namespace attn
}  // namespace tr
