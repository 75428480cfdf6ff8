// One call of latent_prefill_attention, as its kernels take it.
#pragma once

#include "common.cuh"

namespace kvp {

constexpr int kExpandedMaxDim = 512;  // of each of nope_dim, rope_dim and v_dim

struct ExpandedCall {
  const void* q;
  const void* k;
  const void* k_pe;
  const void* v;
  void* out;  // [total_q, H, dv]
  long long q_stride, q_head_stride, k_stride, k_head_stride, k_pe_stride, v_stride, v_head_stride;  // elements
  const int32_t* q_start;
  const int32_t* k_start;
  int B, H, max_q, total_q, total_k, dn, dr, dv;
  float scale;
  int32_t* err;
};

// Request b's rows: queries q0 .. q0 + ql - 1, keys k0 .. k0 + kl - 1. Not ok
// (offsets out of order or past the tensors, more queries than max_q or than
// keys): the request is skipped.
struct ExpandedRequest {
  int q0, ql, k0, kl;
  bool ok;
};

__device__ __forceinline__ ExpandedRequest expanded_request(const ExpandedCall& a, int b) {
  ExpandedRequest r;
  const long long q0 = a.q_start[b], q1 = a.q_start[b + 1], k0 = a.k_start[b], k1 = a.k_start[b + 1];
  r.ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k && q1 - q0 <= a.max_q &&
         q1 - q0 <= k1 - k0;
  r.q0 = (int)q0;
  r.ql = (int)(q1 - q0);
  r.k0 = (int)k0;
  r.kl = (int)(k1 - k0);
  return r;
}

// The tcgen05 kernel (expanded_tc.cu): whether it takes a call, and its launch.
bool expanded_tc_eligible(const ExpandedCall& c, int dtype);
int launch_expanded_tc(const ExpandedCall& c, cudaStream_t stream);

}  // namespace kvp
