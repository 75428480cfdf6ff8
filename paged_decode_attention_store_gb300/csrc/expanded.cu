// Causal attention of ragged prompts in the expanded form of latent attention:
// the general CUDA-core kernel and the C entry point.
//
// Mathematics. Head h's key of token t is [k_t,h | r_t] (its own nope_dim
// entries and rope_dim rotated ones that all heads share), its value v_t,h:
// s_t = scale (<q_nope, k_t,h> + <q_rope, r_t>), o = sum_t softmax(s)_t v_t,h.
// Request b's queries are its last tokens: query j of q_len sits at position
// k_len - q_len + j and attends positions up to its own.
#include "attention.cuh"
#include "expanded.cuh"

namespace kvp {

namespace {

constexpr int kExpWarps = 8;
constexpr int kExpPer = kExpandedMaxDim / 32;

__device__ __forceinline__ float exp_f(float x) { return x; }
__device__ __forceinline__ float exp_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T exp_t(float x);
template <>
__device__ __forceinline__ float exp_t<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 exp_t<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One block per (request, query token, head), for fp32 and the shapes the
// tensor-core kernel does not take: warp w takes keys w, w + 8, ..., lanes
// over the entries, an online softmax per warp, joined through shared memory.
template <typename T>
__global__ void __launch_bounds__(32 * kExpWarps) expanded_general_kernel(const ExpandedCall a) {
  __shared__ float qs[2 * kExpandedMaxDim];
  __shared__ float part[kExpWarps][kExpandedMaxDim];
  __shared__ float pm[kExpWarps], pl[kExpWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (int)(blockIdx.x % a.H), j = (int)((blockIdx.x / a.H) % a.max_q);
  const int b = (int)(blockIdx.x / ((long long)a.H * a.max_q));
  const ExpandedRequest r = expanded_request(a, b);
  if (!r.ok) {
    if (h == 0 && j == 0 && threadIdx.x == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
    return;
  }
  if (j >= r.ql) return;
  const T* q = static_cast<const T*>(a.q) + (size_t)(r.q0 + j) * a.q_stride + (size_t)h * a.q_head_stride;
  const int width = a.dn + a.dr;
  for (int d = threadIdx.x; d < width; d += 32 * kExpWarps) qs[d] = exp_f(q[d]);
  __syncthreads();
  const int n = r.kl - r.ql + j + 1;
  float acc[kExpPer];
#pragma unroll
  for (int i = 0; i < kExpPer; ++i) acc[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  const float sl2 = a.scale * 1.4426950408889634f;
  for (int t = warp; t < n; t += kExpWarps) {
    const size_t tok = (size_t)(r.k0 + t);
    const T* k = static_cast<const T*>(a.k) + tok * a.k_stride + (size_t)h * a.k_head_stride;
    const T* pe = static_cast<const T*>(a.k_pe) + tok * a.k_pe_stride;
    const T* v = static_cast<const T*>(a.v) + tok * a.v_stride + (size_t)h * a.v_head_stride;
    float dot = 0.f;
    for (int d = lane; d < a.dn; d += 32) dot = fmaf(qs[d], exp_f(k[d]), dot);
    for (int d = lane; d < a.dr; d += 32) dot = fmaf(qs[a.dn + d], exp_f(pe[d]), dot);
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, sh);
    const float s = dot * sl2;
    const float mn = fmaxf(m, s);
    const bool none = s == -INFINITY && m == -INFINITY;  // nothing yet: its value still meets a weight of 0
    const float alpha = none ? 1.f : exp2f(m - mn), p = none ? 0.f : exp2f(s - mn);
    l = l * alpha + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < kExpPer; ++i)
      if (lane + 32 * i < a.dv) acc[i] = fmaf(p, exp_f(v[lane + 32 * i]), acc[i] * alpha);
  }
#pragma unroll
  for (int i = 0; i < kExpPer; ++i)
    if (lane + 32 * i < a.dv) part[warp][lane + 32 * i] = acc[i];
  if (lane == 0) {
    pm[warp] = m;
    pl[warp] = l;
  }
  __syncthreads();
  float mx = pm[0];
#pragma unroll
  for (int w = 1; w < kExpWarps; ++w) mx = fmaxf(mx, pm[w]);
  float f[kExpWarps], tot = 0.f;
#pragma unroll
  for (int w = 0; w < kExpWarps; ++w) {
    f[w] = pm[w] == -INFINITY ? 0.f : exp2f(pm[w] - mx);
    tot += f[w] * pl[w];
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  T* out = static_cast<T*>(a.out) + ((size_t)(r.q0 + j) * a.H + h) * a.dv;
  for (int d = threadIdx.x; d < a.dv; d += 32 * kExpWarps) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kExpWarps; ++w) o = fmaf(f[w], part[w][d], o);
    out[d] = exp_t<T>(o * inv);
  }
}

}  // namespace

}  // namespace kvp

using namespace kvp;

extern "C" int latent_prefill_attention(const void* q, long long q_stride, long long q_head_stride, const void* k,
                                        long long k_stride, long long k_head_stride, const void* k_pe,
                                        long long k_pe_stride, const void* v, long long v_stride,
                                        long long v_head_stride, const int32_t* q_start, const int32_t* k_start,
                                        int batch, int num_heads, int max_q, int total_q, int total_k, int nope_dim,
                                        int rope_dim, int v_dim, int dtype, float scale, void* out,
                                        int32_t* error_word, void* stream) {
  if (!q_start || !k_start || batch <= 0 || num_heads <= 0 || max_q < 0 || total_q < 0 || total_k < 0)
    return KVP_ERR_INVALID_ARG;
  if (nope_dim <= 0 || rope_dim < 0 || v_dim <= 0 || nope_dim > kExpandedMaxDim || rope_dim > kExpandedMaxDim ||
      v_dim > kExpandedMaxDim)
    return KVP_ERR_INVALID_ARG;
  if (dtype != KVP_F32 && dtype != KVP_BF16) return KVP_ERR_INVALID_ARG;
  if (!(scale - scale == 0.f)) return KVP_ERR_INVALID_ARG;
  if (max_q == 0 || total_q == 0) return KVP_OK;  // no query
  if (!q || !k || !v || !out || (rope_dim > 0 && !k_pe)) return KVP_ERR_INVALID_ARG;
  // inputs are only read: rows and heads may lie in any order, or be the same (a stride of zero)
  if (q_stride < 0 || q_head_stride < 0 || k_stride < 0 || k_head_stride < 0 || v_stride < 0 || v_head_stride < 0 ||
      (rope_dim > 0 && k_pe_stride < 0))
    return KVP_ERR_INVALID_ARG;
  const uintptr_t em = dtype == KVP_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(k_pe) | reinterpret_cast<uintptr_t>(out)) & em)
    return KVP_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVP_ERR_CUDA;
  for (const void* p : {q, k, k_pe, v, static_cast<const void*>(out), static_cast<const void*>(q_start),
                        static_cast<const void*>(k_start), static_cast<const void*>(error_word)}) {  // another device's memory
    cudaPointerAttributes at;
    if (!p) continue;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) return KVP_ERR_CUDA;
    if (at.type == cudaMemoryTypeDevice && at.device != dev) return KVP_ERR_INVALID_ARG;
  }
  if (max_q > total_q) max_q = total_q;
  ExpandedCall a;
  a.q = q;
  a.k = k;
  a.k_pe = k_pe;
  a.v = v;
  a.out = out;
  a.q_stride = q_stride;
  a.q_head_stride = q_head_stride;
  a.k_stride = k_stride;
  a.k_head_stride = k_head_stride;
  a.k_pe_stride = k_pe_stride;
  a.v_stride = v_stride;
  a.v_head_stride = v_head_stride;
  a.q_start = q_start;
  a.k_start = k_start;
  a.B = batch;
  a.H = num_heads;
  a.max_q = max_q;
  a.total_q = total_q;
  a.total_k = total_k;
  a.dn = nope_dim;
  a.dr = rope_dim;
  a.dv = v_dim;
  a.scale = scale;
  a.err = error_word;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (expanded_tc_eligible(a, dtype)) return launch_expanded_tc(a, st);
  const long long blocks = (long long)batch * max_q;
  if (blocks > 0x7fffffffLL / num_heads) return KVP_ERR_INVALID_ARG;
  const unsigned grid = (unsigned)(blocks * num_heads);
  if (dtype == KVP_F32) expanded_general_kernel<float><<<grid, 32 * kExpWarps, 0, st>>>(a);
  else expanded_general_kernel<__nv_bfloat16><<<grid, 32 * kExpWarps, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}
