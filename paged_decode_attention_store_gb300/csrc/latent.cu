// Attention over a paged cache of latent rows, absorbed form: the general
// CUDA-core kernel and the C entry points.
//
// Mathematics. A token's row is x = [c | r]: its latent c (latent_dim) and one
// rotated key part r (rope_dim), shared by all heads. Head h's key is W_h^K c
// with r appended and its value W_h^V c, so with the projections moved to the
// query and the output (q^ = [(W_h^K)^T q_nope | q_rope], o = W_h^V o^) a step is
// multi-query attention: s_t = scale <q^, x_t>, o^ = sum_t softmax(s)_t c_t.
// One row of (latent_dim + rope_dim) elements is read for all heads.
#include "attention.cuh"

namespace kvp {

namespace {

constexpr int kLatWarps = 8;

struct LatGenArgs {
  TableRef T;
  const char* layer;
  const void* q;
  void* out;
  const int32_t* context_lens;
  const int32_t* table_rows;
  const int32_t* q_lens;
  int B, C, H, dc, width, window, sinks;
  float scale_log2;
  int32_t* err;
};

__device__ __forceinline__ float lat_f(float x) { return x; }
__device__ __forceinline__ float lat_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T lat_t(float x);
template <>
__device__ __forceinline__ float lat_t<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 lat_t<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One block per (request, query token, head), for fp32 caches and the shapes
// the tensor-core kernel does not take. Warp w takes rows w, w + 8, ... of the
// span; its lanes hold the row (lane l: elements l, l + 32, ...), so a row is
// read once for its score and its value; each warp keeps an online softmax in
// log2 units and the eight are joined through shared memory. PER: floats a
// lane holds of the latent (32 PER >= latent_dim).
template <typename T, int PER>
__global__ void __launch_bounds__(32 * kLatWarps) latent_general_kernel(const LatGenArgs a) {
  extern __shared__ float lat_smem[];
  float* qs = lat_smem;                   // [width]
  float* part = qs + a.width;             // [warps][dc]
  __shared__ float pm[kLatWarps], pl[kLatWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long wid = blockIdx.x;
  const long long bj = wid / a.H;
  const int b = (int)(bj / a.C), j = (int)(bj % a.C);
  T* out = static_cast<T*>(a.out) + (size_t)wid * a.dc;
  const T* q = static_cast<const T*>(a.q) + (size_t)wid * a.width;
  const int Lr = a.context_lens[b];
  const int row = a.table_rows ? a.table_rows[b] : b;
  const int Mb = a.q_lens ? a.q_lens[b] : a.C;
  if (Mb < 1 || Mb > a.C || Lr < Mb || Lr > table_capacity(a.T) || row < 0 || row >= a.T.rows_total) {
    if (j == 0 && threadIdx.x == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
    for (int d = threadIdx.x; d < a.dc; d += 32 * kLatWarps) out[d] = lat_t<T>(0.f);
    return;
  }
  if (j >= Mb) return;
  const int L = Lr - Mb + j + 1;  // the query token's own context (causal)
  for (int d = threadIdx.x; d < a.width; d += 32 * kLatWarps) qs[d] = lat_f(q[d]);
  __syncthreads();
  const Span sp = attend_span(L, a.window, a.sinks);
  const int n = sp.se + L - sp.lo;
  float acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int o = warp; o < n; o += kLatWarps) {
    const int slot = resolve_slot(a.T, row, span_pos(sp, o), a.err);
    if (slot < 0) continue;
    const T* x = reinterpret_cast<const T*>(a.layer) + (size_t)slot * a.width;
    float xr[PER];
    float dot = 0.f, odd = 0.f;  // odd: NaN once an entry is not finite, whatever it meets in q
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int d = lane + 32 * i;
      xr[i] = d < a.dc ? lat_f(x[d]) : 0.f;
      if (d < a.dc) dot = fmaf(qs[d], xr[i], dot);
      odd = fmaf(xr[i], 0.f, odd);
    }
    for (int d = a.dc + lane; d < a.width; d += 32) {
      const float y = lat_f(x[d]);
      dot = fmaf(qs[d], y, dot);
      odd = fmaf(y, 0.f, odd);
    }
    dot += odd;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, sh);
    const float s = dot * a.scale_log2;
    const float mn = fmaxf(m, s);
    if (s == -INFINITY && m == -INFINITY) continue;  // a NaN goes on
    const float alpha = exp2f(m - mn), p = exp2f(s - mn);
    l = l * alpha + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = fmaf(p, xr[i], acc[i] * alpha);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (lane + 32 * i < a.dc) part[warp * a.dc + lane + 32 * i] = acc[i];
  if (lane == 0) {
    pm[warp] = m;
    pl[warp] = l;
  }
  __syncthreads();
  float mx = pm[0];
#pragma unroll
  for (int w = 1; w < kLatWarps; ++w) mx = fmaxf(mx, pm[w]);
  float f[kLatWarps], tot = 0.f;
#pragma unroll
  for (int w = 0; w < kLatWarps; ++w) {
    f[w] = pm[w] == -INFINITY ? 0.f : exp2f(pm[w] - mx);
    tot += f[w] * pl[w];
  }
  // a NaN row sum is the answer of a NaN score, not an empty row
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  for (int d = threadIdx.x; d < a.dc; d += 32 * kLatWarps) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kLatWarps; ++w) o = fmaf(f[w], part[w * a.dc + d], o);
    out[d] = lat_t<T>(o * inv);
  }
}

template <typename T>
void launch_general(const LatGenArgs& a, cudaStream_t st) {
  const unsigned blocks = (unsigned)((long long)a.B * a.C * a.H);
  const size_t smem = sizeof(float) * ((size_t)a.width + (size_t)kLatWarps * a.dc);
  if (a.dc <= 512) latent_general_kernel<T, 16><<<blocks, 32 * kLatWarps, smem, st>>>(a);
  else latent_general_kernel<T, 32><<<blocks, 32 * kLatWarps, smem, st>>>(a);
}

}  // namespace

}  // namespace kvp

using namespace kvp;

extern "C" int paged_latent_attention_workspace_size(const kvp_pool* pool, int batch, int chunk, int num_q_heads,
                                                     size_t* bytes) {
  if (!pool || !pool->latent_dim || !bytes || batch <= 0 || chunk <= 0 || num_q_heads <= 0) return KVP_ERR_INVALID_ARG;
  // the general kernel needs no scratch
  *bytes = latent_tc_eligible(pool, chunk, num_q_heads) ? latent_tc_workspace(pool, chunk, num_q_heads) : 256;
  return KVP_OK;
}

extern "C" int paged_latent_attention(const kvp_pool* pool, int layer, const void* q, int batch, int chunk,
                                      int num_q_heads, const int32_t* q_lens, const int32_t* table,
                                      int table_rows_total, int table_cols, int table_mode, const int32_t* table_rows,
                                      const int32_t* context_lens, int window, int sinks, float scale, void* out,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!pool || !pool->latent_dim || !q || !table || !context_lens || !out) return KVP_ERR_INVALID_ARG;
  if (layer < 0 || layer >= pool->num_layers || batch <= 0 || chunk <= 0 || num_q_heads <= 0) return KVP_ERR_INVALID_ARG;
  if (table_rows_total <= 0 || table_cols <= 0) return KVP_ERR_INVALID_ARG;
  if (table_mode != KVP_BLOCK_TABLE && table_mode != KVP_RAW_LOCATIONS) return KVP_ERR_INVALID_ARG;
  if (!(scale - scale == 0.f)) return KVP_ERR_INVALID_ARG;
  if (sinks < 0 || (window > 0 && sinks >= window)) return KVP_ERR_INVALID_ARG;
  // a window that holds every context the table can hold is none
  if (window <= 0 || window >= (long long)table_cols * (table_mode == KVP_RAW_LOCATIONS ? 1 : pool->page_size))
    window = sinks = 0;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return KVP_ERR_INVALID_ARG;
  if ((long long)batch * chunk > 0x7fffffffLL / num_q_heads) return KVP_ERR_INVALID_ARG;
  size_t need = 0;
  const int rc = paged_latent_attention_workspace_size(pool, batch, chunk, num_q_heads, &need);
  if (rc != KVP_OK) return rc;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need) return KVP_ERR_INVALID_ARG;
  if (!pool_device_current(pool)) return KVP_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (scale > 0.f && latent_tc_eligible(pool, chunk, num_q_heads)) {  // its row maxima are of unscaled scores
    LatentCall c;
    c.pool = pool;
    c.layer = layer;
    c.q = q;
    c.out = out;
    c.B = batch;
    c.C = chunk;
    c.H = num_q_heads;
    c.q_lens = q_lens;
    c.T = make_table(pool, table, table_rows_total, table_cols, table_mode);
    c.table_rows = table_rows;
    c.context_lens = context_lens;
    c.window = window;
    c.sinks = sinks;
    c.scale = scale;
    c.workspace = workspace;
    return launch_latent_tc(c, st);
  }
  LatGenArgs g;
  g.T = make_table(pool, table, table_rows_total, table_cols, table_mode);
  g.layer = pool->buf + (size_t)layer * pool->layer_bytes;
  g.q = q;
  g.out = out;
  g.context_lens = context_lens;
  g.table_rows = table_rows;
  g.q_lens = q_lens;
  g.B = batch;
  g.C = chunk;
  g.H = num_q_heads;
  g.dc = pool->latent_dim;
  g.width = pool->head_dim;
  g.window = window;
  g.sinks = sinks;
  g.scale_log2 = scale * 1.4426950408889634f;
  g.err = pool->err;
  if (pool->dtype == KVP_F32) launch_general<float>(g, st);
  else launch_general<__nv_bfloat16>(g, st);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}
