// Four-bit pools (fp4.cuh): the rows of given slots, the general attention
// kernel, and the entry points of paged_fp4_attention.
//
// Mathematics: as attention.cu, over K and V entries code * scale * g. The
// general kernel takes every type and width: one block per query token and
// head, its warps take 32 positions in turn; a lane scores one position (its
// K row is its own 8-byte loads), then the lanes take V's entries and the
// positions' weights come by shuffles; the warps' running maxima, sums and
// outputs are joined at the end. It is bound by instructions: a row is read
// again for every query head.
#include <cstring>

#include "attention.cuh"
#include "fp4.cuh"

namespace kvp {

namespace {

constexpr int kLoadThreads = 256;

__device__ __forceinline__ float2 half2_floats(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// The eight entries of four code bytes under one scale (e4m3 code) and g.
__device__ __forceinline__ void fp4_entries(uint32_t codes, uint32_t scale, float g, float (&x)[8]) {
  uint32_t h[4];
  e2m1x8_to_half(codes, h);
  const float s = half2_floats(e4m3x2_to_half(scale)).x * g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = half2_floats(h[i]);
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
}

__device__ __forceinline__ void put8(float* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void put8(__nv_bfloat16* dst, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Rows of slots: a thread turns four code bytes into eight entries; a warp reads the 128 bytes of a head of 128 and
// writes 256 bytes of K and of V. Bytes bound it: 9 / 16 read, 2 written (bf16) an entry.
template <typename T>
__global__ void __launch_bounds__(kLoadThreads) load_fp4_kernel(const char* __restrict__ codes,
                                                                 const char* __restrict__ scales, int heads, int d,
                                                                 const int32_t* __restrict__ slots, int n, int num_slots,
                                                                 float gk, float gv, T* __restrict__ k, T* __restrict__ v,
                                                                 int32_t* err) {
  const int per_head = d / 4;  // words of four code bytes: half of them K's
  const long long total = (long long)n * heads * per_head;
  for (long long u = blockIdx.x * (long long)kLoadThreads + threadIdx.x; u < total; u += (long long)gridDim.x * kLoadThreads) {
    const int w = (int)(u % per_head);
    const long long rest = u / per_head;
    const int h = (int)(rest % heads);
    const long long i = rest / heads;
    const int part = w >= per_head / 2, e0 = (w - part * (per_head / 2)) * 8;
    const int slot = __ldg(slots + i);
    float x[8] = {};
    if ((unsigned)slot < (unsigned)num_slots) {
      const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes + (size_t)slot * heads * d + (size_t)h * d) + w);
      const uint8_t* s = reinterpret_cast<const uint8_t*>(scales) + fp4_scale_offset(slot, h, heads, d);
      fp4_entries(c, __ldg(s + part * (d / 16) + e0 / 16), part ? gv : gk, x);
    } else if (w == 0 && h == 0) {
      set_error(err, KVP_ERR_BAD_INDEX);
    }
    put8((part ? v : k) + ((size_t)i * heads + h) * d + e0, x);
  }
}

constexpr int kGenWarps = 8;

struct GenArgs {
  TableRef T;
  const char* codes;
  const char* scales;
  const void* q;
  void* out;
  const int32_t* context_lens;
  const int32_t* table_rows;
  const int32_t* q_lens;
  int Hq, Hkv, D, C, window, sinks, max_context;
  float scale_log2, gv;  // K's g is in the scale
  int32_t* err;
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put1(float* p, float x) { *p = x; }
__device__ __forceinline__ void put1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T>
__global__ void __launch_bounds__(32 * kGenWarps) fp4_general_kernel(const GenArgs a) {
  __shared__ float qs[kFp4MaxDim];
  __shared__ float part_o[kGenWarps][kFp4MaxDim], part_m[kGenWarps], part_l[kGenWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % a.Hq, bj = blockIdx.x / a.Hq, b = bj / a.C, j = bj % a.C;
  const int kvh = h / (a.Hq / a.Hkv), D = a.D;
  T* out = static_cast<T*>(a.out) + (size_t)blockIdx.x * D;
  const T* q = static_cast<const T*>(a.q) + (size_t)blockIdx.x * D;
  const int Lr = a.context_lens[b], row = a.table_rows ? a.table_rows[b] : b, ql = a.q_lens ? a.q_lens[b] : a.C;
  if (ql < 1 || ql > a.C || Lr < ql || Lr > a.max_context || row < 0 || row >= a.T.rows_total) {
    if (threadIdx.x == 0 && h == 0 && j == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
    for (int d = threadIdx.x; d < D; d += blockDim.x) put1(out + d, 0.f);
    return;
  }
  if (j >= ql) return;
  const int L = Lr - ql + j + 1;  // the query token's own context
  for (int d = threadIdx.x; d < D; d += blockDim.x) qs[d] = as_float(q[d]);
  __syncthreads();
  const Span sp = attend_span(L, a.window, a.sinks);
  const int n = sp.se + L - sp.lo;
  constexpr int kBytes = kFp4MaxDim / 64;  // bytes of V a lane takes
  float acc[2 * kBytes] = {}, m = -INFINITY, l = 0.f;
  for (int o0 = 32 * warp; o0 < n; o0 += 32 * kGenWarps) {
    const int o = o0 + lane;
    int slot = -1;
    float s = -INFINITY;
    if (o < n) {
      slot = resolve_slot(a.T, row, span_pos(sp, o), a.err);
      if (slot >= 0) {
        const uint32_t* kr = reinterpret_cast<const uint32_t*>(a.codes + ((size_t)slot * a.Hkv + kvh) * D);
        const uint8_t* ks = reinterpret_cast<const uint8_t*>(a.scales) + fp4_scale_offset(slot, kvh, a.Hkv, D);
        float dot = 0.f;
        for (int w = 0; w < D / 8; ++w) {
          float x[8];
          fp4_entries(__ldg(kr + w), __ldg(ks + w / 2), 1.f, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(qs[8 * w + i], x[i], dot);
        }
        s = dot * a.scale_log2;
      }
    }
    float mx = s;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
    const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;  // a NaN score passes by the maximum, not by p
    const float alpha = exp2f(m - base), p = exp2f(s - base);
    float ps = p;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, sh);
    l = l * alpha + ps;
    m = mn;
#pragma unroll
    for (int i = 0; i < 2 * kBytes; ++i) acc[i] *= alpha;
    const int nt = min(32, n - o0);
    for (int t = 0; t < nt; ++t) {
      const float pt = __shfl_sync(0xffffffffu, p, t);
      const int st = __shfl_sync(0xffffffffu, slot, t);
      if (st < 0) continue;
      const uint8_t* vr = reinterpret_cast<const uint8_t*>(a.codes) + ((size_t)st * a.Hkv + kvh) * D + D / 2;
      const uint8_t* vs = reinterpret_cast<const uint8_t*>(a.scales) + fp4_scale_offset(st, kvh, a.Hkv, D) + D / 16;
#pragma unroll
      for (int i = 0; i < kBytes; ++i) {
        const int x = lane + 32 * i;
        if (x >= D / 2) break;
        uint32_t hh[4];
        e2m1x8_to_half(__ldg(vr + x), hh);
        const float2 f = half2_floats(hh[0]);
        const float w = half2_floats(e4m3x2_to_half(__ldg(vs + x / 8))).x * pt;
        acc[2 * i] = fmaf(f.x, w, acc[2 * i]);
        acc[2 * i + 1] = fmaf(f.y, w, acc[2 * i + 1]);
      }
    }
  }
  if (lane == 0) {
    part_m[warp] = m;
    part_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < kBytes; ++i) {
    const int x = lane + 32 * i;
    if (x < D / 2) {
      part_o[warp][2 * x] = acc[2 * i];
      part_o[warp][2 * x + 1] = acc[2 * i + 1];
    }
  }
  __syncthreads();
  float M = -INFINITY, Ls = 0.f;
  for (int w = 0; w < kGenWarps; ++w) M = fmaxf(M, part_m[w]);
  const float base = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < kGenWarps; ++w) Ls += exp2f(part_m[w] - base) * part_l[w];
  const float inv = Ls == 0.f ? 0.f : a.gv / Ls;  // no weight at all: zeros; a NaN stays one
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float o = 0.f;
    for (int w = 0; w < kGenWarps; ++w) o += exp2f(part_m[w] - base) * part_o[w][d];
    put1(out + d, o * inv);
  }
}

int launch_general(const Fp4Call& c, cudaStream_t st) {
  GenArgs g;
  g.T = c.T;
  g.codes = c.pool->buf + (size_t)c.layer * c.pool->layer_bytes;
  g.scales = c.pool->fp4_scales + (size_t)c.layer * c.pool->fp4_scale_layer_bytes;
  g.q = c.q;
  g.out = c.out;
  g.context_lens = c.context_lens;
  g.table_rows = c.table_rows;
  g.q_lens = c.q_lens;
  g.Hq = c.H;
  g.Hkv = c.pool->kv_heads;
  g.D = c.pool->head_dim;
  g.C = c.C;
  g.window = c.window;
  g.sinks = c.sinks;
  g.max_context = c.max_context;
  g.scale_log2 = c.scale * c.pool->fp4_globals[c.layer] * 1.4426950408889634f;
  g.gv = c.pool->fp4_globals[c.pool->num_layers + c.layer];
  g.err = c.pool->err;
  const unsigned grid = (unsigned)((long long)c.B * c.C * c.H);
  if (c.pool->dtype == KVP_F32) fp4_general_kernel<float><<<grid, 32 * kGenWarps, 0, st>>>(g);
  else fp4_general_kernel<__nv_bfloat16><<<grid, 32 * kGenWarps, 0, st>>>(g);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

// What both calls about a shape check.
bool shape_ok(const kvp_pool* pool, int batch, int chunk, int num_q_heads, int max_context) {
  return pool && pool->fp4 && batch > 0 && chunk > 0 && num_q_heads > 0 && num_q_heads % pool->kv_heads == 0 &&
         max_context > 0 && (long long)batch * chunk <= 0x7fffffffLL / num_q_heads;
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int load_cache_fp4(const kvp_pool* pool, int layer, const int32_t* slots, int n, void* k, void* v, void* stream) {
  if (!pool || !pool->fp4 || n < 0 || layer < 0 || layer >= pool->num_layers) return KVP_ERR_INVALID_ARG;
  if (n == 0) return KVP_OK;
  if (!slots || !k || !v || ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15))
    return KVP_ERR_INVALID_ARG;
  if (!pool_device_current(pool)) return KVP_ERR_INVALID_ARG;
  const char* codes = pool->buf + (size_t)layer * pool->layer_bytes;
  const char* scales = pool->fp4_scales + (size_t)layer * pool->fp4_scale_layer_bytes;
  const float gk = pool->fp4_globals[layer], gv = pool->fp4_globals[pool->num_layers + layer];
  const long long blocks = ((long long)n * pool->kv_heads * (pool->head_dim / 4) + kLoadThreads - 1) / kLoadThreads;
  const unsigned grid = (unsigned)(blocks < 1 << 22 ? blocks : 1 << 22);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (pool->dtype == KVP_F32)
    load_fp4_kernel<float><<<grid, kLoadThreads, 0, st>>>(codes, scales, pool->kv_heads, pool->head_dim, slots, n,
                                                          pool->num_slots, gk, gv, static_cast<float*>(k),
                                                          static_cast<float*>(v), pool->err);
  else
    load_fp4_kernel<__nv_bfloat16><<<grid, kLoadThreads, 0, st>>>(codes, scales, pool->kv_heads, pool->head_dim, slots, n,
                                                                  pool->num_slots, gk, gv, static_cast<__nv_bfloat16*>(k),
                                                                  static_cast<__nv_bfloat16*>(v), pool->err);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

extern "C" int paged_fp4_attention_workspace_size(const kvp_pool* pool, int batch, int chunk, int num_q_heads,
                                                  int max_context, size_t* bytes) {
  if (!bytes || !shape_ok(pool, batch, chunk, num_q_heads, max_context)) return KVP_ERR_INVALID_ARG;
  const size_t need = fp4_tc_workspace(pool, chunk, num_q_heads);
  *bytes = need ? need : 256;  // the general kernel needs none
  return KVP_OK;
}

extern "C" int paged_fp4_attention(const kvp_pool* pool, int layer, const void* q, int batch, int chunk, int num_q_heads,
                                   const int32_t* q_lens, const int32_t* table, int table_rows_total, int table_cols,
                                   int table_mode, const int32_t* table_rows, const int32_t* context_lens, int max_context,
                                   int window, int sinks, float scale, void* out, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  if (!shape_ok(pool, batch, chunk, num_q_heads, max_context)) return KVP_ERR_INVALID_ARG;
  if (!q || !table || !context_lens || !out || layer < 0 || layer >= pool->num_layers) return KVP_ERR_INVALID_ARG;
  if (table_rows_total <= 0 || table_cols <= 0) return KVP_ERR_INVALID_ARG;
  if (table_mode != KVP_BLOCK_TABLE && table_mode != KVP_RAW_LOCATIONS) return KVP_ERR_INVALID_ARG;
  if (!(scale == scale) || sinks < 0 || (window > 0 && sinks >= window)) return KVP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return KVP_ERR_INVALID_ARG;
  size_t need = 0;
  if (paged_fp4_attention_workspace_size(pool, batch, chunk, num_q_heads, max_context, &need) != KVP_OK)
    return KVP_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need) return KVP_ERR_INVALID_ARG;
  if (!pool_device_current(pool)) return KVP_ERR_INVALID_ARG;
  Fp4Call c;
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
  // a window no context can fill is none: so window + chunk stays within int32
  c.window = window > 0 && window < max_context ? window : 0;
  c.sinks = c.window ? sinks : 0;
  const long long cap = table_capacity(c.T);
  c.max_context = cap < max_context ? (int)cap : max_context;
  c.scale = scale;
  c.workspace = workspace;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return fp4_tc_eligible(pool, chunk, num_q_heads) ? launch_fp4_tc(c, st) : launch_general(c, st);
}
