// Four-bit pools (fp4.cuh): rows turned back into full entries, chunks, the
// general attention kernel of fp32 pools, and the entry points.
//
// Mathematics: as attention.cu, over K and V entries code * scale * g. The
// general kernel takes every fp32 shape: one block per query token and head, its
// warps take 32 positions in turn; a lane scores one position (its K row is its
// own loads), then the lanes take V's entries and the positions' weights come by
// shuffles; the warps' running maxima, sums and outputs are joined at the end.
// It is bound by instructions: a row is read again for every query head (64
// requests of 512-4096 rows, 32 heads on 8 of 128: 810 us).
//
// Chunks (many query tokens a request) are bound by the matrix rate, and every
// key is met by many query tiles: turning it back once a tile costs more than
// once a call (16 chunks of 512 tokens: 975 us by fp4_tile.cu, 258 so). So a call
// turns the attended rows into bf16 (exactly) in its workspace, request b's as
// the one page b of a pool whose pages are as long as the longest context, and
// runs the chunk kernel of bf16 pools (prefill_tc.cu) over them. Bytes: 1.1 KB
// read and 4 KB written a token of eight heads, and read again by the chunk
// kernel, mostly from L2. Of the 258 us the unpacking takes 32, the chunk kernel
// 221, the look for NaN 4; five prompts of 33-600 tokens 48 us (7, 38, 3).
// That kernel multiplies V by weights of zero where a query does not attend, so a
// block that reads as NaN would reach more queries than it should: a request with
// one in its span is noticed on the way and done again (fp4_tile.cu; 383 us with
// one of the 16).
#include <cstring>

#include "attention.cuh"
#include "fp4.cuh"

namespace kvp {

namespace {

constexpr int kLoadThreads = 256;
constexpr int kChunkColumns = 64;

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

constexpr int kUnpackRows = 32;  // rows a block at most

// Chunks: where a request's rows come from, and what the launches after this one read.
struct Chunk {
  TableRef T;
  const int32_t* context_lens;
  const int32_t* q_lens;
  const int32_t* table_rows;
  int C, window, sinks, max_context;
  int blocks;      // of Unpack::rows positions, max_context in all
  long long page;  // rows of a request's page in the workspace
  int32_t* lens;   // [B] context lengths, 0 for invalid requests
  int32_t* table;  // [B] page b
  int32_t* nan;    // [B][blocks] whether a row of the block has a scale NaN; written up to the context's end
};

struct Unpack {
  const char* codes;
  const char* scales;
  int heads, d;
  float gk, gv;
  void* k;
  void* v;
  int32_t* err;
  const int32_t* slots;  // rows of these slots ...
  int n, num_slots, rows;  // ``rows`` a block
  Chunk ch;              // ... or of the requests' spans
};

__device__ __forceinline__ bool request_ok(int L, int ql, int row, int C, int max_context, int rows_total) {
  return ql >= 1 && ql <= C && L >= ql && L <= max_context && row >= 0 && row < rows_total;
}

// Rows back to full entries: a block takes up to 32 rows (their slots first, all at once). A thread has 32 bytes of
// a row's entries, or of several rows side by side, row after row; a bf16 warp reads 256 bytes of two heads of 128 and writes
// 512 bytes of K and of V. Bytes bound it: 9 / 16 read and 2 written (bf16) an entry: 8,192
// rows of 8 heads of 128 12 us (3.5 TB/s; 42 MB, of which the writes stay in L2), 30,011 scattered ones 32 us (4.9 TB/s).
template <typename T, bool CHUNK>
__global__ void __launch_bounds__(kLoadThreads) unpack_kernel(const __grid_constant__ Unpack a) {
  __shared__ int slots[kUnpackRows];
  const int tid = threadIdx.x;
  const size_t row_entries = (size_t)a.heads * a.d;
  size_t out0;  // row of slots[0] in k and v
  int rows;
  if (CHUNK) {
    const Chunk& s = a.ch;
    const int b = blockIdx.y, t0 = blockIdx.x * a.rows;
    const int L = __ldg(s.context_lens + b), ql = s.q_lens ? __ldg(s.q_lens + b) : s.C;
    const int row = s.table_rows ? __ldg(s.table_rows + b) : b;
    const bool ok = request_ok(L, ql, row, s.C, s.max_context, s.T.rows_total);
    if (blockIdx.x == 0 && tid == 0) {
      s.lens[b] = ok ? L : 0;
      s.table[b] = b;
    }
    if (!ok || t0 >= L) return;
    const int wide = s.window > 0 && ql - 1 < 0x7fffffff - s.window ? s.window + ql - 1 : 0;
    const Span u = attend_span(L, wide, s.sinks);
    if (tid < a.rows) {
      const int t = t0 + tid;
      slots[tid] = t < L && (t >= u.lo || t < u.se) ? resolve_slot(s.T, row, t, a.err) : -1;
    }
    rows = min(a.rows, L - t0);
    out0 = (size_t)b * s.page + t0;
  } else {
    const long long i0 = (long long)blockIdx.x * a.rows;
    rows = (int)min((long long)a.rows, a.n - i0);
    if (tid < rows) {
      const int slot = __ldg(a.slots + i0 + tid);
      const bool good = (unsigned)slot < (unsigned)a.num_slots;
      if (!good) set_error(a.err, KVP_ERR_BAD_INDEX);
      slots[tid] = good ? slot : -1;
    }
    out0 = (size_t)i0;
  }
  __syncthreads();
  constexpr int kWords = sizeof(T) == 2 ? 2 : 1;  // words of four code bytes: 32 bytes of entries
  const int units = a.d / 4 / kWords, width = a.heads * units;  // of a token's row, K's first in a head
  const int beside = width < kLoadThreads ? kLoadThreads / width : 1;
  const int r0 = width < kLoadThreads ? tid / width : 0;
  bool nan = false;
  if (r0 < beside)
    for (int hu = tid - r0 * width; hu < width; hu += kLoadThreads) {
      const int h = hu / units, u = hu - h * units, part = u >= units / 2, e0 = (u - part * (units / 2)) * 8 * kWords;
      const float g = part ? a.gv : a.gk;
      T* dst = static_cast<T*>(part ? a.v : a.k) + (size_t)h * a.d + e0;
      const uint8_t* scales = reinterpret_cast<const uint8_t*>(a.scales) + part * (a.d / 16) + e0 / 16;
#pragma unroll 4
      for (int r = r0; r < rows; r += beside) {
        const int slot = slots[r];
        float x[kWords][8] = {};
        if (slot >= 0) {
          const char* from = a.codes + (size_t)slot * row_entries + (size_t)hu * 4 * kWords;
          uint32_t c[2];
          if (kWords == 2) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(from));
            c[0] = w.x;
            c[1] = w.y;
          } else {
            c[0] = __ldg(reinterpret_cast<const uint32_t*>(from));
          }
          const uint32_t s = __ldg(scales + fp4_scale_offset(slot, h, a.heads, a.d));
          nan |= s == kFp4NanScale;
#pragma unroll
          for (int i = 0; i < kWords; ++i) fp4_entries(c[i], s, g, x[i]);
        } else if (CHUNK) {
          continue;  // not attended, or a hole: nothing reads it, or what is read is unspecified
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) put8(dst + (out0 + r) * row_entries + 8 * i, x[i]);
      }
    }
  if (CHUNK) {
    const int any = __syncthreads_or(nan);
    if (tid == 0) a.ch.nan[(size_t)blockIdx.y * a.ch.blocks + blockIdx.x] = any;
  }
}

constexpr int kGenWarps = 8;

struct GenArgs {
  TableRef T;
  const char* codes;
  const char* scales;
  const float* q;
  float* out;
  const int32_t* context_lens;
  const int32_t* table_rows;
  const int32_t* q_lens;
  int Hq, Hkv, D, C, window, sinks, max_context;
  float scale_log2, gv;  // K's g is in the scale
  int32_t* err;
};

// fp32 pools: a block has one query head of one token.
__global__ void __launch_bounds__(32 * kGenWarps) fp4_general_kernel(const __grid_constant__ GenArgs a) {
  const int item = blockIdx.x;
  __shared__ float qs[kFp4MaxDim];
  __shared__ float part_o[kGenWarps][kFp4MaxDim], part_m[kGenWarps], part_l[kGenWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = item % a.Hq, bj = item / a.Hq, b = bj / a.C, j = bj % a.C;
  const int kvh = h / (a.Hq / a.Hkv), D = a.D;
  float* out = a.out + (size_t)item * D;
  const float* q = a.q + (size_t)item * D;
  const int Lr = a.context_lens[b], row = a.table_rows ? a.table_rows[b] : b, ql = a.q_lens ? a.q_lens[b] : a.C;
  if (!request_ok(Lr, ql, row, a.C, a.max_context, a.T.rows_total)) {
    if (threadIdx.x == 0 && h == 0 && j == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
    for (int d = threadIdx.x; d < D; d += blockDim.x) out[d] = 0.f;
    return;
  }
  if (j >= ql) return;
  const int L = Lr - ql + j + 1;  // the query token's own context
  for (int d = threadIdx.x; d < D; d += blockDim.x) qs[d] = q[d];
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
    out[d] = o * inv;
  }
}

GenArgs general_args(const Fp4Call& c) {
  GenArgs g;
  g.T = c.T;
  g.codes = c.pool->buf + (size_t)c.layer * c.pool->layer_bytes;
  g.scales = c.pool->fp4_scales + (size_t)c.layer * c.pool->fp4_scale_layer_bytes;
  g.q = static_cast<const float*>(c.q);
  g.out = static_cast<float*>(c.out);
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
  return g;
}

int launch_general(const Fp4Call& c, cudaStream_t st) {
  const GenArgs g = general_args(c);
  const unsigned grid = (unsigned)((long long)c.B * c.C * c.H);
  fp4_general_kernel<<<grid, 32 * kGenWarps, 0, st>>>(g);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

Unpack unpack_args(const kvp_pool* pool, int layer, void* k, void* v) {
  Unpack u = {};
  u.codes = pool->buf + (size_t)layer * pool->layer_bytes;
  u.scales = pool->fp4_scales + (size_t)layer * pool->fp4_scale_layer_bytes;
  u.heads = pool->kv_heads;
  u.d = pool->head_dim;
  u.gk = pool->fp4_globals[layer];
  u.gv = pool->fp4_globals[pool->num_layers + layer];
  u.k = k;
  u.v = v;
  u.err = pool->err;
  u.num_slots = pool->num_slots;
  return u;
}

// A chunk's workspace for B requests of up to ``longest`` rows.
struct ChunkLayout {
  long long page;  // rows of a request
  int rows, blocks;  // positions a block takes, blocks of a request
  size_t lens, table, nan, kv, plane, total;
};
ChunkLayout chunk_layout(const kvp_pool* pool, int B, int longest) {
  ChunkLayout l;
  l.page = ((long long)longest + 15) / 16 * 16;
  l.rows = kUnpackRows;  // fewer where that would be less than eight blocks an SM (6,000 rows of 8 heads by 32 at a time: 21 us, by 4: 9)
  while (l.rows > 2 && (long long)B * longest / l.rows < 8 * pool->num_sms) l.rows /= 2;
  l.blocks = (longest - 1) / l.rows + 1;
  l.lens = 0;
  l.table = align256(sizeof(int32_t) * (size_t)B);
  l.nan = align256(l.table + sizeof(int32_t) * (size_t)B);
  l.kv = align256(l.nan + sizeof(int32_t) * (size_t)B * (l.page / 2));  // for any ``rows``: larger calls' workspaces fit
  l.plane = (size_t)B * l.page * pool->kv_heads * pool->head_dim * 2;
  l.total = l.kv + 2 * l.plane;
  return l;
}

// The pool that a chunk's rows become: request b's are its page b.
kvp_pool chunk_pool(const kvp_pool* pool, int B, const ChunkLayout& l, char* ws) {
  kvp_pool p = *pool;
  p.fp4 = 0;
  p.planes = 2;
  p.num_layers = 1;
  p.num_pages = B;
  p.page_size = (int)l.page;
  p.num_slots = (int)(B * l.page);
  p.row_bytes = (size_t)p.kv_heads * p.head_dim * 2;
  p.layer_bytes = p.kv_bytes = l.plane;
  p.buf = ws + l.kv;
  p.tmap1_state = 0;  // its maps are made for this call
  p.ev_before = p.ev_after = nullptr;
  return p;
}

// Whether a call goes through the chunk kernel of bf16 pools. Up to 64 (token, head) columns a KV head are the decode
// kernel's, which splits contexts over the SMs; it takes up to 128, and above 64 a CTA has one KV head alone. 64 requests of
// 512-4096 rows, 8 KV heads, decode kernel against chunk kernel: 64 columns 229 and 348 us, 96 397 and 347. Where the chunk
// kernel would have less than a CTA an SM, the decode kernel keeps them all: 4 requests, 128 columns 36 and 46 us.
bool chunk_eligible(const kvp_pool* pool, int B, int C, int H, int longest, float scale) {
  const long long columns = (long long)C * (H / pool->kv_heads);
  const bool few = columns <= kChunkColumns || (long long)B * pool->kv_heads < pool->num_sms;
  if (few && fp4_tc_eligible(pool, C, H)) return false;
  return pool->dtype == KVP_BF16 && (long long)B * (((long long)longest + 15) / 16 * 16) <= 0x7fffffffLL && B <= 65535 &&
         prefill_tc_eligible(pool, H, C, scale);
}

int launch_chunk(const Fp4Call& c, int longest, cudaStream_t st) {
  const kvp_pool* pool = c.pool;
  char* ws = static_cast<char*>(c.workspace);
  const ChunkLayout l = chunk_layout(pool, c.B, longest);
  kvp_pool rows = chunk_pool(pool, c.B, l, ws);
  int32_t* lens = reinterpret_cast<int32_t*>(ws + l.lens);
  int32_t* table = reinterpret_cast<int32_t*>(ws + l.table);
  int32_t* nan = reinterpret_cast<int32_t*>(ws + l.nan);
  Unpack u = unpack_args(pool, c.layer, ws + l.kv, ws + l.kv + l.plane);
  u.ch = {c.T, c.context_lens, c.q_lens, c.table_rows, c.C, c.window, c.sinks, c.max_context, l.blocks, l.page, lens, table,
          nan};
  u.rows = l.rows;
  unpack_kernel<__nv_bfloat16, true><<<dim3(l.blocks, c.B), kLoadThreads, 0, st>>>(u);
  if (cudaGetLastError() != cudaSuccess) return KVP_ERR_CUDA;
  const int rc = launch_prefill_tc(&rows, 0, c.q, c.B, c.C, c.H, c.q_lens, make_table(&rows, table, c.B, 1, KVP_BLOCK_TABLE),
                                   nullptr, lens, c.window, c.sinks, c.scale, c.out, st);
  if (rc != KVP_OK) return rc;
  return launch_fp4_again(c, lens, nan, l.blocks, l.rows, st);
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
  Unpack u = unpack_args(pool, layer, k, v);
  u.slots = slots;
  u.n = n;
  // as many rows a block as leave every SM eight blocks (64 rows by 32 at a time are two blocks, and 12 us)
  u.rows = 1;
  while (u.rows < kUnpackRows && n / (2 * u.rows) >= 8 * pool->num_sms) u.rows *= 2;
  const unsigned grid = (unsigned)(((long long)n + u.rows - 1) / u.rows);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (pool->dtype == KVP_F32) unpack_kernel<float, false><<<grid, kLoadThreads, 0, st>>>(u);
  else unpack_kernel<__nv_bfloat16, false><<<grid, kLoadThreads, 0, st>>>(u);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

extern "C" int paged_fp4_attention_workspace_size(const kvp_pool* pool, int batch, int chunk, int num_q_heads,
                                                  int max_context, size_t* bytes) {
  if (!bytes || !shape_ok(pool, batch, chunk, num_q_heads, max_context)) return KVP_ERR_INVALID_ARG;
  // whatever the scale's sign, which decides between chunk kernel and the others
  size_t need = fp4_tc_workspace(pool, chunk, num_q_heads);
  if (chunk_eligible(pool, batch, chunk, num_q_heads, max_context, 1.f)) {
    const size_t rows = chunk_layout(pool, batch, max_context).total;
    if (rows > need) need = rows;
  }
  *bytes = need ? need : 256;  // the other kernels need none
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
  if (chunk_eligible(pool, batch, chunk, num_q_heads, max_context, scale)) return launch_chunk(c, max_context, st);
  if (fp4_tc_eligible(pool, chunk, num_q_heads)) return launch_fp4_tc(c, st);
  return pool->dtype == KVP_BF16 ? launch_fp4_tile(c, st) : launch_general(c, st);
}
