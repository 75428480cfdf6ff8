// Four-bit pools (fp4.cuh): rows turned back into full entries, chunks, the
// attention kernel of fp32 pools, and the entry points.
//
// Mathematics: as attention.cu, over K and V entries code * scale * g.
//
// Chunks (many query tokens a request) are bound by the matrix rate, and every
// key is met by many query tiles: turning it back once a tile costs more than
// once a call (16 chunks of 512 tokens: 975 us by fp4_tile.cu, 258 so). So a call
// turns the attended rows into bf16 (exactly) in its workspace, request b's as
// the one page b of a pool whose pages are as long as the longest context, and
// runs the chunk kernel of bf16 pools (prefill_tc.cu) over them, for as many
// requests at a time as 4 GiB of rows hold. Bytes: 1.1 KB
// read and 4 KB written a token of eight heads, and read again by the chunk
// kernel, mostly from L2. Of the 258 us the unpacking takes 32, the chunk kernel
// 221, the look for NaN 4; five prompts of 33-600 tokens 48 us (7, 38, 3); called
// one by one, without a graph, 267 and 55.
// That kernel multiplies V by weights of zero where a query does not attend, so a
// block that reads as NaN would reach more queries than it should: a request with
// one in its span is noticed on the way and done again (fp4_tile.cu; 383 us with
// one of the 16).
#include <cooperative_groups.h>

#include <type_traits>

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
          nan |= fp4_is_nan(s);
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

// ---------------------------------------------------------------------------
// fp32 pools. A CTA of eight warps has up to 32 (token, head) columns of one KV head, four a warp. Blocks of 64 positions are
// turned into fp32 rows in shared memory, the next block's codes fetched meanwhile. A lane scores a position for its warp's
// four columns (its K row is its own loads, the queries' are broadcast), then has four entries of V and the columns' weights
// of each position come as one word: 16 multiplications and additions a load either way, so fp32's rate bounds it where there
// are columns enough. With fewer, all eight warps work all the same, on parts of a block's positions: 32, 16 or 8, of which a
// lane then scores a half or a quarter. Where tiles are few a cluster shares
// one, as in fp4_tile.cu. 64 requests of 512-4096 rows, 32 heads on 8 of 128: 380 us (a block a query head
// 810), one of 500 rows 11; four prompts of up to 100 tokens on up to 300 73 us (233).
// ---------------------------------------------------------------------------
namespace cg = cooperative_groups;

constexpr int kF32Rows = 64, kF32Warps = 8, kF32Parts = 8;

struct F32Args {
  TableRef T;
  const char* codes;
  const char* scales;
  const float* q;
  float* out;
  const int32_t* context_lens;
  const int32_t* table_rows;
  const int32_t* q_lens;
  int Hq, Hkv, G, D, C, window, sinks, max_context, tiles;
  float scale_log2, gv;  // K's g is in the scale
  int32_t* err;
};

// I: head_dim over 128, rounded up; CG: warps that have columns of their own.
template <int I, int CG>
__global__ void __launch_bounds__(32 * kF32Warps, I == 1 ? 2 : 1) fp4_f32_kernel(const __grid_constant__ F32Args a) {
  constexpr int kParts = kF32Warps / CG;              // of a block's positions
  constexpr int kPos = CG < 4 ? 8 * CG : 32;           // positions at once, 32 / kPos lanes each
  constexpr int kSubs = kF32Rows / kParts / kPos;
  constexpr int kLanes = 32 / kPos;
  extern __shared__ __align__(16) float f32_smem[];
  __shared__ int pos[kF32Rows];
  __shared__ uint32_t vnan[2][kF32Rows];  // of a row's even and odd blocks
  __shared__ float4 weights[kF32Warps][32];
  __shared__ float part_m[kF32Warps][4], part_l[kF32Warps][4];
  const int D = a.D, pitch = D + 4;
  float* sk = f32_smem;
  float* sv = sk + kF32Rows * pitch;
  float* sq = sv + kF32Rows * pitch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int R = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const long long item = (long long)blockIdx.x / R;
  const int tile = (int)(item % a.tiles), kvh = (int)(item / a.tiles % a.Hkv), b = (int)(item / a.tiles / a.Hkv);
  const int col0 = tile * 4 * CG, cols = a.C * a.G;
  const int L = a.context_lens[b], ql = a.q_lens ? a.q_lens[b] : a.C, row = a.table_rows ? a.table_rows[b] : b;
  auto column = [&](int col) {  // its row of q and out
    const int cj = col / a.G;
    return (((size_t)b * a.C + cj) * a.Hq + (size_t)kvh * a.G + (col - cj * a.G)) * D;
  };
  if (!request_ok(L, ql, row, a.C, a.max_context, a.T.rows_total)) {
    if (rank) return;
    if (tid == 0 && tile == 0 && kvh == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
    for (int i = tid; i < 4 * CG * D; i += 32 * kF32Warps)
      if (col0 + i / D < cols) a.out[column(col0 + i / D) + i % D] = 0.f;
    return;
  }
  const int j0 = col0 / a.G, j1 = min((min(col0 + 4 * CG, cols) - 1) / a.G, ql - 1);
  if (j0 > j1) return;
  const int p0 = L - ql + j0, p1 = L - ql + j1;
  const Span u = attend_span(p1 + 1, a.window > 0 && j1 - j0 < 0x7fffffff - a.window ? a.window + (j1 - j0) : 0, a.sinks);
  const Span newest = attend_span(p1 + 1, a.window, a.sinks);
  const int n = u.se + (p1 + 1) - u.lo, blocks = (n - 1) / kF32Rows + 1;

  // a thread's part of a block: every other block of 16 entries of K or of V of one position
  const int mine = tid & (kF32Rows - 1), odd = tid >> 6 & 1;
  const bool is_v = tid >= 2 * kF32Rows;
  uint2 codes[4 * I];
  uint32_t scales[I];
  int at = 0x7fffffff;
  auto fetch = [&](int o) {
    const int t = o < n ? span_pos(u, o) : 0;
    const int slot = o < n ? resolve_slot(a.T, row, t, a.err) : -1;
    at = slot < 0 ? 0x7fffffff : t;
#pragma unroll
    for (int i = 0; i < I; ++i) scales[i] = 0;
#pragma unroll
    for (int i = 0; i < 4 * I; ++i) {
      codes[i] = make_uint2(0u, 0u);
      const int x = 2 * i + odd;  // block of the row
      if (slot < 0 || 16 * x >= D) continue;
      codes[i] = __ldg(reinterpret_cast<const uint2*>(a.codes + ((size_t)slot * a.Hkv + kvh) * D + (is_v ? D / 2 : 0)) + x);
      scales[i / 4] |= (uint32_t)__ldg(reinterpret_cast<const uint8_t*>(a.scales) + fp4_scale_offset(slot, kvh, a.Hkv, D) +
                                       (is_v ? D / 16 : 0) + x)
                       << (8 * (i & 3));
    }
  };
  if (rank < blocks) fetch(rank * kF32Rows + mine);
  for (int i = tid; i < 4 * CG * D; i += 32 * kF32Warps) {
    const int c = i / D, col = col0 + c;
    sq[c * pitch + i % D] = col < cols && col / a.G <= j1 ? __ldg(a.q + column(col) + i % D) : 0.f;
  }

  const int group = warp % CG, part = warp / CG;
  float4 o[4][I];
  float m[4], l[4];
  int p[4], lo[4], se[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    m[c] = -3.0e38f;
    l[c] = 0.f;
    p[c] = L - ql + min((col0 + 4 * group + c) / a.G, j1);
    const Span s = attend_span(p[c] + 1, a.window, a.sinks);
    lo[c] = s.lo;
    se[c] = s.se;
#pragma unroll
    for (int i = 0; i < I; ++i) o[c][i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const bool live = col0 + 4 * group < cols;
  for (int blk = rank; blk < blocks; blk += R) {
    __syncthreads();  // the block before is done with
    uint32_t bad = 0;
    float* dst = (is_v ? sv : sk) + mine * pitch;
#pragma unroll
    for (int i = 0; i < 4 * I; ++i) {
      const int x = 2 * i + odd;
      if (16 * x >= D) break;
      uint32_t sc = scales[i / 4] >> (8 * (i & 3)) & 0xffu;
      if (is_v && fp4_is_nan(sc)) {
        bad |= 1u << x;
        sc = 0;
      }
      float y[8];
      fp4_entries(codes[i].x, sc, 1.f, y);
      put8(dst + 16 * x, y);
      fp4_entries(codes[i].y, sc, 1.f, y);
      put8(dst + 16 * x + 8, y);
    }
    if (is_v) vnan[odd][mine] = bad;
    else if (!odd) pos[mine] = at;
    // whether some column does not attend some position, or a V block is NaN
    const int special = __syncthreads_or(bad != 0 || at > p0 || at < newest.lo);
    if (blk + R < blocks) fetch((blk + R) * kF32Rows + mine);
    if (!live) continue;
#pragma unroll 1
    for (int sub = 0; sub < kSubs; ++sub) {
      const int first = kPos * (part * kSubs + sub);
      float s[4] = {};
      const float4* kr = reinterpret_cast<const float4*>(sk + (first + lane % kPos) * pitch);
      const float* qr = sq + 4 * group * pitch;
#pragma unroll 4
      for (int w = lane / kPos; w < D / 4; w += kLanes) {
        const float4 kv = kr[w];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 qv = reinterpret_cast<const float4*>(qr + c * pitch)[w];
          s[c] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[c]))));
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int sh = kPos; sh < 32; sh <<= 1) s[c] += __shfl_xor_sync(0xffffffffu, s[c], sh);
      const int t = pos[first + lane % kPos];
      float w4[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float x = special && !(t <= p[c] && (t >= lo[c] || t < se[c])) ? -INFINITY : __fmul_rn(s[c], a.scale_log2);
        float mx = x;
#pragma unroll
        for (int sh = kPos / 2; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
        mx = fminf(fmaxf(mx, m[c]), 3.0e38f);  // finite: a score beyond it becomes a NaN
        const float al = exp2f(m[c] - mx);
        m[c] = mx;
        w4[c] = exp2f(x - mx);
        l[c] = l[c] * al + (lane < kPos ? w4[c] : 0.f);
        if (al != 1.f)
#pragma unroll
          for (int i = 0; i < I; ++i) {
            o[c][i].x *= al;
            o[c][i].y *= al;
            o[c][i].z *= al;
            o[c][i].w *= al;
          }
      }
      __syncwarp();
      if (lane < kPos) weights[warp][lane] = make_float4(w4[0], w4[1], w4[2], w4[3]);
      __syncwarp();
#pragma unroll 4
      for (int y = 0; y < kPos; ++y) {
        const float4 wv = weights[warp][y];
        const float wc[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int e = 4 * (lane + 32 * i);
          if (e >= D) break;
          const float4 v = *reinterpret_cast<const float4*>(sv + (first + y) * pitch + e);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            o[c][i].x = fmaf(wc[c], v.x, o[c][i].x);
            o[c][i].y = fmaf(wc[c], v.y, o[c][i].y);
            o[c][i].z = fmaf(wc[c], v.z, o[c][i].z);
            o[c][i].w = fmaf(wc[c], v.w, o[c][i].w);
          }
        }
      }
      if (special)
        for (int y = first; y < first + kPos; ++y) {
          const uint32_t blocks_of = vnan[0][y] | vnan[1][y];
          if (!blocks_of) continue;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < I; ++i)
              if ((blocks_of >> ((lane + 32 * i) / 4) & 1) && pos[y] <= p[c] && (pos[y] >= lo[c] || pos[y] < se[c])) {
                const float none = __int_as_float(0x7fffffff);
                o[c][i] = make_float4(none, none, none, none);
              }
        }
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], sh);
  // the parts' sums, maxima and outputs to shared memory, over K and V, and their join: a warp a column
  __syncthreads();
  float* po = f32_smem;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (lane == 0) {
      part_m[warp][c] = m[c];
      part_l[warp][c] = l[c];
    }
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (4 * (lane + 32 * i) < D) *reinterpret_cast<float4*>(po + (warp * 4 + c) * D + 4 * (lane + 32 * i)) = o[c][i];
  }
  cluster.sync();
  for (int r = rank + R * warp; r < 4 * CG; r += kF32Warps * R) {
    const int col = col0 + r;
    if (col >= cols || col / a.G > j1) break;  // nor are later ones
    const int parts = kParts * R;
    auto from = [&](int k) { return (k % kParts * CG) * 4 + r; };  // of a CTA's warps' columns
    float M = -3.0e38f, sum = 0.f;
    for (int k = lane; k < parts; k += 32) M = fmaxf(M, cluster.map_shared_rank(&part_m[0][0], k / kParts)[from(k)]);
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, sh));
    for (int k = lane; k < parts; k += 32)
      sum += exp2f(cluster.map_shared_rank(&part_m[0][0], k / kParts)[from(k)] - M) *
             cluster.map_shared_rank(&part_l[0][0], k / kParts)[from(k)];
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
    const float inv = sum == 0.f ? 0.f : a.gv / sum;  // every score minus infinity: zeros, as in the other kernels
    float* dst = a.out + column(col);
    for (int e = 4 * lane; e < D; e += 128) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < parts; ++k) {
        const float w = exp2f(cluster.map_shared_rank(&part_m[0][0], k / kParts)[from(k)] - M);
        const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(po, k / kParts) + from(k) * D + e);
        acc.x = fmaf(w, x.x, acc.x);
        acc.y = fmaf(w, x.y, acc.y);
        acc.z = fmaf(w, x.z, acc.z);
        acc.w = fmaf(w, x.w, acc.w);
      }
      *reinterpret_cast<float4*>(dst + e) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
  }
  cluster.sync();  // the others have read this CTA's parts
}

template <int I, int CG>
cudaError_t launch_f32_one(const F32Args& a, unsigned grid, int R, cudaStream_t st) {
  auto kernel = fp4_f32_kernel<I, CG>;
  auto bytes = [](int D) { return (size_t)(2 * kF32Rows + 4 * CG) * (D + 4) * sizeof(float); };
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(128 * I));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = R;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(32 * kF32Warps);
  cfg.dynamicSmemBytes = bytes(a.D);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

int launch_f32(const Fp4Call& c, cudaStream_t st) {
  const kvp_pool* pool = c.pool;
  F32Args a;
  a.T = c.T;
  a.codes = pool->buf + (size_t)c.layer * pool->layer_bytes;
  a.scales = pool->fp4_scales + (size_t)c.layer * pool->fp4_scale_layer_bytes;
  a.q = static_cast<const float*>(c.q);
  a.out = static_cast<float*>(c.out);
  a.context_lens = c.context_lens;
  a.table_rows = c.table_rows;
  a.q_lens = c.q_lens;
  a.Hq = c.H;
  a.Hkv = pool->kv_heads;
  a.G = c.H / pool->kv_heads;
  a.D = pool->head_dim;
  a.C = c.C;
  a.window = c.window;
  a.sinks = c.sinks;
  a.max_context = c.max_context;
  a.scale_log2 = c.scale * pool->fp4_globals[c.layer] * 1.4426950408889634f;
  a.gv = pool->fp4_globals[pool->num_layers + c.layer];
  a.err = pool->err;
  const long long cols = (long long)c.C * a.G;
  const int CG = cols <= 4 ? 1 : cols <= 8 ? 2 : cols <= 16 ? 4 : 8;
  a.tiles = (int)((cols + 4 * CG - 1) / (4 * CG));
  const long long items = (long long)a.tiles * a.Hkv * c.B;
  // CTAs share a tile while that leaves no SM more than two, and each a block at least
  int R = 1;
  while (R < kF32Parts && 2 * R * items <= 2LL * pool->num_sms && 2 * R * kF32Rows <= c.max_context) R *= 2;
  if (items * R > 0x7fffffffLL) return KVP_ERR_INVALID_ARG;
  const unsigned grid = (unsigned)(items * R);
  cudaError_t e;
  auto launch = [&](auto width) {
    constexpr int I = decltype(width)::value;
    return CG == 1   ? launch_f32_one<I, 1>(a, grid, R, st)
           : CG == 2 ? launch_f32_one<I, 2>(a, grid, R, st)
           : CG == 4 ? launch_f32_one<I, 4>(a, grid, R, st)
                     : launch_f32_one<I, 8>(a, grid, R, st);
  };
  e = a.D <= 128 ? launch(std::integral_constant<int, 1>{}) : launch(std::integral_constant<int, 2>{});
  return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
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

// Rows turned back take 3.6 times the bytes that they have in the pool, and the longest context's for every request. So they
// are bounded, and the requests of a call go through them in groups: 16 chunks of 512 tokens on 131,072 rows 14.8 ms (at once,
// in 8 GiB, 14.7), 64 on 32,768 15.0 (14.5), 64 of 40 tokens on them 5.2 (4.6).
constexpr size_t kChunkBytes = (size_t)4 << 30;

// Requests of a group, 0 where not even one fits.
int chunk_group(const kvp_pool* pool, int B, int longest) {
  const long long page = ((long long)longest + 15) / 16 * 16;
  const size_t each = 2 * sizeof(int32_t) + sizeof(int32_t) * (page / 2) + (size_t)page * pool->kv_heads * pool->head_dim * 4;
  long long n = (long long)((kChunkBytes - 3 * 256) / each);  // the layout's parts are aligned to 256 bytes
  if (n * page > 0x7fffffffLL) n = 0x7fffffffLL / page;
  return (int)(n < 65535 ? (n < B ? n : B) : (B < 65535 ? B : 65535));
}

// Whether the chunk kernel of bf16 pools takes a call's shape.
bool chunk_shape(const kvp_pool* pool, int B, int C, int H, float scale) {
  const long long columns = (long long)C * (H / pool->kv_heads);
  const bool few = columns <= kChunkColumns || (long long)B * pool->kv_heads < pool->num_sms;
  return !(few && fp4_tc_eligible(pool, C, H)) && prefill_tc_eligible(pool, H, C, scale);
}

// Whether a call goes through the chunk kernel. Up to 64 (token, head) columns a KV head are the decode
// kernel's, which splits contexts over the SMs; it takes up to 128, and above 64 a CTA has one KV head alone. 64 requests of
// 512-4096 rows, 8 KV heads, decode kernel against chunk kernel: 64 columns 229 and 348 us, 96 397 and 347. Where the chunk
// kernel would have less than a CTA an SM, the decode kernel keeps them all: 4 requests, 128 columns 36 and 46 us.
// Groups of requests that leave three of four SMs idle are the tile kernel's, which takes 3.8 times as long as the chunk kernel
// on all of them (16 chunks of 512 tokens) and has all requests at once; so is a request whose rows do not fit.
bool chunk_eligible(const kvp_pool* pool, int B, int C, int H, int longest, float scale) {
  if (!chunk_shape(pool, B, C, H, scale)) return false;
  const int group = chunk_group(pool, B, longest), G = H / pool->kv_heads;
  const long long tiles = ((long long)C * G + 127) / 128;
  return group >= B || (group > 0 && 4 * group * tiles * pool->kv_heads >= pool->num_sms);
}

// Few query tokens of few short contexts: the tile kernel's one launch, whose clusters join their parts, before the decode
// kernel's two. Columns up to 16, 8 KV heads: one request of 128 rows 6.9 and 8.7 us, 16 of them 8.6 and 10.4, 4 tokens of
// two requests of 200 rows 11.6 and 13.2, one request of 300 rows 10.1 and 9.9; 64 of 50 rows, more tiles than SMs, 14.6 and
// 11.8; 28 columns of 100 rows 18.6 and 13.5.
bool short_eligible(const kvp_pool* pool, int B, int C, int H, int longest) {
  return pool->dtype == KVP_BF16 && (long long)C * (H / pool->kv_heads) <= 16 && longest <= 256 &&
         (long long)B * pool->kv_heads <= pool->num_sms;
}

// Requests b0 .. b0 + n - 1 of a call as one of its own.
Fp4Call requests_of(const Fp4Call& all, int b0, int n) {
  Fp4Call c = all;
  const size_t at = (size_t)b0 * c.C * c.H * c.pool->head_dim * c.pool->elem;
  c.q = static_cast<const char*>(c.q) + at;
  c.out = static_cast<char*>(c.out) + at;
  c.B = n;
  c.context_lens += b0;
  if (c.q_lens) c.q_lens += b0;
  if (c.table_rows) {
    c.table_rows += b0;
  } else {  // request b's row is b
    c.T.table += (size_t)b0 * c.T.cols;
    c.T.rows_total -= b0;
  }
  return c;
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
  if (chunk_shape(pool, batch, chunk, num_q_heads, 1.f)) {
    // no less than for fewer requests or a lower bound, which may fit where these do not
    const bool fits = chunk_group(pool, batch, max_context) >= batch;
    const size_t rows = fits ? chunk_layout(pool, batch, max_context).total : kChunkBytes;
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
  if (chunk_eligible(pool, batch, chunk, num_q_heads, max_context, scale)) {
    const int group = chunk_group(pool, batch, max_context);
    for (int b0 = 0; b0 < batch; b0 += group) {
      const int rc = launch_chunk(requests_of(c, b0, batch - b0 < group ? batch - b0 : group), max_context, st);
      if (rc != KVP_OK) return rc;
    }
    return KVP_OK;
  }
  if (fp4_tc_eligible(pool, chunk, num_q_heads) && !short_eligible(pool, batch, chunk, num_q_heads, max_context))
    return launch_fp4_tc(c, st);
  return pool->dtype == KVP_BF16 ? launch_fp4_tile(c, st) : launch_f32(c, st);
}
