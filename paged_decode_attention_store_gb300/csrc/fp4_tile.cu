// Attention over a four-bit pool, bf16, on the tensor cores for every head_dim, group size and number of query tokens: what
// neither the decode kernel (fp4_tc.cu) nor the chunk kernel takes (they are for head_dim 128), and few short contexts.
//
// Mathematics: as fp4_tc.cu. K and V entries are code * block scale, exact in fp16; a query row is scaled by a power of two
// and held in fp16; the weights, at most 256 (their sum stays in fp32), are rounded once to fp16.
//
// How. A CTA of four warps has a tile of (token, head) columns of one KV head. Blocks of 64 positions of the tile's span
// are turned into fp16 rows in shared memory, K by half of the threads and V by the other, a row each, the next block's
// codes fetched meanwhile; a warp multiplies 16 columns (mma m16n8k16, columns x positions, then columns x entries of V,
// the weights straight from the accumulators). Up to 16 columns: the warps have 16 positions of each block each; above:
// 16 columns each, 64 in all. Where the tiles are few the CTAs of a cluster share a tile's blocks; parts are joined over
// shared memory in a fixed order.
//
// A row is turned back once for every 64 columns, not once a call as in the chunk path, so long chunks are bound by the
// conversions and by mma's rate; few columns by the loads' latency, which other CTAs of the SM hide. 64 requests of 512-4096
// rows, 32 query heads on 8: head_dim 64 98 us (13 at the memory's rate; a block a query head on CUDA cores 474), 256 307
// (51; 1537). 16 chunks of 512 tokens on up to 2048 rows, head_dim 64: 532 us (29,107; some 45 at the matrix rate). Rows come
// by one thread's plain loads a row, one block ahead, between two barriers a block; a ring of asynchronous copies, as the decode
// kernel's, has not been built for these widths.
//
// A block of V that reads as NaN counts as zero; the columns that attend it get the NaN by hand.
#include <cooperative_groups.h>

#include "attention.cuh"
#include "fp4.cuh"

namespace kvp {

namespace {

namespace cg = cooperative_groups;

constexpr int kRows = 64;  // positions a block
constexpr int kTileThreads = 128;
constexpr int kMaxParts = 8;  // CTAs that share a tile

struct TileArgs {
  TableRef T;
  const char* codes;
  const char* scales;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const int32_t* context_lens;
  const int32_t* table_rows;
  const int32_t* q_lens;
  int Hq, Hkv, G, D, C, window, sinks, max_context, tiles;
  float scale_log2, gv;  // K's g is in the scale
  int32_t* err;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A thread's row of a block: K's or V's codes and scales of one position.
template <int DT>
struct Row {
  uint4 codes[DT / 32];
  uint32_t scales[DT / 64];
  int pos;  // INT_MAX: none, or a hole
};

template <int DT>
__device__ __forceinline__ void fetch(const TileArgs& a, const Span& u, int n, int row, int kvh, int o, bool v, Row<DT>& r) {
  const int t = o < n ? span_pos(u, o) : 0;
  const int slot = o < n ? resolve_slot(a.T, row, t, a.err) : -1;
  r.pos = slot < 0 ? 0x7fffffff : t;
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) r.codes[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < DT / 64; ++i) r.scales[i] = 0;
  if (slot < 0) return;
  const int D = a.D;
  const char* c = a.codes + ((size_t)slot * a.Hkv + kvh) * D + (v ? D / 2 : 0);
  const uint8_t* s = reinterpret_cast<const uint8_t*>(a.scales) + fp4_scale_offset(slot, kvh, a.Hkv, D) + (v ? D / 16 : 0);
  if (D % 64 == 0) {  // 16-byte rows, scales in words
#pragma unroll
    for (int i = 0; i < DT / 32; ++i)
      if (32 * i < D) r.codes[i] = __ldg(reinterpret_cast<const uint4*>(c) + i);
#pragma unroll
    for (int i = 0; i < DT / 64; ++i)
      if (64 * i < D) r.scales[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
  } else {
#pragma unroll
    for (int i = 0; i < DT / 16; ++i)
      if (16 * i < D) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(c) + i);
        if (i & 1) r.codes[i / 2].z = x.x, r.codes[i / 2].w = x.y;
        else r.codes[i / 2].x = x.x, r.codes[i / 2].y = x.y;
        r.scales[i / 4] |= (uint32_t)__ldg(s + i) << (8 * (i & 3));
      }
  }
}

// Row r as fp16 entries to ``dst``; V's blocks of NaN as zeros. Returns which of V's they are.
template <int DT>
__device__ __forceinline__ uint32_t turn(const Row<DT>& r, int D, bool v, unsigned char* dst) {
  uint32_t nan = 0;
#pragma unroll
  for (int i = 0; i < DT / 16; ++i) {
    if (16 * i >= D) break;
    const uint4 c = r.codes[i / 2];
    uint32_t s = r.scales[i / 4] >> (8 * (i & 3)) & 0xffu;
    if (v && fp4_is_nan(s)) {
      nan |= 1u << i;
      s = 0;
    }
    const uint32_t s2 = e4m3x2_to_half(s | s << 8);
    uint32_t h[4], g[4];
    e2m1x8_to_half(i & 1 ? c.z : c.x, h);
    e2m1x8_to_half(i & 1 ? c.w : c.y, g);
    reinterpret_cast<uint4*>(dst)[2 * i] =
        make_uint4(mul_half2(h[0], s2), mul_half2(h[1], s2), mul_half2(h[2], s2), mul_half2(h[3], s2));
    reinterpret_cast<uint4*>(dst)[2 * i + 1] =
        make_uint4(mul_half2(g[0], s2), mul_half2(g[1], s2), mul_half2(g[2], s2), mul_half2(g[3], s2));
  }
  return nan;
}

// Tile ``item`` of the call's. DT: head_dim rounded up to 64, 128 or 256. CT: tiles of 16 columns a CTA, 1 or 4.
template <int DT, int CT>
__device__ __forceinline__ void tile_item(const TileArgs& a, unsigned char* smem, long long item, cg::cluster_group cluster) {
  constexpr int kWarpRows = kRows * CT / 4;  // positions of a block that a warp has
  constexpr int kParts = 4 / CT;
  __shared__ int pos[kRows];
  __shared__ uint32_t vnan[kRows];
  __shared__ float factor[16 * CT], part_m[4][16], part_l[4][16];
  const int D = a.D, pitch = 2 * D + 16;
  unsigned char* sk = smem;
  unsigned char* sv = sk + kRows * pitch;
  unsigned char* sq = sv + kRows * pitch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tile = (int)(item % a.tiles), kvh = (int)(item / a.tiles % a.Hkv), b = (int)(item / a.tiles / a.Hkv);
  const int col0 = tile * 16 * CT, cols = a.C * a.G;

  const int L = a.context_lens[b], ql = a.q_lens ? a.q_lens[b] : a.C, row = a.table_rows ? a.table_rows[b] : b;
  auto column_out = [&](int col) {
    const int cj = col / a.G;
    return a.out + (((size_t)b * a.C + cj) * a.Hq + (size_t)kvh * a.G + (col - cj * a.G)) * D;
  };
  if (ql < 1 || ql > a.C || L < ql || L > a.max_context || row < 0 || row >= a.T.rows_total) {
    if (rank) return;
    if (tid == 0 && tile == 0 && kvh == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
    for (int i = tid; i < 16 * CT * (D / 8); i += kTileThreads) {
      const int col = col0 + i / (D / 8);
      if (col < cols) reinterpret_cast<uint4*>(column_out(col))[i % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int j0 = col0 / a.G, j1 = min((min(col0 + 16 * CT, cols) - 1) / a.G, ql - 1);
  if (j0 > j1) return;
  const int p0 = L - ql + j0, p1 = L - ql + j1;
  const Span u = attend_span(p1 + 1, a.window > 0 && j1 - j0 < 0x7fffffff - a.window ? a.window + (j1 - j0) : 0, a.sinks);
  const Span newest = attend_span(p1 + 1, a.window, a.sinks);
  const int n = u.se + (p1 + 1) - u.lo, blocks = (n - 1) / kRows + 1;

  const int mine = tid & (kRows - 1);
  const bool is_v = tid >= kRows;
  Row<DT> next;
  if (rank < blocks) fetch<DT>(a, u, n, row, kvh, rank * kRows + mine, is_v, next);

  // queries: 2^e <= a row's largest < 2^(e + 1), times 2^-e and the scale's sign; rows that are not finite as they are
  for (int r = warp; r < 16 * CT; r += 4) {
    const int col = col0 + r;
    const bool live = col < cols && col / a.G <= j1;
    const uint32_t* src =
        reinterpret_cast<const uint32_t*>(a.q + (((size_t)b * a.C + (live ? col / a.G : 0)) * a.Hq + (size_t)kvh * a.G +
                                                 (live ? col % a.G : 0)) * D);
    uint32_t x[DT / 64], mx = 0;
#pragma unroll
    for (int i = 0; i < DT / 64; ++i) {
      const int w = lane + 32 * i;
      x[i] = live && w < D / 2 ? __ldg(src + w) : 0u;
      mx = max(mx, max(x[i] << 16 & 0x7fff0000u, x[i] & 0x7fff0000u));
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    const int e = mx >= kInfBits ? 0 : max((int)(mx >> 23), 1) - 127;
    const float down = (e == 127 ? 0x1p-127f : __uint_as_float((uint32_t)(127 - e) << 23)) * (a.scale_log2 < 0.f ? -1.f : 1.f);
    const float up = e == -126 ? 0x1p-126f : __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int i = 0; i < DT / 64; ++i) {
      const int w = lane + 32 * i;
      if (w < D / 2) reinterpret_cast<uint32_t*>(sq + r * pitch)[w] = half2_of(bf16_lo(x[i]) * down, bf16_hi(x[i]) * down);
    }
    if (lane == 0) factor[r] = fminf(fabsf(a.scale_log2) * up, 3.0e38f);
  }

  const int ct = warp % CT, part = warp / CT, g = lane >> 2, c = lane & 3;
  float o[DT / 8][4], m[2] = {-3.0e38f, -3.0e38f}, l[2] = {0.f, 0.f}, f[2];
  int p[2], lo[2], se[2];
#pragma unroll
  for (int i = 0; i < DT / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    p[y] = L - ql + min((col0 + 16 * ct + g + 8 * y) / a.G, j1);
    const Span s = attend_span(p[y] + 1, a.window, a.sinks);
    lo[y] = s.lo;
    se[y] = s.se;
  }
  const uint32_t q_at = smem_u32(sq) + (16 * ct + (lane & 15)) * pitch + (lane >> 4) * 16;
  const uint32_t k_at = smem_u32(sk) + (part * kWarpRows + (lane & 7) + (lane >> 4) * 8) * pitch + (lane >> 3 & 1) * 16;
  const uint32_t v_at = smem_u32(sv) + (part * kWarpRows + (lane & 15)) * pitch + (lane >> 4) * 16;

  for (int i = rank; i < blocks; i += R) {
    const Row<DT> now = next;
    __syncthreads();  // the block before is done with
    const uint32_t bad = turn<DT>(now, D, is_v, (is_v ? sv : sk) + mine * pitch);
    if (is_v) vnan[mine] = bad;
    else pos[mine] = now.pos;
    // whether some column does not attend some position, or a V block is NaN
    const int special = __syncthreads_or(bad != 0 || now.pos > p0 || now.pos < newest.lo);
    if (i + R < blocks) fetch<DT>(a, u, n, row, kvh, (i + R) * kRows + mine, is_v, next);

    f[0] = factor[16 * ct + g];
    f[1] = factor[16 * ct + g + 8];
    float s[kWarpRows / 8][4];
#pragma unroll
    for (int x = 0; x < kWarpRows / 8; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < DT / 16; ++kk) {
      if (16 * kk >= D) break;
      uint32_t qa[4];
      ldmatrix_x4(qa, q_at + 32 * kk);
#pragma unroll
      for (int x = 0; x < kWarpRows / 16; ++x) {
        uint32_t kb[4];
        ldmatrix_x4(kb, k_at + 16 * x * pitch + 32 * kk);
        mma_f16(s[2 * x], qa, kb[0], kb[1]);
        mma_f16(s[2 * x + 1], qa, kb[2], kb[3]);
      }
    }
    // products rounded, so that a score minus the maximum is what it says however large both are
#pragma unroll
    for (int x = 0; x < kWarpRows / 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[x][e] = __fmul_rn(s[x][e], f[e >> 1]);
    if (special)
#pragma unroll
      for (int x = 0; x < kWarpRows / 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = pos[part * kWarpRows + 8 * x + 2 * c + (e & 1)], y = e >> 1;
          if (!(t <= p[y] && (t >= lo[y] || t < se[y]))) s[x][e] = -INFINITY;
        }
    float al[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float mx = m[y];
#pragma unroll
      for (int x = 0; x < kWarpRows / 8; ++x) mx = fmaxf(mx, fmaxf(s[x][2 * y], s[x][2 * y + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fminf(fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)), 3.0e38f);  // finite: a score beyond it becomes a NaN
      al[y] = exp2_of(m[y] - mx);
      m[y] = mx;
      l[y] *= al[y];
    }
    if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f))
#pragma unroll
      for (int x = 0; x < DT / 8; ++x) {
        o[x][0] *= al[0];
        o[x][1] *= al[0];
        o[x][2] *= al[1];
        o[x][3] *= al[1];
      }
#pragma unroll
    for (int x = 0; x < kWarpRows / 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[x][e] = exp2_of((s[x][e] - m[e >> 1]) + 8.f);  // at most 256: few of fp16's lowest
        l[e >> 1] += s[x][e];
      }
#pragma unroll
    for (int x = 0; x < kWarpRows / 16; ++x) {
      const uint32_t pa[4] = {half2_of(s[2 * x][0], s[2 * x][1]), half2_of(s[2 * x][2], s[2 * x][3]),
                              half2_of(s[2 * x + 1][0], s[2 * x + 1][1]), half2_of(s[2 * x + 1][2], s[2 * x + 1][3])};
#pragma unroll
      for (int d = 0; d < DT / 16; ++d) {
        if (16 * d >= D) break;
        uint32_t vb[4];
        ldmatrix_x4_trans(vb, v_at + 16 * x * pitch + 32 * d);
        mma_f16(o[2 * d], pa, vb[0], vb[1]);
        mma_f16(o[2 * d + 1], pa, vb[2], vb[3]);
      }
    }
    if (special)
      for (int x = part * kWarpRows; x < (part + 1) * kWarpRows; ++x) {
        const uint32_t blocks_of = vnan[x];
        if (!blocks_of) continue;
        const int t = pos[x];
#pragma unroll
        for (int d = 0; d < DT / 8; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int y = e >> 1;
            if ((blocks_of >> (d / 2) & 1) && t <= p[y] && (t >= lo[y] || t < se[y])) o[d][e] = __int_as_float(0x7fffffff);
          }
      }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
  }
  if (kParts * R == 1) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int col = col0 + 16 * ct + g + 8 * y;
      if (col >= cols || col / a.G > j1) continue;
      const float inv = l[y] == 0.f ? 0.f : a.gv / l[y];  // every score minus infinity: zeros, as in the other kernels
      uint32_t* dst = reinterpret_cast<uint32_t*>(column_out(col));
#pragma unroll
      for (int d = 0; d < DT / 8; ++d)
        if (8 * d < D) dst[4 * d + c] = pack_bf16(o[d][2 * y] * inv, o[d][2 * y + 1] * inv);
    }
    return;
  }
  // the parts' sums, maxima and outputs to shared memory, over K and V, and their join
  __syncthreads();
  float* po = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int r = g + 8 * y;
    if (c == 0) {
      part_m[warp][r] = m[y];
      part_l[warp][r] = l[y];
    }
#pragma unroll
    for (int d = 0; d < DT / 8; ++d)
      if (8 * d < D)
        *reinterpret_cast<float2*>(po + (warp * 16 + r) * D + 8 * d + 2 * c) = make_float2(o[d][2 * y], o[d][2 * y + 1]);
  }
  cluster.sync();
  // a warp a column: lane k has part k's maximum and sum, then the parts' outputs come four at a time
  for (int r = rank + R * warp; r < 16 * CT; r += 4 * R) {
    const int col = col0 + r;
    if (col >= cols || col / a.G > j1) break;  // nor are later ones
    const int parts = kParts * R, w0 = (r / 16) * 16 + r % 16;
    auto at = [&](int k) { return k % kParts * CT * 16 + w0; };  // of a CTA's warps' columns
    float mk = -3.0e38f, lk = 0.f;
    if (lane < parts) {
      mk = cluster.map_shared_rank(&part_m[0][0], lane / kParts)[at(lane)];
      lk = cluster.map_shared_rank(&part_l[0][0], lane / kParts)[at(lane)];
    }
    float M = mk;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, sh));
    const float wk = exp2_of(mk - M);
    float sum = wk * lk;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
    float2 acc[DT / 64];
#pragma unroll
    for (int i = 0; i < DT / 64; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float scale = __shfl_sync(0xffffffffu, wk, k);
      const float2* src = reinterpret_cast<const float2*>(cluster.map_shared_rank(po, k / kParts) + at(k) * D);
#pragma unroll
      for (int i = 0; i < DT / 64; ++i)
        if (lane + 32 * i < D / 2) {
          const float2 x = src[lane + 32 * i];
          acc[i].x += scale * x.x;
          acc[i].y += scale * x.y;
        }
    }
    const float inv = sum == 0.f ? 0.f : a.gv / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(column_out(col));
#pragma unroll
    for (int i = 0; i < DT / 64; ++i)
      if (lane + 32 * i < D / 2) dst[lane + 32 * i] = pack_bf16(acc[i].x * inv, acc[i].y * inv);
  }
  cluster.sync();  // the others have read this CTA's parts
}

template <int DT, int CT>
__global__ void __launch_bounds__(kTileThreads, DT == 64 ? 4 : DT == 128 ? 3 : 2)
    fp4_tile_kernel(const __grid_constant__ TileArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  cg::cluster_group cluster = cg::this_cluster();
  tile_item<DT, CT>(a, smem, blockIdx.x / cluster.num_blocks(), cluster);
}

// Chunks: the requests with a scale NaN in their spans, all their query heads again. The other calls' cost is one look
// through the marks (4 us).
__global__ void __launch_bounds__(kTileThreads, 3)
    fp4_again_kernel(const __grid_constant__ TileArgs a, int B, const int32_t* lens, const int32_t* nan, int blocks, int rows) {
  extern __shared__ __align__(128) unsigned char smem[];
  int any = 0;
#pragma unroll 8
  for (unsigned u = threadIdx.x; u < (unsigned)(B * blocks); u += kTileThreads) {  // 2^30 at most
    const unsigned b = u / (unsigned)blocks, first = (u - b * blocks) * rows;
    const int mark = nan[u];  // past the context's end whatever lay there
    any |= first < (unsigned)lens[b] ? mark : 0;
  }
  if (!__syncthreads_or(any)) return;
  const long long per = (long long)a.tiles * a.Hkv;
  for (int b = 0; b < B; ++b) {
    const int n = lens[b] == 0 ? 0 : (lens[b] - 1) / rows + 1;
    int hit = 0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) hit |= nan[(size_t)b * blocks + i];
    if (!__syncthreads_or(hit)) continue;
    for (long long i = blockIdx.x; i < per; i += gridDim.x) {
      tile_item<128, 4>(a, smem, b * per + i, cg::this_cluster());
      __syncthreads();  // its shared memory is the next one's
    }
  }
}

size_t tile_smem(int D, int CT) { return (size_t)(2 * kRows + 16 * CT) * (2 * D + 16); }

template <int DT, int CT>
cudaError_t launch_one(const TileArgs& a, unsigned grid, int R, size_t smem, cudaStream_t st) {
  auto kernel = fp4_tile_kernel<DT, CT>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tile_smem(DT, CT));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = R;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ``columns``: of a tile.
TileArgs tile_args(const Fp4Call& c, int columns) {
  const kvp_pool* pool = c.pool;
  TileArgs a;
  a.T = c.T;
  a.codes = pool->buf + (size_t)c.layer * pool->layer_bytes;
  a.scales = pool->fp4_scales + (size_t)c.layer * pool->fp4_scale_layer_bytes;
  a.q = static_cast<const __nv_bfloat16*>(c.q);
  a.out = static_cast<__nv_bfloat16*>(c.out);
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
  a.tiles = (int)(((long long)c.C * a.G + columns - 1) / columns);
  return a;
}

}  // namespace

int launch_fp4_tile(const Fp4Call& c, cudaStream_t st) {
  const kvp_pool* pool = c.pool;
  const int CT = (long long)c.C * (c.H / pool->kv_heads) <= 16 ? 1 : 4;
  const TileArgs a = tile_args(c, 16 * CT);
  const long long items = (long long)a.tiles * a.Hkv * c.B;
  // CTAs share a tile while that leaves no SM more than four, and each a block at least, or four where they join 64 columns
  // (head_dim 64: one request of 500 rows 8.9 us, with four each 13.3; a chunk of 256 tokens 20.8 us, with one each 24.4)
  int R = 1;
  const long long least = (CT == 1 ? 1 : 4) * kRows;
  while (R < kMaxParts && 2 * R * items <= 4LL * pool->num_sms && 2 * R * least <= c.max_context) R *= 2;
  if (items * R > 0x7fffffffLL) return KVP_ERR_INVALID_ARG;
  const size_t smem = tile_smem(a.D, CT);
  const unsigned grid = (unsigned)(items * R);
  cudaError_t e;
  if (a.D <= 64) e = CT == 1 ? launch_one<64, 1>(a, grid, R, smem, st) : launch_one<64, 4>(a, grid, R, smem, st);
  else if (a.D <= 128) e = CT == 1 ? launch_one<128, 1>(a, grid, R, smem, st) : launch_one<128, 4>(a, grid, R, smem, st);
  else e = CT == 1 ? launch_one<256, 1>(a, grid, R, smem, st) : launch_one<256, 4>(a, grid, R, smem, st);
  return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

int launch_fp4_again(const Fp4Call& c, const int32_t* lens, const int32_t* nan, int blocks, int rows, cudaStream_t st) {
  const TileArgs a = tile_args(c, 64);
  const size_t smem = tile_smem(a.D, 4);
  if (a.D != 128 || cudaFuncSetAttribute(fp4_again_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return KVP_ERR_CUDA;
  fp4_again_kernel<<<3 * c.pool->num_sms, kTileThreads, smem, st>>>(a, c.B, lens, nan, blocks, rows);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

}  // namespace kvp
