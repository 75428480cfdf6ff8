// Causal attention of ragged prompts in expanded form on the fifth-generation
// tensor cores: bf16, nope_dim 128, rope_dim 64, v_dim 128.
//
// Mathematics (expanded.cu): s = scale (<q_nope, k> + <q_rope, r>), o = sum
// softmax(s) v per head; the rotated part r of a key is one row for all heads, so
// S = Q K^T over 192 entries takes k from the head's rows and r from the shared
// ones, as a third 64-entry chunk of the same operand.
//
// What bounds it: the tensor cores, and the loads that feed them. A tile is 128
// query rows of one (request, head); a block of 128 keys is 12 MMAs (M 128 N 128 K
// 16, 33 ns each) for S and 8 for O, 0.65 us, on 80 KB of K and V. Measured: 0.9 us a
// block (48 KB of K take 1.0 us to come in and S 0.5 us on two stages; the softmax
// takes 0.75 us), 1.5 us more a tile (its Q waits for the tile before); 164 us,
// 1170 TFLOP/s on 512-token chunks of 16 requests with 32 heads (GPU time in a short
// CUDA graph; 183 us under the power limit of a longer run).
//  * TMEM: two S buffers of 128 columns, O (128), two P buffers (64 columns, two
//    bf16 keys each). S(i + 1) and O += P(i) V(i) run while the softmax works:
//    four threads a row in one warp, 32 keys each (the 16-lane forms of the TMEM
//    load and store), online softmax in log2 units, O rescaled only when a row's
//    maximum grows by more than 8 (P <= 256). P is rounded to bf16 once (half a step,
//    2^-8, at most), as an operand has to be; the row sums keep it in fp32. Against 64
//    bits the output is off by 1.2 to 1.4 times what its own last rounding costs.
//  * Operands by TMA under the 128-byte swizzle: 64-entry chunks of 128 rows (16
//    KB): Q 3, K 3 a stage (two of k, one of r), V 2 a stage, two stages each.
//    Rows past the request's last key are another request's: their scores are
//    masked, their V rows zeroed in shared memory (0 times what they hold must
//    be 0).
//  * One CTA an SM keeps running: it takes the next tile off the grid by
//    cluster launch control (a waiting block's launch is cancelled and its index
//    taken over), so that the next tile's K, Q and V load while this one's last
//    block and epilogue run, and the SMs stay balanced over prompts of any
//    lengths. The loader alone decodes indices, skips tiles without rows and hands
//    the others on through shared memory: code that runs once a tile comes from
//    the instruction cache's slow levels. Tiles of a request and head are adjacent,
//    the longest first.
//  * The epilogue has warps of its own and turns its rows around in shared memory:
//    stores of 32 rows an instruction held up the softmax for 1.3 us a tile (173 us
//    where this takes 164).
//  * Slower on the same chunk: two tiles a CTA sharing K and V (half the loads, but
//    no second S buffer), Q in TMEM with P over S (S(i + 2) waits for O += P V(i)),
//    most of Q in TMEM with one P buffer, a barrier per chunk of K (176 us), softmax
//    warps in two groups that take blocks in turn, a part of the exponentials as a
//    polynomial (172 us before the epilogue's change, 171 without).
//
// Warps: 0 takes tiles and loads K and Q, 1 issues S, 2 issues O, 3 loads V, 4..11
// run the softmax (16 rows each: quadrant warp % 4, its lower or upper half), 12..15
// the epilogue.
#include "expanded.cuh"
#include "tcgen05.cuh"

namespace kvp {

namespace {

constexpr int kTile = 128, kKeys = 128;
constexpr int kDn = 128, kDr = 64, kDv = 128;
constexpr uint32_t kChunk = 16384;  // 128 rows x 128 B
constexpr int kQChunks = (kDn + kDr) / 64, kVChunks = kDv / 64;
constexpr int kKS = 2, kVS = 2;
constexpr int kThreads = 512;
constexpr int kSoft0 = 4, kSoftWarps = 8;
constexpr int kEpi0 = 12, kEpiWarps = 4;
constexpr uint64_t kWaitNs = 2000000000ull;
// For the loader's next tile: it may come by 2^31 tiles without rows before (a long prompt among many requests), 0.5 us
// each and CTA, 7 s in all. What the loader itself waits for is bounded as above and ends these waits too.
constexpr uint64_t kTileWaitNs = 20000000000ull;
constexpr size_t kSmem = (kQChunks + kKS * kQChunks + kVS * kVChunks + 1) * kChunk;

struct ExpArgs {
  CUtensorMap qmap;   // (d, head, token), box (64, 1, 128); likewise the others
  CUtensorMap kmap;
  CUtensorMap pemap;  // (d, token), box (64, 128)
  CUtensorMap vmap;
  ExpandedCall c;
  int tiles;          // of max_q
  float scale_log2;
};

// A tile's rows as the loader hands them on; nblk 0: no more tiles.
struct Tile {
  int h, jn;          // head, query rows
  int q0, k0, kl;     // first query row (of the tensor), first key row, the request's keys
  int shift;          // query row j of the tile sits at position shift + j
  int nblk;
};

struct ExpBars {
  uint64_t q_full, q_free;
  uint64_t k_full[kKS], k_empty[kKS];
  uint64_t v_full[kVS], v_empty[kVS];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t l_full[2], l_free[2];    // a tile's row sums are in ``sums``; read
  uint64_t o_free, drain, vtail;
  uint64_t answer;                  // cluster launch control -> loader
  uint64_t tile_full[2], tile_free[2];
  uint32_t taddr;
  int abort, late;
  alignas(16) uint32_t next[4];     // cluster launch control's answer
  Tile tile[2];
  // Values that are not finite (see the epilogue). Rings of four tiles: the V loader is two
  // blocks ahead of the products, at most three tiles ahead of the epilogue.
  int careful;                      // such values have been met: V's masked blocks are looked through
  int looked[4], cleared[4];        // per tile: they were; such values were found
  uint32_t first[4][kDv / 4];       // per tile: of an entry (a byte), the first key cleared, from the first row's own on; 255: none
  int again, again_bits, epilogues; // tiles to do once more; by their index mod 32; warps' tiles done
  Tile redo[8];
  float sums[2][kTile];
};

__device__ __forceinline__ bool ewait(uint64_t* bar, int k, volatile int* abort_flag, int32_t* err) {
  return mbar_wait_bounded(bar, (uint32_t)(k & 1), abort_flag, err, kWaitNs);
}

__device__ __forceinline__ void tma_2d(void* dst, const void* tmap, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// Zeros in place of the infinities and NaNs in a V stage's rows r0 .. r1 - 1 (a warp: a lane has four entries).
// ``first``: per entry (a byte) the smallest r - r0 + base with one, 255: none. Returns whether there are any.
__device__ __noinline__ bool clear_not_finite(unsigned char* stage, int r0, int r1, int base, uint32_t* first, int lane) {
  uint32_t any = 0, mine = first[lane];
  for (int r = r0; r < r1; ++r) {
    uint32_t* at = reinterpret_cast<uint32_t*>(stage + (lane >> 4) * kChunk + r * 128 + ((((lane & 15) >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8);
    uint32_t cleared = 0;  // a byte for each of the four entries
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t w = at[x];
      const bool lo = (w & 0x7f80u) == 0x7f80u, hi = (w & 0x7f800000u) == 0x7f800000u;
      if (lo || hi) at[x] = w & (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
      cleared |= (lo ? 0xffu : 0u) << (16 * x) | (hi ? 0xff00u : 0u) << (16 * x);
    }
    if (cleared) {
      any = 1;
      mine = __vminu4(mine, (~cleared) | (uint32_t)(r - r0 + base) * 0x01010101u);
    }
  }
  first[lane] = mine;
  return __any_sync(0xffffffffu, any);
}

// Ask for the index of a block that has not started; 16 bytes into ``dst``, counted on ``bar``.
__device__ __forceinline__ void take_next(uint32_t* dst, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(dst)),
               "r"(smem_u32(bar))
               : "memory");
}
// The index taken, or -1 when no block was waiting.
__device__ __forceinline__ long long taken(const uint32_t* src) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(src))
      : "memory");
  return ok ? (long long)x : -1;
}

__device__ __forceinline__ Tile tile_of(const ExpArgs& a, uint32_t idx) {
  Tile t;
  const uint32_t bh = idx / (uint32_t)a.tiles;
  const int tile = a.tiles - 1 - (int)(idx - bh * (uint32_t)a.tiles);
  const uint32_t b = bh / (uint32_t)a.c.H;
  t.h = (int)(bh - b * (uint32_t)a.c.H);
  const ExpandedRequest r = expanded_request(a.c, (int)b);
  const int j0 = tile * kTile;
  t.jn = r.ok ? max(0, min(kTile, r.ql - j0)) : 0;
  t.q0 = r.q0 + j0;
  t.k0 = r.k0;
  t.kl = r.kl;
  t.shift = r.kl - r.ql + j0;
  t.nblk = t.jn ? (t.shift + t.jn + kKeys - 1) / kKeys : 0;
  if (!r.ok && t.h == 0 && tile == 0 && threadIdx.x == 0) set_error(a.c.err, KVP_ERR_BAD_INDEX);
  return t;
}

__global__ void __launch_bounds__(kThreads, 1) expanded_tc_kernel(const __grid_constant__ ExpArgs a) {
  extern __shared__ __align__(1024) unsigned char exp_raw[];
  __shared__ ExpBars sb;
  unsigned char* sQ = exp_raw;
  unsigned char* sK = sQ + kQChunks * kChunk;
  unsigned char* sV = sK + kKS * kQChunks * kChunk;
  unsigned char* sO = sV + kVS * kVChunks * kChunk;  // 64 entries of the tile's rows of O
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sb.abort;
  int32_t* err = a.c.err;

  if (tid == 0) {
    mbar_init(&sb.q_full, 1);
    mbar_init(&sb.q_free, 1);
    for (int s = 0; s < kKS; ++s) {
      mbar_init(&sb.k_full[s], 1);
      mbar_init(&sb.k_empty[s], 1);
    }
    for (int s = 0; s < kVS; ++s) {
      mbar_init(&sb.v_full[s], 1);
      mbar_init(&sb.v_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sb.s_full[x], 1);
      mbar_init(&sb.s_free[x], kSoftWarps);
      mbar_init(&sb.p_full[x], kSoftWarps);
      mbar_init(&sb.pv_done[x], 1);
      mbar_init(&sb.tile_full[x], 1);
      mbar_init(&sb.tile_free[x], 3 + kSoftWarps + kEpiWarps);
      mbar_init(&sb.l_full[x], kSoftWarps + 1);
      mbar_init(&sb.l_free[x], kEpiWarps);
    }
    mbar_init(&sb.answer, 1);
    mbar_init(&sb.o_free, kEpiWarps);
    mbar_init(&sb.drain, 2);
    mbar_init(&sb.vtail, 1);
    sb.abort = sb.late = 0;
    sb.careful = sb.again = sb.again_bits = sb.epilogues = 0;
    fence_mbar_init();
  }
  if (warp == 0) tc5::alloc512(&sb.taddr);
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  // TMEM: S buffers at columns 0 and 128, O at 256, P buffers at 384 and 448
  const uint32_t tbase = sb.taddr;
  const uint32_t tO = tbase + 256u;

  // This CTA's k-th tile, from slot k % 2; false: none, or a wait gave up.
  auto get_tile = [&](int k, Tile& t) -> bool {
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&sb.tile_full[k & 1], (uint32_t)((k >> 1) & 1), abort_flag, err, kTileWaitNs)))
      return false;
    t = sb.tile[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sb.tile_free[k & 1]);
    return t.nblk > 0;
  };

  if (warp == 0) {
    // ======================= tiles, Q and K ===================================
    int n = 0, nq = 0, asked = 0;
    bool ok = true;
    auto ask = [&]() {
      if (lane == 0) take_next(sb.next, &sb.answer);
      ++asked;
      __syncwarp();
    };
    auto publish = [&](int k, const Tile& t) {
      if (k >= 2) ok = ok && __all_sync(0xffffffffu, ewait(&sb.tile_free[k & 1], (k >> 1) - 1, abort_flag, err));
      if (!ok) return;
      if (lane == 0) {
        sb.tile[k & 1] = t;
        mbar_arrive(&sb.tile_full[k & 1]);  // release: the tile is seen by who waits
      }
      __syncwarp();
    };
    Tile t;
    t.nblk = 0;
    bool looking = true;  // for the next tile: at first this block's own, then what is asked for
    int redo = -1;        // >= 0: the grid is done
    for (int k = -1; ok; ++k) {
      Tile nx;
      nx.nblk = 0;
      if (k >= 0 && !t.nblk) {
        if (redo < 0) {  // the tiles that have to be done again are known once all epilogues are through
          const uint64_t t0 = global_timer_ns();
          while (*(volatile int*)&sb.epilogues < k * kEpiWarps && !*abort_flag) {
            if (global_timer_ns() - t0 > kWaitNs) {
              set_error(err, KVP_ERR_TIMEOUT);
              sb.abort = 1;
            }
            __nanosleep(64);
          }
          __syncwarp();
          redo = 0;
        }
        // one lane's reading for all; after a wait that gave up the list may be half written
        const int again = __shfl_sync(0xffffffffu, *(volatile int*)&sb.again, 0);
        ok = ok && __all_sync(0xffffffffu, !*abort_flag);
        if (ok && redo < min(again, 8)) t = sb.redo[redo++];
        publish(k, t);
        if (!t.nblk) break;
      }
      if (k >= 0 && redo < 0) {
        ask();
        looking = true;
      }
      for (int i = 0; i < t.nblk || looking;) {
        if (i < t.nblk) {
          const int st = n % kKS;
          if (n >= kKS) ok = __all_sync(0xffffffffu, ewait(&sb.k_empty[st], n / kKS - 1, abort_flag, err));
          if (!ok) break;
          if (lane == 0) {
            unsigned char* dst = sK + st * kQChunks * kChunk;
            mbar_arrive_expect_tx(&sb.k_full[st], kQChunks * kChunk);
            tc5::tma_3d(dst, &a.kmap, 0, t.h, t.k0 + i * kKeys, &sb.k_full[st]);
            tc5::tma_3d(dst + kChunk, &a.kmap, 64, t.h, t.k0 + i * kKeys, &sb.k_full[st]);
            tma_2d(dst + 2 * kChunk, &a.pemap, 0, t.k0 + i * kKeys, &sb.k_full[st]);
          }
          __syncwarp();
          if (i == 0) {  // behind the first block's K, which need not wait for the tile before
            if (nq > 0) ok = __all_sync(0xffffffffu, ewait(&sb.q_free, nq - 1, abort_flag, err));
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(&sb.q_full, kQChunks * kChunk);
              for (int c = 0; c < kQChunks; ++c) tc5::tma_3d(sQ + c * kChunk, &a.qmap, 64 * c, t.h, t.q0, &sb.q_full);
            }
            ++nq;
            __syncwarp();
          }
          ++i;
          ++n;
        }
        // With the stages full, the next tile is decoded and handed on; where it has no rows, the look for another one
        // does not hold up this one's blocks: a long prompt may have millions of tiles without rows behind it.
        if (!looking || i < min(kKS, t.nblk)) continue;
        long long idx = blockIdx.x;
        if (k >= 0 || asked > 0) {
          if (i == kKS || i == t.nblk) ok = __all_sync(0xffffffffu, ewait(&sb.answer, asked - 1, abort_flag, err));
          else if (!__all_sync(0xffffffffu, mbar_test_wait(&sb.answer, (uint32_t)((asked - 1) & 1)))) continue;
          if (!ok) break;
          idx = taken(sb.next);
          fence_proxy_async_smem();  // the next answer comes through the async proxy
          __syncwarp();
        }
        if (idx >= 0) nx = tile_of(a, (uint32_t)idx);
        looking = idx >= 0 && !nx.nblk;
        if (looking) ask();
        if (nx.nblk) publish(k + 1, nx);
        if (!ok) break;
      }
      t = nx;
    }
    // what was issued has landed (bounded) before the shared memory goes away
    if (nq > 0) ewait(&sb.q_full, nq - 1, &sb.late, err);
    for (int s = 0; s < kKS; ++s) {
      const int cnt = (n + kKS - 1 - s) / kKS;
      if (cnt > 0) ewait(&sb.k_full[s], cnt - 1, &sb.late, err);
    }
    if (asked > 0) ewait(&sb.answer, asked - 1, &sb.late, err);
    __syncwarp();
  } else if (warp == 3) {
    // ======================= V ================================================
    int n = 0, ntail = 0;
    bool ok = true;
    Tile t;
    for (int k = 0; ok && get_tile(k, t); ++k) {
      // one lane's reading for all: an epilogue warp may set it at this moment
      const bool careful = __shfl_sync(0xffffffffu, *(volatile int*)&sb.careful, 0);
      if (lane == 0) {
        sb.looked[k & 3] = careful;
        sb.cleared[k & 3] = 0;
      }
      sb.first[k & 3][lane] = 0xffffffffu;
      __syncwarp();
      for (int i = 0; i < t.nblk; ++i, ++n) {
        const int st = n % kVS;
        if (n >= kVS) ok = __all_sync(0xffffffffu, ewait(&sb.v_empty[st], n / kVS - 1, abort_flag, err));
        if (!ok) break;
        unsigned char* dst = sV + st * kVChunks * kChunk;
        const int rows = t.kl - i * kKeys;  // of this request
        const bool look = careful && min(t.kl, (i + 1) * kKeys) - 1 > t.shift;  // the tile's first row does not attend all
        uint64_t* bar = rows < kKeys || look ? &sb.vtail : &sb.v_full[st];
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, kVChunks * kChunk);
          for (int c = 0; c < kVChunks; ++c) tc5::tma_3d(dst + c * kChunk, &a.vmap, 64 * c, t.h, t.k0 + i * kKeys, bar);
        }
        __syncwarp();
        if (rows < kKeys || look) {
          ok = __all_sync(0xffffffffu, ewait(&sb.vtail, ntail, abort_flag, err));
          ++ntail;
          if (!ok) break;
          for (int x = rows * 8 + lane; x < kKeys * 8; x += 32)
            for (int c = 0; c < kVChunks; ++c)
              *reinterpret_cast<uint4*>(dst + c * kChunk + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          if (look) {
            // the keys after the tile's first row's own: fewer than a tile has rows, over at most two blocks
            const int r0 = t.shift + 1 - i * kKeys;
            if (clear_not_finite(dst, max(r0, 0), min(rows, kKeys), max(r0, 0) - r0, sb.first[k & 3], lane) && lane == 0)
              sb.cleared[k & 3] = 1;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sb.v_full[st]);
          __syncwarp();
        }
      }
    }
    if (ntail > 0) ewait(&sb.vtail, ntail - 1, &sb.late, err);
    for (int s = 0; ok && s < kVS; ++s) {
      const int cnt = (n + kVS - 1 - s) / kVS;
      if (cnt > 0) ewait(&sb.v_full[s], cnt - 1, &sb.late, err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= S issuer =========================================
    int n = 0;
    bool ok = true;
    constexpr uint32_t id = tc5::idesc(kTile, kKeys, 0, 0);
    const uint64_t dq = tc5::desc(smem_u32(sQ), 16, 1024);
    Tile t;
    for (int k = 0; ok && get_tile(k, t); ++k) {
      ok = __all_sync(0xffffffffu, ewait(&sb.q_full, k, abort_flag, err));
      for (int i = 0; ok && i < t.nblk; ++i, ++n) {
        const int st = n % kKS, buf = n & 1;
        ok = __all_sync(0xffffffffu, ewait(&sb.k_full[st], n / kKS, abort_flag, err));
        if (ok && n >= 2) ok = __all_sync(0xffffffffu, ewait(&sb.s_free[buf], (n >> 1) - 1, abort_flag, err));
        if (!ok) break;
        tc5::fence_after();
        const uint64_t dk = tc5::desc(smem_u32(sK) + st * kQChunks * kChunk, 16, 1024);
        if (tc5::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4 * kQChunks; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * kChunk + (kk & 3) * 32) >> 4);
            tc5::mma_ss(tbase + 128u * (uint32_t)buf, dq + off, dk + off, id, kk > 0);
          }
          tc5::commit(&sb.s_full[buf]);
          tc5::commit(&sb.k_empty[st]);
          if (i + 1 == t.nblk) tc5::commit(&sb.q_free);
        }
        __syncwarp();
      }
    }
    if (tc5::elect_one()) tc5::commit(&sb.drain);
    __syncwarp();
  } else if (warp == 2) {
    // ======================= O issuer =========================================
    int n = 0;
    bool ok = true;
    constexpr uint32_t id = tc5::idesc(kTile, kDv, 0, 1);
    Tile t;
    for (int k = 0; ok && get_tile(k, t); ++k) {
      if (k > 0) ok = __all_sync(0xffffffffu, ewait(&sb.o_free, k - 1, abort_flag, err));
      for (int i = 0; ok && i < t.nblk; ++i, ++n) {
        const int st = n % kVS, buf = n & 1;
        ok = __all_sync(0xffffffffu, ewait(&sb.v_full[st], n / kVS, abort_flag, err));
        if (ok) ok = __all_sync(0xffffffffu, ewait(&sb.p_full[buf], n >> 1, abort_flag, err));
        if (!ok) break;
        tc5::fence_after();
        const uint64_t dv = tc5::desc(smem_u32(sV) + st * kVChunks * kChunk, kChunk, 1024);
        const uint32_t tP = tbase + 384u + 64u * (uint32_t)buf;
        const bool first = i == 0;
        if (tc5::elect_one()) {
#pragma unroll
          for (int m = 0; m < kKeys / 16; ++m)
            tc5::mma_ts(tO, tP + (uint32_t)m * 8u, dv + (uint64_t)((m * 2048) >> 4), id, (first && m == 0) ? 0u : 1u);
          tc5::commit(&sb.pv_done[buf]);
          tc5::commit(&sb.v_empty[st]);
          if (i + 1 == t.nblk) mbar_arrive(&sb.l_full[k & 1]);  // the V loader's word on the tile is in
        }
        __syncwarp();
      }
    }
    if (tc5::elect_one()) tc5::commit(&sb.drain);
    __syncwarp();
  } else if (warp < kEpi0) {
    // ======================= softmax ==========================================
    // A warp has 16 query rows: lane l the rows row0 = l / 4 and row0 + 8 of its 16, of
    // every eight keys the two from 2 (l % 4) on, so that a row lies in four lanes.
    const uint32_t lanes = (uint32_t)(32 * (warp & 3) + 16 * ((warp - kSoft0) >> 2)) << 16;
    const int row0 = (int)(lanes >> 16) + (lane >> 2);
    const float sl2 = a.scale_log2;
    int n = 0;
    bool ok = true;
    Tile t;
    for (int k = 0; ok && get_tile(k, t); ++k) {
      // last key a row attends
      const int p0 = row0 < t.jn ? t.shift + row0 : -1, p1 = row0 + 8 < t.jn ? t.shift + row0 + 8 : -1;
      float m[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
      for (int i = 0; i < t.nblk; ++i, ++n) {
        const int buf = n & 1;
        ok = __all_sync(0xffffffffu, ewait(&sb.s_full[buf], n >> 1, abort_flag, err));
        if (!ok) break;
        tc5::fence_after();
        float sv[2][32];
        const uint32_t ts = tbase + 128u * (uint32_t)buf + lanes;
        tc5::ld_rows16(ts, sv[0], sv[1]);
        tc5::ld_rows16(ts + 64, sv[0] + 16, sv[1] + 16);
        tc5::wait_ld();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sb.s_free[buf]);
        const int kb = i * kKeys + 2 * (lane & 3);
        if (!__all_sync(0xffffffffu, min(p0, p1) >= i * kKeys + kKeys - 1)) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int key = kb + 8 * (c / 2) + c % 2;
            if (key > p0) sv[0][c] = -INFINITY;
            if (key > p1) sv[1][c] = -INFINITY;
          }
        }
        float f[2], msub[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mt[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float* v = sv[x] + 8 * q;
            mt[q] = tc5::max3(tc5::max3(v[0], v[1], v[2]), tc5::max3(v[3], v[4], v[5]), fmaxf(v[6], v[7]));
          }
          float mx = fmaxf(tc5::max3(mt[0], mt[1], mt[2]), mt[3]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sl2;  // scale > 0
          const bool grow = mx > m[x] + 8.f;
          f[x] = grow && m[x] > -INFINITY ? exp2f(m[x] - mx) : 1.f;
          if (grow) m[x] = mx;
          msub[x] = m[x] == -INFINITY ? 0.f : m[x];
        }
        uint32_t w[32];  // as the 16-lane store takes them: row row0, row row0 + 8 of every eight keys
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            float y0, y1;
            tc5::fma2(y0, y1, sv[x][2 * q], sv[x][2 * q + 1], sl2, -msub[x]);
            const float e0 = tc5::ex2(y0), e1 = tc5::ex2(y1);
            w[2 * q + x] = pack_bf16(e0, e1);
            tc5::add2(ps0, ps1, e0, e1);
          }
          lsum[x] = lsum[x] * f[x] + (ps0 + ps1);
        }
        if (n >= 2) {  // P buffer buf is free once O += P V of the block two before is done
          ok = __all_sync(0xffffffffu, ewait(&sb.pv_done[buf], (n >> 1) - 1, abort_flag, err));
          if (!ok) break;
          tc5::fence_after();
        }
        tc5::st_pairs16(tbase + 384u + 64u * (uint32_t)buf + lanes, w);
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {  // O holds this tile's blocks before i: scale them once they are in
          ok = __all_sync(0xffffffffu, ewait(&sb.pv_done[buf ^ 1], (n - 1) >> 1, abort_flag, err));
          if (!ok) break;
          tc5::fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < kDv; c0 += 64) {
            float o0[16], o1[16];
            tc5::ld_rows16(tO + lanes + (uint32_t)c0, o0, o1);
            tc5::wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) o0[c] *= f[0], o1[c] *= f[1];
            tc5::st_rows16(tO + lanes + (uint32_t)c0, o0, o1);
          }
        }
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sb.p_full[buf]);
      }
      if (!ok) break;
      // ---- the row sums go to the epilogue
      if (k >= 2) ok = __all_sync(0xffffffffu, ewait(&sb.l_free[k & 1], (k >> 1) - 1, abort_flag, err));
      if (!ok) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        lsum[x] += __shfl_xor_sync(0xffffffffu, lsum[x], 1);
        lsum[x] += __shfl_xor_sync(0xffffffffu, lsum[x], 2);
        if ((lane & 3) == 0) sb.sums[k & 1][row0 + 8 * x] = lsum[x];
      }
      __threadfence_block();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.l_full[k & 1]);
    }
  } else {
    // ======================= epilogue: O / l to the output =====================
    const int quad = warp & 3, row = 32 * quad + lane;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    int n = 0;
    bool ok = true;
    Tile t;
    for (int k = 0; ok && get_tile(k, t); ++k) {
      n += t.nblk;
      // The sums come after the softmax has seen all products but the last two of
      // the tile, so the parity of the last one's phase is unambiguous from then on.
      ok = __all_sync(0xffffffffu, ewait(&sb.l_full[k & 1], k >> 1, abort_flag, err));
      if (ok) ok = __all_sync(0xffffffffu, ewait(&sb.pv_done[(n - 1) & 1], (n - 1) >> 1, abort_flag, err));
      if (!ok) break;
      tc5::fence_after();
      const float tot = *(volatile float*)&sb.sums[k & 1][row];
      const bool met = *(volatile int*)&sb.cleared[k & 3];
      // a NaN sum is the answer of a NaN score
      const float inv = tot == 0.f ? 0.f : 1.f / tot;
      float odd = 0.f;  // NaN once an entry of O is not finite
      // all of O to registers, packed, before the stores: the next tile's first product waits for it
      uint32_t w[kDv / 2];
#pragma unroll
      for (int c = 0; c < kDv; c += 16) {
        float ov[16];
        tc5::ld16(tO + lanes + c, ov);
        tc5::wait_ld();
#pragma unroll
        for (int q = 0; q < 8; ++q) w[c / 2 + q] = pack_bf16(ov[2 * q] * inv, ov[2 * q + 1] * inv);
#pragma unroll
        for (int q = 0; q < 16; ++q) odd = fmaf(ov[q], 0.f, odd);
      }
      if (met) {  // NaN where an entry met a value that was cleared, one of a key up to the row's own
#pragma unroll
        for (int q = 0; q < kDv / 4; ++q) {
          const uint32_t hit = __vcmpltu4(*(volatile uint32_t*)&sb.first[k & 3][q], (uint32_t)row * 0x01010101u);
          w[2 * q] |= __byte_perm(hit, 0, 0x1100) & 0x7fff7fffu;
          w[2 * q + 1] |= __byte_perm(hit, 0, 0x3322) & 0x7fff7fffu;
        }
      }
      // A weight of 0 does not keep an infinity or a NaN of V out of O. It is rare enough
      // that a look through V's masked blocks, which cost 14 %, waits until an O that is no
      // number shows up under a sum that is one: from then on such values that some row
      // does not attend become zeros (that entry of the rows that do becomes NaN here), and
      // the tiles that were already under way are done again.
      if (__any_sync(0xffffffffu, odd != odd && tot == tot && row < t.jn && !*(volatile int*)&sb.looked[k & 3]) && lane == 0) {
        sb.careful = 1;
        if (!(atomicOr(&sb.again_bits, 1 << (k & 31)) >> (k & 31) & 1)) {
          const int x = atomicAdd(&sb.again, 1);
          if (x < 8) sb.redo[x] = t;  // four at most: see above
        }
        __threadfence_block();
      }
      tc5::fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sb.o_free);
        mbar_arrive(&sb.l_free[k & 1]);
      }
      // To rows of 16-byte pieces side by side through shared memory, 64 entries at a
      // time: stored row by row from here, 32 lines an instruction, they held up the
      // softmax warps' accesses for 1.3 us a tile.
      unsigned char* so = sO + quad * 32 * 128;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int x = 32 * c + 4 * q;
          *reinterpret_cast<uint4*>(so + lane * 128 + ((q ^ (lane & 7)) << 4)) = make_uint4(w[x], w[x + 1], w[x + 2], w[x + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const int r = 4 * y + (lane >> 3), q = lane & 7;
          const uint4 v = *reinterpret_cast<const uint4*>(so + r * 128 + ((q ^ (r & 7)) << 4));
          if (32 * quad + r < t.jn)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.c.out) +
                                      ((size_t)(t.q0 + 32 * quad + r) * a.c.H + t.h) * kDv + 64 * c + 8 * q) = v;
        }
      }
      __threadfence_block();
      __syncwarp();
      if (lane == 0) atomicAdd(&sb.epilogues, 1);
    }
  }
  // everything issued is done (bounded) before TMEM goes back
  {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(&sb.drain, 0u))
      if (global_timer_ns() - t0 > 2 * kWaitNs) {
        set_error(err, KVP_ERR_TIMEOUT);
        break;
      }
  }
  tc5::fence_before();
  __syncthreads();
  if (warp == 0) tc5::dealloc512(tbase);
}

// A map (d, head, token) of a strided bf16 tensor, boxes of 64 entries of 128 tokens of a head.
bool encode_heads(CUtensorMap* m, const void* p, int width, int heads, int tokens, long long stride, long long head_stride) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t d[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t s[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)stride * 2};
  const cuuint32_t b[3] = {64, 1, 128}, one[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A tensor map's address is a multiple of 16 bytes, its strides are too, positive and below 2^40.
bool mappable(const void* p, long long stride, long long head_stride) {
  const long long lim = 1ll << 38;
  return !(reinterpret_cast<uintptr_t>(p) & 15) && stride > 0 && head_stride > 0 && !(stride & 7) && !(head_stride & 7) &&
         stride < lim && head_stride < lim;
}

}  // namespace

bool expanded_tc_eligible(const ExpandedCall& c, int dtype) {
  return dtype == KVP_BF16 && c.dn == kDn && c.dr == kDr && c.dv == kDv && c.scale > 0.f &&
         !(reinterpret_cast<uintptr_t>(c.out) & 15) && mappable(c.q, c.q_stride, c.q_head_stride) &&
         mappable(c.k, c.k_stride, c.k_head_stride) && mappable(c.v, c.v_stride, c.v_head_stride) &&
         mappable(c.k_pe, c.k_pe_stride, 8) && c.total_k > 0;
}

int launch_expanded_tc(const ExpandedCall& c, cudaStream_t stream) {
  ExpArgs a;
  a.c = c;
  a.tiles = (c.max_q + kTile - 1) / kTile;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  const long long grid = (long long)a.tiles * c.B * c.H;
  if (grid > 0x7fffffffLL) return KVP_ERR_INVALID_ARG;
  const auto encode = tensor_map_encoder();
  if (!encode) return KVP_ERR_CUDA;
  const cuuint64_t d[2] = {kDr, (cuuint64_t)c.total_k};
  const cuuint64_t s[1] = {(cuuint64_t)c.k_pe_stride * 2};
  const cuuint32_t b[2] = {64, 128}, one[2] = {1, 1};
  if (!encode_heads(&a.qmap, c.q, kDn + kDr, c.H, c.total_q, c.q_stride, c.q_head_stride) ||
      !encode_heads(&a.kmap, c.k, kDn, c.H, c.total_k, c.k_stride, c.k_head_stride) ||
      !encode_heads(&a.vmap, c.v, kDv, c.H, c.total_k, c.v_stride, c.v_head_stride) ||
      encode(&a.pemap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(c.k_pe), d, s, b, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return KVP_ERR_CUDA;
  // set at every call: it belongs to the current context
  if (cudaFuncSetAttribute(expanded_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
    return KVP_ERR_CUDA;
  expanded_tc_kernel<<<(unsigned)grid, kThreads, kSmem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

}  // namespace kvp
