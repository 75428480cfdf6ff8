// Absorbed latent attention on the fifth-generation tensor cores: bf16 rows of
// latent_dim 512 + rope_dim 64, any head count, decode, verify and chunks.
//
// Mathematics (latent.cu): every (token, head) row of a request's queries
// attends the same rows x_t = [c_t | r_t]: s = scale <q, x_t>, o = sum
// softmax(s)_t c_t. A row of 1152 bytes does 2 (576 + 512) flops per query row:
// 1.9 flops a byte and query row. With the measured 281 flops a byte between the
// tensor cores' rate and the memory's, up to about 150 query rows per latent
// row are bound by memory, more by the tensor cores.
//
// Shape. A tile is R query rows (16, 32 or 64: the least that holds chunk *
// heads, else 64) of one request in one CTA; keys come in blocks of 64.
//  * S (64 x 64) = Q X^T: 36 M 64 N 64 K 16 MMAs (16 ns each, 0.59 us a block).
//    Query rows lie on TMEM lanes (16 a warp quadrant), so a row's maximum and
//    sum stay within four lanes of a warp. When R < 64 the A tile reads past Q into the
//    next bytes of shared memory: those rows of S are never read.
//  * O^T (512 x R) += X_c^T P^T: latent entries on the M axis, four M 128 blocks
//    of N = R, so that O takes 4 R <= 256 TMEM columns on all 128 lanes (O with
//    rows on the lanes would take all 512 columns at M 64) and a small R costs
//    little. X's block in shared memory serves both products: K-major for S,
//    MN-major for O^T. 16 MMAs of 20-25 ns, 0.32-0.40 us a block.
//  * What an SM does in a block at R = 64: 1.0 us of tensor time; 316 KB through
//    shared memory (the two products' operands and the block's arrival), 1.3 us at
//    128 bytes a clock; 1.65 us as its share of the memory rate when no other CTA
//    reads the same rows. Measured: 1.65 us a block in either case, with the tensor
//    pipe 45 % and shared memory about 65 % busy over the call: neither is what holds
//    a tile that shares its rows. Two block stages are all that fits beside Q (227
//    KB), so a block's way (load 1.0 us, S 0.75, softmax 0.5, O 0.5, two at a time)
//    shows; finer stages of 32 keys or of a third of the entries gave nothing back
//    (more, smaller boxes and products).
//  * The softmax weights are rounded to bf16 once, half a step (2^-8) each at most,
//    as the operand of the second product has to be; their sum keeps them in fp32.
//    Against 64 bits the output is off by 1.1 to 1.3 times what its own last
//    rounding costs.
//  * Layout of a block: groups of 8 keys, 9 KB each: 9 chunks of 64 entries, 8
//    rows of 128 bytes (128-byte swizzle). Eight consecutive slots are one TMA
//    box; any other rows are copied with 16-byte asynchronous copies (TMA row
//    gathers of 4 x 128 bytes took 41 ns each, 6 us a block), rows past the span
//    and behind holes as zeros: whatever lies in their place must not meet a
//    weight of 0.
//  * One warp finds the rows of up to four blocks ahead, four warps load them, two
//    groups of a block each: one warp for both was 6 % slower on a long context.
//    Prefetches to L2 beyond the two stages only got in the way of other CTAs' loads
//    (64 requests of about 2300 rows, 32 heads: 49.4 us with, 45.7 without).
//  * Code that runs once a block or a piece comes from the instruction cache's slow
//    levels: the walk over pieces lives in one warp, which hands them on, and the
//    issue and epilogue loops stay rolled (10 % at the smallest calls).
//
// Work split. A request's tiles are taken ``Gs`` at a time; such an item's key
// blocks, the union over its tiles, laid end to end over all items (with a block or
// two more for an item's start and end), are divided evenly over NG = SMs / Gs
// groups of Gs CTAs: CTA (g, t) walks group g's range for tile t, the CTAs of a
// group read the same rows at the same time (L2 serves all but one). A cut item
// leaves fp32 partials (slot 0: the group's first piece, slot 1: its last), which
// latent_combine_kernel joins in block order.
//
// Warps: 0 walks the pieces and names the blocks' rows, 1 issues S, 2 issues O, 3
// loads Q, 4..7 run the softmax (16 query rows each, TMEM quadrant = warp % 4),
// 8..11 look for rows that are not finite and scale O when a row's maximum grew, 4..11
// together the epilogue, 12..15 load the blocks.
// Measured (bf16, GPU time of the whole call with its combine in a CUDA graph): one
// request of 777 rows, 16 heads: 12.5 us (two launches); 64 requests of 512 .. 4096
// rows, 32 heads: 45.6 us, 4.1 TB/s (6 us until the first block is in, 4 us of
// combine); 32 requests of 8192 .. 32768 scattered rows, 128 heads: 234 us, 735
// TFLOP/s; four tokens of 64 heads on 64 requests: 128 us, 666 TFLOP/s.
// Every wait is bounded (2 s), as in the other kernels.
#include <cstring>

#include "attention.cuh"
#include "tcgen05.cuh"

namespace kvp {

namespace {

constexpr int kDc = 512, kDr = 64, kW = kDc + kDr;
constexpr int kChunks = kW / 64;
constexpr int kKeys = 64;                          // keys per block
constexpr uint32_t kGroup = 8 * kW * 2;            // 8 keys
constexpr uint32_t kStage = kKeys / 8 * kGroup;    // 73,728
constexpr int kStages = 2;
constexpr int kThreads = 512;
constexpr int kCopiers = 4, kCopy0 = 12;
constexpr int kPieces = 4;  // pieces published ahead
constexpr int kNamed = 4;   // blocks named ahead of their loads
constexpr int kSoft0 = 4, kScale0 = 8, kScaleWarps = 4;  // softmax: R / 16 of 4 warps
constexpr int kMaxR = 64;
constexpr int kMaxGs = 8;
// Blocks of time that an item's start and end cost: without them ranges of many
// items end last (four-token verify: 131 us at 0, 128 at 2; 32 heads: 45.7 at 0,
// 45.2 at 1, 46.1 at 2).
template <int R>
constexpr int kOver = R > 32 ? 2 : 1;
constexpr uint64_t kWaitNs = 2000000000ull;

struct LatArgs {
  CUtensorMap qmap;  // q as (d % 64, row, d / 64), box (64, R, 9)
  CUtensorMap box;   // the pool's lat_box
  TableRef T;
  int layer;
  const char* rows;  // the layer's slot 0
  int page_shift;    // log2 of the page size, -1: no power of two
  __nv_bfloat16* out;
  const int32_t* context_lens;
  const int32_t* table_rows;
  const int32_t* q_lens;
  int B, C, H, Gs, NG, window, sinks;
  float scale_log2;
  int4* merge;      // [CTAs]: the item a CTA starts and does not finish: {first output row, rows, last group of
                    // CTAs, slot of the first piece}; x = -1: none
  float2* part_ml;  // [CTAs][2][R]
  float* part_o;    // [CTAs][2][R][512]
  int32_t* err;
};

// A piece of the range as the namer hands it on: key blocks k0 .. k1 - 1 of a tile; k1 0: no more.
struct Piece {
  int k0, k1;
  int out_row, rows;    // first row of q and out, rows
  int r0, p0;           // the tile's first row in its request; the request's first query position
  Span u;
  int slot, last;       // -1: the whole item; else the partial's slot and, if the item starts here, its last group
};

struct LatBars {
  uint64_t piece_full[kPieces], piece_free[kPieces];
  uint64_t q_full, q_free;
  uint64_t named[kNamed], named_free[kNamed];  // namer -> loaders: a block's slots; they have been read
  uint64_t full[kStages];   // loaders (boxes' bytes, and each when its rows are in) -> issuers: the block is in
  uint64_t empty[kStages];  // O issuer (commit) -> loaders
  uint64_t s_full[2], s_free[2];
  uint64_t f_full[2];       // softmax -> scaling warps: the block's factors are in ``factor``
  uint64_t p_full[2];       // by blocks in turn: a scaling warp with nothing to do may be a block ahead of the slowest
  uint64_t pv_done, o_free, drain, sums;
  uint32_t taddr;
  int abort;
  int late;  // raised by a wait for copies in flight that ran out
  int b0;
  long long off0;
  int slots[kNamed][kKeys];  // -1: nothing to read
  int boxes[kNamed];         // mask of groups that come as boxes; -1: no more blocks
  Piece piece[kPieces];
  uint32_t row_bad[2];      // of a piece: its rows that attend a key that is not finite
  float factor[2][kMaxR];   // of a block: what O's rows have to be scaled by before it
  float row_m[kMaxR], row_l[kMaxR], row_i[kMaxR];  // of a piece: maximum, sum, what O is multiplied by
};

__device__ __forceinline__ bool lwait(uint64_t* bar, int k, volatile int* abort_flag, int32_t* err) {
  return mbar_wait_bounded(bar, (uint32_t)(k & 1), abort_flag, err, kWaitNs);
}

// Request b's lengths; q tokens 0 when it is invalid.
struct LatReq {
  int L, ql, row;
};
__device__ __forceinline__ LatReq request(const LatArgs& a, int b) {
  LatReq r;
  r.L = __ldg(a.context_lens + b);
  r.ql = a.q_lens ? __ldg(a.q_lens + b) : a.C;
  r.row = a.table_rows ? __ldg(a.table_rows + b) : b;
  if (r.ql < 1 || r.ql > a.C || r.L < r.ql || r.L > table_capacity(a.T) || r.row < 0 || r.row >= a.T.rows_total) r.ql = 0;
  return r;
}

// An item's keys: the union of the spans of its query tokens j0 .. j1.
struct LatItem {
  Span u;
  int n_keys, nblk;
};
template <int R>
__device__ __forceinline__ LatItem item_of(const LatArgs& a, const LatReq& r, int tg) {
  const int rows = r.ql * a.H, per = a.Gs * R;
  const int j0 = a.C == 1 ? 0 : tg * per / a.H, j1 = a.C == 1 ? 0 : (min((tg + 1) * per, rows) - 1) / a.H;
  const int p0 = r.L - r.ql + j0, p1 = r.L - r.ql + j1;
  LatItem it;
  it.u = attend_span(p1 + 1, a.window > 0 ? a.window + (p1 - p0) : 0, a.sinks);
  it.n_keys = it.u.se + (p1 + 1 - it.u.lo);
  it.nblk = (it.n_keys + kKeys - 1) / kKeys;
  return it;
}
template <int R>
__device__ __forceinline__ int groups_of(const LatArgs& a, int ql) {
  const int per = a.Gs * R;
  return ql * a.H <= per ? (ql > 0) : (ql * a.H + per - 1) / per;
}

// Walks the pieces of this CTA's range.
template <int R>
struct Pieces {
  const LatArgs& a;
  int b, tg, ng, t;
  long long off, left, all;
  LatReq r;
  // the current piece
  LatItem it;
  int k0, k1, tile, slot;
  long long end;  // of its item, from the range's start
  bool first = true;
  __device__ Pieces(const LatArgs& args, int t_, int b0, long long off0, long long n)
      : a(args), b(b0), tg(0), t(t_), off(off0), left(n), all(n) {
    r = request(a, b);
    ng = groups_of<R>(a, r.ql);
  }
  // The next piece whose tile exists; false at the range's end.
  __device__ bool next() {
    while (left > 0) {
      while (tg >= ng) {
        if (++b >= a.B) return false;
        r = request(a, b);
        ng = groups_of<R>(a, r.ql);
        tg = 0;
      }
      it = item_of<R>(a, r, tg);
      const int cost = it.nblk + kOver<R>;
      if (off >= cost) {  // only before the first piece: the range starts in a later item of the request
        off -= cost;
        ++tg;
        continue;
      }
      const long long to = off + left < cost ? off + left : cost;
      k0 = off > kOver<R> ? (int)off - kOver<R> : 0;
      k1 = to > kOver<R> ? (int)to - kOver<R> : 0;
      end = all - left - off + cost;
      left -= to - off;
      off = 0;
      slot = first ? 0 : 1;
      first = false;
      tile = tg * a.Gs + t;
      ++tg;
      if (k0 == k1) continue;  // only the item's overhead
      if (tile * R < r.ql * a.H) return true;
    }
    return false;
  }
};

// resolve_slot with the page size's shift where it is a power of two.
__device__ __forceinline__ int slot_of(const LatArgs& a, int row, int t) {
  if (a.T.raw || a.page_shift < 0) return resolve_slot(a.T, row, t, a.err);
  const int page = __ldg(a.T.table + (size_t)row * a.T.cols + (t >> a.page_shift));
  if ((unsigned)page >= (unsigned)a.T.num_pages) {
    set_error(a.err, KVP_ERR_BAD_INDEX);
    return -1;
  }
  return (page << a.page_shift) + (t & (a.T.page_size - 1));
}

// Row rr of a tile attends key offsets [0, se) and [wb, we] of its item's span; rows past the tile's end: none.
struct RowSpan {
  int se, wb, we;
  __device__ __forceinline__ RowSpan(const LatArgs& a, const Piece& pc, int rr) {
    const bool rv = rr < pc.rows;
    const int p = pc.p0 + (a.C == 1 ? 0 : (pc.r0 + rr) / a.H);
    const Span u = pc.u, sr = attend_span(p + 1, a.window, a.sinks);
    se = rv ? sr.se : 0;
    wb = rv ? u.se + (sr.lo - u.lo) : 1 << 30;
    we = rv ? u.se + (p - u.lo) : -1;
  }
  __device__ __forceinline__ bool attends(int o) const { return o < se || (o >= wb && o <= we); }
};

// Zeros in place of those of a block's rows key0 .. key0 + n - 1 that hold an infinity or a NaN (a warp; 9 x 128
// bytes a row); who of the tile attends one goes into ``row_bad``. ``o0``: offset of the block's first key.
template <int R>
__device__ __noinline__ void clear_not_finite(const LatArgs& a, const Piece& pc, unsigned char* block, uint32_t* row_bad,
                                              int key0, int n, int o0) {
  const int lane = threadIdx.x & 31;
  for (int key = key0; key < key0 + n; ++key) {
    unsigned char* row = block + (key >> 3) * kGroup + (key & 7) * 128 + lane * 4;
    uint32_t odd = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) odd |= tc5::not_finite2(*reinterpret_cast<const uint32_t*>(row + c * 1024));
    if (!__any_sync(0xffffffffu, odd)) continue;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) *reinterpret_cast<uint32_t*>(row + c * 1024) = 0u;
    for (int rr = lane; rr < R; rr += 32)
      if (RowSpan(a, pc, rr).attends(o0 + key)) atomicOr(&row_bad[rr >> 5], 1u << (rr & 31));
  }
  fence_proxy_async_smem();  // before the product reads them
}

__device__ __forceinline__ long long range_start(long long total, int g, int NG) { return NG ? total * g / NG : 0; }

template <int R>
constexpr size_t lat_smem() {
  return (size_t)R * kW * 2 + kStages * kStage + R * 128;
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1) latent_tc_kernel(const __grid_constant__ LatArgs a) {
  extern __shared__ __align__(1024) unsigned char lat_raw[];
  __shared__ LatBars sb;
  unsigned char* sQ = lat_raw;               // [9][R][128 B]
  unsigned char* sP = sQ + R * kW * 2;       // [R][128 B]
  unsigned char* sX = sP + R * 128;          // stages
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sb.abort;
  const int cta = blockIdx.x, g = cta / a.Gs, t = cta % a.Gs;

  // before the wait for the stream's previous kernel: nothing here touches global memory
  if (tid == 32) {
    tc5::prefetch_map(&a.qmap);
    tc5::prefetch_map(&a.box);
  }
  if (tid == 0) {
    mbar_init(&sb.q_full, 1);
    mbar_init(&sb.q_free, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sb.full[s], 2 * kCopiers);
      mbar_init(&sb.empty[s], 1);
    }
    for (int x = 0; x < kPieces; ++x) {
      mbar_init(&sb.piece_full[x], 1);
      mbar_init(&sb.piece_free[x], kCopy0 - 1);  // warps 1 .. 11
    }
    for (int x = 0; x < kNamed; ++x) {
      mbar_init(&sb.named[x], 1);
      mbar_init(&sb.named_free[x], kCopiers);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sb.s_full[x], 1);
      mbar_init(&sb.s_free[x], 2 * (R / 16));  // softmax warps and the scaling warps that look at their rows
      mbar_init(&sb.f_full[x], R / 16);
      mbar_init(&sb.p_full[x], R / 16 + kScaleWarps);
    }
    mbar_init(&sb.pv_done, 1);
    mbar_init(&sb.o_free, 4 + kScaleWarps);
    mbar_init(&sb.drain, 2);
    mbar_init(&sb.sums, R / 16);
    sb.abort = sb.late = 0;
    sb.row_bad[0] = sb.row_bad[1] = 0;
    fence_mbar_init();
  }
  if (warp == 0) tc5::alloc512(&sb.taddr);
  griddep_wait();
  griddep_launch_dependents();

  // ---- invalid requests: error word, rows of zeros -------------------------
  for (int b = cta; b < a.B; b += gridDim.x) {
    if (request(a, b).ql) continue;
    if (tid == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
    uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)b * a.C * a.H * kDc);
    for (size_t x = tid; x < (size_t)a.C * a.H * (kDc / 8); x += kThreads) o[x] = make_uint4(0u, 0u, 0u, 0u);
  }

  // ---- this group's range of key blocks ------------------------------------
  auto blocks_of = [&](int b) -> long long {
    long long n = 0;
    if (b < a.B) {
      const LatReq r = request(a, b);
      const int ng = groups_of<R>(a, r.ql);
      for (int tg = 0; tg < ng; ++tg) n += item_of<R>(a, r, tg).nblk + kOver<R>;
    }
    return n;
  };
  const long long n0 = blocks_of(tid);
  long long total, before0 = block_exclusive_scan(n0, &total);
  for (int c0 = kThreads; c0 < a.B; c0 += kThreads) {
    long long sum;
    block_exclusive_scan(blocks_of(c0 + tid), &sum);
    total += sum;
  }
  // no more groups than blocks: the groups in use are the first ones
  const int ng_used = a.NG < total ? a.NG : (int)total;
  const long long r0 = range_start(total, g, ng_used), r1 = range_start(total, g + 1, ng_used);
  const bool busy = g < ng_used;
  // the request the range starts in
  long long base = 0;
  for (int c0 = 0; busy && c0 < a.B && base <= r0; c0 += kThreads) {
    long long n = n0, before = before0, sum = total;
    if (a.B > kThreads) {
      n = c0 ? blocks_of(c0 + tid) : n0;
      before = base + block_exclusive_scan(n, &sum);
    }
    if (r0 >= before && r0 < before + n) {
      sb.b0 = c0 + tid;
      sb.off0 = r0 - before;
    }
    base += sum;
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  if (!busy) {
    if (tid == 0) a.merge[cta] = make_int4(-1, 0, 0, 0);
    if (warp == 0) tc5::dealloc512(sb.taddr);
    return;
  }
  // TMEM: O^T at columns 0 .. 4 R - 1 (block j of 128 entries at j R), S buffers at 256 and 320
  const uint32_t tbase = sb.taddr;
  // This CTA's k-th piece; false: none, or a wait gave up.
  auto get_piece = [&](int k, Piece& pc) -> bool {
    const int x = k % kPieces;
    if (!__all_sync(0xffffffffu, lwait(&sb.piece_full[x], k / kPieces, abort_flag, a.err))) return false;
    pc = sb.piece[x];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sb.piece_free[x]);
    return pc.k1 > 0;
  };
  // Rows leave L2 first: a step streams more of them than it holds, and would
  // put out the kernels' own code, which then comes from memory again, a line at a
  // time (64 requests of 2304 rows, 32 heads: 52.5 us without, 47.1 with).
  const uint64_t once = policy_evict_first();

  if (warp == 0) {
    // ======================= namer ============================================
    // Finds each block's rows. Lane l has the slots of keys 2 l and 2 l + 1 (group gi
    // is lanes 4 gi .. 4 gi + 3).
    int n = 0, np = 0;
    bool ok = true;
    Pieces<R> pc(a, t, sb.b0, sb.off0, r1 - r0);
    auto publish = [&](const Piece& v) {
      const int x = np % kPieces;
      if (np >= kPieces) ok = __all_sync(0xffffffffu, lwait(&sb.piece_free[x], np / kPieces - 1, abort_flag, a.err));
      if (!ok) return;
      if (lane == 0) {
        sb.piece[x] = v;
        mbar_arrive(&sb.piece_full[x]);  // release: the piece is seen by who waits
      }
      ++np;
      __syncwarp();
    };
    // Eight consecutive positions of a block table whose pages hold a multiple
    // of eight, from a multiple of eight on, lie in one page: one table read.
    const bool paged8 = !a.T.raw && (a.T.page_size & 7) == 0;
    while (ok && pc.next()) {
      const Span u = pc.it.u;
      const int nk = pc.it.n_keys;
      auto describe = [&]() {
        Piece v;
        v.k0 = pc.k0;
        v.k1 = pc.k1;
        v.out_row = pc.b * a.C * a.H + pc.tile * R;
        v.rows = min(R, pc.r.ql * a.H - pc.tile * R);
        v.r0 = pc.tile * R;
        v.p0 = pc.r.L - pc.r.ql;
        v.u = u;
        v.slot = v.last = -1;
        if (pc.k0 > 0 || pc.k1 < pc.it.nblk) {
          v.slot = pc.slot;
          if (pc.k0 == 0) {
            // this group starts the item: the last group is the first whose range reaches the item's end
            v.last = g;
            while (range_start(total, v.last + 1, ng_used) < r0 + pc.end) ++v.last;
          }
        }
        publish(v);
      };
      if (n) describe();
      for (int i = pc.k0; i < pc.k1; ++i, ++n) {
        const int o0 = i * kKeys, x = n % kNamed;
        int s0 = -1, s1 = -1;
        unsigned boxes = 0;
        if (paged8) {
          const int og = o0 + 8 * lane;
          int s = -1;
          if (lane < 8 && og + 7 < nk && (og >= u.se || og + 7 < u.se)) {
            const int p = span_pos(u, og);
            if ((p & 7) == 0) s = slot_of(a, pc.r.row, p);
          }
          boxes = __ballot_sync(0xffffffffu, s >= 0) & 0xFFu;
          s0 = __shfl_sync(0xffffffffu, s, lane >> 2) + 2 * (lane & 3);
          s1 = s0 + 1;
        }
        if (boxes != 0xFFu) {
          int sl[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int o = o0 + 2 * lane + k;
            sl[k] = o < nk ? slot_of(a, pc.r.row, span_pos(u, o)) : -1;
          }
          s0 = sl[0];
          s1 = sl[1];
          const int g0 = __shfl_sync(0xffffffffu, sl[0], lane & ~3);
          const unsigned run = __ballot_sync(0xffffffffu, sl[0] >= 0 && sl[1] == sl[0] + 1 && sl[0] == g0 + 2 * (lane & 3));
          boxes = 0;
#pragma unroll
          for (int gi = 0; gi < 8; ++gi)
            if (((run >> (4 * gi)) & 0xFu) == 0xFu) boxes |= 1u << gi;
        }
        if (n >= kNamed) ok = __all_sync(0xffffffffu, lwait(&sb.named_free[x], n / kNamed - 1, abort_flag, a.err));
        if (!ok) break;
        sb.slots[x][2 * lane] = s0;
        sb.slots[x][2 * lane + 1] = s1;
        if (lane == 0) sb.boxes[x] = (int)boxes;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sb.named[x]);
        if (n == 0) describe();  // behind the first block, whose rows are what takes longest
      }
    }
    if (ok && n >= kNamed) ok = __all_sync(0xffffffffu, lwait(&sb.named_free[n % kNamed], n / kNamed - 1, abort_flag, a.err));
    if (lane == 0) {
      sb.boxes[n % kNamed] = -1;
      mbar_arrive(&sb.named[n % kNamed]);
    }
    __syncwarp();
    Piece none;
    none.k1 = 0;
    if (ok) publish(none);
  } else if (warp == 3) {
    // ======================= Q ================================================
    int np = 0;
    bool ok = true;
    Piece pc;
    while (ok && get_piece(np, pc)) {
      if (np > 0) ok = __all_sync(0xffffffffu, lwait(&sb.q_free, np - 1, abort_flag, a.err));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sb.q_full, (uint32_t)R * kW * 2);
        tc5::tma_3d(sQ, &a.qmap, 0, pc.out_row, 0, &sb.q_full);
      }
      ++np;
      __syncwarp();
    }
    // what was issued has landed (bounded) before the shared memory goes away
    if (np > 0) lwait(&sb.q_full, np - 1, &sb.late, a.err);
    __syncwarp();
  } else if (warp >= kCopy0) {
    // ======================= loaders ==========================================
    // Each loads two groups of a block: as boxes, or row by row. Copies still on
    // their way when the next block can be loaded are handed on after that one's are
    // issued, else at once.
    const int w = warp - kCopy0;
    int n = 0;
    bool ok = true;
    int before = -1;  // the stage whose copies are on their way
    auto hand_on = [&]() {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.full[before]);
      before = -1;
    };
    for (;; ++n) {
      const int x = n % kNamed, st = n % kStages;
      if (before >= 0 &&
          !__all_sync(0xffffffffu, mbar_test_wait(&sb.named[x], (uint32_t)(n / kNamed) & 1) &&
                                       (n < kStages || mbar_test_wait(&sb.empty[st], (uint32_t)(n / kStages - 1) & 1)))) {
        cp_async_wait<0>();
        hand_on();
      }
      ok = __all_sync(0xffffffffu, lwait(&sb.named[x], n / kNamed, abort_flag, a.err));
      if (!ok) break;
      int boxes = *(volatile int*)&sb.boxes[x];
      if (boxes < 0) break;
      boxes = (boxes >> (2 * w)) & 3;
      const int s8 = *(volatile int*)&sb.slots[x][16 * w + 8 * (lane & 1)];  // lane < 2: the group's first slot
      if (n >= kStages) ok = __all_sync(0xffffffffu, lwait(&sb.empty[st], n / kStages - 1, abort_flag, a.err));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sb.full[st], (uint32_t)__popc(boxes) * kGroup);
        if (boxes == 3) mbar_arrive(&sb.full[st]);
      }
      __syncwarp();
      if (lane < 2 && ((boxes >> lane) & 1))
        tc5::tma_4d(sX + st * kStage + (2 * w + lane) * kGroup, &a.box, 0, s8, 0, a.layer, &sb.full[st], once);
      if (boxes != 3) {
        // a copy is 4 rows x 128 bytes a warp: lane = 8 row + 16-byte piece
        const int piece = lane & 7;
        for (int h = 4 * w; h < 4 * w + 4; ++h) {
          if ((boxes >> ((h >> 1) & 1)) & 1) continue;
          const int key = 4 * h + (lane >> 3), r = key & 7;
          const int s = *(volatile int*)&sb.slots[x][key];
          const char* src = a.rows + (size_t)max(s, 0) * (kW * 2) + piece * 16;
          const uint32_t dst = smem_u32(sX) + st * kStage + (uint32_t)(key >> 3) * kGroup + r * 128 + ((piece ^ r) << 4);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tc5::cp_async16(dst + c * 1024, src + c * 128, s < 0 ? 0 : 16, once);
        }
        cp_async_commit();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.named_free[x]);
      if (before >= 0) {
        if (boxes != 3) cp_async_wait<1>();
        else cp_async_wait<0>();
        hand_on();
      }
      if (boxes != 3) before = st;
    }
    cp_async_wait<0>();
    if (before >= 0) hand_on();
    // the boxes too have landed (bounded) before the shared memory goes away
    for (int s = 0; s < kStages; ++s) {
      const int cnt = (n + kStages - 1 - s) / kStages;
      if (cnt > 0) lwait(&sb.full[s], cnt - 1, &sb.late, a.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= S issuer =========================================
    int n = 0, np = 0;
    bool ok = true;
    constexpr uint32_t id = tc5::idesc(64, kKeys, 0, 0);
    const uint64_t dq = tc5::desc(smem_u32(sQ), 16, 1024);
    Piece pc;
    while (ok && get_piece(np, pc)) {
      ok = __all_sync(0xffffffffu, lwait(&sb.q_full, np, abort_flag, a.err));
      ++np;
      for (int i = pc.k0; ok && i < pc.k1; ++i, ++n) {
        const int st = n % kStages, buf = n & 1;
        ok = __all_sync(0xffffffffu, lwait(&sb.full[st], n / kStages, abort_flag, a.err));
        if (ok && n >= 2) ok = __all_sync(0xffffffffu, lwait(&sb.s_free[buf], n / 2 - 1, abort_flag, a.err));
        if (!ok) break;
        tc5::fence_after();
        const uint64_t dx = tc5::desc(smem_u32(sX) + st * kStage, 16, kGroup);
        const uint32_t ts = tbase + 256u + 64u * (uint32_t)buf;
        if (tc5::elect_one()) {
#pragma unroll 4
          for (int kk = 0; kk < kW / 16; ++kk)
            tc5::mma_ss(ts, dq + (uint64_t)(((kk >> 2) * R * 128 + (kk & 3) * 32) >> 4),
                        dx + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id, kk > 0);
          tc5::commit(&sb.s_full[buf]);
          if (i + 1 == pc.k1) tc5::commit(&sb.q_free);
        }
        __syncwarp();
      }
    }
    if (tc5::elect_one()) tc5::commit(&sb.drain);
    __syncwarp();
  } else if (warp == 2) {
    // ======================= O issuer =========================================
    int n = 0, np = 0;
    bool ok = true;
    constexpr uint32_t id = tc5::idesc(128, R, 1, 0);
    const uint64_t dp = tc5::desc(smem_u32(sP), 16, 1024);
    Piece pc;
    while (ok && get_piece(np, pc)) {
      if (np > 0) ok = __all_sync(0xffffffffu, lwait(&sb.o_free, np - 1, abort_flag, a.err));
      ++np;
      for (int i = pc.k0; ok && i < pc.k1; ++i, ++n) {
        const int st = n % kStages;
        ok = __all_sync(0xffffffffu, lwait(&sb.full[st], n / kStages, abort_flag, a.err));
        if (ok) ok = __all_sync(0xffffffffu, lwait(&sb.p_full[n & 1], n >> 1, abort_flag, a.err));
        if (!ok) break;
        tc5::fence_after();
        const uint64_t dx = tc5::desc(smem_u32(sX) + st * kStage, 1024, kGroup);
        const uint32_t first = i == pc.k0;
        if (tc5::elect_one()) {
#pragma unroll 1
          for (int ks = 0; ks < kKeys / 16; ++ks)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc5::mma_ss(tbase + (uint32_t)(j * R), dx + (uint64_t)((2 * j * 1024 + ks * 2 * kGroup) >> 4),
                          dp + (uint64_t)((ks * 32) >> 4), id, (first && ks == 0) ? 0u : 1u);
          tc5::commit(&sb.empty[st]);
          tc5::commit(&sb.pv_done);
        }
        __syncwarp();
      }
    }
    if (tc5::elect_one()) tc5::commit(&sb.drain);
    __syncwarp();
  } else {
    // ======================= softmax, and the scaling of O ====================
    // A softmax warp has 16 query rows: lane l rows row0 = 16 quadrant + l / 4 and
    // row0 + 8, of every eight keys the two from 2 (l % 4) on (the 16-lane form of
    // tcgen05.ld), so that no lane idles and a row lies in four lanes of one warp.
    // The scaling warps hold back P until O has been scaled, when a maximum grew.
    const int quad = warp & 3, part = (warp - kSoft0) >> 2;
    const bool softmax = warp < kScale0 && quad < R / 16;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const int row0 = 16 * quad + (lane >> 2);
    const float sl2 = a.scale_log2;
    int n = 0, np = 0;  // blocks, pieces
    int4 merge = make_int4(-1, 0, 0, 0);
    bool ok = true;
    Piece pc;
    while (ok && get_piece(np, pc)) {
      if (softmax) {
        const RowSpan sp[2] = {RowSpan(a, pc, row0), RowSpan(a, pc, row0 + 8)};
        float m[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
        for (int i = pc.k0; i < pc.k1; ++i, ++n) {
          const int buf = n & 1;
          ok = __all_sync(0xffffffffu, lwait(&sb.s_full[buf], n >> 1, abort_flag, a.err));
          if (!ok) break;
          tc5::fence_after();
          float sv[2][16];  // [row][key 8 (c / 2) + 2 (l % 4) + c % 2]
          tc5::ld_rows16(tbase + 256u + 64u * (uint32_t)buf + lanes, sv[0], sv[1]);
          tc5::wait_ld();
          tc5::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sb.s_free[buf]);
          const int o0 = i * kKeys;
          if (!__all_sync(0xffffffffu, max(sp[0].wb, sp[1].wb) <= o0 && min(sp[0].we, sp[1].we) >= o0 + kKeys - 1)) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (!sp[x].attends(o0 + 8 * (c / 2) + 2 * (lane & 3) + c % 2)) sv[x][c] = -INFINITY;
          }
          float f[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float* v = sv[x];
            float mx = tc5::max3(tc5::max3(tc5::max3(v[0], v[1], v[2]), tc5::max3(v[3], v[4], v[5]), v[15]),
                                 tc5::max3(v[6], v[7], v[8]),
                                 tc5::max3(tc5::max3(v[9], v[10], v[11]), tc5::max3(v[12], v[13], v[14]), -INFINITY));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sl2;  // scale > 0
            // a new maximum once it is 8 above the old (P <= 256 fits bf16's exponent with ease)
            f[x] = 1.f;
            if (mx > m[x] + 8.f) {
              if (m[x] > -INFINITY) f[x] = exp2f(m[x] - mx);
              m[x] = mx;
            }
            if ((lane & 3) == 0) sb.factor[buf][row0 + 8 * x] = f[x];
          }
          __threadfence_block();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sb.f_full[buf]);
          uint32_t w[2][8];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float msub = m[x] == -INFINITY ? 0.f : m[x];  // nothing kept yet: 2^-inf = 0
            float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              float y0, y1;
              tc5::fma2(y0, y1, sv[x][2 * q], sv[x][2 * q + 1], sl2, -msub);
              const float p0 = tc5::ex2(y0), p1 = tc5::ex2(y1);
              w[x][q] = pack_bf16(p0, p1);
              tc5::add2(ps0, ps1, p0, p1);
            }
            lsum[x] = lsum[x] * f[x] + (ps0 + ps1);
          }
          if (n > 0) {  // O += P X of the block before is done: P's buffer is free
            ok = __all_sync(0xffffffffu, lwait(&sb.pv_done, n - 1, abort_flag, a.err));
            if (!ok) break;
          }
          {
            const int rw = 16 * quad + (lane & 15);
            const uint32_t dst = smem_u32(sP) + rw * 128;
#pragma unroll
            for (int q = 0; q < 8; q += 2)
              tc5::store_8x8x4(dst + (((q + (lane >> 4)) ^ (rw & 7)) << 4), w[0][q], w[1][q], w[0][q + 1], w[1][q + 1]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sb.p_full[buf]);
        }
        if (!ok) break;
        ok = __all_sync(0xffffffffu, lwait(&sb.pv_done, n - 1, abort_flag, a.err));
        if (!ok) break;
        tc5::fence_after();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          lsum[x] += __shfl_xor_sync(0xffffffffu, lsum[x], 1);
          lsum[x] += __shfl_xor_sync(0xffffffffu, lsum[x], 2);
          if ((*(volatile uint32_t*)&sb.row_bad[(row0 + 8 * x) >> 5] >> ((row0 + 8 * x) & 31)) & 1) lsum[x] = __int_as_float(0x7fffffff);
          if ((lane & 3) == 0) {
            sb.row_m[row0 + 8 * x] = m[x];
            sb.row_l[row0 + 8 * x] = lsum[x];
            // a NaN sum is the answer of a NaN score; a sum of zero belongs to a row that attends nothing here
            sb.row_i[row0 + 8 * x] = lsum[x] == 0.f ? 0.f : 1.f / lsum[x];
          }
        }
        __syncwarp();
        // read above by all lanes; nobody sets it again before this piece's epilogue
        if (lane == 0) atomicAnd(&sb.row_bad[quad >> 1], quad & 1 ? 0x0000ffffu : 0xffff0000u);
        __threadfence_block();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sb.sums);
      } else if (warp >= kScale0) {
        for (int i = pc.k0; i < pc.k1; ++i, ++n) {
          const int buf = n & 1;
          ok = __all_sync(0xffffffffu, lwait(&sb.f_full[buf], n >> 1, abort_flag, a.err));
          if (!ok) break;
          if (quad < R / 16) {
            // A row of the cache that holds an infinity or a NaN makes NaN who attends it, whatever their scores
            // (minus infinity would weigh 0), and nobody else (a weight of 0 would not keep it out of O). Its score
            // with any query at all is not finite: this warp looks at its share of the block's keys, each with one
            // query row, while the softmax takes its exponentials. (Every score, and in the softmax's own chain,
            // cost 4 .. 8 %.) A query that is not finite only makes it look in vain.
            constexpr int kOwn = kKeys / (R / 16);
            float sv[kOwn / 4], z0 = 0.f, z1 = 0.f;
            tc5::fence_after();
            const uint32_t ts = tbase + 256u + 64u * (uint32_t)buf + lanes + (uint32_t)(quad * kOwn);
            if constexpr (kOwn == 16) {
              tc5::ld_rows8x16(ts, sv);
            } else if constexpr (kOwn == 32) {
              tc5::ld_rows8x32(ts, sv);
            } else {
              float other[16];
              tc5::ld_rows16(ts, sv, other);
            }
            tc5::wait_ld();
#pragma unroll
            for (int q = 0; q < kOwn / 8; ++q) tc5::fma2_acc(z0, z1, sv[2 * q], sv[2 * q + 1], 0.f);
            if (__any_sync(0xffffffffu, z0 + z1 != 0.f)) {  // NaN
              ok = __all_sync(0xffffffffu, lwait(&sb.full[n % kStages], n / kStages, abort_flag, a.err));
              if (!ok) break;
              const Piece copy = pc;  // pc itself stays in registers
              clear_not_finite<R>(a, copy, sX + (n % kStages) * kStage, sb.row_bad, quad * kOwn, kOwn, i * kKeys);
              __syncwarp();
            }
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.s_free[buf]);
          }
          volatile float* fac = sb.factor[buf];
          const float f0 = lane < R ? fac[lane] : 1.f, f1 = R > 32 ? fac[lane + 32] : 1.f;
          if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
            // Only rows with a maximum before, so O holds blocks of this piece. P(n - 1) has been
            // written, so the product before that is done and the parity is unambiguous.
            ok = __all_sync(0xffffffffu, lwait(&sb.pv_done, n - 1, abort_flag, a.err));
            if (!ok) break;
            tc5::fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < 4 * R; c0 += 16) {
              float ov[16];
              tc5::ld16(tbase + lanes + (uint32_t)c0, ov);
              tc5::wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) ov[c] *= fac[c0 % R + c];
              tc5::st16(tbase + lanes + (uint32_t)c0, ov);
            }
            tc5::wait_st();
            tc5::fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sb.p_full[buf]);
        }
        if (!ok) break;
      }
      // ---- the piece's end, once its last product is done: O / l to the output, or (m, l, O) to a partial
      ok = __all_sync(0xffffffffu, lwait(&sb.sums, np, abort_flag, a.err));
      if (!ok) break;
      ++np;
      tc5::fence_after();
      const bool whole = pc.slot < 0;
      const int rows = pc.rows;
      const size_t pbase = (size_t)(2 * cta + max(pc.slot, 0)) * R;
      if (!whole && warp == kSoft0) {
        for (int r = lane; r < R; r += 32)
          a.part_ml[pbase + r] = make_float2(*(volatile float*)&sb.row_m[r], *(volatile float*)&sb.row_l[r]);
        if (pc.last >= 0) merge = make_int4(pc.out_row, rows, pc.last, pc.slot);
      }
      __nv_bfloat16* orow = a.out + (size_t)pc.out_row * kDc;
      float* prow = a.part_o + pbase * kDc;
#pragma unroll 1
      for (int jj = 0; jj < 2; ++jj) {
        const int d = 128 * (2 * part + jj) + 32 * quad + lane;
#pragma unroll 1
        for (int c0 = 0; c0 < R; c0 += 16) {
          float ov[16];
          tc5::ld16(tbase + lanes + (uint32_t)((2 * part + jj) * R + c0), ov);
          tc5::wait_ld();
          if (whole) {
#pragma unroll
            for (int c = 0; c < 16; ++c) ov[c] *= *(volatile float*)&sb.row_i[c0 + c];
            // lanes 2 i and 2 i + 1 trade columns, so that each stores two entries of one row
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const bool odd = lane & 1;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? ov[c] : ov[c + 1], 1);
              const uint32_t v = odd ? pack_bf16(got, ov[c + 1]) : pack_bf16(ov[c], got);
              const int rw = c0 + c + (odd ? 1 : 0);
              if (rw < rows) *reinterpret_cast<uint32_t*>(orow + (size_t)rw * kDc + (d & ~1)) = v;
            }
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (c0 + c < rows) prow[(size_t)(c0 + c) * kDc + d] = ov[c];
          }
        }
      }
      tc5::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.o_free);
    }
    if (warp == kSoft0 && lane == 0) a.merge[cta] = merge;
  }
  // everything issued is done (bounded) before TMEM goes back
  {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(&sb.drain, 0u))
      if (global_timer_ns() - t0 > 2 * kWaitNs) {
        set_error(a.err, KVP_ERR_TIMEOUT);
        break;
      }
  }
  tc5::fence_before();
  __syncthreads();
  if (warp == 0) tc5::dealloc512(tbase);
}

// Joins the partials of the items that a range boundary cut. With SPLIT (few
// items, many pieces each) block (x, y) takes row y of the x-th cut item, its eight
// warps every eighth piece, joined through shared memory; else rows 8 y .. 8 y + 7
// of the item that CTA x cut, a warp each. A lane holds 16 of a row's 512 entries.
constexpr int kCombWarps = 8;
template <int R, bool SPLIT>
__global__ void __launch_bounds__(32 * kCombWarps) latent_combine_kernel(const LatArgs a) {
  __shared__ int counts[SPLIT ? kCombWarps : 1];
  __shared__ int4 rec;
  __shared__ int rec_cta;
  __shared__ float sm[SPLIT ? kCombWarps : 1], sl[SPLIT ? kCombWarps : 1];
  __shared__ float4 so[SPLIT ? kCombWarps : 1][SPLIT ? kDc / 4 : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  // the stream's next kernel may set itself up; it waits for this one before it touches memory
  griddep_launch_dependents();
  int4 mg;  // {first output row, rows, last group, slot of the first piece}
  int from;
  if (SPLIT) {
    const int ctas = a.NG * a.Gs;
    int seen = 0;
    if (tid == 0) rec_cta = -1;
    for (int c0 = 0; c0 < ctas; c0 += 32 * kCombWarps) {
      const int c = c0 + tid;
      const int4 m = c < ctas ? a.merge[c] : make_int4(-1, 0, 0, 0);
      const unsigned has = __ballot_sync(0xffffffffu, m.x >= 0);
      __syncthreads();
      if (lane == 0) counts[warp] = __popc(has);
      __syncthreads();
      int before = seen;
      for (int w = 0; w < kCombWarps; ++w) {
        if (w < warp) before += counts[w];
        seen += counts[w];
      }
      if (m.x >= 0 && before + __popc(has & ((1u << lane) - 1)) == (int)blockIdx.x) {
        rec = m;
        rec_cta = c;
      }
    }
    __syncthreads();
    from = rec_cta;
    mg = rec;
    if (from < 0) return;
  } else {
    from = blockIdx.x;
    mg = a.merge[from];
    if (mg.x < 0) return;
  }
  const int t = from % a.Gs, g = from / a.Gs, n = mg.z - g + 1;
  const int r = SPLIT ? (int)blockIdx.y : kCombWarps * (int)blockIdx.y + warp;
  if (r >= mg.y) return;  // SPLIT: the whole block
  auto at = [&](int k) { return (size_t)(2 * ((g + k) * a.Gs + t) + (k ? 0 : mg.w)) * R + r; };
  float m = -INFINITY, l = 0.f;
  float4 o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int step = SPLIT ? kCombWarps : 1;
  const int mine = SPLIT ? (n - warp + kCombWarps - 1) / kCombWarps : n;  // pieces of this warp: first + step i
  const int first = SPLIT ? warp : 0;
  for (int k0 = 0; k0 < mine; k0 += 32) {
    // 32 pieces' maxima and sums at once, then their entries
    const float2 ml = k0 + lane < mine ? a.part_ml[at(first + step * (k0 + lane))] : make_float2(-INFINITY, 0.f);
    float mx = ml.x;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
    const float mn = fmaxf(m, mx);
    const float old = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mn);
    m = mn;
    l *= old;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q].x *= old, o[q].y *= old, o[q].z *= old, o[q].w *= old;
    float ls = f * ml.y;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, sh);
    l += ls;
    const int nk = min(32, mine - k0);
#pragma unroll 4
    for (int k = 0; k < nk; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      const float4* x = reinterpret_cast<const float4*>(a.part_o + at(first + step * (k0 + k)) * kDc) + lane;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 v = x[32 * q];
        o[q].x = fmaf(fk, v.x, o[q].x);
        o[q].y = fmaf(fk, v.y, o[q].y);
        o[q].z = fmaf(fk, v.z, o[q].z);
        o[q].w = fmaf(fk, v.w, o[q].w);
      }
    }
  }
  __nv_bfloat16* out = a.out + ((size_t)mg.x + r) * kDc;
  if (!SPLIT) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      reinterpret_cast<uint2*>(out)[lane + 32 * q] =
          make_uint2(pack_bf16(o[q].x * inv, o[q].y * inv), pack_bf16(o[q].z * inv, o[q].w * inv));
    return;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int q = 0; q < 4; ++q) so[warp][lane + 32 * q] = o[q];
  __syncthreads();
  if (tid >= kDc / 4) return;
  float mx = sm[0];
#pragma unroll
  for (int w = 1; w < kCombWarps; ++w) mx = fmaxf(mx, sm[w]);
  float tot = 0.f;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kCombWarps; ++w) {
    const float f = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - mx);
    const float4 v = so[w][tid];
    tot = fmaf(f, sl[w], tot);
    s.x = fmaf(f, v.x, s.x);
    s.y = fmaf(f, v.y, s.y);
    s.z = fmaf(f, v.z, s.z);
    s.w = fmaf(f, v.w, s.w);
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  reinterpret_cast<uint2*>(out)[tid] = make_uint2(pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv));
}

struct LatShape {
  int R, Gs, NG;
};

// The least tile that holds a request's rows, else 64. A request's tiles are
// walked together, up to eight at a time: of 8 .. 5, the number that leaves
// the fewest CTAs idle in a request's last group.
LatShape lat_shape(const kvp_pool* pool, int C, int H) {
  LatShape s;
  const long long rows = (long long)C * H;
  s.R = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  const long long tiles = (rows + s.R - 1) / s.R;
  s.Gs = (int)(tiles < kMaxGs ? tiles : kMaxGs);
  if (tiles > kMaxGs) {
    long long best = -1;
    for (int gs = kMaxGs; gs > kMaxGs / 2; --gs) {
      const long long idle = (tiles + gs - 1) / gs * gs - tiles;
      if (best < 0 || idle < best) {
        best = idle;
        s.Gs = gs;
      }
    }
  }
  if (s.Gs > pool->num_sms) s.Gs = pool->num_sms;
  s.NG = pool->num_sms / s.Gs;
  return s;
}

struct LatWs {
  size_t merge, part_ml, part_o, total;
};
LatWs lat_ws(const LatShape& s) {
  LatWs w;
  const size_t ctas = (size_t)s.Gs * s.NG;
  w.merge = 0;
  w.part_ml = align256(ctas * sizeof(int4));
  w.part_o = align256(w.part_ml + ctas * 2 * s.R * sizeof(float2));
  w.total = align256(w.part_o + ctas * 2 * s.R * kDc * sizeof(float));
  return w;
}

template <int R>
cudaError_t launch_lat(const LatArgs& a, int ctas, cudaStream_t stream) {
  // set at every call: it belongs to the current context
  cudaError_t e = cudaFuncSetAttribute(latent_tc_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)lat_smem<R>());
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)ctas);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = lat_smem<R>();
  c.stream = stream;
  c.attrs = at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, latent_tc_kernel<R>, a);
  if (e != cudaSuccess) return e;
  // at most one cut item per boundary between ranges and per tile of a group, and no more than there are items
  const long long items = (long long)a.B * (((long long)a.C * a.H + (long long)a.Gs * R - 1) / ((long long)a.Gs * R));
  const unsigned cut = (unsigned)((items < a.NG ? items : a.NG) * a.Gs);
  c.blockDim = dim3(32 * kCombWarps);
  c.dynamicSmemBytes = 0;
  if (items * 8 <= a.NG) {  // about eight pieces an item or more: a block per row
    c.gridDim = dim3(cut, R);
    return cudaLaunchKernelEx(&c, latent_combine_kernel<R, true>, a);
  }
  c.gridDim = dim3((unsigned)ctas, R / kCombWarps);
  return cudaLaunchKernelEx(&c, latent_combine_kernel<R, false>, a);
}

}  // namespace

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult qr;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qr) ==
                        cudaSuccess &&
                    qr == cudaDriverEntryPointSuccess;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ok ? fn : nullptr);
  }();
  return encode;
}

// The pool's map (see common.cuh), for the shapes the kernel takes.
void latent_encode_map(kvp_pool* pool) {
  pool->lat_map_ok = 0;
  if (pool->dtype != KVP_BF16 || pool->latent_dim != kDc || pool->head_dim != kW) return;
  const auto encode = tensor_map_encoder();
  if (!encode) return;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const cuuint64_t bd[4] = {64, (cuuint64_t)pool->num_slots, kChunks, (cuuint64_t)pool->num_layers};
  const cuuint64_t bs[3] = {kW * 2, 128, (cuuint64_t)pool->layer_bytes};
  const cuuint32_t bb[4] = {64, 8, kChunks, 1};
  if (encode(&pool->lat_box, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool->buf, bd, bs, bb, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return;
  pool->lat_map_ok = 1;
}

bool latent_tc_eligible(const kvp_pool* pool, int C, int H) {
  // row indices of a request stay in int
  return pool->lat_map_ok == 1 && (long long)C * H <= 0x3fffffffLL;
}

size_t latent_tc_workspace(const kvp_pool* pool, int C, int H) { return lat_ws(lat_shape(pool, C, H)).total; }

int launch_latent_tc(const LatentCall& c, cudaStream_t stream) {
  const LatShape s = lat_shape(c.pool, c.C, c.H);
  const LatWs w = lat_ws(s);
  LatArgs a;
  const auto encode = tensor_map_encoder();
  if (!encode) return KVP_ERR_CUDA;
  const cuuint32_t one[3] = {1, 1, 1};
  const cuuint64_t qd[3] = {64, (cuuint64_t)c.B * c.C * c.H, kChunks};
  const cuuint64_t qs[2] = {kW * 2, 128};
  const cuuint32_t qb[3] = {64, (cuuint32_t)s.R, kChunks};
  if (encode(&a.qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(c.q), qd, qs, qb, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return KVP_ERR_CUDA;
  a.box = c.pool->lat_box;
  a.T = c.T;
  a.layer = c.layer;
  a.rows = c.pool->buf + (size_t)c.layer * c.pool->layer_bytes;
  a.page_shift = -1;
  if (!(c.T.page_size & (c.T.page_size - 1)))
    for (a.page_shift = 0; (1 << a.page_shift) < c.T.page_size; ++a.page_shift) {
    }
  a.out = static_cast<__nv_bfloat16*>(c.out);
  a.context_lens = c.context_lens;
  a.table_rows = c.table_rows;
  a.q_lens = c.q_lens;
  a.B = c.B;
  a.C = c.C;
  a.H = c.H;
  a.Gs = s.Gs;
  a.NG = s.NG;
  a.window = c.window;
  a.sinks = c.sinks;
  a.scale_log2 = c.scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(c.workspace);
  a.merge = reinterpret_cast<int4*>(ws + w.merge);
  a.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  a.err = c.pool->err;
  const int ctas = s.Gs * s.NG;
  const cudaError_t e = s.R == 16   ? launch_lat<16>(a, ctas, stream)
                        : s.R == 32 ? launch_lat<32>(a, ctas, stream)
                                    : launch_lat<64>(a, ctas, stream);
  return e == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

}  // namespace kvp
