// Attention over a four-bit pool for few query tokens (decode, verify), bf16, head_dim 128, on the tensor cores.
//
// Mathematics. s_t = scale * g_k * <q, k_t>, softmax over t, sum of p_t v_t * g_v, over k and v entries code * block
// scale. Such an entry has six significant bits at most and lies between 2^-10 and 2688: exact in fp16, so both products
// run on fp16 operands with fp32 accumulators, K and V without any rounding. A query row is scaled by a power of two to
// at most 2 and held in fp16 (its eight bits fit; entries below 2^-14 of the largest are off by 2^-25 of it, as the fp32
// sums are). The weights are rounded once to fp16 (half a step, 2^-11; they are an operand of the second product), their
// sum keeps them in fp32.
//
// What bounds it. A token and head is 144 bytes, K and V, and its 256 entries have to become fp16 pairs: 128
// conversions, 128 multiplications by scales and 64 permutations that put two tokens' values side by side, a lane and
// instruction each, beside the products. An SM streams 23 bytes a clock (45 GB/s of 6.8 TB/s), 98 clocks for 16 tokens of
// a head; conversions and permutations issue at 64 lanes a clock and take 48 of those, everything together about 65 of
// its issue slots. So bytes bound it as long as nothing waits, and what is laid out here is laid out to need few
// instructions:
// * K is operand A of S^T = K Q^T (mma m16n8k16, tokens x heads) straight from 16-byte shared loads: which entries of d a
//   k step takes is free as long as Q agrees, so a lane's 16 bytes (32 entries, two blocks) are its part of all eight k
//   steps of its token's row. No transposing loads.
// * V^T is operand A of O^T += V^T P^T. A lane takes 16 entries (one block: one scale) of four tokens, and rows 2 i of d
//   are the entries' even ones, so that a lane ends with 16 consecutive outputs.
// * Which token is row r of a tile is free too: r for even r, r ^ 4 for odd ones, so that with the 128-byte swizzle both
//   K's loads (two tokens at a time) and V's (four) touch different banks.
// * Softmax over 32 tokens at once; the running maximum is raised only when it grows by more than 8 (in log2), as P <=
//   256 fits fp16, so O is seldom rescaled.
//
// How. The work is the batch's blocks of 32 positions (aligned, of the union of the request's queries' spans) laid end to
// end and divided evenly over the CTAs; a cut request leaves fp32 partials that a second launch joins in CTA order, so
// results do not depend on timing. One producer warp fills a ring of such blocks: a group of 16 slots that lie together
// and aligned comes by one tensor copy (all heads of the CTA, head-major, swizzled) and one copy of its scales, whole
// even if only some of its rows are attended (they lie in the pool; masks drop the others); other rows come one by one
// (a kilobyte of codes each, scales by 16-byte asynchronous copies). A consumer warp takes one KV head and up to 16
// (token, head) columns.
//
// A block of V that reads as NaN may be attended by some of the columns only: 0 * NaN would reach the others, so when a
// lane sees a NaN scale (a compare, and only with several query tokens) its scale counts as zero and the columns that
// attend it get the NaN by hand.
//
// Every wait is bounded (2 s): on timeout the CTA records KVP_ERR_TIMEOUT, waits (bounded) for its own copies and
// returns.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "attention.cuh"
#include "fp4.cuh"

namespace kvp {

namespace {

constexpr int kTok = 32;      // positions a stage: two groups of 16
constexpr int kD = 128;
constexpr int kHeadBytes = kD;       // codes of one token and head: K, then V
constexpr int kScaleBytes = kD / 8;  // scales of one token and head
constexpr int kMaxStages = 6;
constexpr int kAhead = 2;     // stages whose table entries are fetched ahead of their copies
constexpr int kQueue = 4;     // > kAhead
constexpr int kMaxConsumers = 8;
constexpr int kThreads = 32 * (kMaxConsumers + 1);
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr size_t kSmemPerSm = 227 * 1024;  // what the CTAs of an SM share, 1 KB of each one's is the system's

struct Args {
  CUtensorMap map;  // codes as (byte of a head, slot, head, layer), box (128, 16, HG, 1), 128-byte swizzle
  int use_map, layer;
  TableRef T;
  const char* codes;   // of this layer
  const char* scales;
  size_t row_bytes;    // one token, all heads
  const __nv_bfloat16* q;  // [B, C, Hq, 128]
  __nv_bfloat16* out;
  const int32_t* q_lens;
  const int32_t* context_lens;
  const int32_t* table_rows;
  int B, C, Hq, Hkv, G, HG, n_groups, tiles, CW, stages, num_ctas;
  int window, sinks, max_context;
  float scale_log2, gv;
  int4* merge;    // [num_ctas] the cut request whose last piece is here: request and group, first CTA, its slot, last CTA
  float* part_ml; // [2 * num_ctas][HG * C * G][2]
  float* part_o;  // [2 * num_ctas][HG * C * G][128]
  int32_t* err;
};

struct __align__(16) Hdr {
  int live;
  int t0;      // first position of the stage
  int valid;   // bit j: position t0 + j is in the span and its row is here
  int flags;   // 1 first stage of the piece, 2 last, 4 masks needed, 8 and 16: the groups' rows lie token by token
  int b, group, part, L;
  int ql, pad0, pad1, pad2;
};

struct Smem {
  int code_group, scale_group, stage, pitch;
  unsigned char* stages;
  Hdr* queue;    // [kQueue]
  int* entries;  // [kQueue][kTok]
  Hdr* hdr;      // [stages]
  uint64_t* full;
  uint64_t* empty;
  volatile int* abort_flag;
};

// Bytes of a group's codes: swizzled [head][token][128], or by rows at a pitch that spreads them over the banks.
__host__ __device__ __forceinline__ int code_group_bytes(int HG) { return (16 * (HG * kHeadBytes + 16) + 1023) & ~1023; }
__host__ __device__ __forceinline__ int stage_bytes(int HG) {
  return (2 * (code_group_bytes(HG) + HG * 16 * kScaleBytes) + 1023) & ~1023;
}
__host__ __forceinline__ size_t smem_bytes(int HG, int S) {
  return 1024 + (size_t)S * stage_bytes(HG) + (kQueue + S) * sizeof(Hdr) + kQueue * kTok * sizeof(int) +
         2 * S * sizeof(uint64_t) + 16;
}

__device__ __forceinline__ Smem map_smem(unsigned char* raw, int HG, int S) {
  Smem s;
  s.code_group = code_group_bytes(HG);
  s.scale_group = HG * 16 * kScaleBytes;
  s.stage = stage_bytes(HG);
  s.pitch = HG * kHeadBytes + 16;
  s.stages = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  s.queue = reinterpret_cast<Hdr*>(s.stages + (size_t)S * s.stage);
  s.hdr = s.queue + kQueue;
  s.entries = reinterpret_cast<int*>(s.hdr + S);
  s.full = reinterpret_cast<uint64_t*>(s.entries + kQueue * kTok);
  s.empty = s.full + S;
  s.abort_flag = reinterpret_cast<volatile int*>(s.empty + S);
  return s;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// This thread's arrival once its asynchronous copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// A request's part of the work: its span (of all its queries) in stages of 32 aligned positions, the sink rows' first.
struct Request {
  int L, ql, row, lo, se, n_sink, n;  // n = 0: invalid
};

__device__ __forceinline__ Request request_of(const Args& a, int b) {
  Request r;
  r.L = __ldg(a.context_lens + b);
  r.ql = a.q_lens ? __ldg(a.q_lens + b) : a.C;
  r.row = a.table_rows ? __ldg(a.table_rows + b) : b;
  r.n = 0;
  if (r.ql < 1 || r.ql > a.C || r.L < r.ql || r.L > a.max_context || r.row < 0 || r.row >= a.T.rows_total) return r;
  // the first query reaches furthest back; a.window < max_context, and a window that wide with its queries is none
  const int wide = a.window > 0 && r.ql - 1 < 0x7fffffff - a.window ? a.window + r.ql - 1 : 0;
  const Span sp = attend_span(r.L, wide, a.sinks);
  r.lo = sp.lo;
  r.se = sp.se;
  r.n_sink = (sp.se + kTok - 1) / kTok;
  r.n = r.n_sink + (r.L - 1) / kTok - sp.lo / kTok + 1;
  return r;
}

// This CTA's share of the batch's stages, found by the whole CTA.
struct Plan {
  long long R0, R1, Sv;  // the share, and where its first request and group begin
  int active, b, g;
};

__device__ void make_plan(const Args& a, Plan* pl, bool* any_bad) {
  const int per = (a.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  long long mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int n = request_of(a, b).n;
    mine += n;
    bad |= n == 0;
  }
  if (threadIdx.x == 0) pl->active = 0;
  long long total;
  long long at = block_exclusive_scan(mine, &total);
  const long long T = total * a.n_groups, Ne = min((long long)a.num_ctas, T), k = blockIdx.x;
  if (threadIdx.x == 0) a.merge[k] = make_int4(-1, 0, 0, 0);
  __syncthreads();
  if (k < Ne) {
    const long long R0 = k * T / Ne, R1 = (k + 1) * T / Ne;
    if (at * a.n_groups <= R0 && R0 < (at + mine) * a.n_groups) {  // the first request is one of this thread's
      for (int b = b0; b < b1; ++b) {
        const int n = request_of(a, b).n;
        const long long first = at * a.n_groups;
        if (R0 < first + (long long)n * a.n_groups) {
          const int g = (int)((R0 - first) / n);
          const long long Sv = first + (long long)g * n;
          pl->R0 = R0;
          pl->R1 = R1;
          pl->Sv = Sv;
          pl->b = b;
          pl->g = g;
          pl->active = 1;
          if (Sv < R0 && Sv + n <= R1) {  // cut, and its last piece is here
            const long long ka = ((Sv + 1) * Ne + T - 1) / T - 1;  // the CTA of its first piece
            a.merge[k] = make_int4(b * a.n_groups + g, (int)ka, (int)(ka * T / Ne == Sv ? 2 * ka : 2 * ka + 1), (int)k);
          }
          break;
        }
        at += n;
      }
    }
  }
  *any_bad = __syncthreads_or(bad);
}

// ---------------------------------------------------------------------------
// The producer warp: table entries kAhead stages ahead, then the copies.
// ---------------------------------------------------------------------------
__device__ void produce(const Args& a, const Smem& s, const Plan& pl, int lane) {
  const int HG = a.HG, S = a.stages;
  const uint32_t row_copy = (uint32_t)(HG * kHeadBytes);
  long long x = pl.R0, Sv = pl.Sv;  // stream position of the next stage to queue, and of its request and group
  int b = pl.b, g = pl.g;
  bool done = !pl.active, fresh = true;
  Request r;
  if (!done) r = request_of(a, b);
  int queued = 0;
  auto queue_next = [&]() {
    Hdr* h = s.queue + queued % kQueue;
    if (!done) {
      const int i = (int)(x - Sv);
      const bool sink = i < r.n_sink;
      const int t0 = (sink ? i : r.lo / kTok + i - r.n_sink) * kTok;
      const int first = sink ? 0 : r.lo, end = sink ? r.se : r.L;
      const int t = t0 + lane;
      const bool in = t >= first && t < end;
      if (in)
        cp_async4(&s.entries[queued % kQueue * kTok + lane],
                  a.T.table + (size_t)r.row * a.T.cols + (a.T.raw ? t : t / a.T.page_size));
      const bool last_of_request = x + 1 == Sv + r.n, last = last_of_request || x + 1 == pl.R1;
      const unsigned inside = __ballot_sync(0xffffffffu, in);
      if (lane == 0) {
        h->live = 1;
        h->t0 = t0;
        h->valid = (int)inside;
        // every query attends the whole stage: it ends before the first query's position, and lies in the last one's
        // window or in the first one's sinks
        const int p0 = r.L - r.ql;
        const Span sl = attend_span(r.L, a.window, a.sinks), sf = attend_span(p0 + 1, a.window, a.sinks);
        const bool whole = inside == 0xffffffffu && t0 + kTok - 1 <= p0 && (t0 >= sl.lo || t0 + kTok <= sf.se);
        h->flags = (fresh ? 1 : 0) | (last ? 2 : 0) | (whole ? 0 : 4);
        h->b = b;
        h->group = g;
        const bool cut = Sv < pl.R0 || Sv + r.n > pl.R1;
        h->part = cut ? (Sv <= pl.R0 ? 2 * (int)blockIdx.x : 2 * (int)blockIdx.x + 1) : -1;
        h->L = r.L;
        h->ql = r.ql;
      }
      fresh = last;
      if (++x >= pl.R1) {
        done = true;
      } else if (last_of_request) {
        Sv = x;
        if (++g == a.n_groups) {
          g = 0;
          do r = request_of(a, ++b);  // the share ends within a valid request
          while (r.n == 0 && b + 1 < a.B);
        }
      }
    } else if (lane == 0) {
      h->live = 0;
    }
    cp_async_commit();
    ++queued;
  };
  for (int k = 0; k < kAhead; ++k) queue_next();
  int k = 0;
  bool ok = true;
  for (;; ++k) {
    queue_next();
    cp_async_wait<kAhead>();
    __syncwarp();
    const Hdr h = s.queue[k % kQueue];
    const int st = k % S;
    if (k >= S) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s.empty[st], (uint32_t)((k / S - 1) & 1), s.abort_flag, a.err, kWaitNs));
      if (!ok) break;
    }
    if (!h.live) {
      if (lane == 0) {
        s.hdr[st].live = 0;
        mbar_arrive_n(&s.full[st], 33);
      }
      break;
    }
    const int t = h.t0 + lane, grp = lane >> 4, j = lane & 15;
    int slot = -1;
    if (h.valid >> lane & 1) {
      const int e = s.entries[k % kQueue * kTok + lane];
      const bool good = a.T.raw ? (unsigned)e < (unsigned)a.T.num_slots : (unsigned)e < (unsigned)a.T.num_pages;
      if (good) slot = a.T.raw ? e : e * a.T.page_size + t % a.T.page_size;
      else set_error(a.err, KVP_ERR_BAD_INDEX);
    }
    const unsigned here = __ballot_sync(0xffffffffu, slot >= 0);
    const unsigned mine = here >> (16 * grp) & 0xffffu;
    const int lead = mine ? __ffs(mine) - 1 : 0;
    const int base = __shfl_sync(0xffffffffu, slot, 16 * grp + lead) - lead;
    const unsigned off = __ballot_sync(0xffffffffu, slot >= 0 && slot - j != base);
    const bool together = a.use_map && mine && (base & 15) == 0 && base >= 0 && (off >> (16 * grp) & 0xffffu) == 0;
    const unsigned tg = __ballot_sync(0xffffffffu, together), lin = __ballot_sync(0xffffffffu, mine && !together);
    const bool t0g = tg & 1, t1g = tg >> 16 & 1, l0 = lin & 1, l1 = lin >> 16 & 1;
    unsigned char* sbuf = s.stages + (size_t)st * s.stage;
    unsigned char* scb = sbuf + 2 * s.code_group;
    if (lane == 0) {
      Hdr o = h;
      o.valid = (int)here;
      o.flags = h.flags | (l0 ? 8 : 0) | (l1 ? 16 : 0) | (here != 0xffffffffu ? 4 : 0);
      s.hdr[st] = o;
      const uint32_t tx = (uint32_t)((int)t0g + (int)t1g) * (uint32_t)(HG * 16 * (kHeadBytes + kScaleBytes)) +
                          (uint32_t)__popc(here & ((l0 ? 0xffffu : 0u) | (l1 ? 0xffff0000u : 0u))) * row_copy;
      mbar_arrive_expect_tx(&s.full[st], tx);
    }
    __syncwarp();
    if (together && j == 0) {  // lanes 0 and 16
      tma_load_4d(sbuf + grp * s.code_group, &a.map, 0, base, h.group * HG, a.layer, &s.full[st]);
      bulk_g2s(scb + grp * s.scale_group, a.scales + fp4_scale_offset(base, h.group * HG, a.Hkv, kD),
               (uint32_t)s.scale_group, &s.full[st]);
    }
    if (l0 || l1) {
      if ((grp ? l1 : l0) && slot >= 0)
        bulk_g2s(sbuf + grp * s.code_group + j * s.pitch, a.codes + (size_t)slot * a.row_bytes + (size_t)h.group * row_copy,
                 row_copy, &s.full[st]);
      for (int u = lane; u < kTok * HG; u += 32) {  // (token, head): two heads' lines of 16 tokens at a time
        const int tk = u & 31, hh = u >> 5;
        const int sl = __shfl_sync(0xffffffffu, slot, tk);
        if ((tk < 16 ? l0 : l1) && sl >= 0)
          cp_async16(scb + (tk >> 4) * s.scale_group + (hh * 16 + (tk & 15)) * kScaleBytes,
                     a.scales + fp4_scale_offset(sl, h.group * HG + hh, a.Hkv, kD));
      }
      cp_async_arrive(&s.full[st]);
    } else if (lane == 0) {
      mbar_arrive_n(&s.full[st], 32);
    }
  }
  cp_async_wait<0>();
  if (!ok) {  // let the copies land before the CTA ends
    *s.abort_flag = 1;
    for (int k2 = k - 1; k2 >= 0 && k2 >= k - S; --k2) {
      const uint64_t t_start = global_timer_ns();
      while (!mbar_try_wait(&s.full[k2 % S], (uint32_t)((k2 / S) & 1)))
        if (global_timer_ns() - t_start > 100000000ull) break;
    }
  }
}

// ---------------------------------------------------------------------------
// Consumer warps: one KV head and 8 NT (token, head) columns each.
// ---------------------------------------------------------------------------
template <int NT>
__device__ void consume(const Args& a, const Smem& s, int w, int lane) {
  const int G = a.G, HG = a.HG, h = w / a.tiles, col0 = (w % a.tiles) * 8 * NT, C = a.C * G;
  const int g = lane >> 2, c = lane & 3;
  const int ktok = g & 1 ? g ^ 4 : g;            // the token of row g; row g + 8: 8 further
  const int vt0 = 2 * c, vt1 = (2 * c + 1) ^ 4;  // the tokens of k 2 c and 2 c + 1, and 8 further
  // offsets in a group: rows of 128 bytes, head-major and swizzled (chunk ^ token % 8), or token by token
  auto swz = [&](int tok, int chunk) { return (uint32_t)((h * 16 + tok) * 128 + ((chunk ^ (tok & 7)) << 4)); };
  auto linr = [&](int tok, int chunk) { return (uint32_t)(tok * s.pitch + h * kHeadBytes + chunk * 16); };
  const int vchunk = 4 + (g >> 1), vin = (g & 1) * 8;
  const uint32_t ks = swz(ktok, c), kl = linr(ktok, c), v0s = swz(vt0, vchunk) + vin, v0l = linr(vt0, vchunk) + vin,
                 v1s = swz(vt1, vchunk) + vin, v1l = linr(vt1, vchunk) + vin;
  const uint32_t ksc = (uint32_t)((h * 16 + ktok) * kScaleBytes + 2 * c),
                 v0sc = (uint32_t)((h * 16 + vt0) * kScaleBytes + 8 + g), v1sc = (uint32_t)((h * 16 + vt1) * kScaleBytes + 8 + g);
  const uint32_t stages = smem_u32(s.stages);

  uint32_t qf[8][NT][2];
  float o[8][NT][4], m[NT][2], l[NT][2], f[NT][2];
  int qp[NT][2];  // positions of the columns' tokens
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = f[nt][0] = f[nt][1] = 0.f;
    qp[nt][0] = qp[nt][1] = 0;
  }

  for (int it = 0, st = 0, phase = 0;; ++it) {
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s.full[st], (uint32_t)phase, s.abort_flag, a.err, kWaitNs))) return;
    const volatile Hdr* hd = &s.hdr[st];
    if (!hd->live) return;
    const int flags = hd->flags;
    const uint32_t sb = stages + (uint32_t)st * (uint32_t)s.stage;

    if (flags & 1) {  // a new piece: its queries in fp16, scaled by powers of two; state
      const int b = hd->b, ql = hd->ql, L = hd->L, grp = hd->group;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = col0 + nt * 8 + g, cj = col / G;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (col < C && cj < ql) {
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + (((size_t)b * a.C + cj) * a.Hq + (size_t)(grp * HG + h) * G + col % G) * kD + 32 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = __ldg(src + i);
        }
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          for (const uint32_t v : {x[i].x, x[i].y, x[i].z, x[i].w}) mx = max(mx, max(v << 16 & 0x7fff0000u, v & 0x7fff0000u));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^e <= the largest < 2^(e + 1); zeros and subnormal rows: the smallest normal exponent; not finite: as it is
        const int e = mx >= kInfBits ? 0 : max((int)(mx >> 23), 1) - 127;
        const float down = e == 127 ? 0x1p-127f : __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int y = 0; y < 4; ++y) qf[2 * i + (y >> 1)][nt][y & 1] = pack_half(bf16_lo(v[y]) * down, bf16_hi(v[y]) * down);
        }
#pragma unroll
        for (int x2 = 0; x2 < 2; ++x2) {
          const int ec = __shfl_sync(0xffffffffu, e, (2 * c + x2) * 4);
          const float up = ec == -126 ? 0x1p-126f : __uint_as_float((uint32_t)(127 + ec) << 23);
          f[nt][x2] = fminf(fmaxf(a.scale_log2 * up, -3.0e38f), 3.0e38f);
          qp[nt][x2] = L - ql + min(col0 + nt * 8 + 2 * c + x2, C - 1) / G;
          m[nt][x2] = -INFINITY;
          l[nt][x2] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
      }
    }

    // S^T = K Q^T, two tiles of 16 tokens
    float x[2][NT][4];
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const bool lin = flags & (8 << tile);
      const uint32_t cb = sb + tile * s.code_group, ab = cb + (lin ? kl : ks);
      const uint32_t scb = sb + 2 * s.code_group + tile * s.scale_group + ksc;
      const uint4 r0 = lds16(ab), r1 = lds16(ab + (lin ? 8 * s.pitch : 1024));
      const uint32_t s0 = e4m3x2_to_half(lds_u16(scb)), s1 = e4m3x2_to_half(lds_u16(scb + 8 * kScaleBytes));
      const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[tile][nt][0] = x[tile][nt][1] = x[tile][nt][2] = x[tile][nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t d0 = __byte_perm(s0, s0, i < 2 ? 0x1010 : 0x3232), d1 = __byte_perm(s1, s1, i < 2 ? 0x1010 : 0x3232);
        uint32_t h0[4], h1[4];
        e2m1x8_to_half(w0[i], h0);
        e2m1x8_to_half(w1[i], h1);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t af[4] = {hmul2(h0[2 * y], d0), hmul2(h1[2 * y], d1), hmul2(h0[2 * y + 1], d0), hmul2(h1[2 * y + 1], d1)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(x[tile][nt], af, qf[2 * i + y][nt][0], qf[2 * i + y][nt][1]);
        }
      }
    }

    // softmax over the 32 tokens: rows g and g + 8 of each tile
    const unsigned valid = (unsigned)hd->valid;
    const int t0 = hd->t0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int tile = 0; tile < 2; ++tile)
#pragma unroll
        for (int y = 0; y < 4; ++y) x[tile][nt][y] *= f[nt][y & 1];
      if (flags & 4) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Span sp = attend_span(qp[nt][e] + 1, a.window, a.sinks);
#pragma unroll
          for (int tile = 0; tile < 2; ++tile)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int jt = tile * 16 + y * 8 + ktok, t = t0 + jt;
              const bool in = (valid >> jt & 1) && t <= qp[nt][e] && (t >= sp.lo || t < sp.se);
              if (!in) x[tile][nt][2 * y + e] = -INFINITY;
            }
        }
      }
    }
    float mx[NT][2];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = fmaxf(fmaxf(x[0][nt][e], x[0][nt][2 + e]), fmaxf(x[1][nt][e], x[1][nt][2 + e]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, sh));
        mx[nt][e] = v;
        grow |= v > m[nt][e] + 8.f;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[nt][e], mx[nt][e]);
          const float al = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - mn);
          m[nt][e] = mn;
          l[nt][e] *= al;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i][nt][e] *= al;
            o[i][nt][2 + e] *= al;
          }
        }
    }
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
        const float p0 = ex2(x[tile][nt][0] - m0), p1 = ex2(x[tile][nt][1] - m1), p2 = ex2(x[tile][nt][2] - m0),
                    p3 = ex2(x[tile][nt][3] - m1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        pb[tile][nt][0] = movmatrix_trans(pack_half(p0, p1));
        pb[tile][nt][1] = movmatrix_trans(pack_half(p2, p3));
      }
    }

    // O^T += V^T P^T
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const bool lin = flags & (8 << tile);
      const uint32_t cb = sb + tile * s.code_group, eight = lin ? 8 * s.pitch : 1024;
      const uint32_t a0 = cb + (lin ? v0l : v0s), a1 = cb + (lin ? v1l : v1s);
      const uint32_t scb = sb + 2 * s.code_group + tile * s.scale_group;
      const uint2 r[4] = {lds8(a0), lds8(a1), lds8(a0 + eight), lds8(a1 + eight)};
      uint32_t sc[4] = {lds_u8(scb + v0sc), lds_u8(scb + v1sc), lds_u8(scb + v0sc + 8 * kScaleBytes),
                        lds_u8(scb + v1sc + 8 * kScaleBytes)};
      if (flags & 4) {  // rows that are not there count zero times
        const unsigned vm = valid >> (16 * tile);
        if (!(vm >> vt0 & 1)) sc[0] = 0;
        if (!(vm >> vt1 & 1)) sc[1] = 0;
        if (!(vm >> (vt0 + 8) & 1)) sc[2] = 0;
        if (!(vm >> (vt1 + 8) & 1)) sc[3] = 0;
        const bool nan = sc[0] == kFp4NanScale || sc[1] == kFp4NanScale || sc[2] == kFp4NanScale || sc[3] == kFp4NanScale;
        if (__any_sync(0xffffffffu, nan)) {
          // the tokens whose block g is NaN, for the columns that attend them; their scale is zero from here on
          uint32_t who = 0;
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (sc[y] == kFp4NanScale) {
              who |= 1u << ((y & 1 ? vt1 : vt0) + (y & 2 ? 8 : 0));
              sc[y] = 0;
            }
          who |= __shfl_xor_sync(0xffffffffu, who, 1);
          who |= __shfl_xor_sync(0xffffffffu, who, 2);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const Span sp = attend_span(qp[nt][e] + 1, a.window, a.sinks);
              bool hit = false;
              for (int jt = 0; jt < 16; ++jt) {
                const int t = t0 + 16 * tile + jt;
                hit |= (who >> jt & 1) && t <= qp[nt][e] && (t >= sp.lo || t < sp.se);
              }
              if (hit)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i][nt][e] = o[i][nt][2 + e] = __int_as_float(0x7fffffff);
            }
        }
      }
      uint32_t d[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) d[y] = e4m3x2_to_half(sc[y] * 0x101u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t hv[4][4];
#pragma unroll
        for (int y = 0; y < 4; ++y) e2m1x8_to_half(i ? r[y].y : r[y].x, hv[y]);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint32_t y0 = hmul2(hv[0][z], d[0]), y1 = hmul2(hv[1][z], d[1]), y2 = hmul2(hv[2][z], d[2]),
                         y3 = hmul2(hv[3][z], d[3]);
          const uint32_t af[4] = {__byte_perm(y0, y1, 0x5410), __byte_perm(y0, y1, 0x7632), __byte_perm(y2, y3, 0x5410),
                                  __byte_perm(y2, y3, 0x7632)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[4 * i + z][nt], af, pb[tile][nt][0], pb[tile][nt][1]);
        }
      }
    }
    const int b = hd->b, grp = hd->group, part = hd->part, ql = hd->ql;
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.empty[st]);
    if (++st == a.stages) {
      st = 0;
      phase ^= 1;
    }

    if (flags & 2) {  // the piece's end: entries 16 g .. 16 g + 15 of columns 2 c and 2 c + 1
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float ls = l[nt][e];
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, sh);
          const int col = col0 + nt * 8 + 2 * c + e, cj = col / G;
          if (col >= C || cj >= ql) continue;
          float v[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[2 * i] = o[i][nt][e];
            v[2 * i + 1] = o[i][nt][2 + e];
          }
          if (part < 0) {
            const float inv = ls == 0.f ? 0.f : a.gv / ls;
            uint4* dst = reinterpret_cast<uint4*>(
                a.out + (((size_t)b * a.C + cj) * a.Hq + (size_t)(grp * HG + h) * G + col % G) * kD + 16 * g);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dst[i] = make_uint4(pack_bf16(v[8 * i] * inv, v[8 * i + 1] * inv), pack_bf16(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                                  pack_bf16(v[8 * i + 4] * inv, v[8 * i + 5] * inv),
                                  pack_bf16(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
          } else {
            const size_t at = (size_t)part * HG * C + (size_t)h * C + col;
            float4* dst = reinterpret_cast<float4*>(a.part_o + at * kD + 16 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            if (g == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m[nt][e], ls);
          }
        }
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) fp4_decode_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  __shared__ Plan pl;
  const Smem s = map_smem(raw, a.HG, a.stages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&s.full[i], 33);
      mbar_init(&s.empty[i], a.CW);
    }
    *s.abort_flag = 0;
    fence_mbar_init();
  }
  griddep_wait();  // the previous kernel's writes are visible from here on
  griddep_launch_dependents();
  bool any_bad;
  make_plan(a, &pl, &any_bad);
  if (any_bad) {  // invalid requests: recorded, their rows zero
    for (int b = blockIdx.x; b < a.B; b += a.num_ctas) {
      if (request_of(a, b).n) continue;
      if (threadIdx.x == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)b * a.C * a.Hq * kD);
      for (int i = threadIdx.x; i < a.C * a.Hq * (kD / 8); i += blockDim.x) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (!pl.active) return;
  if (warp == a.CW) produce(a, s, pl, lane);
  else consume<NT>(a, s, warp, lane);
}

// Joins the pieces of the request that CTA blockIdx.x recorded, in CTA order: one warp a column.
__global__ void __launch_bounds__(128) fp4_combine_kernel(const __grid_constant__ Args a) {
  griddep_wait();
  const int4 mg = a.merge[blockIdx.x];
  if (mg.x < 0) return;
  const int b = mg.x / a.n_groups, grp = mg.x % a.n_groups, C = a.C * a.G, lane = threadIdx.x & 31;
  const int ql = a.q_lens ? __ldg(a.q_lens + b) : a.C;
  for (int u = blockIdx.y * 4 + (threadIdx.x >> 5); u < a.HG * C; u += 4 * gridDim.y) {
    const int h = u / C, col = u % C, cj = col / a.G;
    if (cj >= ql) continue;
    const int pieces = 1 + mg.w - mg.y;
    auto at = [&](int i) { return (size_t)(i ? 2 * (mg.y + i) : mg.z) * a.HG * C + u; };
    float M = -INFINITY;
    for (int i = lane; i < pieces; i += 32) M = fmaxf(M, __ldcg(a.part_ml + at(i) * 2));
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, sh));
    const float base = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    for (int i = 0; i < pieces; ++i) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + at(i) * 2));
      const float wgt = ex2(ml.x - base);
      L += wgt * ml.y;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + at(i) * kD) + lane);
      acc.x += wgt * v.x;
      acc.y += wgt * v.y;
      acc.z += wgt * v.z;
      acc.w += wgt * v.w;
    }
    const float inv = L == 0.f ? 0.f : a.gv / L;
    uint2* dst = reinterpret_cast<uint2*>(
        a.out + (((size_t)b * a.C + cj) * a.Hq + (size_t)(grp * a.HG + h) * a.G + col % a.G) * kD) + lane;
    *dst = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
}

// How the columns of a KV head go to warps, and the CTAs to an SM.
struct Shape {
  int NT, tiles, HG, CW, ctas_per_sm, stages;
};

bool shape_for(const kvp_pool* pool, int C, int H, Shape* o) {
  if (!pool->fp4 || pool->dtype != KVP_BF16 || pool->head_dim != kD) return false;
  const long long cols = (long long)C * (H / pool->kv_heads);
  if (cols > 16 * kMaxConsumers) return false;
  o->NT = cols > 8 ? 2 : 1;
  o->tiles = (int)((cols + 8 * o->NT - 1) / (8 * o->NT));
  o->HG = kMaxConsumers / o->tiles;
  while (pool->kv_heads % o->HG) --o->HG;
  o->CW = o->HG * o->tiles;
  // 18 warps an SM at 112 registers a thread, 9 at twice as many columns
  o->ctas_per_sm = (o->NT == 1 ? 18 : 9) / (o->CW + 1);
  if (o->ctas_per_sm > 8) o->ctas_per_sm = 8;
  o->stages = kMaxStages;
  while (o->stages > 2 && smem_bytes(o->HG, o->stages) + 2048 > kSmemPerSm / o->ctas_per_sm) --o->stages;
  return true;
}

struct Layout {
  size_t merge, ml, o, total;
};
Layout layout_for(const kvp_pool* pool, const Shape& sh, int C, int H) {
  const size_t ctas = (size_t)pool->num_sms * sh.ctas_per_sm, cols = (size_t)sh.HG * C * (H / pool->kv_heads);
  Layout l;
  l.merge = 0;
  l.ml = align256(ctas * sizeof(int4));
  l.o = align256(l.ml + 2 * ctas * cols * 2 * sizeof(float));
  l.total = align256(l.o + 2 * ctas * cols * kD * sizeof(float));
  return l;
}

bool encode_map(const kvp_pool* pool, int HG, CUtensorMap* out) {
  cudaDriverEntryPointQueryResult q;
  void* fn = nullptr;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return false;
  const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  cuuint64_t dims[4] = {kHeadBytes, (cuuint64_t)pool->num_slots, (cuuint64_t)pool->kv_heads, (cuuint64_t)pool->num_layers};
  cuuint64_t strides[3] = {pool->row_bytes, kHeadBytes, pool->layer_bytes};
  cuuint32_t box[4] = {kHeadBytes, 16, (cuuint32_t)HG, 1}, each[4] = {1, 1, 1, 1};
  return encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pool->buf, dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool fp4_tc_eligible(const kvp_pool* pool, int C, int H) {
  Shape sh;
  return shape_for(pool, C, H, &sh);
}

size_t fp4_tc_workspace(const kvp_pool* pool, int C, int H) {
  Shape sh;
  return shape_for(pool, C, H, &sh) ? layout_for(pool, sh, C, H).total : 0;
}

int launch_fp4_tc(const Fp4Call& c, cudaStream_t stream) {
  kvp_pool* pool = const_cast<kvp_pool*>(c.pool);
  Shape sh;
  if (!shape_for(pool, c.C, c.H, &sh)) return KVP_ERR_INVALID_ARG;
  const Layout lay = layout_for(pool, sh, c.C, c.H);
  char* ws = static_cast<char*>(c.workspace);
  Args a;
  if (pool->fp4_map_hg != sh.HG && pool->fp4_map_hg != -sh.HG)
    pool->fp4_map_hg = encode_map(pool, sh.HG, &pool->fp4_map) ? sh.HG : -sh.HG;
  a.use_map = pool->fp4_map_hg == sh.HG;
  if (a.use_map) a.map = pool->fp4_map;
  else memset(&a.map, 0, sizeof(a.map));
  a.layer = c.layer;
  a.T = c.T;
  a.codes = pool->buf + (size_t)c.layer * pool->layer_bytes;
  a.scales = pool->fp4_scales + (size_t)c.layer * pool->fp4_scale_layer_bytes;
  a.row_bytes = pool->row_bytes;
  a.q = static_cast<const __nv_bfloat16*>(c.q);
  a.out = static_cast<__nv_bfloat16*>(c.out);
  a.q_lens = c.q_lens;
  a.context_lens = c.context_lens;
  a.table_rows = c.table_rows;
  a.B = c.B;
  a.C = c.C;
  a.Hq = c.H;
  a.Hkv = pool->kv_heads;
  a.G = c.H / pool->kv_heads;
  a.HG = sh.HG;
  a.n_groups = pool->kv_heads / sh.HG;
  a.tiles = sh.tiles;
  a.CW = sh.CW;
  a.stages = sh.stages;
  a.num_ctas = pool->num_sms * sh.ctas_per_sm;
  a.window = c.window;
  a.sinks = c.sinks;
  a.max_context = c.max_context;
  a.scale_log2 = c.scale * pool->fp4_globals[c.layer] * 1.4426950408889634f;
  a.gv = pool->fp4_globals[pool->num_layers + c.layer];
  a.merge = reinterpret_cast<int4*>(ws + lay.merge);
  a.part_ml = reinterpret_cast<float*>(ws + lay.ml);
  a.part_o = reinterpret_cast<float*>(ws + lay.o);
  a.err = pool->err;
  auto kernel = sh.NT == 1 ? fp4_decode_kernel<1> : fp4_decode_kernel<2>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(sh.HG, sh.stages)) !=
      cudaSuccess)
    return KVP_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_ctas);
  cfg.blockDim = dim3(32 * (sh.CW + 1));
  cfg.dynamicSmemBytes = smem_bytes(sh.HG, sh.stages);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return KVP_ERR_CUDA;
  cfg.gridDim = dim3(a.num_ctas, (sh.HG * a.C * a.G + 3) / 4);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fp4_combine_kernel, a) == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

}  // namespace kvp
