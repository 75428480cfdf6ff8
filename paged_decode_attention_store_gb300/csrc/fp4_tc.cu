// Attention over a four-bit pool for few query tokens (decode, verify), bf16, head_dim 128, on the tensor cores.
//
// Mathematics. s_t = scale * g_k * <q, k_t>, softmax over t, sum of p_t v_t * g_v, over k and v entries code * block
// scale. Such an entry has six significant bits at most and lies between 2^-10 and 2688: exact in fp16, so both products
// run on fp16 operands with fp32 accumulators, K and V without any rounding. A query row is scaled by a power of two to
// at most 2 and held in fp16 (its eight bits fit; entries below 2^-14 of the largest are off by 2^-25 of it, as the fp32
// sums are). The weights are rounded once to fp16 (half a step, 2^-11, or 2^-32 of the largest if that is more; they are an
// operand of the second product), their sum keeps them in fp32.
//
// What bounds it. A token and head is 144 bytes, K and V, and its 256 entries have to become fp16 pairs. An SM streams 23
// bytes a clock (45 GB/s of 6.8 TB/s): 32 positions of eight heads in 1,660 clocks, 0.80 us. For such a stage each of the
// eight consumer warps, two on a scheduler, has 128 conversions, 128 multiplications by scales and 32 mma a lane; fp16
// multiplications and mma share a port, and in a loop of nothing else two warps took 551 clocks each way. With the shared
// loads, the permutations that put two tokens' values side by side and the softmax a stage takes 0.95 us: issue slots and
// that port bound it (0.73 of the memory's rate over a long batch), and every choice here is for fewer instructions:
// * K is operand A of S^T = K Q^T (mma m16n8k16, tokens x heads) straight from 16-byte shared loads: which entries of d a
//   k step takes is free as long as Q agrees, so a lane's 16 bytes (32 entries, two blocks) are its part of all eight k
//   steps of its token's row. No transposing loads.
// * V^T is operand A of O^T += V^T P^T. A lane takes 16 entries (one block: one scale) of four tokens, and rows 2 i of d
//   are the entries' even ones, so that a lane ends with 16 consecutive outputs.
// * Which token is row r of a tile is free too: r for even r, r ^ 4 for odd ones, so that with the 128-byte swizzle both
//   K's loads (two tokens at a time) and V's (four) touch different banks.
// * Softmax over 32 tokens at once; weights are taken against a reference, the maximum less 7 (in log2), that is raised only
//   when a score is more than 15 above it, as 2^15 fits fp16: O is seldom rescaled, and a weight still counts down to 2^-32 of
//   the largest (against the maximum itself, thousands of rows at 2^-26 of one were lost from O while the sum had them).
//
// How. The work is the batch's blocks of 32 positions (aligned, of the union of the request's queries' spans) laid end to
// end and divided evenly over the CTAs; a cut request leaves fp32 partials that a second launch joins in CTA order, so
// results do not depend on timing. Twelve warps an SM at 168 registers: eight that compute, one KV head and up to 16 (token,
// head) columns each, and up to four that fill a ring of five blocks or so. A group of 16 slots that lie together and aligned
// comes by one tensor copy (all heads of the CTA, head-major, swizzled) and one copy of its scales, whole even if only some
// of its rows are attended (they lie in the pool; masks drop the others): one warp issues all of these. Other rows come one
// by one (a kilobyte of codes each, scales by 16-byte asynchronous copies), the blocks dealt to the four warps. A warp that
// computes works on the next block's scores beside this one's values: two chains of instructions that hide each other's
// latencies (139 us instead of 185 for 256 requests).
//
// Measured (8 KV heads of 128, pages of 16): 256 requests of 512-4096 rows, 32 query heads, 136 us (0.73 of a copy's rate);
// 64 of them 46.8 us (0.57); with 4 tokens each 62 us; one of 777 rows 11 us, of which about 2 us are the work split, 1 the
// table, 3 the first rows' way and 3.5 the join: chains of memory latencies, as in the other small calls. 32 requests of
// 8,192-32,768 scattered rows, 64 query heads, 192 us (0.61; 116 at a copy's rate): a row's scales, 16 bytes a head, cost a
// sector of 32 each, 31 us of that (161 with the scales left out); what the other 44 are, the rows' single copies or their
// issue, has not been measured.
//
// A block of V that reads as NaN may be attended by some of the columns only: 0 * NaN would reach the others, so when a
// lane sees a NaN scale (a compare, and only with several query tokens) its scale counts as zero and the columns that
// attend it get the NaN by hand.
//
// Every wait is bounded (2 s): on timeout the CTA records KVP_ERR_TIMEOUT and returns; its producers wait (4 s) for the copies
// that they issued, whoever gave up.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "attention.cuh"
#include "fp4.cuh"

namespace kvp {

namespace {

constexpr int kTok = 32;      // positions a stage: two groups of 16
constexpr int kD = 128;
constexpr int kHeadBytes = kD;       // codes of one token and head: K, then V
constexpr int kScaleBytes = kD / 8;  // scales of one token and head
constexpr int kMaxStages = 6;
constexpr int kMaxConsumers = 8;
constexpr int kThreads = 32 * (kMaxConsumers + kMaxConsumers / 2);
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr size_t kSmemPerSm = 227 * 1024;  // what the CTAs of an SM share
constexpr size_t kSmemRest = 2048;         // of each: 1 KB is the system's, the rest the kernel's static part

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
  int B, C, Hq, Hkv, G, HG, n_groups, tiles, CW, PW, stages, num_ctas;
  int by_request;  // records are numbered by request and group (there are at most num_ctas), else by CTA
  int window, sinks, max_context;
  float scale_log2, gv;
  int4* merge;    // records of cut requests: request and group (-1: none), CTA and slot of the first piece, last CTA
  float* part_ml; // [2 * num_ctas][HG * C * G][2]
  float* part_o;  // [2 * num_ctas][HG * C * G][128]
  int32_t* err;
};

struct __align__(16) Hdr {
  int flags;   // 1 first stage of the piece, 2 last, 4 masks needed, 8 and 16: the groups' rows lie token by token
  int valid;   // bit j: position t0 + j is in the span and its row is here
  int t0;      // first position of the stage
  int b, group, part, L, ql;
};

struct Smem {
  int code_group, scale_group, stage, pitch;
  unsigned char* stages;
  unsigned char* queries;  // [warp][nt][4][lane] 16 bytes: each warp's queries as operand B, two k steps of it a word
  Hdr* hdr;  // [stages]
  uint64_t* full;
  uint64_t* empty;
  volatile int* abort_flag;
};

// Bytes of a group's codes: swizzled [head][token][128], or by rows at a pitch that spreads them over the banks.
__host__ __device__ __forceinline__ int code_group_bytes(int HG) { return (16 * (HG * kHeadBytes + 16) + 1023) & ~1023; }
__host__ __device__ __forceinline__ int stage_bytes(int HG) {
  return (2 * (code_group_bytes(HG) + HG * 16 * kScaleBytes) + 1023) & ~1023;
}
constexpr int kQueryBytes = 2048;  // of a warp's eight columns
__host__ __forceinline__ size_t smem_bytes(int HG, int S, int CW, int NT) {
  return 1024 + (size_t)S * (stage_bytes(HG) + sizeof(Hdr) + 2 * sizeof(uint64_t)) + (size_t)CW * NT * kQueryBytes + 16;
}

__device__ __forceinline__ Smem map_smem(unsigned char* raw, int HG, int S, int CW, int NT) {
  Smem s;
  s.code_group = code_group_bytes(HG);
  s.scale_group = HG * 16 * kScaleBytes;
  s.stage = stage_bytes(HG);
  s.pitch = HG * kHeadBytes + 16;
  s.stages = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  s.queries = s.stages + (size_t)S * s.stage;
  s.hdr = reinterpret_cast<Hdr*>(s.queries + CW * NT * kQueryBytes);
  s.full = reinterpret_cast<uint64_t*>(s.hdr + S);
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same without a sum to begin with.
__device__ __forceinline__ void mma_f16_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// movmatrix_trans that the compiler may move.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// (a & mask) | (b & ~mask)
template <uint32_t MASK>
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xb8;" : "=r"(r) : "r"(b), "r"(MASK), "r"(a));
  return r;
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

// a / b of numbers that are not negative: in 32 bits where they fit, as they nearly always do (64 take a hundred
// instructions, and four of them lie one after another at every CTA's start).
__device__ __forceinline__ long long quotient_of(long long a, long long b) {
  if (((unsigned long long)(a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

// This CTA's share of the batch's stages, found by the whole CTA.
struct Plan {
  long long R0, R1, Sv;  // the share, and where its first request and group begin
  int active, b, g, ql;
  int4 cut;  // the record of that one if its last piece is here and it began before
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
  if (threadIdx.x == 0 && !a.by_request) a.merge[k] = make_int4(-1, 0, 0, 0);
  __syncthreads();
  if (k < Ne) {
    const long long R0 = quotient_of(k * T, Ne), R1 = quotient_of((k + 1) * T, Ne);
    if (at * a.n_groups <= R0 && R0 < (at + mine) * a.n_groups) {  // the first request is one of this thread's
      for (int b = b0; b < b1; ++b) {
        const Request r = request_of(a, b);
        const int n = r.n;
        const long long first = at * a.n_groups;
        if (R0 < first + (long long)n * a.n_groups) {
          const int g = a.n_groups == 1 ? 0 : (int)quotient_of(R0 - first, n);
          const long long Sv = first + (long long)g * n;
          pl->R0 = R0;
          pl->R1 = R1;
          pl->Sv = Sv;
          pl->b = b;
          pl->g = g;
          pl->active = 1;
          pl->ql = r.ql;
          pl->cut = make_int4(-1, 0, 0, 0);
          if (Sv < R0 && Sv + n <= R1) {  // cut, and its last piece is here
            const long long ka = quotient_of((Sv + 1) * Ne + T - 1, T) - 1;  // the CTA of its first piece
            pl->cut = make_int4(b * a.n_groups + g, (int)ka, (int)(quotient_of(ka * T, Ne) == Sv ? 2 * ka : 2 * ka + 1), (int)k);
            if (!a.by_request) a.merge[k] = pl->cut;
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
// The producers. They take the share's stages 32 at a time, a lane each: every lane finds its stage's request and group
// (from 32 requests' sizes and their sums), and in a block table whose pages are whole groups also the two slots that its
// copies start at, all while the 32 stages before are on their way. Issuing such a stage is then one lane's work: two
// tensor copies and two of scales. Of other tables each lane fetches one position's entry, a stage ahead, and copies that
// row where the group does not lie together. (Planning a stage at a time with the whole warp set the pace: 55 us for 64
// requests that take 47 now.)
// ---------------------------------------------------------------------------
struct Lane {   // a stage, in one lane's registers
  Hdr h;
  int row;      // of the table
  int e0, e1;   // table entries of its two groups (block tables of whole groups)
};

// Stages x0 .. x0 + 31 of the stream, lane by lane; (b, g, Sv) is the request and group of x0 or an earlier one, and
// becomes that of stage x0 + 31 or the last. ``n``: the share's stages from x0 on.
__device__ __forceinline__ void prepare(const Args& a, const Plan& pl, long long x0, int n, int& b, int& g, long long& Sv,
                                        bool paged, int shift, int lane, Lane& o) {
  const int want = min(lane, n - 1);  // lanes past the end repeat the last stage
  bool found = false;
  int fb = 0, fg = 0;
  long long fS = 0;
  Request r;
  for (;;) {
    // requests b .. b + 31: their stages over all groups (of b, those from group g on), and the sums before them
    r = request_of(a, min(b + lane, a.B - 1));
    long long size = b + lane < a.B ? (long long)r.n * (lane ? a.n_groups : a.n_groups - g) : 0, sum = size;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += y;
    }
    const long long target = x0 + want - Sv;  // from the first one's start
    int i = 0;
    for (; i < 32; ++i) {
      const long long end = __shfl_sync(0xffffffffu, sum, i);
      if (!found && target < end) {
        found = true;
        fb = b + i;
        fS = Sv + end;  // its end, for now
      }
      if (__all_sync(0xffffffffu, found)) break;
    }
    if (__all_sync(0xffffffffu, found)) break;
    const long long all = __shfl_sync(0xffffffffu, sum, 31);
    Sv += all;
    b += 32;
    g = 0;
    if (b >= a.B) break;  // cannot happen within the share
  }
  r = request_of(a, fb);
  const long long x = x0 + want;
  const int back = a.n_groups == 1 ? 0 : (int)quotient_of(max(fS - x - 1, 0ll), max(r.n, 1));  // groups after this stage's: fS is the end of all
  fg = a.n_groups - 1 - back;
  fS -= (long long)(back + 1) * r.n;                   // this group's first stage
  const int i = (int)(x - fS);
  const bool sink = i < r.n_sink;
  const int t0 = (sink ? i : r.lo / kTok + i - r.n_sink) * kTok;
  const int first = max((sink ? 0 : r.lo) - t0, 0), end = min((sink ? r.se : r.L) - t0, kTok);  // positions t0 + first ..
  const unsigned inside = !found ? 0u : (end >= 32 ? 0xffffffffu : (1u << end) - 1u) & ~((1u << first) - 1u);
  // every query attends the whole stage: it ends before the first query's position, and lies in the last one's window or
  // in the first one's sinks
  const int p0 = r.L - r.ql;
  const Span sl = attend_span(r.L, a.window, a.sinks), sf = attend_span(p0 + 1, a.window, a.sinks);
  const bool whole = inside == 0xffffffffu && t0 + kTok - 1 <= p0 && (t0 >= sl.lo || t0 + kTok <= sf.se);
  const bool cut = fS < pl.R0 || fS + r.n > pl.R1;
  o.h.flags = (x == max(fS, pl.R0) ? 1 : 0) | (x + 1 == min(fS + r.n, pl.R1) ? 2 : 0) | (whole ? 0 : 4);
  o.h.valid = (int)inside;
  o.h.t0 = t0;
  o.h.b = fb;
  o.h.group = fg;
  o.h.part = cut ? (fS <= pl.R0 ? 2 * (int)blockIdx.x : 2 * (int)blockIdx.x + 1) : -1;
  o.h.L = r.L;
  o.h.ql = r.ql;
  o.row = r.row;
  if (a.by_request && found && lane < n && x + 1 == fS + r.n)  // the request's last stage: its record is this CTA's to write
    a.merge[fb * a.n_groups + fg] = fS < pl.R0 ? pl.cut : make_int4(-1, 0, 0, 0);
  o.e0 = o.e1 = -1;
  if (paged) {
    const int32_t* row = a.T.table + (size_t)r.row * a.T.cols;
    if (inside & 0xffffu) o.e0 = __ldg(row + (shift >= 0 ? t0 >> shift : t0 / a.T.page_size));
    if (inside >> 16) o.e1 = __ldg(row + (shift >= 0 ? (t0 + 16) >> shift : (t0 + 16) / a.T.page_size));
  }
  b = __shfl_sync(0xffffffffu, fb, 31);
  g = __shfl_sync(0xffffffffu, fg, 31);
  Sv = __shfl_sync(0xffffffffu, fS, 31);
}

// A stage's copies by the whole warp, rows that lie together by groups, others one by one; ``e``: the lane's table entry.
__device__ __forceinline__ void load_rows(const Args& a, const Smem& s, Hdr h, int e, int st, int shift, int lane) {
  const int HG = a.HG, P = a.T.page_size;
  const uint32_t row_copy = (uint32_t)(HG * kHeadBytes);
  const int t = h.t0 + lane, grp = lane >> 4, j = lane & 15;
  int slot = -1;
  if (h.valid >> lane & 1) {
    const bool good = a.T.raw ? (unsigned)e < (unsigned)a.T.num_slots : (unsigned)e < (unsigned)a.T.num_pages;
    if (good) slot = a.T.raw ? e : e * P + (shift >= 0 ? t & (P - 1) : t % P);
    else set_error(a.err, KVP_ERR_BAD_INDEX);
  }
  const unsigned here = __ballot_sync(0xffffffffu, slot >= 0);
  const unsigned mine = here >> (16 * grp) & 0xffffu;
  const int lead = mine ? __ffs(mine) - 1 : 0;
  const int base = __shfl_sync(0xffffffffu, slot, 16 * grp + lead) - lead;
  const unsigned off = __ballot_sync(0xffffffffu, slot >= 0 && slot - j != base);
  const bool together = a.use_map && mine && (base & 15) == 0 && base >= 0 && (off >> (16 * grp) & 0xffffu) == 0;
  const unsigned tg = __ballot_sync(0xffffffffu, together), lin = __ballot_sync(0xffffffffu, mine && !together);
  unsigned char* sbuf = s.stages + (size_t)st * s.stage;
  unsigned char* scb = sbuf + 2 * s.code_group;
  uint64_t* full = &s.full[st];
  if (lane == 0) {
    h.valid = (int)here;
    h.flags |= (lin & 1 ? 8 : 0) | (lin >> 16 & 1 ? 16 : 0) | (here != 0xffffffffu ? 4 : 0);
    s.hdr[st] = h;
    mbar_arrive_expect_tx(full, ((tg & 1) + (tg >> 16 & 1)) * (uint32_t)(HG * 16 * (kHeadBytes + kScaleBytes)) +
                                    (uint32_t)__popc(here & lin) * row_copy);
  }
  __syncwarp();
  if (together && j == 0) {  // lanes 0 and 16
    fence_proxy_async_smem();  // the buffer's scales may have come by cp.async before, and these are another proxy's writes
    tma_load_4d(sbuf + grp * s.code_group, &a.map, 0, base, h.group * HG, a.layer, full);
    bulk_g2s(scb + grp * s.scale_group, a.scales + fp4_scale_offset(base, h.group * HG, a.Hkv, kD), (uint32_t)s.scale_group,
             full);
  }
  if (lin) {
    if ((lin >> lane & 1) && slot >= 0) {
      bulk_g2s(sbuf + grp * s.code_group + j * s.pitch, a.codes + (size_t)slot * a.row_bytes + (size_t)h.group * row_copy,
               row_copy, full);
      const char* src = a.scales + fp4_scale_offset(slot, h.group * HG, a.Hkv, kD);
      unsigned char* dst = scb + grp * s.scale_group + j * kScaleBytes;
      for (int hh = 0; hh < HG; ++hh) cp_async16(dst + hh * 16 * kScaleBytes, src + hh * 16 * kScaleBytes);
    }
    cp_async_arrive(full);
  } else if (lane == 0) {
    mbar_arrive_n(full, 32);
  }
}

// The copies of a stage of whole groups, by one lane.
__device__ __forceinline__ void load_groups(const Args& a, const Smem& s, Lane& o, int st, int shift) {
  const int HG = a.HG, P = a.T.page_size;
  const uint32_t codes = (uint32_t)(HG * 16 * kHeadBytes);
  int base[2] = {-1, -1};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = i ? o.e1 : o.e0, t = o.h.t0 + 16 * i;
    if (!(o.h.valid >> (16 * i) & 0xffff)) continue;
    if ((unsigned)e < (unsigned)a.T.num_pages) {
      base[i] = e * P + (shift >= 0 ? t & (P - 1) : t % P);
    } else {
      set_error(a.err, KVP_ERR_BAD_INDEX);
      o.h.valid &= i ? 0xffff : (int)0xffff0000u;
      o.h.flags |= 4;
    }
  }
  uint64_t* full = &s.full[st];
  s.hdr[st] = o.h;
  mbar_arrive_expect_tx(full, ((base[0] >= 0) + (base[1] >= 0)) * (codes + (uint32_t)s.scale_group));
  unsigned char* sbuf = s.stages + (size_t)st * s.stage;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (base[i] >= 0) {
      tma_load_4d(sbuf + i * s.code_group, &a.map, 0, base[i], o.h.group * HG, a.layer, full);
      bulk_g2s(sbuf + 2 * s.code_group + i * s.scale_group, a.scales + fp4_scale_offset(base[i], o.h.group * HG, a.Hkv, kD),
               (uint32_t)s.scale_group, full);
    }
  mbar_arrive_n(full, 32);
}

__device__ __forceinline__ Hdr from_lane(const Hdr& h, int j) {
  Hdr o;
  o.flags = __shfl_sync(0xffffffffu, h.flags, j);
  o.valid = __shfl_sync(0xffffffffu, h.valid, j);
  o.t0 = __shfl_sync(0xffffffffu, h.t0, j);
  o.b = __shfl_sync(0xffffffffu, h.b, j);
  o.group = __shfl_sync(0xffffffffu, h.group, j);
  o.part = __shfl_sync(0xffffffffu, h.part, j);
  o.L = __shfl_sync(0xffffffffu, h.L, j);
  o.ql = __shfl_sync(0xffffffffu, h.ql, j);
  return o;
}

__device__ void produce(const Args& a, const Smem& s, const Plan& pl, int me, int lane) {
  const int S = a.stages, P = a.T.page_size;
  const int shift = (P & (P - 1)) == 0 ? __ffs(P) - 1 : -1;
  const bool paged = a.use_map && !a.T.raw && (P & 15) == 0;
  if (paged && me) return;
  const int PW = paged ? 1 : a.PW;  // each has every PW-th stage
  int b = pl.b, g = pl.g;
  long long Sv = pl.Sv, x = pl.R0;
  Lane cur, nxt;
  prepare(a, pl, x, (int)min(pl.R1 - x, (long long)32), b, g, Sv, paged, shift, lane, cur);
  bool ok = true;
  int st = me % S, phase = 1 ^ (me / S & 1), k = me;  // stage k goes to buffer st; a buffer's first wait passes at once
  int e = 0;
  auto fetch = [&](const Hdr& h, int row) {  // the lane's table entry of a stage
    if (!(h.valid >> lane & 1)) return 0;
    const int t = h.t0 + lane;
    return __ldg(a.T.table + (size_t)row * a.T.cols + (a.T.raw ? t : shift >= 0 ? t >> shift : t / P));
  };
  if (!paged && me < pl.R1 - pl.R0) e = fetch(from_lane(cur.h, me), __shfl_sync(0xffffffffu, cur.row, me));
  while (ok) {
    const int n = (int)min(pl.R1 - x, (long long)32);
    const bool more = pl.R1 - x > 32;
    if (more) prepare(a, pl, x + 32, (int)min(pl.R1 - x - 32, (long long)32), b, g, Sv, paged, shift, lane, nxt);
    for (int j = me; j < n && ok; j += PW) {  // PW divides 32
      if (paged) {
        if (lane == j) {
          ok = mbar_wait_bounded(&s.empty[st], (uint32_t)phase, s.abort_flag, a.err, kWaitNs);
          if (ok) load_groups(a, s, cur, st, shift);
        }
        ok = __all_sync(0xffffffffu, ok);
      } else {
        const Hdr h = from_lane(cur.h, j);
        const int mine = e;
        if (j + PW < n) e = fetch(from_lane(cur.h, j + PW), __shfl_sync(0xffffffffu, cur.row, j + PW));
        else if (more && me < pl.R1 - x - 32) e = fetch(from_lane(nxt.h, me), __shfl_sync(0xffffffffu, nxt.row, me));
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s.empty[st], (uint32_t)phase, s.abort_flag, a.err, kWaitNs));
        if (ok) load_rows(a, s, h, mine, st, shift, lane);
      }
      if (!ok) break;
      k += PW;
      for (st += PW; st >= S; st -= S) phase ^= 1;
    }
    x += 32;
    if (!more) break;
    cur = nxt;
  }
  if (!ok) *s.abort_flag = 1;
  // The copies land (bounded) before the CTA ends, also when all of them went out: a consumer may give up and leave later. The
  // last ones of each buffer; older ones' buffers were filled again.
  const long long from = ok ? pl.R1 - pl.R0 - S : (long long)k - PW - S + 1;
  const uint64_t start = global_timer_ns();
  for (int k2 = k - PW; k2 >= 0 && k2 >= from; k2 -= PW)
    while (!mbar_try_wait(&s.full[k2 % S], (uint32_t)(k2 / S & 1)))
      if (global_timer_ns() - start > 2 * kWaitNs) return;
}

// ---------------------------------------------------------------------------
// Consumer warps: one KV head and 8 NT (token, head) columns each.
// ---------------------------------------------------------------------------

// Whether the query token of column ``col`` attends position t (the stage's masks allow for rows that are not there).
struct Column {
  int p, lo, se;
};
__device__ __forceinline__ Column column_of(const Args& a, const Hdr* h, int col) {
  Column q;
  q.p = h->L - h->ql + min(col, a.C * a.G - 1) / a.G;
  const Span sp = attend_span(q.p + 1, a.window, a.sinks);
  q.lo = sp.lo;
  q.se = sp.se;
  return q;
}
__device__ __forceinline__ bool attends(const Column& q, int t) { return t <= q.p && (t >= q.lo || t < q.se); }

// What a warp keeps from stage to stage.
template <int NT>
struct State {
  float o[8][NT][4];                  // O^T
  // of its columns: the reference (log2: the running maximum less 7, 8 further behind at most), this lane's part of the sum
  // of weights 2^(score - reference), the score's factor
  float m[NT][2], l[NT][2], f[NT][2];
};

// Where a lane's K and V of the first tile lie: rows of 128 bytes, head-major and swizzled (chunk ^ token % 8), or token by
// token. A tile's tokens 8 to 15 lie ``eight`` further.
struct Place {
  uint32_t k, v0, v1, eight;
};

// What a lane knows of its part in every stage.
struct Part {
  Place swz, lin;
  uint32_t ksc, vsc;       // its scales in a group's
  uint32_t queries;        // its operand words
  int col, ktok, vt0, vt1; // its first column, its row's token, its tokens of k 2 c and 2 c + 1
};

// A stage that is being worked on.
struct Stage {
  const Hdr* hd;
  uint32_t flags, valid, sb;
  int t0;
};

// The phases of a stage. LIN: 0 both groups swizzled, 1 both token by token, 2 as the flags say; MASKED: the flags' masks
// count.
template <int NT, int LIN>
__device__ __forceinline__ void scores(const Smem& s, const Stage& g, const Part& p, float (&x)[2][NT][4]) {
  // S^T = K Q^T, two tiles of 16 tokens
#pragma unroll
  for (int tile = 0; tile < 2; ++tile) {
    const bool by_row = LIN == 1 || (LIN == 2 && (g.flags & (8 << tile)));
    const uint32_t ab = g.sb + tile * s.code_group + (by_row ? p.lin.k : p.swz.k);
    const uint32_t scb = g.sb + 2 * s.code_group + tile * s.scale_group + p.ksc;
    const uint4 r0 = lds16(ab), r1 = lds16(ab + (by_row ? p.lin.eight : 1024));
    const uint32_t s0 = e4m3x2_to_half(lds_u16(scb)), s1 = e4m3x2_to_half(lds_u16(scb + 8 * kScaleBytes));
    const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t d0 = __byte_perm(s0, s0, i < 2 ? 0x1010 : 0x3232), d1 = __byte_perm(s1, s1, i < 2 ? 0x1010 : 0x3232);
      uint32_t h0[4], h1[4];
      e2m1x8_to_half(w0[i], h0);
      e2m1x8_to_half(w1[i], h1);
      // read again for every tile: sixteen registers less, and no spills at 96
      uint4 q[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) q[nt] = lds16(p.queries + nt * kQueryBytes + i * 512);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t af[4] = {hmul2(h0[2 * y], d0), hmul2(h1[2 * y], d1), hmul2(h0[2 * y + 1], d0), hmul2(h1[2 * y + 1], d1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (i == 0 && y == 0) mma_f16_new(x[tile][nt], af, q[nt].x, q[nt].y);
          else mma_f16(x[tile][nt], af, y ? q[nt].z : q[nt].x, y ? q[nt].w : q[nt].y);
        }
      }
    }
  }
}

template <int NT, bool MASKED>
__device__ __forceinline__ void weights(const Args& a, const Stage& g, const Part& p, float (&x)[2][NT][4],
                                        uint32_t (&pb)[2][NT][2], State<NT>& z) {
  // softmax over the 32 tokens: rows g and g + 8 of each tile
  if (MASKED) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const Column q = column_of(a, g.hd, p.col + nt * 8 + e);
#pragma unroll
        for (int tile = 0; tile < 2; ++tile)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int jt = tile * 16 + y * 8 + p.ktok;
            if (!((g.valid >> jt & 1) && attends(q, g.t0 + jt))) x[tile][nt][2 * y + e] = -INFINITY;
          }
      }
  }
  constexpr float kBelow = 7.f, kMost = 15.f;
  float mx[NT][2];
  bool grow = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = fmaxf(fmaxf(x[0][nt][e], x[0][nt][2 + e]), fmaxf(x[1][nt][e], x[1][nt][2 + e]));
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, sh));
      mx[nt][e] = fminf(__fmul_rn(v, z.f[nt][e]), 3.0e38f);  // finite: a product beyond it gives an infinite weight, and a NaN
      grow |= mx[nt][e] - z.m[nt][e] > kMost;  // the difference is exact where scores are large; a sum is not
    }
  if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(z.m[nt][e], mx[nt][e] - kBelow);
        const float al = z.m[nt][e] == -INFINITY ? 0.f : ex2(z.m[nt][e] - mn);
        z.m[nt][e] = mn;
        z.l[nt][e] *= al;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          z.o[i][nt][e] *= al;
          z.o[i][nt][2 + e] *= al;
        }
      }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    // the product rounded before the difference, as in the maximum: one rounding of both would leave 2^-24 of a score,
    // more than all of an exponent where scores are large
    const float m0 = fmaxf(z.m[nt][0], -3.0e38f), m1 = fmaxf(z.m[nt][1], -3.0e38f);  // nothing attended: 2^-inf, not NaN
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const float p0 = ex2(__fmul_rn(x[tile][nt][0], z.f[nt][0]) - m0), p1 = ex2(__fmul_rn(x[tile][nt][1], z.f[nt][1]) - m1),
                  p2 = ex2(__fmul_rn(x[tile][nt][2], z.f[nt][0]) - m0), p3 = ex2(__fmul_rn(x[tile][nt][3], z.f[nt][1]) - m1);
      z.l[nt][0] += p0 + p2;
      z.l[nt][1] += p1 + p3;
      pb[tile][nt][0] = transposed(pack_half(p0, p1));
      pb[tile][nt][1] = transposed(pack_half(p2, p3));
    }
  }
}

template <int NT, int LIN, bool MASKED>
__device__ __forceinline__ void values(const Args& a, const Smem& s, const Stage& g, const Part& p,
                                       const uint32_t (&pb)[2][NT][2], State<NT>& z) {
  // O^T += V^T P^T. Codes of two tokens are put side by side in a byte, so that a conversion gives the pair that a fragment
  // holds.
#pragma unroll
  for (int tile = 0; tile < 2; ++tile) {
    const bool by_row = LIN == 1 || (LIN == 2 && (g.flags & (8 << tile)));
    const uint32_t cb = g.sb + tile * s.code_group, eight = by_row ? p.lin.eight : 1024;
    const uint32_t a0 = cb + (by_row ? p.lin.v0 : p.swz.v0), a1 = cb + (by_row ? p.lin.v1 : p.swz.v1);
    const uint32_t scb = g.sb + 2 * s.code_group + tile * s.scale_group + p.vsc, one = (uint32_t)((p.vt1 - p.vt0) * kScaleBytes);
    const uint2 r[4] = {lds8(a0), lds8(a1), lds8(a0 + eight), lds8(a1 + eight)};
    uint32_t sc0 = lds_u8(scb) + 256u * lds_u8(scb + one),
             sc1 = lds_u8(scb + 8 * kScaleBytes) + 256u * lds_u8(scb + one + 8 * kScaleBytes);
    if (MASKED) {  // rows that are not there count zero times
      const unsigned vm = g.valid >> (16 * tile);
      if (!(vm >> p.vt0 & 1)) sc0 &= 0xff00u;
      if (!(vm >> p.vt1 & 1)) sc0 &= 0xffu;
      if (!(vm >> (p.vt0 + 8) & 1)) sc1 &= 0xff00u;
      if (!(vm >> (p.vt1 + 8) & 1)) sc1 &= 0xffu;
      const uint32_t two = sc0 | sc1 << 16;
      uint32_t who = 0;  // tokens whose block g is NaN; their scale is zero from here on
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (fp4_is_nan(two >> (8 * y))) {
          who |= 1u << ((y & 1 ? p.vt1 : p.vt0) + (y & 2 ? 8 : 0));
          if (y < 2) sc0 &= y ? 0xffu : 0xff00u;
          else sc1 &= y & 1 ? 0xffu : 0xff00u;
        }
      if (__any_sync(0xffffffffu, who != 0)) {
        who |= __shfl_xor_sync(0xffffffffu, who, 1);
        who |= __shfl_xor_sync(0xffffffffu, who, 2);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const Column q = column_of(a, g.hd, p.col + nt * 8 + e);
            bool hit = false;
            for (int jt = 0; jt < 16; ++jt) hit |= (who >> jt & 1) && attends(q, g.t0 + 16 * tile + jt);
            if (hit)
#pragma unroll
              for (int i = 0; i < 8; ++i) z.o[i][nt][e] = z.o[i][nt][2 + e] = __int_as_float(0x7fffffff);
          }
      }
    }
    const uint32_t d0 = e4m3x2_to_half(sc0), d1 = e4m3x2_to_half(sc1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t y0 = i ? r[0].y : r[0].x, y1 = i ? r[1].y : r[1].x, y2 = i ? r[2].y : r[2].x, y3 = i ? r[3].y : r[3].x;
      constexpr uint32_t kLow = 0x0f0f0f0fu;
      uint32_t e0[4], o0[4], e1[4], o1[4];  // even and odd entries of tokens 2 c, 2 c + 1 and of 2 c + 8, 2 c + 9
      e2m1x8_to_half(select_bits<kLow>(y0, y1 << 4), e0);
      e2m1x8_to_half(select_bits<kLow>(y0 >> 4, y1), o0);
      e2m1x8_to_half(select_bits<kLow>(y2, y3 << 4), e1);
      e2m1x8_to_half(select_bits<kLow>(y2 >> 4, y3), o1);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t af[4] = {hmul2(e0[u], d0), hmul2(o0[u], d0), hmul2(e1[u], d1), hmul2(o1[u], d1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(z.o[4 * i + u][nt], af, pb[tile][nt][0], pb[tile][nt][1]);
      }
    }
  }
}

// A new piece's queries, on their way: entries 32 c .. 32 c + 31 of column g of each eight.
template <int NT>
struct Queries {
  uint4 x[NT][4];
};
template <int NT>
__device__ __forceinline__ void fetch_queries(const Args& a, int b, int grp, int ql, int h, int col0, int lane, Queries<NT>& q) {
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = col0 + nt * 8 + g, cj = a.C == 1 ? 0 : col / a.G;
#pragma unroll
    for (int i = 0; i < 4; ++i) q.x[nt][i] = make_uint4(0u, 0u, 0u, 0u);
    if (col < a.C * a.G && cj < ql) {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (((size_t)b * a.C + cj) * a.Hq + (size_t)(grp * a.HG + h) * a.G + col - cj * a.G) * kD + 32 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) q.x[nt][i] = __ldg(src + i);
    }
  }
}

// They turn to fp16, scaled by powers of two; nothing is attended yet.
template <int NT>
__device__ __forceinline__ void begin(const Args& a, const Queries<NT>& q, unsigned char* queries, int lane, State<NT>& z) {
  const int c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      for (const uint32_t v : {q.x[nt][i].x, q.x[nt][i].y, q.x[nt][i].z, q.x[nt][i].w})
        mx = max(mx, max(v << 16 & 0x7fff0000u, v & 0x7fff0000u));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // 2^e <= the largest < 2^(e + 1); zeros and subnormal rows: the smallest normal exponent; not finite: as it is
    const int e = mx >= kInfBits ? 0 : max((int)(mx >> 23), 1) - 127;
    // the sign of the scale goes to the queries: f is positive, and the largest score has the largest product
    const float down = (e == 127 ? 0x1p-127f : __uint_as_float((uint32_t)(127 - e) << 23)) * (a.scale_log2 < 0.f ? -1.f : 1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v[4] = {q.x[nt][i].x, q.x[nt][i].y, q.x[nt][i].z, q.x[nt][i].w};
      uint32_t y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) y[u] = pack_half(bf16_lo(v[u]) * down, bf16_hi(v[u]) * down);
      reinterpret_cast<uint4*>(queries + nt * kQueryBytes)[i * 32 + lane] = make_uint4(y[0], y[1], y[2], y[3]);  // its own lane's
    }
#pragma unroll
    for (int x2 = 0; x2 < 2; ++x2) {
      const int ec = __shfl_sync(0xffffffffu, e, (2 * c + x2) * 4);
      const float up = ec == -126 ? 0x1p-126f : __uint_as_float((uint32_t)(127 + ec) << 23);
      // not zero, as masked products are -inf, and finite
      z.f[nt][x2] = fminf(fmaxf(fabsf(a.scale_log2) * up, 1e-37f), 3.0e38f);
      z.m[nt][x2] = -INFINITY;
      z.l[nt][x2] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z.o[i][nt][0] = z.o[i][nt][1] = z.o[i][nt][2] = z.o[i][nt][3] = 0.f;
  }
}

// The piece's end: entries 16 g .. 16 g + 15 of columns 2 c and 2 c + 1, the result or a partial one.
template <int NT>
__device__ __forceinline__ void finish(const Args& a, const Hdr* hd, int h, int col0, int lane, const State<NT>& z) {
  const int g = lane >> 2, c = lane & 3, C = a.C * a.G, part = hd->part, ql = hd->ql;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float ls = z.l[nt][e];
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, sh);
      const int col = col0 + nt * 8 + 2 * c + e, cj = a.C == 1 ? 0 : col / a.G;
      if (col >= C || cj >= ql) continue;
      float v[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[2 * i] = z.o[i][nt][e];
        v[2 * i + 1] = z.o[i][nt][2 + e];
      }
      if (part < 0) {
        const float inv = ls == 0.f ? 0.f : a.gv / ls;
        uint4* dst = reinterpret_cast<uint4*>(
            a.out + (((size_t)hd->b * a.C + cj) * a.Hq + (size_t)(hd->group * a.HG + h) * a.G + col - cj * a.G) * kD + 16 * g);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          dst[i] = make_uint4(pack_bf16(v[8 * i] * inv, v[8 * i + 1] * inv), pack_bf16(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                              pack_bf16(v[8 * i + 4] * inv, v[8 * i + 5] * inv),
                              pack_bf16(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
      } else {
        const size_t at = (size_t)part * a.HG * C + (size_t)h * C + col;
        float4* dst = reinterpret_cast<float4*>(a.part_o + at * kD + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if (g == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(z.m[nt][e], ls);
      }
    }
}

template <int NT>
__device__ void consume(const Args& a, const Smem& s, const Plan& pl, int w, int lane) {
  const int h = w / a.tiles, col0 = (w % a.tiles) * 8 * NT;
  const int g = lane >> 2, c = lane & 3;
  const int vchunk = 4 + (g >> 1), vin = (g & 1) * 8;
  auto swz = [&](int tok, int chunk) { return (uint32_t)((h * 16 + tok) * 128 + ((chunk ^ (tok & 7)) << 4)); };
  auto row = [&](int tok, int chunk) { return (uint32_t)(tok * s.pitch + h * kHeadBytes + chunk * 16); };
  unsigned char* queries = s.queries + (size_t)w * NT * kQueryBytes;
  Part p;
  p.col = col0 + 2 * c;
  p.ktok = g & 1 ? g ^ 4 : g;     // the token of row g; row g + 8: 8 further
  p.vt0 = 2 * c;                  // the tokens of k 2 c and 2 c + 1, and 8 further
  p.vt1 = (2 * c + 1) ^ 4;
  p.swz = {swz(p.ktok, c), swz(p.vt0, vchunk) + vin, swz(p.vt1, vchunk) + vin, 1024u};
  p.lin = {row(p.ktok, c), row(p.vt0, vchunk) + vin, row(p.vt1, vchunk) + vin, 8u * s.pitch};
  p.ksc = (uint32_t)((h * 16 + p.ktok) * kScaleBytes + 2 * c);
  p.vsc = (uint32_t)((h * 16 + p.vt0) * kScaleBytes + 8 + g);
  p.queries = smem_u32(queries) + 16 * lane;
  const uint32_t stages = smem_u32(s.stages);
  State<NT> z;
  Queries<NT> q;
  fetch_queries<NT>(a, pl.b, pl.g, pl.ql, h, col0, lane, q);  // the first piece's, while its rows are on their way
  begin<NT>(a, q, queries, lane, z);

  int st = 0, phase = 0;  // the buffer of the next stage to wait for, and that wait's parity
  auto next = [&](Stage& o) {
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s.full[st], (uint32_t)phase, s.abort_flag, a.err, kWaitNs))) return false;
    o.hd = &s.hdr[st];
    const uint4 head = lds16(smem_u32(o.hd));  // flags, valid, t0, request
    o.flags = head.x;
    o.valid = head.y;
    o.t0 = (int)head.z;
    o.sb = stages + (uint32_t)st * (uint32_t)s.stage;
    if (++st == a.stages) {
      st = 0;
      phase ^= 1;
    }
    return true;
  };
  auto release = [&](const Stage& o) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.empty[(int)(o.hd - s.hdr)]);
  };
  long long left = pl.R1 - pl.R0;
  Stage cur;
  if (!next(cur)) return;
  for (;;) {
    // plain stages of a piece, all swizzled or all token by token: the next one's scores beside this one's values, two
    // streams of instructions that wait for each other only through the weights
    float x[2][NT][4];
    uint32_t pb[2][NT][2];
    const uint32_t kind = cur.flags & 28;
    Stage ahead;
    if (kind == 0) {
      scores<NT, 0>(s, cur, p, x);
      for (;;) {
        weights<NT, false>(a, cur, p, x, pb, z);
        if ((cur.flags & 2) && left == 1) break;
        if (!next(ahead)) return;
        if ((cur.flags & 2) || (ahead.flags & 28)) break;
        scores<NT, 0>(s, ahead, p, x);
        values<NT, 0, false>(a, s, cur, p, pb, z);
        release(cur);
        cur = ahead;
        --left;
      }
      if (NT == 1 && (ahead.flags & 1) && left > 1) fetch_queries<NT>(a, ahead.hd->b, ahead.hd->group, ahead.hd->ql, h, col0, lane, q);
      values<NT, 0, false>(a, s, cur, p, pb, z);
    } else if (kind == 24) {
      scores<NT, 1>(s, cur, p, x);
      for (;;) {
        weights<NT, false>(a, cur, p, x, pb, z);
        if ((cur.flags & 2) && left == 1) break;
        if (!next(ahead)) return;
        if ((cur.flags & 2) || (ahead.flags & 28) != 24) break;
        scores<NT, 1>(s, ahead, p, x);
        values<NT, 1, false>(a, s, cur, p, pb, z);
        release(cur);
        cur = ahead;
        --left;
      }
      if (NT == 1 && (ahead.flags & 1) && left > 1) fetch_queries<NT>(a, ahead.hd->b, ahead.hd->group, ahead.hd->ql, h, col0, lane, q);
      values<NT, 1, false>(a, s, cur, p, pb, z);
    } else {
      scores<NT, 2>(s, cur, p, x);
      weights<NT, true>(a, cur, p, x, pb, z);
      if (left > 1 && !next(ahead)) return;
      if (NT == 1 && (ahead.flags & 1) && left > 1) fetch_queries<NT>(a, ahead.hd->b, ahead.hd->group, ahead.hd->ql, h, col0, lane, q);
      values<NT, 2, true>(a, s, cur, p, pb, z);
    }
    const bool last = cur.flags & 2;
    if (last) finish<NT>(a, cur.hd, h, col0, lane, z);
    release(cur);
    if (--left == 0) return;
    if (last) {
      if (NT > 1) fetch_queries<NT>(a, ahead.hd->b, ahead.hd->group, ahead.hd->ql, h, col0, lane, q);
      begin<NT>(a, q, queries, lane, z);
    }
    cur = ahead;
  }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) fp4_decode_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) unsigned char raw[];
  __shared__ Plan pl;
  const Smem s = map_smem(raw, a.HG, a.stages, a.CW, NT);
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
      if (a.by_request)
        for (int i = threadIdx.x; i < a.n_groups; i += blockDim.x) a.merge[b * a.n_groups + i] = make_int4(-1, 0, 0, 0);
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)b * a.C * a.Hq * kD);
      for (int i = threadIdx.x; i < a.C * a.Hq * (kD / 8); i += blockDim.x) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (!pl.active) return;
  if (warp >= a.CW) produce(a, s, pl, warp - a.CW, lane);
  else consume<NT>(a, s, pl, warp, lane);
}

// Joins the pieces of a cut request, in CTA order, six loads on their way at a time: a warp a column, or, of more pieces, a
// block a column, its four warps a quarter of the pieces each, then the quarters in order.
constexpr int kJoin = 6;
struct Joined {
  float4 o;
  float m, l;
};
__device__ __forceinline__ void join(Joined& j, float m, float l, const float4& o) {
  const float w = ex2(m - j.m);
  j.l += w * l;
  j.o.x += w * o.x;
  j.o.y += w * o.y;
  j.o.z += w * o.z;
  j.o.w += w * o.w;
}
__device__ __forceinline__ void raise(Joined& j, float m) {
  const float al = ex2(j.m - m);
  j.m = m;
  j.l *= al;
  j.o = make_float4(j.o.x * al, j.o.y * al, j.o.z * al, j.o.w * al);
}
__global__ void __launch_bounds__(128, 8) fp4_combine_kernel(const __grid_constant__ Args a) {
  __shared__ float4 sum[4][32];
  __shared__ float2 weight[4];  // a quarter's maximum and sum
  griddep_wait();
  const int4 mg = a.merge[blockIdx.x];
  if (mg.x < 0) return;
  const int b = mg.x / a.n_groups, grp = mg.x % a.n_groups, C = a.C * a.G, cols = a.HG * C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ql = a.q_lens ? __ldg(a.q_lens + b) : a.C, pieces = 1 + mg.w - mg.y;
  const bool alone = pieces <= kJoin;  // a warp has a column's pieces
  const int per = alone ? pieces : (pieces + 3) / 4;
  const int i0 = alone ? 0 : min(pieces, warp * per), i1 = min(pieces, i0 + per), beside = alone ? 4 : 1;
  for (int u0 = blockIdx.y * beside; u0 < cols; u0 += gridDim.y * beside) {
    const int u = alone ? u0 + warp : u0;
    if (u >= cols) break;
    const int h = u / C, col = u - h * C, cj = a.C == 1 ? 0 : col / a.G;
    if (cj >= ql) continue;
    Joined j = {make_float4(0.f, 0.f, 0.f, 0.f), -3.0e38f, 0.f};
    for (int i = i0; i < i1; i += kJoin) {
      float2 ml[kJoin];
      float4 v[kJoin];
#pragma unroll
      for (int y = 0; y < kJoin; ++y) {
        ml[y] = make_float2(-INFINITY, 0.f);
        v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + y < i1) {
          const size_t at = (size_t)(i + y ? 2 * (mg.y + i + y) : mg.z) * cols + u;
          ml[y] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + at * 2));
          v[y] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * kD) + lane);
        }
      }
      float mn = j.m;
#pragma unroll
      for (int y = 0; y < kJoin; ++y) mn = fmaxf(mn, ml[y].x);
      raise(j, mn);
#pragma unroll
      for (int y = 0; y < kJoin; ++y) join(j, ml[y].x, ml[y].y, v[y]);
    }
    if (!alone) {
      sum[warp][lane] = j.o;
      if (lane == 0) weight[warp] = make_float2(j.m, j.l);
      __syncthreads();
      if (warp == 0) {
        raise(j, fmaxf(fmaxf(j.m, weight[1].x), fmaxf(weight[2].x, weight[3].x)));
#pragma unroll
        for (int i = 1; i < 4; ++i) join(j, weight[i].x, weight[i].y, sum[i][lane]);
      }
      __syncthreads();
    }
    if (alone || warp == 0) {
      const float inv = j.l == 0.f ? 0.f : a.gv / j.l;
      uint2* dst = reinterpret_cast<uint2*>(
          a.out + (((size_t)b * a.C + cj) * a.Hq + (size_t)(grp * a.HG + h) * a.G + col - cj * a.G) * kD) + lane;
      *dst = make_uint2(pack_bf16(j.o.x * inv, j.o.y * inv), pack_bf16(j.o.z * inv, j.o.w * inv));
    }
  }
}

// How the columns of a KV head go to warps, and the CTAs to an SM (one with eight heads; fewer heads make smaller CTAs).
struct Shape {
  int NT, tiles, HG, CW, PW, ctas_per_sm, stages;
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
  o->PW = o->CW > 4 ? 4 : o->CW > 2 ? 2 : 1;
  o->ctas_per_sm = kThreads / 32 / (o->CW + o->PW);  // twelve warps an SM, 168 registers a thread
  o->stages = kMaxStages;
  while (o->stages > 2 && smem_bytes(o->HG, o->stages, o->CW, o->NT) + kSmemRest > kSmemPerSm / o->ctas_per_sm) --o->stages;
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
  {
    static std::mutex encoding;  // host threads may call at once, with other shapes
    std::lock_guard<std::mutex> lock(encoding);
    int& state = pool->fp4_map_state[sh.HG - 1];
    if (state == 0) state = encode_map(pool, sh.HG, &pool->fp4_map[sh.HG - 1]) ? 1 : -1;
    a.use_map = state == 1;
    a.map = pool->fp4_map[sh.HG - 1];
  }
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
  a.PW = sh.PW;
  a.stages = sh.stages;
  a.num_ctas = pool->num_sms * sh.ctas_per_sm;
  a.by_request = (long long)c.B * a.n_groups <= a.num_ctas;
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
  // the most that a shape takes, whatever this one does: host threads may call at once, with other shapes
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kSmemPerSm - kSmemRest)) != cudaSuccess)
    return KVP_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_ctas);
  cfg.blockDim = dim3(32 * (sh.CW + sh.PW));
  cfg.dynamicSmemBytes = smem_bytes(sh.HG, sh.stages, sh.CW, sh.NT);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return KVP_ERR_CUDA;
  // a block a column, no more than run at once
  const int records = a.by_request ? c.B * a.n_groups : a.num_ctas;
  const int columns = sh.HG * a.C * a.G, most = 16 * pool->num_sms / records;
  cfg.gridDim = dim3(records, most < 1 ? 1 : most < columns ? most : columns);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fp4_combine_kernel, a) == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

}  // namespace kvp
