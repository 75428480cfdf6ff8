// Rotary positions of a step's queries and keys, and the write of the rotated
// keys (and of the values, or of the latents) to their slots of the paged
// cache, in one pass over the data.
//
// Mathematics. Pair i of a head's first ``rotary_dim`` entries is a complex
// number z; the token at position p gets z * attn * exp(i p theta_i). The pair
// is entries (i, i + rotary_dim / 2) in the half layout and (2 i, 2 i + 1) in
// the interleaved one. The angle p theta_i reaches 10^6 radians and more, where
// 32-bit floats are off by 0.03 rad and more, so it is kept as turns in 64-bit
// fixed point: f_i = theta_i / 2 pi mod 1 scaled by 2^64, p * f_i mod 2^64 is
// the exact fraction of a turn (the product wraps as turns do), for every int32
// position, negative ones too. The nearest quarter turn is taken off it in
// integers and put back by exchanging sine and cosine and their signs; what is
// left, pi / 4 at most, is rounded to float once, relative to itself, so that
// sines and cosines are good to two units in the last place near their zeros too
// (the whole fraction rounded to float was off by 2^-25 of half a turn: 1.3 times
// the fp32 store's error). One 64-bit multiplication replaces both double
// arithmetic and a table of angles.
//
// What bounds it: bytes. Each token is read and written once (q, k, v) and
// there are 3 flops per byte at most. A block takes 1 to 4 tokens: its threads
// compute the tokens' rotary_dim / 2 (cos, sin) pairs into shared memory once for
// all heads, then move 16-byte chunks: a unit is the two chunks of eight pairs in
// the half layout, one chunk of four in the interleaved one; a group of threads
// takes one head of one token, the groups stride over the tokens' heads. Loads run
// ahead of what they wait for: v and the first heads are on their way while
// positions, slots and sines are found, later heads two at a time.
// Measured (GPU time in a CUDA graph, bf16 unless said, 8 key heads): 64 tokens of 32
// heads 3.6 us; 8,192 of them 34.0 us (5.9 TB/s, 0.87 of a copy's rate); 65,537 of 64
// heads, half of each turned, 410 us (6.6 TB/s, 0.97); 3,001 fp32 tokens of 16 heads 8.1
// us; 16,461 latent rows with 32 heads' rotated parts 32.2 us (5.4 TB/s, 0.79). Positions
// of three axes: 64 tokens 3.7 us; 8,205 tokens of 32 heads 35.3 us (0.84).
//
// Four-bit pools (rotary_store_fp4) take the same pass; keys and values are rounded on
// the way (fp4.cuh) and leave 9 bytes for 32. Measured, queries of 32 heads included:
// 64 tokens 5.3 us (queries alone 2.5, as one launch with chains for both); 8,192 tokens
// 37 us (3.8 TB/s; queries 23.8, keys and values alone 25.2, of which bytes need 6.3); 30,011
// tokens of 64 heads, half of each turned, slot by slot, 231 us (158 and 82). Keys and values
// wait for this code's instructions (over two thirds of the issue slots), and not for the turn's:
// rows as they are take 23. What of them the rounding cannot do without has not been measured.
#include "fp4.cuh"

#include <cmath>

namespace kvp {

namespace {

constexpr int kRotThreads = 128;
constexpr int kRotMaxPairs = 512;  // (cos, sin) pairs a block holds: tokens * rotary_dim / 2
constexpr int kRotMaxTokens = 4;

struct RotArgs {
  const char* q;
  char* q_out;
  long long q_tok, q_head, qo_tok, qo_head;  // strides in bytes
  const char* k;
  long long k_tok;
  const char* v;  // copied as it is: the values, or the latents
  long long v_tok;
  char* k_dst;  // slot 0's first rotated key entry
  char* v_dst;  // slot 0's first copied entry
  size_t row_bytes;
  const int32_t* positions;
  const int32_t* out_loc;
  const uint64_t* freqs;
  int n, tokens, hq, hk, d, rot, v_elems, num_slots;
  float attn;
  int32_t* err;
  const uint8_t* pair_axis;  // positions of several axes: pair i's axis; axis x of token t at positions[x * pos_axis + t]
  long long pos_axis;
  int axes;
  char* scales;  // four-bit pools: the layer's block scales; k_dst and v_dst are codes
  float gk, gv;
  int kv_tokens, kv_blocks;  // tokens a block of keys and values takes, and how many such blocks there are
};

// The position by which pair i of token tok turns.
template <bool AXES>
__device__ __forceinline__ int position_of(const RotArgs& a, size_t tok, int i) {
  if (!AXES) return __ldg(a.positions + tok);
  int x = __ldg(a.pair_axis + i);
  if (x >= a.axes) {
    set_error(a.err, KVP_ERR_BAD_INDEX);
    x = 0;
  }
  return __ldg(a.positions + x * a.pos_axis + tok);
}

// (cos, sin) * attn of position p and the pair's frequency f (turns * 2^64).
__device__ __forceinline__ float2 turn_of(int p, uint64_t f, float attn) {
  const uint64_t t = (uint64_t)(int64_t)p * f;
  const uint32_t quarters = ((uint32_t)(t >> 32) + (1u << 29)) >> 30;
  // [-1/4, 1/4]: the rest's angle / pi, its bits down to 2^-34 of a turn (bits 30 to 61 with bit 61 as the sign: it is
  // the one that rounded ``quarters`` up)
  const float half_turns = (float)(int32_t)(uint32_t)(t >> 30) * 0x1p-33f;
  float s, c;
  sincospif(half_turns, &s, &c);
  const bool odd = quarters & 1;  // (c, s) -> (-s, c) a quarter
  const float x = odd ? s : c, y = odd ? c : s;
  return make_float2(((quarters + 1) & 2 ? -x : x) * attn, (quarters & 2 ? -y : y) * attn);
}

__device__ __forceinline__ double exact_value(float x) { return x; }
__device__ __forceinline__ double exact_value(__nv_bfloat16 x) { return __bfloat162float(x); }

// The cosine and sine of turn t (of 2^64) in 62-bit fixed point, good to 2^-57: the Taylor series of both on [-pi/4, pi/4]
// around the nearest quarter turn. In integers, as they run at full rate here: 64-bit floats run at a 64th of it.
__device__ __forceinline__ void turn_exact(uint64_t t, int64_t* cosine, int64_t* sine) {
  // (-1)^k / (2 k)! and (-1)^k / (2 k + 1)!, times 2^62, k = 8 .. 0
  constexpr int64_t kOne = 1ll << 62;
  constexpr int64_t kCos[9] = {kOne / 20922789888000ll, -kOne / 87178291200ll, kOne / 479001600ll, -kOne / 3628800ll,
                               kOne / 40320ll, -kOne / 720ll, kOne / 24ll, -kOne / 2ll, kOne};
  constexpr int64_t kSin[9] = {kOne / 355687428096000ll, -kOne / 1307674368000ll, kOne / 6227020800ll, -kOne / 39916800ll,
                               kOne / 362880ll, -kOne / 5040ll, kOne / 120ll, -kOne / 6ll, kOne};
  const uint32_t quarters = ((uint32_t)(t >> 32) + (1u << 29)) >> 30;
  const int64_t r = (int64_t)(t - ((uint64_t)quarters << 62));  // a quarter turn is 2^62
  const int64_t angle = __mul64hi(r, 7244019458077122842ll) << 2;  // r * pi / 2^63, times 2^62: by pi * 2^61
  const int64_t z = __mul64hi(angle, angle) << 2;
  int64_t c = kCos[0], s = kSin[0];
#pragma unroll
  for (int k = 1; k < 9; ++k) {
    c = kCos[k] + (__mul64hi(c, z) << 2);
    s = kSin[k] + (__mul64hi(s, z) << 2);
  }
  s = __mul64hi(s, angle) << 2;
  const bool odd = quarters & 1;  // (c, s) -> (-s, c) a quarter
  const int64_t x = odd ? s : c, y = odd ? c : s;
  *cosine = (quarters + 1) & 2 ? -x : x;
  *sine = quarters & 2 ? -y : y;
}

// Entry e of a head at src, turned, to 52 bits: what decides a rounding to four bits when 32 leave it open.
template <typename T, bool AXES>
__device__ __noinline__ double exact_entry(const RotArgs& a, const T* src, size_t tok, int e, bool half) {
  if (e >= a.rot) return exact_value(src[e]);
  const int pairs = a.rot / 2, i = half ? (e < pairs ? e : e - pairs) : e / 2;
  const bool first = half ? e < pairs : !(e & 1);
  const double x = exact_value(src[half ? i : 2 * i]), y = exact_value(src[half ? i + pairs : 2 * i + 1]);
  const uint64_t t = (uint64_t)(int64_t)position_of<AXES>(a, tok, i) * __ldg(a.freqs + i);
  int64_t ci, si;
  turn_exact(t, &ci, &si);
  const double c = (double)ci * 0x1p-62, s = (double)si * 0x1p-62;
  return (first ? x * c - y * s : y * c + x * s) * (double)a.attn;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& w, float* x) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 put(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& w, float* x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(v[i]);
      x[2 * i + 1] = bf16_hi(v[i]);
    }
  }
  static __device__ __forceinline__ uint4 put(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
};

// One unit of one head of one token: the chunks, where they go, the pairs' turns.
template <typename T, bool HALF>
struct RotUnit {
  uint4 w0, w1;
  char* dst;  // nullptr: nothing to do (past the last head, or a key without a slot)
  const float4* f;  // two pairs' turns, the next two ``rot_units`` further
};

// 16-byte chunks: every row, stride and half of a pair block starts on 16 bytes. The fp32 interleaved form is held to
// 48 registers, ten blocks an SM (the 56 it takes by itself: 9.1 us for 8.1 at 3,001 tokens); bounds cost the others.
template <typename T, bool HALF, bool AXES, bool KEYS>
__device__ __forceinline__ void rotary_body(const RotArgs& a, int block) {
  constexpr int N = Vec<T>::N;
  constexpr int kV = 2;  // chunks of v a thread loads ahead
  constexpr int PU = HALF ? N : N / 2;  // pairs of a unit
  // A token's turns lie two pairs by two, unit after unit: the threads of a head
  // read 16 bytes each side by side (pair after pair they met in the same banks
  // eight at a time, which cost more than the memory did).
  __shared__ float4 cs[kRotMaxPairs / 2];
  __shared__ int slots[kRotMaxTokens];
  const int tid = threadIdx.x;
  const int pairs = a.rot / 2;
  const int t0 = block * a.tokens;
  const int nt = min(a.tokens, a.n - t0);
  // units of a head: rotated ones first (HALF: chunk u and chunk u + rot / 2 N), then the rest of the head, one chunk each
  const int rot_units = HALF ? a.rot / (2 * N) : a.rot / N;
  const int units = rot_units + (a.d - a.rot) / N;
  const int upar = max(1, min(units, kRotThreads));  // no units: rows without a rotated part
  const int groups = kRotThreads / upar;
  const int g = tid / upar, u0 = tid - g * upar;
  const int heads = KEYS ? a.hq + a.hk : a.hq;
  const int jobs = g < groups ? nt * heads : 0;  // (token, head)
  const int v_chunks = KEYS && a.k ? a.v_elems / N : 0, v_jobs = nt * v_chunks;

  // Loads the unit u of job j; its slot is looked up in store().
  auto load = [&](int j, int u, RotUnit<T, HALF>& x, int& key_of) {
    x.dst = nullptr;
    key_of = -1;
    if (j >= jobs) return;
    const int t = j / heads, h = j - t * heads;
    const size_t tok = (size_t)(t0 + t);
    const bool is_q = h < a.hq, turn = u < rot_units;
    const int e0 = HALF ? (turn ? u * N : a.rot + (u - rot_units) * N) : u * N;
    const char* src = is_q ? a.q + tok * a.q_tok + (size_t)h * a.q_head
                           : a.k + tok * a.k_tok + (size_t)(h - a.hq) * a.d * sizeof(T);
    // plain loads: q_out may be q itself
    x.w0 = *reinterpret_cast<const uint4*>(src + (size_t)e0 * sizeof(T));
    if (HALF && turn) x.w1 = *reinterpret_cast<const uint4*>(src + (size_t)(e0 + pairs) * sizeof(T));
    x.f = cs + t * (pairs / 2) + (turn ? u : 0);
    if (is_q) {
      x.dst = a.q_out + tok * a.qo_tok + (size_t)h * a.qo_head + (size_t)e0 * sizeof(T);
    } else {
      x.dst = a.k_dst + ((size_t)(h - a.hq) * a.d + e0) * sizeof(T);
      key_of = t;
    }
  };
  auto store = [&](const RotUnit<T, HALF>& x, int u, int key_of) {
    if (!x.dst) return;
    char* dst = x.dst;
    if (KEYS && key_of >= 0) {
      const int slot = slots[key_of];
      if (slot < 0) return;
      dst += (size_t)slot * a.row_bytes;
    }
    if (u >= rot_units) {
      *reinterpret_cast<uint4*>(dst) = x.w0;
      return;
    }
    float v[N];
    Vec<T>::get(x.w0, v);
    if (HALF) {
      float y[N], r0[N], r1[N];
      Vec<T>::get(x.w1, y);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float4 f = x.f[i / 2 * rot_units];
        r0[i] = v[i] * f.x - y[i] * f.y;
        r1[i] = y[i] * f.x + v[i] * f.y;
        r0[i + 1] = v[i + 1] * f.z - y[i + 1] * f.w;
        r1[i + 1] = y[i + 1] * f.z + v[i + 1] * f.w;
      }
      *reinterpret_cast<uint4*>(dst) = Vec<T>::put(r0);
      *reinterpret_cast<uint4*>(dst + (size_t)pairs * sizeof(T)) = Vec<T>::put(r1);
    } else {
      float r[N];
#pragma unroll
      for (int i = 0; i < N / 2; i += 2) {
        const float4 f = x.f[i / 2 * rot_units];
        r[2 * i] = v[2 * i] * f.x - v[2 * i + 1] * f.y;
        r[2 * i + 1] = v[2 * i + 1] * f.x + v[2 * i] * f.y;
        r[2 * i + 2] = v[2 * i + 2] * f.z - v[2 * i + 3] * f.w;
        r[2 * i + 3] = v[2 * i + 3] * f.z + v[2 * i + 2] * f.w;
      }
      *reinterpret_cast<uint4*>(dst) = Vec<T>::put(r);
    }
  };
  auto v_src = [&](int c) {
    const int t = KEYS ? c / v_chunks : 0;
    return reinterpret_cast<const uint4*>(a.v + (size_t)(t0 + t) * a.v_tok) + (c - t * v_chunks);
  };
  auto v_put = [&](int c, const uint4& w) {
    const int t = KEYS ? c / v_chunks : 0, slot = slots[t];
    if (slot >= 0) reinterpret_cast<uint4*>(a.v_dst + (size_t)slot * a.row_bytes)[c - t * v_chunks] = w;
  };

  uint4 vw[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (tid + i * kRotThreads < v_jobs) vw[i] = __ldg(v_src(tid + i * kRotThreads));
  RotUnit<T, HALF> x0, x1;
  int k0, k1;
  load(g, u0, x0, k0);
  load(g + groups, u0, x1, k1);
  if (KEYS && a.k && tid < nt) {
    const int slot = __ldg(a.out_loc + t0 + tid);
    const bool good = (unsigned)slot < (unsigned)a.num_slots;
    if (!good) set_error(a.err, KVP_ERR_BAD_INDEX);
    slots[tid] = good ? slot : -1;
  }
  for (int x = tid; x < nt * pairs; x += kRotThreads) {
    const int t = x / pairs, i = x - t * pairs;
    const int u = i / PU, r = i % PU;
    reinterpret_cast<float2*>(cs)[t * pairs + 2 * (r / 2 * rot_units + u) + (r & 1)] =
        turn_of(AXES ? position_of<AXES>(a, (size_t)(t0 + t), i) : __ldg(a.positions + t0 + t), __ldg(a.freqs + i), a.attn);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (tid + i * kRotThreads < v_jobs) v_put(tid + i * kRotThreads, vw[i]);
  for (int c = tid + kV * kRotThreads; c < v_jobs; c += kRotThreads) v_put(c, __ldg(v_src(c)));
  for (int u = u0; u < units; u += upar) {  // more than one round only for heads of more than 128 units
    for (int j = g; j < jobs; j += 2 * groups) {
      if (j != g || u != u0) {
        load(j, u, x0, k0);
        load(j + groups, u, x1, k1);
      }
      store(x0, u, k0);
      store(x1, u, k1);
    }
  }
}

template <typename T, bool HALF, bool AXES>
__global__ void __launch_bounds__(kRotThreads, !HALF && sizeof(T) == 4 && !AXES ? 10 : 0) rotary_store_kernel(const RotArgs a) {
  rotary_body<T, HALF, AXES, true>(a, blockIdx.x);
}

// Keys and values into a four-bit pool (fp4.cuh): a block takes up to four tokens. A thread has one place in a token's row
// for all of them, a whole block of V (16 entries) or what the rotated form calls a unit of K. K's blocks lie in 16 / N
// neighbouring threads, which agree on the largest entry by shuffles.
// The rotation's error (2^-21 of a pair's size; 2^-20 is reckoned with) leaves one rounding in some ten thousand open:
// those entries are turned again to 52 bits, so that codes and scales are those of the 64-bit formula.
template <typename T, bool HALF, bool AXES>
__device__ __forceinline__ void fp4_body(const RotArgs& a, int block) {
  constexpr int N = Vec<T>::N;
  constexpr int PU = HALF ? N : N / 2;   // pairs of a unit
  constexpr int kChunks = kFp4Block / N;  // of a block of V; also the threads of a block of K
  constexpr int kMost = kChunks > 2 ? kChunks : 2;
  __shared__ float4 cs[kRotMaxPairs / 2];  // laid out as in rotary_body
  __shared__ int slots[kRotMaxTokens];
  const int tid = threadIdx.x, t0 = block * a.kv_tokens, nt = min(a.kv_tokens, a.n - t0);
  const int pairs = a.rot / 2, rot_units = HALF ? a.rot / (2 * N) : a.rot / N, units = rot_units + (a.d - a.rot) / N;
  const int v_units = a.hk * (a.d / kFp4Block), all = v_units + a.hk * units;
  const unsigned mask = ((1u << kChunks) - 1u) << (tid & 31 & ~(kChunks - 1));
  const float inv_gk = 1.f / a.gk, inv_gv = 1.f / a.gv, off = fabsf(a.attn) * 0x1p-20f;

  uint4 w[kMost];
  // where a unit lies: head, first entry, whether it turns
  auto place = [&](int x, int& h, int& u, int& e0) {
    if (x < v_units) {
      h = x / (a.d / kFp4Block);
      u = x - h * (a.d / kFp4Block);
      e0 = u * kFp4Block;
    } else {
      h = (x - v_units) / units;
      u = x - v_units - h * units;
      e0 = HALF && u >= rot_units ? a.rot + (u - rot_units) * N : u * N;
    }
  };
  auto load = [&](int x, int t) {
    int h, u, e0;
    place(x, h, u, e0);
    const size_t tok = (size_t)(t0 + t);
    if (x < v_units) {
      const uint4* src = reinterpret_cast<const uint4*>(a.v + tok * a.v_tok + ((size_t)h * a.d + e0) * sizeof(T));
#pragma unroll
      for (int i = 0; i < kChunks; ++i) w[i] = __ldg(src + i);
    } else {
      const char* src = a.k + tok * a.k_tok + ((size_t)h * a.d + e0) * sizeof(T);
      w[0] = __ldg(reinterpret_cast<const uint4*>(src));
      if (HALF && u < rot_units) w[1] = __ldg(reinterpret_cast<const uint4*>(src + (size_t)pairs * sizeof(T)));
    }
  };
  if (tid < all) load(tid, 0);
  if (tid < nt) {
    const int slot = __ldg(a.out_loc + t0 + tid);
    const bool good = (unsigned)slot < (unsigned)a.num_slots;
    if (!good) set_error(a.err, KVP_ERR_BAD_INDEX);
    slots[tid] = good ? slot : -1;
  }
  for (int x = tid; x < nt * pairs; x += kRotThreads) {
    const int t = x / pairs, i = x - t * pairs;
    const int u = i / PU, r = i % PU;
    reinterpret_cast<float2*>(cs)[t * pairs + 2 * (r / 2 * rot_units + u) + (r & 1)] =
        turn_of(AXES ? position_of<AXES>(a, (size_t)(t0 + t), i) : __ldg(a.positions + t0 + t), __ldg(a.freqs + i), a.attn);
  }
  __syncthreads();
  for (int x = tid; x < all; x += kRotThreads) {
    int h, u, e0;
    place(x, h, u, e0);
    for (int t = 0; t < nt; ++t) {
      if (x != tid || t) load(x, t);
      const int slot = slots[t];
      if (slot < 0) continue;
      char* row = a.k_dst + (size_t)slot * a.row_bytes + (size_t)h * a.d;
      char* scales = a.scales + fp4_scale_offset(slot, h, a.hk, a.d);
      uint32_t codes, scale;
      if (x < v_units) {
        float v[kFp4Block];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) Vec<T>::get(w[i], v + N * i);
        uint32_t lo, hi;
        fp4_block16(v, a.gv, inv_gv, lo, hi, scale);
        *reinterpret_cast<uint2*>(row + a.d / 2 + e0 / 2) = make_uint2(lo, hi);
        scales[a.d / 16 + u] = (char)scale;
        continue;
      }
      auto put = [&](int e) {
        if (N == 8) *reinterpret_cast<uint32_t*>(row + e / 2) = codes;
        else *reinterpret_cast<uint16_t*>(row + e / 2) = (uint16_t)codes;
        if (e % kFp4Block == 0) scales[e / kFp4Block] = (char)scale;
      };
      float v[N];
      Vec<T>::get(w[0], v);
      if (u >= rot_units) {
        fp4_block<N>(v, a.gk, inv_gk, mask, codes, scale);
        put(e0);
        continue;
      }
      const T* src = reinterpret_cast<const T*>(a.k + (size_t)(t0 + t) * a.k_tok) + (size_t)h * a.d;
      const float4* f = cs + t * (pairs / 2) + u;
      auto entry = [&](int e) { return exact_entry<T, AXES>(a, src, (size_t)(t0 + t), e, HALF); };
      float er = 0.f;  // what the rotation may be off by, in any of the unit's entries
      if (HALF) {
        float y[N], r0[N], r1[N];
        Vec<T>::get(w[1], y);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float4 c = f[i / 2 * rot_units];
          r0[i] = v[i] * c.x - y[i] * c.y;
          r1[i] = y[i] * c.x + v[i] * c.y;
          r0[i + 1] = v[i + 1] * c.z - y[i + 1] * c.w;
          r1[i + 1] = y[i + 1] * c.z + v[i + 1] * c.w;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) er = fmaxf(er, fabsf(v[i]) + fabsf(y[i]));
        er *= off;
        fp4_block_within<N>(r0, er, a.gk, inv_gk, mask, [&](int i) { return entry(e0 + i); }, codes, scale);
        put(e0);
        fp4_block_within<N>(r1, er, a.gk, inv_gk, mask, [&](int i) { return entry(e0 + pairs + i); }, codes, scale);
        put(e0 + pairs);
      } else {
        float r[N];
#pragma unroll
        for (int i = 0; i < N / 2; i += 2) {
          const float4 c = f[i / 2 * rot_units];
          r[2 * i] = v[2 * i] * c.x - v[2 * i + 1] * c.y;
          r[2 * i + 1] = v[2 * i + 1] * c.x + v[2 * i] * c.y;
          r[2 * i + 2] = v[2 * i + 2] * c.z - v[2 * i + 3] * c.w;
          r[2 * i + 3] = v[2 * i + 3] * c.z + v[2 * i + 2] * c.w;
        }
#pragma unroll
        for (int i = 0; i < N; i += 2) er = fmaxf(er, fabsf(v[i]) + fabsf(v[i + 1]));
        er *= off;
        fp4_block_within<N>(r, er, a.gk, inv_gk, mask, [&](int i) { return entry(e0 + i); }, codes, scale);
        put(e0);
      }
    }
  }
}

// A step into a four-bit pool in one launch: the first a.kv_blocks blocks have keys and values, the others queries.
template <typename T, bool HALF, bool AXES>
__global__ void __launch_bounds__(kRotThreads, 10) fp4_store_kernel(const __grid_constant__ RotArgs a) {
  if ((int)blockIdx.x < a.kv_blocks) fp4_body<T, HALF, AXES>(a, blockIdx.x);
  else rotary_body<T, HALF, AXES, false>(a, blockIdx.x - a.kv_blocks);
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Any alignment and any even rotary_dim: one block per token, element by
// element (a thread owns a whole pair, so q_out may be q itself).
template <typename T, bool AXES>
__global__ void __launch_bounds__(kRotThreads) rotary_store_elem_kernel(const RotArgs a, int half) {
  const size_t tok = blockIdx.x;
  const int tid = threadIdx.x, pairs = a.rot / 2, per = pairs + (a.d - a.rot);
  const int p = AXES ? 0 : __ldg(a.positions + tok);
  char* krow = nullptr;
  if (a.k) {
    const int slot = __ldg(a.out_loc + tok);
    if ((unsigned)slot < (unsigned)a.num_slots) {
      krow = a.k_dst + (size_t)slot * a.row_bytes;
      const T* src = reinterpret_cast<const T*>(a.v + tok * a.v_tok);
      T* dst = reinterpret_cast<T*>(a.v_dst + (size_t)slot * a.row_bytes);
      for (int c = tid; c < a.v_elems; c += kRotThreads) dst[c] = src[c];
    } else if (tid == 0) {
      set_error(a.err, KVP_ERR_BAD_INDEX);
    }
  }
  const long long work = (long long)(a.hq + (krow ? a.hk : 0)) * per;
  for (long long x = tid; x < work; x += kRotThreads) {
    const int h = (int)(x / per), i = (int)(x % per);
    const bool is_q = h < a.hq;
    const T* src = reinterpret_cast<const T*>(is_q ? a.q + tok * a.q_tok + (size_t)h * a.q_head
                                                   : a.k + tok * a.k_tok + (size_t)(h - a.hq) * a.d * sizeof(T));
    T* dst = reinterpret_cast<T*>(is_q ? a.q_out + tok * a.qo_tok + (size_t)h * a.qo_head
                                       : krow + (size_t)(h - a.hq) * a.d * sizeof(T));
    if (i >= pairs) {
      dst[a.rot + i - pairs] = src[a.rot + i - pairs];
      continue;
    }
    const float2 f = turn_of(AXES ? position_of<AXES>(a, tok, i) : p, __ldg(a.freqs + i), a.attn);
    const int e0 = half ? i : 2 * i, e1 = half ? i + pairs : 2 * i + 1;
    const float x0 = ld1(src + e0), x1 = ld1(src + e1);
    st1(dst + e0, x0 * f.x - x1 * f.y);
    st1(dst + e1, x1 * f.x + x0 * f.y);
  }
}

// Keys and values into a four-bit pool, any alignment and any even rotary_dim, entry by entry: two neighbouring threads make
// one block, as in fp4_body, with a sine a pair and head (64 tokens of 8 heads of 128: 7.4 us, 8,192 tokens 49 us).
template <typename T, bool AXES>
__global__ void __launch_bounds__(kRotThreads) fp4_store_elem_kernel(const __grid_constant__ RotArgs a, int half) {
  constexpr int N = kFp4Block / 2;
  const int blocks = a.d / kFp4Block, per = 2 * a.hk * blocks, pairs = a.rot / 2;
  const long long stride = (long long)gridDim.x * kRotThreads;
  const unsigned mask = 3u << (threadIdx.x & 30);
  const float off = fabsf(a.attn) * 0x1p-20f;
  for (long long id = (long long)blockIdx.x * kRotThreads + threadIdx.x; id < 2LL * a.n * per; id += stride) {
    const size_t tok = (size_t)(id / (2 * per));
    const int x = (int)(id / 2 % per), part = x / (a.hk * blocks), h = x / blocks % a.hk;
    const int e0 = x % blocks * kFp4Block + (int)(id & 1) * N;
    const int slot = __ldg(a.out_loc + tok);
    if ((unsigned)slot >= (unsigned)a.num_slots) {
      if (x == 0) set_error(a.err, KVP_ERR_BAD_INDEX);
      continue;
    }
    const T* src = reinterpret_cast<const T*>(part ? a.v + tok * a.v_tok : a.k + tok * a.k_tok) + (size_t)h * a.d;
    const float g = part ? a.gv : a.gk, inv_g = 1.f / g;
    float v[N];
    uint32_t codes, scale;
    if (part || e0 >= a.rot) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = ld1(src + e0 + i);
    }
    // K's blocks that turn, or the halves of one, agree on the way they take
    if (part || e0 - (int)(id & 1) * N >= a.rot) {
      fp4_block<N>(v, g, inv_g, mask, codes, scale);
    } else {
      float er = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = e0 + i;
        if (e >= a.rot) {
          v[i] = ld1(src + e);
          continue;
        }
        const int pair = half ? (e < pairs ? e : e - pairs) : e / 2;
        const bool first = half ? e < pairs : !(e & 1);
        const float x0 = ld1(src + (half ? pair : 2 * pair)), x1 = ld1(src + (half ? pair + pairs : 2 * pair + 1));
        const float2 f = turn_of(position_of<AXES>(a, tok, pair), __ldg(a.freqs + pair), a.attn);
        v[i] = first ? x0 * f.x - x1 * f.y : x1 * f.x + x0 * f.y;
        er = fmaxf(er, fabsf(x0) + fabsf(x1));
      }
      fp4_block_within<N>(v, er * off, g, inv_g, mask, [&](int i) { return exact_entry<T, AXES>(a, src, tok, e0 + i, half); },
                          codes, scale);
    }
    char* dst = a.k_dst + (size_t)slot * a.row_bytes + (size_t)h * a.d + part * (a.d / 2) + e0 / 2;
    *reinterpret_cast<uint32_t*>(dst) = codes;
    if (!(id & 1)) a.scales[fp4_scale_offset(slot, h, a.hk, a.d) + part * blocks + e0 / 16] = (char)scale;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, bool HALF>
void launch_vec(const RotArgs& a, bool fp4, unsigned grid, cudaStream_t st) {
  if (fp4) {
    if (a.pair_axis) fp4_store_kernel<T, HALF, true><<<grid, kRotThreads, 0, st>>>(a);
    else fp4_store_kernel<T, HALF, false><<<grid, kRotThreads, 0, st>>>(a);
  } else {
    if (a.pair_axis) rotary_store_kernel<T, HALF, true><<<grid, kRotThreads, 0, st>>>(a);
    else rotary_store_kernel<T, HALF, false><<<grid, kRotThreads, 0, st>>>(a);
  }
}
template <typename T>
void launch_layout(const RotArgs& a, bool half, bool fp4, unsigned grid, cudaStream_t st) {
  if (half) launch_vec<T, true>(a, fp4, grid, st);
  else launch_vec<T, false>(a, fp4, grid, st);
}
template <typename T>
void launch_elem(const RotArgs& a, bool half, cudaStream_t st) {
  if (a.pair_axis) rotary_store_elem_kernel<T, true><<<a.n, kRotThreads, 0, st>>>(a, half);
  else rotary_store_elem_kernel<T, false><<<a.n, kRotThreads, 0, st>>>(a, half);
}
template <typename T>
void launch_fp4_elem(const RotArgs& a, bool half, cudaStream_t st) {
  const long long blocks = ((long long)a.n * 4 * a.hk * (a.d / kFp4Block) + kRotThreads - 1) / kRotThreads;
  const unsigned grid = (unsigned)(blocks < 1 << 20 ? blocks : 1 << 20);
  if (a.pair_axis) fp4_store_elem_kernel<T, true><<<grid, kRotThreads, 0, st>>>(a, half);
  else fp4_store_elem_kernel<T, false><<<grid, kRotThreads, 0, st>>>(a, half);
}

int launch_rotary(const kvp_pool* pool, RotArgs& a, int layout, cudaStream_t st) {
  const int es = pool->elem, N = 16 / es;
  const bool half = layout == KVP_ROTARY_HALF, fp4 = pool->fp4 && a.k;
  const int span = half ? a.rot / 2 : a.rot;  // contiguous elements of a rotated block
  // four bits: threads that share a block of 16 all turn it or all do not
  bool vec = a.d % N == 0 && span % (fp4 ? kFp4Block : N) == 0 && a.rot / 2 <= kRotMaxPairs;
  bool vec_q = true;
  if (a.q) vec_q = aligned16(a.q) && aligned16(a.q_out) && !((a.q_tok | a.q_head | a.qo_tok | a.qo_head) & 15);
  bool vec_k = true;
  if (a.k)
    vec_k = aligned16(a.k) && aligned16(a.v) && !((a.k_tok | a.v_tok) & 15) && a.v_elems % N == 0 &&
            (fp4 || (aligned16(a.k_dst) && aligned16(a.v_dst))) && a.row_bytes % 16 == 0;
  if (fp4 && a.q && !(vec && vec_q && vec_k)) {  // the queries by themselves, then keys and values
    RotArgs q = a;
    q.k = q.v = nullptr;
    q.hk = 0;
    const int rc = launch_rotary(pool, q, layout, st);
    if (rc != KVP_OK) return rc;
    a.q = nullptr;
    a.hq = 0;
    vec_q = true;
  }
  vec = vec && vec_q && vec_k;
  if (!vec) {
    if (fp4) {
      if (es == 4) launch_fp4_elem<float>(a, half, st);
      else launch_fp4_elem<__nv_bfloat16>(a, half, st);
    } else {
      if (es == 4) launch_elem<float>(a, half, st);
      else launch_elem<__nv_bfloat16>(a, half, st);
    }
    return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
  }
  // as many tokens a block as its shared memory's pairs allow, up to 4, once
  // that still leaves every SM eight blocks
  int tokens = 1;
  while (tokens < kRotMaxTokens && 2 * tokens * (a.rot / 2) <= kRotMaxPairs && a.n / (2 * tokens) >= pool->num_sms * 8) tokens *= 2;
  a.tokens = tokens;
  long long grid = fp4 && !a.q ? 0 : ((long long)a.n + tokens - 1) / tokens;
  if (fp4) {
    a.kv_tokens = tokens;
    a.kv_blocks = (int)(((long long)a.n + tokens - 1) / tokens);
    grid += a.kv_blocks;
    if (grid > 0x7fffffffLL) return KVP_ERR_INVALID_ARG;
  }
  if (es == 4) launch_layout<float>(a, half, fp4, (unsigned)grid, st);
  else launch_layout<__nv_bfloat16>(a, half, fp4, (unsigned)grid, st);
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

// Positions of several axes: their number, the axis of each pair (device; not read for one axis), the distance of two
// axes' positions in entries.
struct Axes {
  int count;
  const uint8_t* of_pair;
  long long stride;
};
constexpr Axes kOneAxis = {1, nullptr, 0};

// The checks the entry points share. ``width``: entries of a query head.
bool rotary_args_ok(const kvp_pool* pool, int layer, const void* q, long long q_stride, long long q_head_stride, int hq,
                    int width, const void* k, long long k_stride, const void* v, long long v_stride,
                    const int32_t* positions, const int32_t* out_loc, int n, const uint64_t* freqs,
                    int rotary_dim, int layout, float attn, const void* q_out, long long qo_stride,
                    long long qo_head_stride, const Axes& ax) {
  if (layer < 0 || layer >= pool->num_layers || n < 0) return false;
  if (layout != KVP_ROTARY_HALF && layout != KVP_ROTARY_INTERLEAVED) return false;
  if (rotary_dim < 0 || rotary_dim % 2 || rotary_dim > width || !(attn == attn)) return false;
  if (ax.count < 1 || ax.count > KVP_ROTARY_MAX_AXES) return false;
  if (n == 0) return true;  // empty tensors may have no address
  if ((k == nullptr) != (v == nullptr) || (!q && !k)) return false;
  // rows as they are into a four-bit pool need no positions; the kernels of other pools read them whatever turns
  if ((!positions && (!pool->fp4 || q || rotary_dim > 0)) || (rotary_dim > 0 && !freqs)) return false;
  if (ax.count != 1 && (rotary_dim > 0 && !ax.of_pair)) return false;
  if (ax.count > 1 && ax.stride < n) return false;
  if (k && (!out_loc || k_stride < 0 || v_stride < 0)) return false;
  if (q) {
    if (!q_out || hq <= 0 || q_stride < 0 || q_head_stride < 0) return false;
    // the outputs do not overlap: heads within a token's row, or tokens within a head's
    if (qo_head_stride < width || qo_stride < width) return false;
    if (qo_stride < (hq - 1) * qo_head_stride + width && qo_head_stride < (n - 1) * qo_stride + width) return false;
    if (q_out == q && (q_stride != qo_stride || q_head_stride != qo_head_stride)) return false;
  }
  const uintptr_t em = pool->elem - 1;
  return !((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(k) |
            reinterpret_cast<uintptr_t>(v)) & em);
}

}  // namespace

bool pool_device_current(const kvp_pool* pool) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == pool->device;
}

}  // namespace kvp

extern "C" int kvp_rotary_frequencies(int rotary_dim, double base, int scaling, double factor, double original_len,
                                      double low_turns, double high_turns, uint64_t* freqs) {
  if (!freqs || rotary_dim <= 0 || rotary_dim % 2 || !(base > 0.0) || !std::isfinite(base)) return KVP_ERR_INVALID_ARG;
  if (scaling < KVP_ROTARY_PLAIN || scaling > KVP_ROTARY_BY_PARTS) return KVP_ERR_INVALID_ARG;
  if (scaling != KVP_ROTARY_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return KVP_ERR_INVALID_ARG;
  if (scaling == KVP_ROTARY_NTK && rotary_dim == 2) return KVP_ERR_INVALID_ARG;  // its exponent d / (d - 2)
  if (scaling == KVP_ROTARY_BY_PARTS &&
      (!(original_len > 0.0) || !std::isfinite(original_len) || !(low_turns < high_turns)))
    return KVP_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  if (scaling == KVP_ROTARY_NTK) base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == KVP_ROTARY_LINEAR) {
      f /= factor;
    } else if (scaling == KVP_ROTARY_BY_PARTS) {
      double keep = (original_len * f / two_pi - low_turns) / (high_turns - low_turns);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = keep * f + (1.0 - keep) * (f / factor);
    }
    if (!std::isfinite(f)) return KVP_ERR_INVALID_ARG;
    double turns = f / two_pi;
    turns -= std::floor(turns);
    // turns < 1 has 53 bits; the top 2^-53 would round up to 2^64
    const double scaled = std::ldexp(turns, 64);
    freqs[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
  }
  return KVP_OK;
}

namespace kvp {
namespace {

// Every entry point's arguments; two rows a token: K and V, or the shared key part and the latent.
struct RotaryCall {
  const void* q;
  long long q_stride, q_head_stride;
  int num_q_heads;
  const void* k;
  long long k_stride;
  const void* v;
  long long v_stride;
  const int32_t* positions;
  const int32_t* out_loc;
  int n;
  const uint64_t* freqs;
  int rotary_dim, layout;
  float attn_factor;
  void* q_out;
  long long q_out_stride, q_out_head_stride;
  Axes axes;
};

bool call_ok(const kvp_pool* pool, int layer, const RotaryCall& c, int width) {
  return rotary_args_ok(pool, layer, c.q, c.q_stride, c.q_head_stride, c.num_q_heads, width, c.k, c.k_stride, c.v,
                        c.v_stride, c.positions, c.out_loc, c.n, c.freqs, c.rotary_dim, c.layout, c.attn_factor, c.q_out,
                        c.q_out_stride, c.q_out_head_stride, c.axes);
}

// What does not depend on the pool's kind.
RotArgs common_args(const kvp_pool* pool, const RotaryCall& c) {
  const long long es = pool->elem;
  RotArgs a = {};
  a.q = static_cast<const char*>(c.q);
  a.q_out = static_cast<char*>(c.q_out);
  a.q_tok = c.q_stride * es;
  a.q_head = c.q_head_stride * es;
  a.qo_tok = c.q_out_stride * es;
  a.qo_head = c.q_out_head_stride * es;
  a.k = static_cast<const char*>(c.k);
  a.k_tok = c.k_stride * es;
  a.v = static_cast<const char*>(c.v);
  a.v_tok = c.v_stride * es;
  a.row_bytes = pool->row_bytes;
  a.positions = c.positions;
  a.out_loc = c.out_loc;
  a.freqs = c.freqs;
  a.n = c.n;
  a.hq = c.q ? c.num_q_heads : 0;
  a.rot = c.rotary_dim;
  a.num_slots = pool->num_slots;
  a.attn = c.attn_factor;
  a.err = pool->err;
  if (c.axes.count > 1) {
    a.pair_axis = c.axes.of_pair;
    a.pos_axis = c.axes.stride;
    a.axes = c.axes.count;
  }
  return a;
}

int store_planes(const kvp_pool* pool, int layer, const RotaryCall& c, void* stream) {
  if (!pool || !pool->kv_rows()) return KVP_ERR_INVALID_ARG;
  if (!call_ok(pool, layer, c, pool->head_dim)) return KVP_ERR_INVALID_ARG;
  if (c.n == 0) return KVP_OK;
  if (!pool_device_current(pool)) return KVP_ERR_INVALID_ARG;
  RotArgs a = common_args(pool, c);
  a.k_dst = pool->buf + (size_t)layer * pool->layer_bytes;
  a.v_dst = a.k_dst + pool->kv_bytes;
  a.hk = c.k ? pool->kv_heads : 0;
  a.d = pool->head_dim;
  a.v_elems = pool->kv_heads * pool->head_dim;
  return launch_rotary(pool, a, c.layout, static_cast<cudaStream_t>(stream));
}

int store_fp4(const kvp_pool* pool, int layer, const RotaryCall& c, void* stream) {
  if (!pool || !pool->fp4) return KVP_ERR_INVALID_ARG;
  if (!call_ok(pool, layer, c, pool->head_dim)) return KVP_ERR_INVALID_ARG;
  if (c.n == 0) return KVP_OK;
  if (!pool_device_current(pool)) return KVP_ERR_INVALID_ARG;
  RotArgs a = common_args(pool, c);
  a.k_dst = pool->buf + (size_t)layer * pool->layer_bytes;
  a.v_dst = a.k_dst + pool->head_dim / 2;
  a.scales = pool->fp4_scales + (size_t)layer * pool->fp4_scale_layer_bytes;
  a.gk = pool->fp4_globals[layer];
  a.gv = pool->fp4_globals[pool->num_layers + layer];
  a.hk = c.k ? pool->kv_heads : 0;
  a.d = pool->head_dim;
  a.v_elems = pool->kv_heads * pool->head_dim;
  return launch_rotary(pool, a, c.layout, static_cast<cudaStream_t>(stream));
}

int store_latent(const kvp_pool* pool, int layer, RotaryCall c, void* stream) {
  if (!pool || !pool->latent_dim) return KVP_ERR_INVALID_ARG;
  const int dc = pool->latent_dim, dr = pool->head_dim - dc;
  if (dr == 0) {  // rows without a rotated part: no queries, and k_pe may have no address
    c.q = nullptr;
    c.k = c.v;
    c.k_stride = c.v_stride;
    if (!c.v) return c.n == 0 ? KVP_OK : KVP_ERR_INVALID_ARG;
  }
  if (!call_ok(pool, layer, c, dr)) return KVP_ERR_INVALID_ARG;
  if (c.n == 0) return KVP_OK;
  if (!pool_device_current(pool)) return KVP_ERR_INVALID_ARG;
  RotArgs a = common_args(pool, c);
  a.v_dst = pool->buf + (size_t)layer * pool->layer_bytes;
  a.k_dst = a.v_dst + (size_t)dc * pool->elem;
  a.hk = c.k && dr > 0 ? 1 : 0;
  a.d = dr;
  a.v_elems = dc;
  return launch_rotary(pool, a, c.layout, static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace kvp

extern "C" int rotary_store_cache(const kvp_pool* pool, int layer, const void* q, long long q_stride,
                                  long long q_head_stride, int num_q_heads, const void* k, long long k_stride,
                                  const void* v, long long v_stride, const int32_t* positions, const int32_t* out_loc,
                                  int n, const uint64_t* freqs, int rotary_dim, int layout, float attn_factor,
                                  void* q_out, long long q_out_stride, long long q_out_head_stride, void* stream) {
  return kvp::store_planes(pool, layer,
                           {q, q_stride, q_head_stride, num_q_heads, k, k_stride, v, v_stride, positions, out_loc, n, freqs,
                            rotary_dim, layout, attn_factor, q_out, q_out_stride, q_out_head_stride, kvp::kOneAxis},
                           stream);
}

extern "C" int rotary_store_cache_axes(const kvp_pool* pool, int layer, const void* q, long long q_stride,
                                       long long q_head_stride, int num_q_heads, const void* k, long long k_stride,
                                       const void* v, long long v_stride, const int32_t* positions,
                                       long long position_stride, const int32_t* out_loc, int n, const uint64_t* freqs,
                                       const uint8_t* pair_axis, int num_axes, int rotary_dim, int layout,
                                       float attn_factor, void* q_out, long long q_out_stride,
                                       long long q_out_head_stride, void* stream) {
  return kvp::store_planes(pool, layer,
                           {q, q_stride, q_head_stride, num_q_heads, k, k_stride, v, v_stride, positions, out_loc, n, freqs,
                            rotary_dim, layout, attn_factor, q_out, q_out_stride, q_out_head_stride,
                            {num_axes, pair_axis, position_stride}},
                           stream);
}

extern "C" int rotary_store_fp4(const kvp_pool* pool, int layer, const void* q, long long q_stride,
                                long long q_head_stride, int num_q_heads, const void* k, long long k_stride,
                                const void* v, long long v_stride, const int32_t* positions, long long position_stride,
                                const int32_t* out_loc, int n, const uint64_t* freqs, const uint8_t* pair_axis,
                                int num_axes, int rotary_dim, int layout, float attn_factor, void* q_out,
                                long long q_out_stride, long long q_out_head_stride, void* stream) {
  return kvp::store_fp4(pool, layer,
                        {q, q_stride, q_head_stride, num_q_heads, k, k_stride, v, v_stride, positions, out_loc, n, freqs,
                         rotary_dim, layout, attn_factor, q_out, q_out_stride, q_out_head_stride,
                         {num_axes, pair_axis, position_stride}},
                        stream);
}

extern "C" int rotary_store_latent(const kvp_pool* pool, int layer, const void* q_pe, long long q_stride,
                                   long long q_head_stride, int num_q_heads, const void* latent,
                                   long long latent_stride, const void* k_pe, long long k_pe_stride,
                                   const int32_t* positions, const int32_t* out_loc, int n, const uint64_t* freqs,
                                   int rotary_dim, int layout, float attn_factor, void* q_pe_out,
                                   long long q_out_stride, long long q_out_head_stride, void* stream) {
  return kvp::store_latent(pool, layer,
                           {q_pe, q_stride, q_head_stride, num_q_heads, k_pe, k_pe_stride, latent, latent_stride, positions,
                            out_loc, n, freqs, rotary_dim, layout, attn_factor, q_pe_out, q_out_stride, q_out_head_stride,
                            kvp::kOneAxis},
                           stream);
}

extern "C" int rotary_store_latent_axes(const kvp_pool* pool, int layer, const void* q_pe, long long q_stride,
                                        long long q_head_stride, int num_q_heads, const void* latent,
                                        long long latent_stride, const void* k_pe, long long k_pe_stride,
                                        const int32_t* positions, long long position_stride, const int32_t* out_loc, int n,
                                        const uint64_t* freqs, const uint8_t* pair_axis, int num_axes, int rotary_dim,
                                        int layout, float attn_factor, void* q_pe_out, long long q_out_stride,
                                        long long q_out_head_stride, void* stream) {
  return kvp::store_latent(pool, layer,
                           {q_pe, q_stride, q_head_stride, num_q_heads, k_pe, k_pe_stride, latent, latent_stride, positions,
                            out_loc, n, freqs, rotary_dim, layout, attn_factor, q_pe_out, q_out_stride, q_out_head_stride,
                            {num_axes, pair_axis, position_stride}},
                           stream);
}
