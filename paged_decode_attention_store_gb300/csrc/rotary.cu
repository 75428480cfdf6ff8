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
// us; 16,461 latent rows with 32 heads' rotated parts 32.2 us (5.4 TB/s, 0.79).
#include "common.cuh"

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
};

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
template <typename T, bool HALF>
__global__ void __launch_bounds__(kRotThreads, !HALF && sizeof(T) == 4 ? 10 : 0) rotary_store_kernel(const RotArgs a) {
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
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, a.n - t0);
  // units of a head: rotated ones first (HALF: chunk u and chunk u + rot / 2 N), then the rest of the head, one chunk each
  const int rot_units = HALF ? a.rot / (2 * N) : a.rot / N;
  const int units = rot_units + (a.d - a.rot) / N;
  const int upar = max(1, min(units, kRotThreads));  // no units: rows without a rotated part
  const int groups = kRotThreads / upar;
  const int g = tid / upar, u0 = tid - g * upar;
  const int heads = a.hq + a.hk;
  const int jobs = g < groups ? nt * heads : 0;  // (token, head)
  const int v_chunks = a.k ? a.v_elems / N : 0, v_jobs = nt * v_chunks;

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
    if (key_of >= 0) {
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
    const int t = c / v_chunks;
    return reinterpret_cast<const uint4*>(a.v + (size_t)(t0 + t) * a.v_tok) + (c - t * v_chunks);
  };
  auto v_put = [&](int c, const uint4& w) {
    const int t = c / v_chunks, slot = slots[t];
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
  if (a.k && tid < nt) {
    const int slot = __ldg(a.out_loc + t0 + tid);
    const bool good = (unsigned)slot < (unsigned)a.num_slots;
    if (!good) set_error(a.err, KVP_ERR_BAD_INDEX);
    slots[tid] = good ? slot : -1;
  }
  for (int x = tid; x < nt * pairs; x += kRotThreads) {
    const int t = x / pairs, i = x - t * pairs;
    const int u = i / PU, r = i % PU;
    reinterpret_cast<float2*>(cs)[t * pairs + 2 * (r / 2 * rot_units + u) + (r & 1)] =
        turn_of(__ldg(a.positions + t0 + t), __ldg(a.freqs + i), a.attn);
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

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Any alignment and any even rotary_dim: one block per token, element by
// element (a thread owns a whole pair, so q_out may be q itself).
template <typename T>
__global__ void __launch_bounds__(kRotThreads) rotary_store_elem_kernel(const RotArgs a, int half) {
  const size_t tok = blockIdx.x;
  const int tid = threadIdx.x, pairs = a.rot / 2, per = pairs + (a.d - a.rot);
  const int p = __ldg(a.positions + tok);
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
    const float2 f = turn_of(p, __ldg(a.freqs + i), a.attn);
    const int e0 = half ? i : 2 * i, e1 = half ? i + pairs : 2 * i + 1;
    const float x0 = ld1(src + e0), x1 = ld1(src + e1);
    st1(dst + e0, x0 * f.x - x1 * f.y);
    st1(dst + e1, x1 * f.x + x0 * f.y);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int launch_rotary(const kvp_pool* pool, RotArgs& a, int layout, cudaStream_t st) {
  const int es = pool->elem, N = 16 / es;
  const bool half = layout == KVP_ROTARY_HALF;
  const int span = half ? a.rot / 2 : a.rot;  // contiguous elements of a rotated block
  bool vec = a.d % N == 0 && span % N == 0 && a.rot / 2 <= kRotMaxPairs;
  if (a.q)
    vec = vec && aligned16(a.q) && aligned16(a.q_out) && !((a.q_tok | a.q_head | a.qo_tok | a.qo_head) & 15);
  if (a.k)
    vec = vec && aligned16(a.k) && aligned16(a.v) && !((a.k_tok | a.v_tok) & 15) && a.v_elems % N == 0 &&
          aligned16(a.k_dst) && aligned16(a.v_dst) && a.row_bytes % 16 == 0;
  if (!vec) {
    if (es == 4) rotary_store_elem_kernel<float><<<a.n, kRotThreads, 0, st>>>(a, half);
    else rotary_store_elem_kernel<__nv_bfloat16><<<a.n, kRotThreads, 0, st>>>(a, half);
    return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
  }
  // as many tokens a block as its shared memory's pairs allow, up to 4, once
  // that still leaves every SM eight blocks
  int tokens = 1;
  while (tokens < kRotMaxTokens && 2 * tokens * (a.rot / 2) <= kRotMaxPairs && a.n / (2 * tokens) >= pool->num_sms * 8) tokens *= 2;
  a.tokens = tokens;
  const unsigned grid = (unsigned)(((long long)a.n + tokens - 1) / tokens);
  if (es == 4) {
    if (half) rotary_store_kernel<float, true><<<grid, kRotThreads, 0, st>>>(a);
    else rotary_store_kernel<float, false><<<grid, kRotThreads, 0, st>>>(a);
  } else {
    if (half) rotary_store_kernel<__nv_bfloat16, true><<<grid, kRotThreads, 0, st>>>(a);
    else rotary_store_kernel<__nv_bfloat16, false><<<grid, kRotThreads, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? KVP_OK : KVP_ERR_CUDA;
}

// The checks both entry points share. ``width``: entries of a query head.
bool rotary_args_ok(const kvp_pool* pool, int layer, const void* q, long long q_stride, long long q_head_stride, int hq,
                    int width, const void* k, long long k_stride, const void* v, long long v_stride,
                    const int32_t* positions, const int32_t* out_loc, int n, const uint64_t* freqs,
                    int rotary_dim, int layout, float attn, const void* q_out, long long qo_stride,
                    long long qo_head_stride) {
  if (layer < 0 || layer >= pool->num_layers || n < 0) return false;
  if (layout != KVP_ROTARY_HALF && layout != KVP_ROTARY_INTERLEAVED) return false;
  if (rotary_dim < 0 || rotary_dim % 2 || rotary_dim > width || !(attn == attn)) return false;
  if (n == 0) return true;  // empty tensors may have no address
  if ((k == nullptr) != (v == nullptr) || (!q && !k)) return false;
  if (!positions || (rotary_dim > 0 && !freqs)) return false;
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

extern "C" int rotary_store_cache(const kvp_pool* pool, int layer, const void* q, long long q_stride,
                                  long long q_head_stride, int num_q_heads, const void* k, long long k_stride,
                                  const void* v, long long v_stride, const int32_t* positions, const int32_t* out_loc,
                                  int n, const uint64_t* freqs, int rotary_dim, int layout, float attn_factor,
                                  void* q_out, long long q_out_stride, long long q_out_head_stride, void* stream) {
  if (!pool || pool->latent_dim) return KVP_ERR_INVALID_ARG;
  const int row = pool->kv_heads * pool->head_dim;
  if (!kvp::rotary_args_ok(pool, layer, q, q_stride, q_head_stride, num_q_heads, pool->head_dim, k, k_stride, v, v_stride,
                           positions, out_loc, n, freqs, rotary_dim, layout, attn_factor, q_out,
                           q_out_stride, q_out_head_stride))
    return KVP_ERR_INVALID_ARG;
  if (n == 0) return KVP_OK;
  if (!kvp::pool_device_current(pool)) return KVP_ERR_INVALID_ARG;
  const long long es = pool->elem;
  kvp::RotArgs a = {};
  a.q = static_cast<const char*>(q);
  a.q_out = static_cast<char*>(q_out);
  a.q_tok = q_stride * es;
  a.q_head = q_head_stride * es;
  a.qo_tok = q_out_stride * es;
  a.qo_head = q_out_head_stride * es;
  a.k = static_cast<const char*>(k);
  a.k_tok = k_stride * es;
  a.v = static_cast<const char*>(v);
  a.v_tok = v_stride * es;
  a.k_dst = pool->buf + (size_t)layer * pool->layer_bytes;
  a.v_dst = a.k_dst + pool->kv_bytes;
  a.row_bytes = pool->row_bytes;
  a.positions = positions;
  a.out_loc = out_loc;
  a.freqs = freqs;
  a.n = n;
  a.hq = q ? num_q_heads : 0;
  a.hk = k ? pool->kv_heads : 0;
  a.d = pool->head_dim;
  a.rot = rotary_dim;
  a.v_elems = row;
  a.num_slots = pool->num_slots;
  a.attn = attn_factor;
  a.err = pool->err;
  return kvp::launch_rotary(pool, a, layout, static_cast<cudaStream_t>(stream));
}

extern "C" int rotary_store_latent(const kvp_pool* pool, int layer, const void* q_pe, long long q_stride,
                                   long long q_head_stride, int num_q_heads, const void* latent,
                                   long long latent_stride, const void* k_pe, long long k_pe_stride,
                                   const int32_t* positions, const int32_t* out_loc, int n, const uint64_t* freqs,
                                   int rotary_dim, int layout, float attn_factor, void* q_pe_out,
                                   long long q_out_stride, long long q_out_head_stride, void* stream) {
  if (!pool || !pool->latent_dim) return KVP_ERR_INVALID_ARG;
  const int dc = pool->latent_dim, dr = pool->head_dim - dc;
  if (dr == 0) {  // rows without a rotated part: no queries, and k_pe may have no address
    q_pe = nullptr;
    k_pe = latent;
    k_pe_stride = latent_stride;
    if (!latent) return n == 0 ? KVP_OK : KVP_ERR_INVALID_ARG;
  }
  if (!kvp::rotary_args_ok(pool, layer, q_pe, q_stride, q_head_stride, num_q_heads, dr, k_pe, k_pe_stride, latent,
                           latent_stride, positions, out_loc, n, freqs, rotary_dim, layout, attn_factor, q_pe_out,
                           q_out_stride, q_out_head_stride))
    return KVP_ERR_INVALID_ARG;
  if (n == 0) return KVP_OK;
  if (!kvp::pool_device_current(pool)) return KVP_ERR_INVALID_ARG;
  const long long es = pool->elem;
  kvp::RotArgs a = {};
  a.q = static_cast<const char*>(q_pe);
  a.q_out = static_cast<char*>(q_pe_out);
  a.q_tok = q_stride * es;
  a.q_head = q_head_stride * es;
  a.qo_tok = q_out_stride * es;
  a.qo_head = q_out_head_stride * es;
  a.k = static_cast<const char*>(k_pe);
  a.k_tok = k_pe_stride * es;
  a.v = static_cast<const char*>(latent);
  a.v_tok = latent_stride * es;
  a.v_dst = pool->buf + (size_t)layer * pool->layer_bytes;
  a.k_dst = a.v_dst + (size_t)dc * pool->elem;
  a.row_bytes = pool->row_bytes;
  a.positions = positions;
  a.out_loc = out_loc;
  a.freqs = freqs;
  a.n = n;
  a.hq = q_pe ? num_q_heads : 0;
  a.hk = k_pe && dr > 0 ? 1 : 0;
  a.d = dr;
  a.rot = rotary_dim;
  a.v_elems = dc;
  a.num_slots = pool->num_slots;
  a.attn = attn_factor;
  a.err = pool->err;
  return kvp::launch_rotary(pool, a, layout, static_cast<cudaStream_t>(stream));
}
