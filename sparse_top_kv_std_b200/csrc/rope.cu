// Queries, keys and values of new tokens, from the projection's token-major layout to the
// library's head-major one, in one pass: an RMS norm of every query and key head, the
// position rotation, and the append of K and V to the cache.
//
//   y_i = w_i x_i / sqrt(mean_j x_j^2 + eps)                   (skipped where w is NULL)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[pair]
//
// The pass reads and writes every value once and does about ten operations on it, so HBM
// bounds it.  Sixteen lanes hold one head of one token, d / 16 neighbouring channels each:
// the sum of squares is four shuffles, a rotation partner half the rotated width away is one
// shuffle (that width is a multiple of d / 16), an adjacent partner sits in the same lane.
// Angles are formed once for each token and shared by all its heads: position times frequency
// in 64 bits, in turns, reduced to [-1/2, 1/2] before they are rounded to 32 (at position
// 140,000 a 32-bit product would be off by up to 8e-3 rad).  Norms and rotations are float32;
// the result is rounded once, to the output type.
#include "common.cuh"
#include "internal.h"

#include <type_traits>

namespace stdb {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsAtOnce = kThreads / 16;

template <int BYTES>
struct Vec {  // BYTES contiguous bytes moved in 16- or 8-byte pieces
  static constexpr int PIECE = BYTES % 16 == 0 ? 16 : 8;
  static constexpr int N = BYTES / PIECE;
  uint32_t w[BYTES / 4];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (PIECE == 16) {
        const uint4 v = __ldcs(static_cast<const uint4*>(p) + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      } else {
        const uint2 v = __ldcs(static_cast<const uint2*>(p) + i);
        w[2 * i] = v.x; w[2 * i + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void store(void* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (PIECE == 16) {
        static_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      } else {
        static_cast<uint2*>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
      }
    }
  }
};

template <typename T, int E>
__device__ __forceinline__ void unpack(const Vec<E * sizeof(T)>& v, float (&x)[E]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = __uint_as_float(v.w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      x[2 * j] = __uint_as_float(v.w[j] << 16);
      x[2 * j + 1] = __uint_as_float(v.w[j] & 0xffff0000u);
    }
  }
}

template <typename T, int E>
__device__ __forceinline__ void pack(const float (&x)[E], Vec<E * sizeof(T)>& v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < E; ++j) v.w[j] = __float_as_uint(x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < E / 2; ++j) v.w[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
  }
}

constexpr int64_t kNoToken = INT64_MIN;
constexpr int kBatch = 4;  // heads a half-warp has in flight

// What a half-warp does of one part (q, k or v) of its token: n heads, from src / dst on, a head apart
// by d / dst_step.
template <typename T>
struct Part {
  const T* src;
  T* dst;
  int64_t dst_step;
  int n;
  const T* w;  // weights of the norm, or NULL
};

template <typename T, int E>
__device__ __forceinline__ void load_heads(Vec<E * sizeof(T)> (&v)[kBatch], const Part<T>& p, int h, int e0) {
#pragma unroll
  for (int i = 0; i < kBatch; ++i)
    if (h + i < p.n) v[i].load(p.src + (h + i) * (16 * E) + e0);
}

// The heads of one part, the first kBatch of them loaded.  Channel j of a lane becomes
//   x_j (c_j w_j) inv + x_partner (s_j w_partner) inv
// so the weights join the cosines and signed sines, once for all heads, and the partner's value travels as it
// was read, two bf16 in a shuffle.  Past the rotated channels (of which ALL has none: 2 us of the prompt below) c
// is 1 and the second product left out, whatever it is.
template <typename T, int E, bool ROTATE, bool ALL>
__device__ __forceinline__ void run_heads(Vec<E * sizeof(T)> (&v)[kBatch], const Part<T>& p, const float2* cs, int half,
                                          bool interleaved, float eps, int e0, uint32_t mask) {
  constexpr int D = 16 * E;
  using V = Vec<E * sizeof(T)>;
  float c[E], s[E];
  int partner = threadIdx.x & 31;
  const bool past = !ALL && e0 >= 2 * half;
  if constexpr (ROTATE) {
    // (E divides half, so a lane lies wholly in the first half, the second, or past both)
    const bool first = e0 < half, second = !first && e0 < 2 * half;
    const int shift = interleaved ? 0 : first ? half : second ? -half : 0;  // channels to the partner's
    partner += shift / E;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int q = interleaved ? (e0 + j) >> 1 : first ? e0 + j : e0 - half + j;
      const float2 f = first || second ? cs[q] : make_float2(1.f, 0.f);
      c[j] = f.x;
      s[j] = (interleaved ? !(j & 1) : first) ? -f.y : f.y;
    }
    if (p.w) {
      V wv, wp;
      wv.load(p.w + e0);
      wp.load(p.w + e0 + shift);
      float x[E], y[E];
      unpack<T, E>(wv, x);
      unpack<T, E>(wp, y);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        c[j] *= x[j];
        s[j] *= interleaved ? y[j ^ 1] : y[j];
      }
    }
  }
  for (int h = 0;;) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= p.n) break;
      if constexpr (ROTATE) {
        float x[E], y[E];
        unpack<T, E>(v[i], x);
        if (interleaved) {
#pragma unroll
          for (int j = 0; j < E; ++j) y[j] = x[j ^ 1];
        } else {
          V o;
#pragma unroll
          for (int j = 0; j < (int)(E * sizeof(T) / 4); ++j) o.w[j] = __shfl_sync(mask, v[i].w[j], partner);
          unpack<T, E>(o, y);
        }
        float inv = 1.f;
        if (p.w) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < E; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
          inv = rsqrtf(ss * (1.f / D) + eps);
        }
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = (x[j] * c[j] + (past ? -0.f : y[j] * s[j])) * inv;
        pack<T, E>(x, v[i]);
      }
      v[i].store(p.dst + (h + i) * p.dst_step + e0);
    }
    h += kBatch;
    if (h >= p.n) break;
    load_heads<T, E>(v, p, h, e0);
  }
}

// One CTA: TOK neighbouring tokens of one (layer, sequence), or (SHARED) of all of them, 16 / TOK half-warps
// on each; `count` is the chunks of TOK tokens of a sequence, or all tokens.  It takes one of
// `head_parts` equal shares of their heads.  E = d / 16 channels a lane.  A lane keeps its cosines and
// sines for all heads of its token and has kBatch heads' loads in flight, the first ones before the
// angles are formed.  33,024 tokens of 28 + 4 + 4 heads, d = 128, bf16: 124 us, 4.9 TB/s of 6.46; eight
// tokens a CTA took 205 us with cosines and sines read from shared memory for each head, 173 with a
// shuffle for each normalised channel, 148 as it is.
template <typename T, int E, int TOK, bool SHARED>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && TOK > 1 ? 3 : 1) qk_norm_rope_kernel(const RopeArgs a, int count, int head_parts) {
  __shared__ float2 cs[TOK][8 * E];
  __shared__ int64_t at[SHARED ? TOK : 1];
  pdl_wait();  // memory of earlier kernels in the stream is visible from here on
  pdl_trigger();
  constexpr int D = 16 * E, HS = kHeadsAtOnce / TOK;
  const int part = blockIdx.x % head_parts, rest = blockIdx.x / head_parts;
  const int hw = threadIdx.x >> 4, e0 = (threadIdx.x & 15) * E;
  const uint32_t mask = 0xffffu << (threadIdx.x & 16);
  // this half-warp's token: row r of sequence b in layer l, cache row base + r
  const int t = hw / HS;
  const int tok = rest * TOK + t;  // (SHARED)
  const int lb = SHARED ? (tok < count ? tok / a.rows : 0) : rest / count;
  const int r = SHARED ? tok - lb * a.rows : (rest - lb * count) * TOK + t;
  const int l = lb / a.B, b = lb - l * a.B;
  bool ok = !SHARED || tok < count;
  int64_t base = 0;
  int n = 0;
  if (ok) {
    n = a.n_rows ? a.n_rows[b] : a.rows;
    base = (a.len ? (int64_t)a.len[b] : 0) + a.pos_offset;
    const bool counted = n >= 0 && n <= a.rows;
    const bool fits = !(a.k_in || a.v_in) || (base >= 0 && base + n <= a.cap);
    if (!(counted && fits) && r == 0 && part == 0 && (threadIdx.x & 15) == 0)
      flag_error(a.err, counted ? STD_DEVERR_CAPACITY : STD_DEVERR_LENGTH);
    ok = counted && fits && r < n;
    if (!SHARED && !(counted && fits && r - t < n)) return;  // (the same for the CTA: none of its tokens)
    if (ok && (a.k_in || a.v_in)) ok = STD_DCHECK(base >= 0 && base + r < a.cap, a.err);
  }
  // its place in `pos`, or its position
  if constexpr (SHARED) {
    if ((threadIdx.x & 15) == 0 && hw % HS == 0) at[t] = !ok ? kNoToken : a.pos ? (int64_t)b * a.rows + r : base + r;
  }

  // its share of the heads, in the order q, k, v
  const int nq = a.q_in ? a.Hq : 0, nk = a.k_in ? a.Hkv : 0, nv = a.v_in ? a.Hkv : 0;
  const int heads = nq + nk + nv, shares = HS * head_parts, share = part * HS + hw % HS;
  const int h0 = (int)((int64_t)heads * share / shares);
  const int h1 = ok ? (int)((int64_t)heads * (share + 1) / shares) : h0;
  auto part_of = [&](int which) {  // 0, 1, 2: q, k, v
    const int64_t tok = (int64_t)lb * a.rows + r;
    Part<T> p;
    if (which == 0) {
      p.src = static_cast<const T*>(a.q_in) + tok * a.q_stride + h0 * D;
      p.dst = static_cast<T*>(a.q_out) + (((int64_t)lb * a.Hq + h0) * a.rows + r) * D;
      p.dst_step = (int64_t)a.rows * D;
      p.n = min(h1, nq) - h0;
      p.w = static_cast<const T*>(a.q_w);
    } else {
      const int off = which == 1 ? nq : nq + nk, h = max(h0 - off, 0);
      p.src = static_cast<const T*>(which == 1 ? a.k_in : a.v_in) + tok * (which == 1 ? a.k_stride : a.v_stride) + h * D;
      p.dst = static_cast<T*>(which == 1 ? a.k_cache : a.v_cache) + (((int64_t)lb * a.Hkv + h) * a.cap + base + r) * D;
      p.dst_step = a.cap * D;
      p.n = min(h1 - off, which == 1 ? nk : nv) - h;
      p.w = which == 1 ? static_cast<const T*>(a.k_w) : nullptr;
    }
    if (p.w) p.w += (int64_t)l * D;
    return p;
  };
  // the first loads go out before the angles are formed
  Vec<E * sizeof(T)> x[kBatch];
  const int start = h0 < nq ? 0 : h0 < nq + nk ? 1 : 2;
  if (h0 < h1) load_heads<T, E>(x, part_of(start), 0, e0);

  const int half = a.rot_dim >> 1;
  if (SHARED && !__syncthreads_or(ok)) return;
  const int filled = SHARED ? TOK : min(TOK, n - (r - t));
  for (int i = threadIdx.x; i < filled * half; i += kThreads) {
    const int tt = i / half, p = i - tt * half;
    if (SHARED && at[tt] == kNoToken) continue;
    const int axis = p < a.sec_end[0] ? 0 : p < a.sec_end[1] ? 1 : 2;
    const int64_t x = SHARED ? at[tt] : (a.pos ? (int64_t)b * a.rows : base) + (r - t + tt);
    const double where = a.pos ? (double)a.pos[(int64_t)axis * a.B * a.rows + x] : (double)x;
    double turns = where * a.inv_freq[p] * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    cs[tt][p] = make_float2(c, s);
  }
  __syncthreads();

  if (h0 >= h1) return;
#pragma unroll 1
  for (int which = start; which < 2; ++which) {
    const Part<T> p = part_of(which);
    if (p.n <= 0) continue;
    if (which != start) load_heads<T, E>(x, p, 0, e0);
    if (a.rot_dim == D)
      run_heads<T, E, true, true>(x, p, cs[t], half, a.interleaved, a.eps, e0, mask);
    else
      run_heads<T, E, true, false>(x, p, cs[t], half, a.interleaved, a.eps, e0, mask);
  }
  const Part<T> p = part_of(2);
  if (p.n > 0) {  // (values are copied bit for bit)
    if (start != 2) load_heads<T, E>(x, p, 0, e0);
    run_heads<T, E, false, true>(x, p, cs[t], half, a.interleaved, a.eps, e0, mask);
  }
}

template <typename T, int E>
cudaError_t launch(const RopeArgs& a, int sms, cudaStream_t s) {
  const int heads = (a.q_in ? a.Hq : 0) + (a.k_in ? a.Hkv : 0) + (a.v_in ? a.Hkv : 0);
  const int64_t tokens = (int64_t)a.L * a.B * a.rows;
  // Tokens of a CTA: as few as fill the device about twice (once for few heads).  The fewer a CTA takes,
  // the more half-warps share a token's heads and the sooner it is done; but each works out the token's
  // coefficients for itself, which many CTAs feel.  28 + 4 + 4 heads, d = 128, bf16, us with 1 / 2 / 4 / 8 /
  // 16 tokens a CTA: 8 tokens 3.3 / 4.7 / 7.3 / 9.9 / 11.7; 700 tokens 21.9 / 7.0 / 9.1 / 11.0 / 14.7; 2,800 tokens
  // 83 / 25.5 / 22.6 / 18.8 / 21.2; 11,200 tokens 323 / 83 / 73 / 62 / 49.
  const int64_t most = (int64_t)sms * (heads > kHeadsAtOnce ? 12 : 6) / 5;
  auto go = [&](auto tok) {
    constexpr int TOK = decltype(tok)::value;
    // Sequences of few tokens share CTAs where chunks of their own would leave more than a tenth of the places
    // empty.  28 + 4 + 4 heads, d = 128, bf16, us with chunks of their own / shared: 1,024 sequences of one
    // token 22.3 / 11.7, 28 layers x 64 sequences of one 42 / 17, 256 sequences of 9 26.4 / 17.9; where chunks
    // are full the divisions and the table of tokens cost 2 in 100 (33,024 tokens 124.6 / 127.4).
    const int64_t chunks = (a.rows + TOK - 1) / TOK;
    if (10 * (chunks * TOK - a.rows) > chunks * TOK)
      return launch_pdl(qk_norm_rope_kernel<T, E, TOK, true>, dim3((unsigned)((tokens + TOK - 1) / TOK)), dim3(kThreads), 0,
                        s, a, (int)tokens, 1);
    return launch_pdl(qk_norm_rope_kernel<T, E, TOK, false>, dim3((unsigned)((int64_t)a.L * a.B * chunks)), dim3(kThreads),
                      0, s, a, (int)chunks, 1);
  };
  // one token: up to kHeadsAtOnce heads a CTA
  const int parts = (heads + kHeadsAtOnce - 1) / kHeadsAtOnce;
  if (tokens * parts <= most)
    return launch_pdl(qk_norm_rope_kernel<T, E, 1, false>, dim3((unsigned)(tokens * parts)), dim3(kThreads), 0, s, a, a.rows,
                      parts);
  if (tokens <= 2 * most) return go(std::integral_constant<int, 2>());
  if (tokens <= 4 * most) return go(std::integral_constant<int, 4>());
  if (tokens <= 8 * most) return go(std::integral_constant<int, 8>());
  return go(std::integral_constant<int, 16>());
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, int sms, cudaStream_t s) {
  if (a.dtype == STD_F32) {
    switch (a.d) {
      case 32: return launch<float, 2>(a, sms, s);
      case 64: return launch<float, 4>(a, sms, s);
      case 96: return launch<float, 6>(a, sms, s);
      case 128: return launch<float, 8>(a, sms, s);
    }
  } else {
    switch (a.d) {
      case 64: return launch<__nv_bfloat16, 4>(a, sms, s);
      case 128: return launch<__nv_bfloat16, 8>(a, sms, s);
    }
  }
  return cudaErrorInvalidValue;
}

}  // namespace stdb
