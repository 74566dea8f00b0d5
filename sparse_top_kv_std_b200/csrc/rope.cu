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

constexpr int kBatch = 4;  // heads a half-warp has in flight

// Heads [h0, h1) of one part (q, k or v) of one token, every `step`-th, by one half-warp: src and dst are
// the token's head h0, a head apart by src_step / dst_step.  (c, s): cosines and signed sines of the
// lane's channels.
template <typename T, int E, bool ROTATE>
__device__ __forceinline__ void run_heads(const T* src, int64_t src_step, T* dst, int64_t dst_step, int n, const T* w,
                                          float eps, const float (&c)[E], const float (&s)[E], int partner,
                                          bool interleaved, uint32_t mask) {
  constexpr int D = 16 * E;
  using V = Vec<E * sizeof(T)>;
  float wf[E];
  if (ROTATE && w) {
    V v;
    v.load(w);
    unpack<T, E>(v, wf);
  }
  for (int h = 0; h < n; h += kBatch) {
    V v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (h + i < n) v[i].load(src + (h + i) * src_step);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= n) break;
      if constexpr (ROTATE) {
        float x[E];
        unpack<T, E>(v[i], x);
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < E; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
          const float inv = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
          for (int j = 0; j < E; ++j) x[j] = x[j] * inv * wf[j];
        }
        if (interleaved) {
#pragma unroll
          for (int j = 0; j < E; j += 2) {
            const float y = x[j], z = x[j + 1];
            x[j] = y * c[j] + z * s[j];
            x[j + 1] = z * c[j + 1] + y * s[j + 1];
          }
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const float z = __shfl_sync(mask, x[j], partner);
            x[j] = x[j] * c[j] + z * s[j];
          }
        }
        pack<T, E>(x, v[i]);
      }
      v[i].store(dst + (h + i) * dst_step);
    }
  }
}

// One CTA: TOK neighbouring tokens of one (layer, sequence), 16 / TOK half-warps on each, and one of
// `head_parts` equal shares of their heads.  E = d / 16 channels a lane.  A lane keeps the cosines and
// sines of its channels for all heads of its token, and has kBatch heads' loads in flight.
// (33,024 tokens of 28 + 4 + 4 heads, d = 128, bf16: from shared memory for each head 205 us.)
template <typename T, int E, int TOK>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a, int chunks, int head_parts) {
  __shared__ float2 cs[TOK][8 * E];
  pdl_wait();  // memory of earlier kernels in the stream is visible from here on
  pdl_trigger();
  constexpr int D = 16 * E, HS = kHeadsAtOnce / TOK;
  const int part = blockIdx.x % head_parts;
  const int rest = blockIdx.x / head_parts;
  const int lb = rest / chunks, b = lb % a.B, l = lb / a.B;
  const int r0 = (rest % chunks) * TOK;
  const int n = a.n_rows ? a.n_rows[b] : a.rows;
  const int64_t base = (a.len ? (int64_t)a.len[b] : 0) + a.pos_offset;
  if (n < 0 || n > a.rows) {
    if (r0 == 0 && part == 0 && threadIdx.x == 0) flag_error(a.err, STD_DEVERR_LENGTH);
    return;
  }
  if ((a.k_in || a.v_in) && (base < 0 || base + n > a.cap)) {
    if (r0 == 0 && part == 0 && threadIdx.x == 0) flag_error(a.err, STD_DEVERR_CAPACITY);
    return;
  }
  if (r0 >= n) return;
  const int ntok = n - r0 < TOK ? n - r0 : TOK;
  const int half = a.rot_dim >> 1;
  for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
    const int t = i / half, p = i - t * half;
    const int axis = p < a.sec_end[0] ? 0 : p < a.sec_end[1] ? 1 : 2;
    const double at = a.pos ? (double)a.pos[((int64_t)axis * a.B + b) * a.rows + r0 + t] : (double)(base + r0 + t);
    double turns = at * a.inv_freq[p] * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    cs[t][p] = make_float2(c, s);
  }
  __syncthreads();

  const int hw = threadIdx.x >> 4, t = hw / HS;
  if (t >= ntok) return;
  const int lane = threadIdx.x & 15, e0 = lane * E;
  const uint32_t mask = 0xffffu << (threadIdx.x & 16);
  // Channel j of the lane becomes x_j c_j + x_partner s_j; past the rotated channels c = 1, s = 0.
  // (E divides half, so a lane lies wholly in the first half, the second, or past both.)
  float c[E], s[E];
  int partner = threadIdx.x & 31;
  if (a.interleaved) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int p = (e0 + j) >> 1;
      const float2 f = p < half ? cs[t][p] : make_float2(1.f, 0.f);
      c[j] = f.x;
      s[j] = j & 1 ? f.y : -f.y;
    }
  } else {
    const bool first = e0 < half, second = !first && e0 < a.rot_dim;
    const int shift = half / E;
    partner += first ? shift : second ? -shift : 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float2 f = first ? cs[t][e0 + j] : second ? cs[t][e0 - half + j] : make_float2(1.f, 0.f);
      c[j] = f.x;
      s[j] = first ? -f.y : f.y;
    }
  }

  // this half-warp's share of the heads, in the order q, k, v
  const int nq = a.q_in ? a.Hq : 0, nk = a.k_in ? a.Hkv : 0, nv = a.v_in ? a.Hkv : 0;
  const int heads = nq + nk + nv, shares = HS * head_parts, share = part * HS + hw % HS;
  const int h0 = (int)((int64_t)heads * share / shares), h1 = (int)((int64_t)heads * (share + 1) / shares);
  const int64_t tok = (int64_t)lb * a.rows + r0 + t;
  const int64_t row = base + r0 + t, q_step = (int64_t)a.rows * D, c_step = a.cap * D;
  const int q1 = min(h1, nq), k0 = max(h0, nq), k1 = min(h1, nq + nk), v0 = max(h0, nq + nk);
  if (h0 < q1)
    run_heads<T, E, true>(static_cast<const T*>(a.q_in) + tok * a.q_stride + h0 * D + e0, D,
                          static_cast<T*>(a.q_out) + ((int64_t)lb * a.Hq + h0) * q_step + (int64_t)(r0 + t) * D + e0,
                          q_step, q1 - h0, a.q_w ? static_cast<const T*>(a.q_w) + (int64_t)l * D + e0 : nullptr, a.eps, c,
                          s, partner, a.interleaved, mask);
  if (k0 < k1)
    run_heads<T, E, true>(static_cast<const T*>(a.k_in) + tok * a.k_stride + (k0 - nq) * D + e0, D,
                          static_cast<T*>(a.k_cache) + ((int64_t)lb * a.Hkv + k0 - nq) * c_step + row * D + e0, c_step,
                          k1 - k0, a.k_w ? static_cast<const T*>(a.k_w) + (int64_t)l * D + e0 : nullptr, a.eps, c, s,
                          partner, a.interleaved, mask);
  if (v0 < h1)  // (values are copied bit for bit)
    run_heads<T, E, false>(static_cast<const T*>(a.v_in) + tok * a.v_stride + (v0 - nq - nk) * D + e0, D,
                           static_cast<T*>(a.v_cache) + ((int64_t)lb * a.Hkv + v0 - nq - nk) * c_step + row * D + e0,
                           c_step, h1 - v0, nullptr, 0.f, c, s, partner, false, mask);
}

template <typename T, int E>
cudaError_t launch(const RopeArgs& a, int sms, cudaStream_t s) {
  const int heads = (a.q_in ? a.Hq : 0) + (a.k_in ? a.Hkv : 0) + (a.v_in ? a.Hkv : 0);
  const int64_t tokens = (int64_t)a.L * a.B * a.rows;
  constexpr int TOK = 8;
  if (tokens < 4 * (int64_t)sms) {  // few tokens: a CTA takes one token and up to kHeadsAtOnce of its heads
    const int parts = (heads + kHeadsAtOnce - 1) / kHeadsAtOnce;
    return launch_pdl(qk_norm_rope_kernel<T, E, 1>, dim3((unsigned)(tokens * parts)), dim3(kThreads), 0, s, a, a.rows,
                      parts);
  }
  const int chunks = (a.rows + TOK - 1) / TOK;
  return launch_pdl(qk_norm_rope_kernel<T, E, TOK>, dim3((unsigned)((int64_t)a.L * a.B * chunks)), dim3(kThreads), 0, s,
                    a, chunks, 1);
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
