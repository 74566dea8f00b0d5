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

// One CTA: TOK neighbouring tokens of one (layer, sequence), and one of `head_parts` equal
// shares of their heads.  E = d / 16 channels a lane.
template <typename T, int E, int TOK>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a, int chunks, int head_parts) {
  __shared__ float2 cs[TOK][8 * E];
  pdl_wait();  // memory of earlier kernels in the stream is visible from here on
  pdl_trigger();
  constexpr int D = 16 * E;
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

  const int nq = a.q_in ? a.Hq : 0, nk = a.k_in ? a.Hkv : 0, nv = a.v_in ? a.Hkv : 0;
  const int heads = nq + nk + nv;
  const int h0 = (int)((int64_t)heads * part / head_parts), h1 = (int)((int64_t)heads * (part + 1) / head_parts);
  const int items = ntok * (h1 - h0);
  const int lane = threadIdx.x & 15;
  const uint32_t mask = 0xffffu << (threadIdx.x & 16);
  const int e0 = lane * E;
  for (int it = threadIdx.x >> 4; it < items; it += kHeadsAtOnce) {
    const int t = it / (h1 - h0);
    int h = h0 + it - t * (h1 - h0);
    const int64_t tok = (int64_t)lb * a.rows + r0 + t;
    const T* src;
    T* dst;
    const T* w = nullptr;
    bool rotate = true;
    if (h < nq) {
      src = static_cast<const T*>(a.q_in) + tok * a.q_stride + h * D;
      dst = static_cast<T*>(a.q_out) + (((int64_t)lb * a.Hq + h) * a.rows + r0 + t) * D;
      w = static_cast<const T*>(a.q_w);
    } else if (h < nq + nk) {
      h -= nq;
      src = static_cast<const T*>(a.k_in) + tok * a.k_stride + h * D;
      dst = static_cast<T*>(a.k_cache) + (((int64_t)lb * a.Hkv + h) * a.cap + base + r0 + t) * D;
      w = static_cast<const T*>(a.k_w);
    } else {
      h -= nq + nk;
      src = static_cast<const T*>(a.v_in) + tok * a.v_stride + h * D;
      dst = static_cast<T*>(a.v_cache) + (((int64_t)lb * a.Hkv + h) * a.cap + base + r0 + t) * D;
      rotate = false;
    }
    Vec<E * sizeof(T)> v;
    v.load(src + e0);
    if (rotate) {  // (values are copied bit for bit)
      float x[E];
      unpack<T, E>(v, x);
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
        Vec<E * sizeof(T)> wv;
        wv.load(w + (int64_t)l * D + e0);
        float wf[E];
        unpack<T, E>(wv, wf);
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = x[j] * inv * wf[j];
      }
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const int p = lane * (E / 2) + j;
          if (p < half) {
            const float2 f = cs[t][p];
            const float u = x[2 * j], z = x[2 * j + 1];
            x[2 * j] = u * f.x - z * f.y;
            x[2 * j + 1] = z * f.x + u * f.y;
          }
        }
      } else {
        // E divides half, so a lane lies wholly in the first half, the second, or past both
        const int shift = half / E;
        const bool first = e0 < half, second = !first && e0 < a.rot_dim;
        const int partner = (threadIdx.x & 31) + (first ? shift : second ? -shift : 0);
        const float sign = first ? -1.f : 1.f;
        const int p0 = first ? e0 : e0 - half;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const float z = __shfl_sync(mask, x[j], partner);
          if (first || second) {
            const float2 f = cs[t][p0 + j];
            x[j] = x[j] * f.x + sign * z * f.y;
          }
        }
      }
      pack<T, E>(x, v);
    }
    v.store(dst + e0);
  }
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
