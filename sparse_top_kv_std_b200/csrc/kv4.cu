// Rows of a 4-bit K/V cache written from bf16 / fp32 rows and read back (format: kv4.cuh).
//
//   m = bf16(min x),  s = bf16(fl32(max x - m) / 15),  c = clamp(rne(fl32(x - m) / s), 0, 15)
//
// with the quotient rounded as the exact quotient of its two fp32 operands would be, so that a
// code does not depend on how the division is carried out.  A group that holds an infinity or a
// NaN gets m = NaN, s = 0: all its channels read back as NaN.  A group whose range is too
// small for a bf16 scale gets s = 0 and reads back as m.
//
// Both directions stream: 2 d values in, d + d / 8 bytes out for the K and V row of a head.
// A lane holds one code word (8 channels), so the codes of a row are one coalesced store, and a
// group's extremes are three shuffles over its eight lanes.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace stdb {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows a lane group has in flight

__device__ __forceinline__ float min_nan(float a, float b) {  // NaN if either is
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 u = __ldcs(reinterpret_cast<const float4*>(p)), v = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w; x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                              pack_bf16(x[6], x[7]));
  }
}

// The code of one channel: diff / s rounded half to even, exactly.  `k` is within one of the
// answer; diff - k s is exact in fp32 next to a border (k s has at most 12 bits, and both
// terms are multiples of the smaller one's last bit, at most 24 bits apart).
__device__ __forceinline__ float settle(float k, float diff, float s) {
  const float r = fmaf(-k, s, diff), h = 0.5f * s;
  const bool odd = ((int)k & 1) != 0;
  if (r > h || (r == h && odd)) k += 1.f;
  else if (r < -h || (r == -h && odd)) k -= 1.f;
  return k;
}

// Where the rows of one call come from and go to: rows r < count of sequence b.
struct RowSpan {
  int n;        // rows of this sequence
  int64_t pos;  // their first cache row
};
__device__ __forceinline__ bool row_span(const Kv4Args& a, int b, RowSpan* sp) {
  sp->n = a.count ? a.count[b] : a.max_n;
  sp->pos = (a.begin ? (int64_t)a.begin[b] : 0) + a.pos_offset;
  const int64_t limit = a.at_pos && a.rows_cap < a.cap ? a.rows_cap : a.cap;
  return sp->n >= 0 && sp->n <= a.max_n && sp->pos >= 0 && sp->pos + sp->n <= limit;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4Args a, int chunks) {
  constexpr int LPR = D / 8;               // lanes of a row
  constexpr int RPB = kThreads / LPR;      // rows of a CTA at a time
  pdl_wait();  // memory of earlier kernels in the stream is visible from here on
  pdl_trigger();
  const int which = blockIdx.x & 1;
  const int rest = blockIdx.x >> 1;
  const int prob = rest / chunks, chunk = rest - prob * chunks;
  const int b = (prob / a.Hkv) % a.B;
  RowSpan sp;
  if (!row_span(a, b, &sp)) {
    if (chunk == 0 && which == 0 && threadIdx.x == 0) flag_error(a.err, STD_DEVERR_CAPACITY);
    return;
  }
  const T* src = static_cast<const T*>(which ? a.v : a.k);
  uint32_t* codes = static_cast<uint32_t*>(which ? a.v_codes : a.k_codes);
  uint32_t* scales = static_cast<uint32_t*>(which ? a.v_scales : a.k_scales);
  const int w = threadIdx.x % LPR, grp = D == 128 ? w & 1 : 0, j = D == 128 ? w >> 1 : w;
  const int ch = kv4_word_channel<D>(w);
  const int r0 = chunk * RPB * kUnroll + threadIdx.x / LPR;
  float x[kUnroll][8];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int r = r0 + u * RPB;
    if (r < sp.n) {
      load8<T>(src + ((int64_t)prob * a.rows_cap + (a.at_pos ? sp.pos : 0) + r) * D + ch, x[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int r = r0 + u * RPB;
    float lo = x[u][0], hi = x[u][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = min_nan(lo, x[u][i]);
      hi = max_nan(hi, x[u][i]);
    }
#pragma unroll
    for (int o = D == 128 ? 2 : 1; o < LPR; o <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    __nv_bfloat16 mb = __float2bfloat16_rn(lo);
    float m = __bfloat162float(mb);
    const float range = hi - m;
    __nv_bfloat16 sb = __float2bfloat16_rn(range / 15.f);
    float s = __bfloat162float(sb);
    const bool finite = fabsf(range) <= 3.402823466e38f;  // false for a NaN or an infinity
    uint32_t word = 0;
    if (finite && s > 0.f) {
      // keep 1 / s finite for the smallest scales (exact: a power of two)
      const float up = s < 5.421010862e-20f ? 1.208925820e24f : 1.f;  // 2^-64, 2^80
      const float ss = s * up, inv = 1.f / ss;
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        const float diff = (x[u][i] - m) * up;
        float k = fminf(fmaxf(rintf(diff * inv), 0.f), 16.f);
        k = settle(k, diff, ss);
        word = (word << 4) | (uint32_t)fminf(fmaxf(k, 0.f), 15.f);
      }
    } else {
      s = 0.f;
      sb = __float2bfloat16_rn(0.f);
      if (!finite) mb = __float2bfloat16_rn(__uint_as_float(0x7fc00000u));
    }
    if (r < sp.n && STD_DCHECK(sp.pos + r < a.cap, a.err)) {
      const int64_t row = (int64_t)prob * a.cap + sp.pos + r;
      codes[row * LPR + w] = word;
      if (j == 0)
        scales[row * (D / kKv4Group) + grp] =
            (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(mb) << 16);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Args a, int chunks) {
  constexpr int LPR = D / 8;
  constexpr int RPB = kThreads / LPR;
  pdl_wait();  // memory of earlier kernels in the stream is visible from here on
  pdl_trigger();
  const int which = blockIdx.x & 1;
  const int rest = blockIdx.x >> 1;
  const int prob = rest / chunks, chunk = rest - prob * chunks;
  const int b = (prob / a.Hkv) % a.B;
  RowSpan sp;
  if (!row_span(a, b, &sp)) {
    if (chunk == 0 && which == 0 && threadIdx.x == 0) flag_error(a.err, STD_DEVERR_CAPACITY);
    return;
  }
  T* dst = const_cast<T*>(static_cast<const T*>(which ? a.v : a.k));
  const uint32_t* codes = static_cast<const uint32_t*>(which ? a.v_codes : a.k_codes);
  const uint32_t* scales = static_cast<const uint32_t*>(which ? a.v_scales : a.k_scales);
  const int w = threadIdx.x % LPR, grp = D == 128 ? w & 1 : 0;
  const int ch = kv4_word_channel<D>(w);
  const int r0 = chunk * RPB * kUnroll + threadIdx.x / LPR;
  uint32_t word[kUnroll], sc[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int r = r0 + u * RPB;
    word[u] = sc[u] = 0;
    if (r < sp.n) {
      const int64_t row = (int64_t)prob * a.cap + sp.pos + r;
      word[u] = __ldcs(codes + row * LPR + w);
      sc[u] = __ldg(scales + row * (D / kKv4Group) + grp);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int r = r0 + u * RPB;
    if (r >= sp.n) break;
    const float s = __uint_as_float(sc[u] << 16), m = __uint_as_float(sc[u] & 0xffff0000u);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((word[u] >> (4 * i)) & 15u), s, m);
    store8<T>(dst + ((int64_t)prob * a.rows_cap + r) * D + ch, x);
  }
}

template <typename T, int D>
cudaError_t launch(const Kv4Args& a, bool read, cudaStream_t s) {
  constexpr int per_cta = kThreads / (D / 8) * kUnroll;
  const int chunks = (a.max_n + per_cta - 1) / per_cta;
  const dim3 grid((unsigned)(2 * (int64_t)a.L * a.B * a.Hkv * chunks));
  if (read) return launch_pdl(kv4_read_kernel<T, D>, grid, dim3(kThreads), 0, s, a, chunks);
  return launch_pdl(kv4_write_kernel<T, D>, grid, dim3(kThreads), 0, s, a, chunks);
}

}  // namespace

cudaError_t launch_kv4(const Kv4Args& a, bool read, cudaStream_t s) {
  if (a.max_n <= 0) return cudaSuccess;
  if (a.dtype == STD_F32) return a.d == 128 ? launch<float, 128>(a, read, s) : launch<float, 64>(a, read, s);
  return a.d == 128 ? launch<__nv_bfloat16, 128>(a, read, s) : launch<__nv_bfloat16, 64>(a, read, s);
}

}  // namespace stdb
