// Rows of a 4-bit K/V cache written from bf16 / fp32 rows and read back (format: kv4.cuh).
//
//   m = bf16(min x),  s = bf16(fl32(max x - m) / 15),  c = clamp(rne(fl32(x - m) / s), 0, 15)
//
// with the quotient rounded as the exact quotient of its two fp32 operands would be, so that a
// code does not depend on how the division is carried out.  A group that holds an infinity or a
// NaN gets m = NaN, s = 0: all its channels read back as NaN.  A group whose range is too
// small for a bf16 scale gets s = 0 and reads back as m.
//
// Both directions stream: 2 d values in, d + d / 8 bytes out for the K and V row of a head, and the
// instructions on the way are what is hard to hide: at full HBM rate an SM has about 13 issue slots
// for a bf16 channel.  When writing a lane holds 16 channels of a group (four lanes a group: two
// shuffles for each extreme, and a group's scale is worked out four times, not eight), and a code is
// three instructions without a division, a conversion or a branch (code_word).
// 143,616 rows of 4 heads, d = 128, bf16 (377 MB): written in 72.9 us (86.5 with nine instructions a
// code; 78.4 with three CTAs an SM), read back in 58.2, the rate of a copy (61.3 with 8 channels a lane).
// That is 12.8 and 6.7 instructions a channel.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace stdb {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows a lane group has in flight

__device__ __forceinline__ float min_nan(float a, float b, float c) {  // NaN if one is
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 16 channels as they were read.
template <typename T>
struct Raw16 {
  static constexpr int N = 4 * sizeof(T);  // 32-bit words
  uint32_t w[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  }
  __device__ __forceinline__ void get(float (&x)[2][8]) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (sizeof(T) == 4) x[i / 8][i % 8] = __uint_as_float(w[i]);
      else x[i / 8][i % 8] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
};

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

// Codes of 8 channels, as one word, two channels an instruction: d = fl32(x - m), q = d / s, and 1.5 2^23 added
// to q leaves its nearest integer, ties to even, in the last bits.  That is the exact quotient's rounding (a
// product by the reciprocal and one correction by its remainder, after Markstein, 1990):
// q0 = d (1 / s) is off by some units in the last place, its remainder d - q0 s is exact (s has 8 bits), and
// q0 + remainder (1 / s) rounds to the quotient to nearest.  An exact tie T = k + 1/2 comes out as T (d = T s
// has 13 bits).  A d next to T s is at least a unit in the last place off, so q is off by more than
// 2^-24 (1 + 2^-8) of T, as s is at most 255/128 of a power of two; fp32 numbers that round to T are nearer.
template <bool CLAMP>
__device__ __forceinline__ uint32_t code_word(const float (&x)[8], float m, float s, float inv) {
  const f32x2 m2 = f2_make(-m, -m), s2 = f2_make(-s, -s), i2 = f2_make(inv, inv), one = f2_make(12582912.f, 12582912.f);
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    f32x2 d = f2_add(f2_make(x[i], x[i + 4]), m2);
    float a, b;
    if constexpr (CLAMP) {
      f2_split(d, a, b);
      d = f2_make(fmaxf(a, 0.f), fmaxf(b, 0.f));
    }
    const f32x2 q = f2_mul(d, i2);
    f2_split(f2_add(f2_fma(f2_fma(q, s2, d), i2, q), one), a, b);
    lo = lo * 16 + __float_as_uint(a);
    hi = hi * 16 + __float_as_uint(b);
  }
  return lo + hi * 65536 - 0x11111111u * 0x4b400000u;  // less the bits of 1.5 2^23 in every place
}

// The same for a scale so small that 1 / s or the products above leave the normal numbers: scaled up
// by a power of two, quotients and remainders one at a time.
__device__ __noinline__ uint32_t code_word_tiny(const float* diff, float s) {
  const float up = 1.208925820e24f;  // 2^80
  uint32_t word = 0;
  for (int i = 7; i >= 0; --i) {
    const float d = diff[i] * up, t = s * up;
    float k = fminf(rintf(d / t), 16.f);
    const float r = fmaf(-k, t, d), h = 0.5f * t;
    const bool odd = ((int)k & 1) != 0;
    if (r > h || (r == h && odd)) k += 1.f;
    else if (r < -h || (r == -h && odd)) k -= 1.f;
    word = (word << 4) | (uint32_t)fminf(fmaxf(k, 0.f), 15.f);
  }
  return word;
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
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) kv4_write_kernel(const Kv4Args a, int chunks) {
  constexpr int GR = D / kKv4Group;
  constexpr int LPR = D / 16;          // lanes of a row: word pairs (2 j, 2 j + 1) of one group
  constexpr int RPB = kThreads / LPR;  // rows of a CTA at a time
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
  const int j = threadIdx.x % 4, grp = GR == 2 ? threadIdx.x / 4 % 2 : 0;
  const int ch = 64 * grp + 16 * j;
  const int r0 = chunk * RPB * kUnroll + threadIdx.x / LPR;
  if (r0 - threadIdx.x / LPR >= sp.n) return;
  Raw16<T> raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int r = min(r0 + u * RPB, sp.n - 1);  // (past the end: a row that is not stored)
    raw[u].load(src + ((int64_t)prob * a.rows_cap + (a.at_pos ? sp.pos : 0) + r) * D + ch);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if ((r0 & ~(32 / LPR - 1)) + u * RPB >= sp.n) break;  // (none of the warp's rows)
    float x[2][8];
    raw[u].get(x);
    float lo = x[0][0], hi = lo;
#pragma unroll
    for (int i = 1; i < 16; i += 2) {
      const float y = x[i / 8][i % 8], z = x[(i + 1) / 8 % 2][(i + 1) % 8];  // (the last z is the first again)
      lo = min_nan(lo, y, z);
      hi = max_nan(hi, y, z);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, lo, o), z = __shfl_xor_sync(0xffffffffu, hi, o);
      lo = min_nan(lo, lo, y);
      hi = max_nan(hi, hi, z);
    }
    const float m = __bfloat162float(__float2bfloat16_rn(lo));
    const float range = hi - m;
    float s = __bfloat162float(__float2bfloat16_rn(range / 15.f));
    const bool finite = fabsf(range) <= 3.402823466e38f;  // false for a NaN or an infinity
    uint32_t w0 = 0, w1 = 0;
    if (finite && s > 0.f) {
      constexpr bool CLAMP = sizeof(T) == 4;  // (bf16: m is the smallest x)
      if (s >= 7.888609052e-31f) {  // 2^-100
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        w0 = code_word<CLAMP>(x[0], m, s, inv);
        w1 = code_word<CLAMP>(x[1], m, s, inv);
      } else {
        float y[16];  // (a copy: only this path's needs an address)
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = CLAMP ? fmaxf(x[i / 8][i % 8] - m, 0.f) : x[i / 8][i % 8] - m;
        w0 = code_word_tiny(y, s);
        w1 = code_word_tiny(y + 8, s);
      }
    } else {
      s = 0.f;
    }
    const int r = r0 + u * RPB;
    if (r < sp.n && STD_DCHECK(sp.pos + r < a.cap, a.err)) {
      const int64_t row = (int64_t)prob * a.cap + sp.pos + r;
      uint32_t* q = codes + row * (D / 8);
      if constexpr (GR == 2) {
        q[4 * j + grp] = w0;
        q[4 * j + 2 + grp] = w1;
      } else {
        *reinterpret_cast<uint2*>(q + 2 * j) = make_uint2(w0, w1);
      }
      if (j == 0) scales[row * GR + grp] = (__float_as_uint(s) >> 16) | (finite ? __float_as_uint(m) : 0x7fc00000u);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Args a, int chunks) {
  constexpr int GR = D / kKv4Group;
  constexpr int LPR = D / 16;  // a lane reads two words of a row: at d = 128 one of each group
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
  const int w = threadIdx.x % LPR;
  const int r0 = chunk * (RPB * kUnroll) + threadIdx.x / LPR;
  T* dst = const_cast<T*>(static_cast<const T*>(which ? a.v : a.k)) + (int64_t)prob * a.rows_cap * D;
  const int64_t first = (int64_t)prob * a.cap + sp.pos;
  const uint32_t* codes = static_cast<const uint32_t*>(which ? a.v_codes : a.k_codes) + first * (D / 8) + 2 * w;
  const uint32_t* scales = static_cast<const uint32_t*>(which ? a.v_scales : a.k_scales) + first * GR;
  uint2 word[kUnroll];
  uint32_t sc[kUnroll][GR];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int r = r0 + u * RPB;
    if (r < sp.n && STD_DCHECK(sp.pos + r < a.cap, a.err)) {
      word[u] = __ldcs(reinterpret_cast<const uint2*>(codes + (int64_t)r * (D / 8)));
      if constexpr (GR == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(scales + (int64_t)r * 2));
        sc[u][0] = x.x; sc[u][1] = x.y;
      } else {
        sc[u][0] = __ldg(scales + r);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int r = r0 + u * RPB;
    if (r >= sp.n || !STD_DCHECK(r < a.rows_cap && sp.pos + r < a.cap, a.err)) return;
    float x[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t c = i ? word[u].y : word[u].x, sm = sc[u][GR == 2 ? i : 0];
      const float s = __uint_as_float(sm << 16), m = __uint_as_float(sm & 0xffff0000u);
      // 2^23 + c, one byte permutation, less 2^23
      const uint32_t even = c & 0x0f0f0f0fu, odd = (c >> 4) & 0x0f0f0f0fu;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f32x2 f = f2_add(f2_make(__uint_as_float(__byte_perm(even, 0x4b000000u, 0x7550 + k)),
                                       __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7550 + k))),
                               f2_make(-8388608.f, -8388608.f));
        f2_split(f2_fma(f, f2_make(s, s), f2_make(m, m)), x[i][2 * k], x[i][2 * k + 1]);
      }
    }
    T* row = dst + (int64_t)r * D;
    store8<T>(row + kv4_word_channel<D>(2 * w), x[0]);
    store8<T>(row + kv4_word_channel<D>(2 * w + 1), x[1]);
  }
}

template <typename T, int D>
cudaError_t launch(const Kv4Args& a, bool read, cudaStream_t s) {
  const int per_cta = kThreads / (D / 16) * kUnroll;
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
