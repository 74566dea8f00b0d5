// What the kernels of the attention over a 4-bit cache share: the split of the work over the CTAs, the
// layout of their partial results and the kernel that merges those.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "tc100.cuh"

namespace stdb {
namespace {

constexpr int kTile = 128;  // keys of a tile
constexpr float kLimit = 32768.f;  // largest weight x scale x factor that goes to fp16
constexpr float kMostFactor = 1.3292280e36f;  // 2^120: a factor of weights x scales before any was seen
constexpr float kHeadroom = 8.f;  // a new reference puts the largest weight at 2^8

// ---------------------------------------------------------------- codes in the tensor cores
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
// Two codes as fp16 subnormals: c 2^-24 from bits 0-3 and 16-19, c 2^-20 from bits 4-7 and 20-23.
__device__ __forceinline__ uint32_t widen0(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t widen4(uint32_t w) { return w & 0x00f000f0u; }
// Two codes as c - 8, one instruction more: 0x6400 is 1024, whose last ten bits hold a code at bit 0 or 4.
__device__ __forceinline__ uint32_t centre0(uint32_t w) {
  return as_u32(__hsub2(as_h2(widen0(w) | 0x64006400u), __float2half2_rn(1032.f)));
}
__device__ __forceinline__ uint32_t centre4(uint32_t w) {
  return as_u32(__hfma2(as_h2(widen4(w) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-72.f)));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// ---------------------------------------------------------------- work split
// Units are numbered (layer, sequence, KV head, row block).  A unit's tiles are cut into groups of
// `group`, all units' groups form one sequence, and CTA c takes groups [c share, (c + 1) share) of it.
// Long work is cut tile by tile (group = 1): every CTA has the same number of tiles to within one, and
// those that straddle two units pay for it with a second set of queries and a second merge, some 2.5
// us.  Where that is more than the tiles it saves, units are cut into equal parts, one a CTA
// (share = 1).
struct Split {
  int cum[kKv4AttnMaxB + 1];  // groups of the sequences before b, in one (layer, head, row block)
  int group, share, total;
};

struct Unit {
  int l, b, h, rb;
  int first, groups;  // the group within the unit; the unit's groups
};

// Keys that sequence b's last query position attends; -1: not valid.  (Read again from the length
// wherever it is needed: after the first time that is a hit in L1.)
__device__ __forceinline__ int keys_of(const Kv4AttnArgs& a, int b) {
  const int len = a.len[b];
  const int64_t n = (int64_t)len + a.len_off + a.nq - 1;
  return len >= 0 && n <= a.cap ? (int)n : -1;
}
__device__ __forceinline__ int tiles_of(int keys) { return keys < 0 ? 0 : keys < 1 ? 1 : (keys + kTile - 1) / kTile; }

// The split of this call's work over `ctas` CTAs, by one warp.  (The first 32 sequences stay in
// registers: a draft step of a few sequences waits for this.)
__device__ __forceinline__ void plan_split(const Kv4AttnArgs& a, Split* sp, int ctas, int lane, bool flag) {
  const int units = a.Hkv * a.row_blocks * a.L;  // of one sequence
  auto load = [&](int b) {
    if (b >= a.B) return 0;
    const int keys = keys_of(a, b);
    if (keys < 0 && flag) flag_error(a.err, STD_DEVERR_LENGTH);
    return tiles_of(keys);
  };
  const int mine = load(lane);
  int sum = mine;
  for (int b = lane + 32; b < a.B; b += 32) sum += load(b);
  flag = false;
  sum = (a.B == 1 ? __shfl_sync(0xffffffffu, sum, 0) : __reduce_add_sync(0xffffffffu, sum)) * units;
  int share = sum <= ctas ? (sum > 0) : (sum + ctas - 1) / ctas, group = 1;
  if (share > 1 && share <= 32) {
#pragma unroll 1
    for (int s = share; s <= share + 2; ++s) {  // parts of s tiles
      int parts = (mine + s - 1) / s;
      for (int b = lane + 32; b < a.B; b += 32) parts += (load(b) + s - 1) / s;
      parts = __reduce_add_sync(0xffffffffu, parts) * units;
      if (parts <= ctas) {
        group = s;
        share = 1;
        sum = parts;
        break;
      }
    }
  }
  if (lane == 0) {
    sp->cum[0] = 0;
    sp->group = group;
    sp->share = share;
    sp->total = sum;
  }
  int run = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int s = b0 == 0 ? mine : load(b);
    if (group > 1) s = (s + group - 1) / group;
    for (int o = 1; o < 32 && o < a.B; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (b < a.B) sp->cum[b + 1] = run + s;
    run += __shfl_sync(0xffffffffu, s, 31);
  }
}

// The unit that group x of the sequence belongs to.
__device__ __forceinline__ Unit locate(const Kv4AttnArgs& a, const Split& sp, int x) {
  Unit u;
  const int heads = a.Hkv * a.row_blocks;
  const int layer = sp.cum[a.B] * heads;  // groups of a layer
  u.l = a.L == 1 ? 0 : x / layer;
  int r = x - u.l * layer;
  int lo = 0, hi = a.B;  // the last b with cum[b] * heads <= r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sp.cum[mid] * heads <= r) lo = mid; else hi = mid;
  }
  u.b = lo;
  r -= sp.cum[lo] * heads;
  u.groups = sp.cum[lo + 1] - sp.cum[lo];
  const int hr = r / u.groups;
  u.first = r - hr * u.groups;
  u.h = a.row_blocks == 1 ? hr : hr / a.row_blocks;
  u.rb = hr - u.h * a.row_blocks;
  return u;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// A tile in shared memory: K codes, V codes, K scales, V scales, 128 rows each.
template <int D>
struct TileAt {
  static constexpr int CW = D / 2;                     // code bytes of a row
  static constexpr int SW = D / kKv4Group * 4;         // scale bytes of a row
  static constexpr int VC = kTile * CW, KS = 2 * VC, VS = KS + kTile * SW;
  static constexpr int BYTES = VS + kTile * SW;
};

// The next tile of a CTA's range to fetch (touched by one thread at a time).
struct Fetch {
  int fills, next, left, first, keys;
  int64_t row0;  // cache row of the unit's row 0
};

// Fetch it into its stage of the ring; `end`: the end of the CTA's range of groups.
template <int D, int STAGES>
__device__ __forceinline__ void fetch_tile(const Kv4AttnArgs& a, Fetch* f, const Split& sp, uint64_t* full, uint32_t ring,
                                           int end) {
  using At = TileAt<D>;
  while (f->left == 0) {
    const int x = f->next;
    if (x >= end) return;
    const Unit u = locate(a, sp, x);
    const int n = min(u.groups - u.first, end - x);
    const int keys = keys_of(a, u.b), first = u.first * sp.group;
    f->next = x + n;
    f->left = min(n * sp.group, (keys + kTile - 1) / kTile - first);  // (none for a sequence without keys)
    f->first = first * kTile;
    f->keys = keys;
    f->row0 = (((int64_t)u.l * a.B + u.b) * a.Hkv + u.h) * a.cap;
  }
  const int first = f->first, stage = f->fills % STAGES;
  // whole 16-row blocks: the capacity is a multiple of 16, so they end inside the cache
  const uint32_t rows = min(kTile, (f->keys - first + 15) & ~15);
  const int64_t row = f->row0 + first;
  const uint32_t dst = ring + stage * At::BYTES;
  uint64_t* bar = &full[stage];
  if (STD_DCHECK(first >= 0 && first + (int64_t)rows <= a.cap && row >= 0, a.err)) {
    tc::mbar_expect_tx(bar, 2 * rows * (At::CW + At::SW));
    bulk_load(dst, a.k_codes + row * At::CW, rows * At::CW, bar);
    bulk_load(dst + At::KS, a.k_scales + row * At::SW, rows * At::SW, bar);
    bulk_load(dst + At::VC, a.v_codes + row * At::CW, rows * At::CW, bar);
    bulk_load(dst + At::VS, a.v_scales + row * At::SW, rows * At::SW, bar);
  } else {
    tc::mbar_arrive(bar);  // (debug build: the tile is left as it is)
  }
  f->fills += 1;
  f->first = first + kTile;
  f->left -= 1;
}

__device__ __forceinline__ float lo_bf16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  }
}

// Partials of one slot: [8 NT][D] unnormalised sums, then [8 NT][2] (reference, sum of weights).
template <int D>
__host__ __device__ constexpr int64_t slot_floats(int rows) { return (int64_t)rows * (D + 2); }

// Units that several CTAs touched: one CTA for each query row merges their slots.
//   M = max_c m_c,  o = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c
// D / 4 lanes hold a slot's row, blockDim.y slots are read at a time (so that a row's slots come in one or
// two trips to memory), and each lane merges its slots as it goes.
template <int D, int ROWS, typename T>
__global__ void __launch_bounds__(1024) kv4_merge_kernel(const Kv4AttnArgs a, int ctas) {
  constexpr int LPR = D / 4;
  __shared__ Split sp;
  __shared__ float4 part[1024 / LPR][LPR];
  __shared__ float2 stat[1024 / LPR];
  const int lane = threadIdx.x, first = threadIdx.y, tid = first * LPR + lane;
  // The attention kernel lets this one start once it has itself waited for the kernels before it, so the
  // lengths can be read, and the slots found, while it runs.
  if (tid < 32) plan_split(a, &sp, ctas, tid, false);
  __syncthreads();
  int id = blockIdx.x;  // ((l * B + b) * Hkv + h) * rows + r
  const int r = id % a.rows;
  id /= a.rows;
  const int h = id % a.Hkv, lb = id / a.Hkv, b = lb % a.B, l = lb / a.B;
  const int heads = a.Hkv * a.row_blocks, groups = sp.cum[b + 1] - sp.cum[b], share = sp.share;
  const int rb = r / ROWS, n = r - rb * ROWS;
  const int u0 = (l * sp.cum[a.B] + sp.cum[b]) * heads + (h * a.row_blocks + rb) * groups;
  const int c0 = groups ? u0 / share : 0, c1 = groups ? (u0 + groups - 1) / share : 0;
  pdl_wait();  // memory of earlier kernels in the stream is visible from here on
  pdl_trigger();
  if (c0 == c1) return;  // written whole, or not valid
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  float top = -INFINITY, lt = 0.f;
  for (int c = c0 + first; c <= c1; c += 4 * blockDim.y) {
    float2 ml[4];
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ci = c + i * (int)blockDim.y;
      ml[i] = make_float2(-INFINITY, 0.f);
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ci <= c1) {  // (the first CTA's slot 1, unless its range begins with the unit)
        const float* p = a.ws + (2 * (int64_t)ci + (ci > c0 || ci * share == u0 ? 0 : 1)) * slot_floats<D>(ROWS);
        ml[i] = *reinterpret_cast<const float2*>(p + ROWS * D + 2 * n);
        v[i] = *reinterpret_cast<const float4*>(p + n * D + 4 * lane);
      }
    }
    const float m1 = fmaxf(top, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
    const float keep = top == -INFINITY ? 0.f : ex2(top - m1);
    sum.x *= keep; sum.y *= keep; sum.z *= keep; sum.w *= keep;
    lt *= keep;
    top = m1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = ml[i].x == -INFINITY ? 0.f : ex2(ml[i].x - top);
      sum.x = fmaf(f, v[i].x, sum.x); sum.y = fmaf(f, v[i].y, sum.y);
      sum.z = fmaf(f, v[i].z, sum.z); sum.w = fmaf(f, v[i].w, sum.w);
      lt = fmaf(f, ml[i].y, lt);
    }
  }
  part[first][lane] = sum;
  if (lane == 0) stat[first] = make_float2(top, lt);
  __syncthreads();
  if (first == 0) {
    top = -INFINITY;
    for (int i = 0; i < (int)blockDim.y; ++i) top = fmaxf(top, stat[i].x);
    sum = make_float4(0.f, 0.f, 0.f, 0.f);
    lt = 0.f;
#pragma unroll 8
    for (int i = 0; i < (int)blockDim.y; ++i) {
      const float2 ml = stat[i];
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
      const float4 v = part[i][lane];
      sum.x = fmaf(f, v.x, sum.x); sum.y = fmaf(f, v.y, sum.y);
      sum.z = fmaf(f, v.z, sum.z); sum.w = fmaf(f, v.w, sum.w);
      lt = fmaf(f, ml.y, lt);
    }
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
    const int64_t at = (((int64_t)lb * a.Hq + h * a.G) * a.nq + r) * D + 4 * lane;
    store4(static_cast<T*>(a.o) + at, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
  }
}

// The merge's launch, after the attention kernel's with row blocks of ROWS.
template <int D, int ROWS, typename T>
cudaError_t launch_kv4_merge(const Kv4AttnArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.L * a.B * a.Hkv * a.rows;
  // slots of a unit if all are equally long: four for each lane of the merge
  const int slots = a.ctas / (a.L * a.B * a.Hkv * a.row_blocks) + 2;
  int at_once = 128 / (D / 4);
  while (at_once < 1024 / (D / 4) && 4 * at_once < slots) at_once *= 2;
  return launch_pdl(kv4_merge_kernel<D, ROWS, T>, dim3((unsigned)rows), dim3(D / 4, at_once), 0, s, a, a.ctas);
}

}  // namespace
}  // namespace stdb
