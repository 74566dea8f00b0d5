// Attention over a 4-bit K/V cache for more than 16 query rows of a KV head (verify rows): the
// mathematics of kv4_attn.cu on the 5th-generation tensor cores.
//
// 64 query rows share each widened code here, so a tile's codes are widened once, into tensor and shared
// memory, and both products run as tcgen05.mma:
//   S_g^T [128 keys][64 rows] = K codes of group g (tensor memory) x Q_g (shared memory), g = 0, 1
//   O [2 x 64 rows][128 channels] += (P sv_0 over P sv_1) x V codes (both shared memory, read across their rows)
// With keys in the lanes of S a key's scales and minima are a thread's own: it turns its part of S_0 and S_1
// into logits and weights, multiplies them by sv_0 and sv_1 and writes 16-bit rows of the next operand.
// (O's upper 64 rows are valid for group 0's channels, the lower for group 1's: half of the product is thrown away,
// which costs what two half-height products would.)  No maximum is taken on the way: weights are relative to a
// reference of each row, and their products with a group's scales have a factor of the row's and group's own; both
// move only when some product would leave fp16's range, so a tile has one barrier, and the sums of p and p m stay
// in registers, 16 rows a thread, until the unit ends.
//
// A tile at d = 128 is 18 KB; at full HBM rate it would be 760 clocks.  Measured: 28 layers
// x 4 heads x 33,024 keys, 49 rows, 394 us (four blocks of 16 rows in kv4_attn.cu: 748 us; without the factors of rows
// and groups 372, and 403 where a thread widened a group of its key of K and not half a row, which reads all codes
// twice).  Of a tile's 3,490 clocks the tensor cores are busy 770; the phases follow each other.
#include "kv4_attn.cuh"

#include <atomic>

namespace stdb {
namespace {

constexpr int kRows = 64;               // query rows of a block
constexpr int kShare = 16;              // rows of a thread: four threads a key
constexpr int kThreads = kTile * kRows / kShare;
constexpr int kStages = 4;
// The thread that fetches tiles, and the warps that issue the products: of those that widen K, which is less
// work than V.  (The issue of P V blocks its warp until the tensor cores have taken most of it, some 800
// clocks; wg 3 has the fewest rows where a block is short.  On the S issuer's scheduler, warp 12, it is 412 us
// where this is 400.)
constexpr int kFetcher = kThreads - 32, kIssueS = 0, kIssuePV = 13;
static_assert(kIssueS != kIssuePV && kIssueS != kFetcher / 32 && kIssuePV != kFetcher / 32, "one role a warp");
constexpr float kMostWeight = 1.1529215e18f;  // 2^60: a weight above it moves its reference, however small the scales

// Shared memory, from a 1024-byte boundary on: operands in 128-byte swizzled rows, then the ring of 4-bit
// tiles, then tables.
template <int D>
struct Lay {
  static constexpr int GR = D / kKv4Group;
  static constexpr int V = 0;                             // [2][GR][128 keys][64 channels] fp16
  static constexpr int V_GROUP = kTile * 128;
  static constexpr int P = V + 2 * GR * V_GROUP;          // [2][2][128 keys][64 rows] fp16 (one group: the second unused)
  static constexpr int P_GROUP = kTile * 128;
  static constexpr int Q = P + 4 * P_GROUP;          // [GR][64 rows][64 channels] fp16
  static constexpr int Q_GROUP = kRows * 128;
  static constexpr int RING = Q + GR * Q_GROUP;
  static constexpr int TAB = RING + kStages * TileAt<D>::BYTES;
  static constexpr int RED = TAB + 10 * kRows * 4;        // [4 warps][64 rows][3]
  static constexpr int BYTES = RED + 4 * kRows * 3 * 4;
};

struct Ctl {
  uint64_t full[kStages], s_done, pv_done[2];
  Split split;
  Fetch fetch;
  uint32_t tmem;
  volatile int abort;
};

// Tensor memory columns: K codes (two buffers of 32 columns a group), S (two buffers of one 64-column
// accumulator a group), O (a column a channel).
template <int D>
struct Cols {
  static constexpr int GR = D / kKv4Group;
  static constexpr int K = 0, S = 2 * 32 * GR, O = S + 2 * kRows * GR;
  static constexpr int N = 512;
  static_assert(O + D <= N, "tensor memory");
};

constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// tcgen05.mma and its commit by the lane whose `leader` is set; the other operands are the warp's.
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %5, 0;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d), "r"(a_tmem), "l"(b), "r"(id), "r"(add), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %5, 0;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(add), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n"
      ::"r"(smem_u32(bar)), "r"(leader)
      : "memory");
}
// Wait for a phase, by a whole warp.  A wait that gives up raises the CTA's abort flag and the warp goes on,
// within its own buffers, to the next barrier, where every thread sees the flag.
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  if (!__all_sync(0xffffffffu, tc::mbar_try_wait(smem_u32(bar), parity))) {
    tc::mbar_wait(bar, parity, abort, err);
    __syncwarp();
  }
}
// 8 consecutive 32-bit columns of this thread's lane
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait8(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

// Position p of eight in an operand holds code (channel of the word) perm8(p): the order in which masks
// take codes out of a word, (0, 4), (1, 5), (2, 6), (3, 7); the second and fourth pair come at 2^-20.
__device__ __forceinline__ constexpr int perm8(int p) { return (p >> 1) + 4 * (p & 1); }

// Four columns: a word of K.
__device__ __forceinline__ void widen_word(uint32_t x, uint32_t* r) {
  r[0] = widen0(x);
  r[1] = widen4(x);
  r[2] = widen0(x >> 8);
  r[3] = widen4(x >> 8);
}
// Half of a thread's key of K to tensor memory (its lane), 16 columns a group.
template <int D>
__device__ __forceinline__ void widen_k(uint32_t row, uint32_t taddr, int part) {
  uint32_t r[16];
  if constexpr (D == 64) {
    const uint4 v = lds128(row + 16 * part);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) widen_word(w[k], r + 4 * k);
    tc::tmem_st_x16(taddr + 16 * part, r);
    return;
  }
  const uint4 lo = lds128(row + 32 * part), hi = lds128(row + 32 * part + 16);
  const uint32_t w[8] = {lo.x, lo.z, hi.x, hi.z, lo.y, lo.w, hi.y, hi.w};
#pragma unroll
  for (int gr = 0; gr < 2; ++gr) {
#pragma unroll
    for (int k = 0; k < 4; ++k) widen_word(w[4 * gr + k], r + 4 * k);
    tc::tmem_st_x16(taddr + 32 * gr + 16 * part, r);
  }
}

// Half of a thread's key of V to its 128-byte rows of the operand, chunk c of 16 bytes at c ^ (key % 8).
// The order of the 16-byte loads differs from lane to lane so that neither they nor the stores conflict.
template <int D>
__device__ __forceinline__ void widen_v(uint32_t row, uint32_t dst, int key, int part) {
  constexpr int GR = D / kKv4Group;
  const int a = (key >> 1) & 3, turn = ((a << 1) ^ (a >> 1) * 3) & 3;
  uint4 v[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) v[i] = lds128(row + 16 * (D == 128 ? (2 * part + i) ^ turn : part ^ (turn & 1)));
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int c = D == 128 ? (2 * part + i) ^ turn : part ^ (turn & 1);
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int gr = GR == 2 ? k & 1 : 0, chunk = GR == 2 ? 2 * c + (k >> 1) : 4 * c + k;
      sts128(dst + gr * Lay<D>::V_GROUP + key * 128 + ((chunk ^ (key & 7)) << 4), centre0(w[k]), centre4(w[k]),
             centre0(w[k] >> 8), centre4(w[k] >> 8));
    }
  }
}

// A block's queries: the operand (kRows x 64 for each group, fp16, each row scaled by a power of two of its own, K-major
// with swizzled rows), and the rows' tables: the group sums of the scaled queries and the powers of two that undo it.
template <int D>
__device__ __forceinline__ void load_queries(const Kv4AttnArgs& a, const Unit& u, int n0, uint8_t* smem, int tid) {
  constexpr int GR = D / kKv4Group, NC = D / 8;  // channels of a thread: an eighth of a row
  const int r = tid >> 3, part = tid & 7, row = u.rb * kRows + r;
  float x[NC];
  float top = 0.f;
  const int64_t at = ((((int64_t)u.l * a.B + u.b) * a.Hq + u.h * a.G) * a.nq + row) * D + part * NC;
#pragma unroll
  for (int i = 0; i < NC; i += 8) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < a.rows) v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at + i);
    x[i] = lo_bf16(v.x); x[i + 1] = hi_bf16(v.x); x[i + 2] = lo_bf16(v.y); x[i + 3] = hi_bf16(v.y);
    x[i + 4] = lo_bf16(v.z); x[i + 5] = hi_bf16(v.z); x[i + 6] = lo_bf16(v.w); x[i + 7] = hi_bf16(v.w);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (fabsf(x[i + k]) < INFINITY) top = fmaxf(top, fabsf(x[i + k]));
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  int ex = (int)(__float_as_uint(top) >> 23) - 127;
  ex = ex < -100 ? -100 : ex;
  const float mul = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
  float sum = 0.f;
  const int per = 8 / GR, gr = part / per, c0 = part % per * NC;  // threads of a group; channels of the group
  uint8_t* base = smem + Lay<D>::Q + gr * Lay<D>::Q_GROUP + r * 128;
#pragma unroll
  for (int i = 0; i < NC; i += 8) {
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // pair k: channels k and k + 4 of the word
      const float f = mul * (k & 1 ? 0.0625f : 1.f);
      h[k] = as_u32(__floats2half2_rn(x[i + k] * f, x[i + k + 4] * f));
      sum += (x[i + k] + x[i + k + 4]) * mul;
    }
    const int chunk = (c0 + i) >> 3;
    *reinterpret_cast<uint4*>(base + ((chunk ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
  }
  sum *= 5.9604645e-8f;  // 2^-24
#pragma unroll
  for (int o = 1; o < 8 / GR; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float* tab = reinterpret_cast<float*>(smem + Lay<D>::TAB);
  if (part % per == 0) tab[gr * kRows + r] = sum;
  if (part == 1) {
    tab[2 * kRows + r] = INFINITY;  // minus the row's reference
    reinterpret_cast<int*>(tab)[4 * kRows + r] = n0 + (row < a.rows ? row % a.nq : 0);  // keys it attends
    tab[5 * kRows + r] = __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
    tab[6 * kRows + r] = tab[7 * kRows + r] = kMostFactor;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_attn_tc_kernel(const Kv4AttnArgs a) {
  using L = Lay<D>;
  using C = Cols<D>;
  using At = TileAt<D>;
  constexpr int GR = D / kKv4Group;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int wg = warp >> 2, qd = warp & 3, key = tid & 127;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) tc::mbar_init(&ctl.full[s], 1);
    tc::mbar_init(&ctl.s_done, 1);
    tc::mbar_init(&ctl.pv_done[0], 1);
    tc::mbar_init(&ctl.pv_done[1], 1);
    ctl.abort = 0;
    ctl.fetch.fills = ctl.fetch.left = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();  // memory of earlier kernels in the stream is visible from here on
  if (warp == 1) {
    tc::tmem_alloc(&ctl.tmem, C::N);
    tc::tmem_relinquish();
  }
  if (warp == 0) plan_split(a, &ctl.split, gridDim.x, lane, blockIdx.x == 0);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // (only now: a kernel that starts early must not take the tensor memory that this one has yet to get)
  pdl_trigger();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0), lanes = tmem + ((uint32_t)(qd * 32) << 16);
  const int total = ctl.split.total, share = ctl.split.share;
  const int64_t begin64 = (int64_t)share * blockIdx.x;
  const int begin = begin64 < total ? (int)begin64 : total, end = min(begin + share, total);
  const uint32_t ring = sm + L::RING;
  // Of the rows: [0], [1] sums of q (two groups), [2] minus the references, [3] what sums of weights are multiplied
  // with when those move, [4] the keys they attend, [5] their powers of two, [6], [7] the factors of weights x
  // scales (two groups), [8], [9] what the sums of those are multiplied with.
  float* tab = reinterpret_cast<float*>(smem + L::TAB);
  float* red = reinterpret_cast<float*>(smem + L::RED);
  if (tid == kFetcher && begin < end) {
    ctl.fetch.next = begin;
    for (int s = 0; s < kStages; ++s) fetch_tile<D, kStages>(a, &ctl.fetch, ctl.split, ctl.full, ring, end);
  }
  uint32_t leader;  // one lane of each warp
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(leader));
  // (start addresses are in units of 16 bytes and do not carry: shared memory is smaller than the field)
  const uint64_t q_desc = tc::sdesc_sw128(sm + L::Q), v_desc = tc::sdesc_sw128_mn(sm + L::V, L::V_GROUP),
                 p_desc = tc::sdesc_sw128_mn(sm + L::P, L::P_GROUP);
  int tiles_read = 0;      // tiles of the units before this one
  uint32_t s_count = 0;    // S products issued
  uint32_t pv_count = 0;   // P V products issued, in turn on pv_done[0] and [1]
  bool ok = true;

  for (int t = begin; t < end && ok;) {
    const Unit u = locate(a, ctl.split, t);
    const int group = ctl.split.group, keys = keys_of(a, u.b), first = u.first * group;
    const int n = min(u.groups - u.first, end - t);
    const int nt = min(n * group, (keys + kTile - 1) / kTile - first);  // (may be none)
    const int n0 = keys - a.nq + 1;
    load_queries<D>(a, u, n0, smem, tid);
    f32x2 l[kShare / 2], pm[GR][kShare / 2];  // sums of p and of p (mv + 8 sv), two rows together
#pragma unroll
    for (int j = 0; j < kShare / 2; ++j) {
      l[j] = f2_make(0.f, 0.f);
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) pm[gr][j] = f2_make(0.f, 0.f);
    }
    const uint32_t pv0 = pv_count;

    const int live = min(kRows, a.rows - u.rb * kRows);  // rows of the block
    auto stage_of = [&](int i) { return ring + (uint32_t)((tiles_read + i) % kStages) * At::BYTES; };
    auto wait_tile = [&](int i) {
      const int k = tiles_read + i;
      wait_for(&ctl.full[k % kStages], (uint32_t)(k / kStages) & 1u, &ctl.abort, a.err);
    };
    // the P V product `c` (counted from the kernel's start) has finished
    auto wait_pv = [&](uint32_t c) { wait_for(&ctl.pv_done[c & 1], (c >> 1) & 1u, &ctl.abort, a.err); };
    // A whole warp comes here and one lane issues, so that addresses and descriptors are the warp's
    // and not a lane's: a tcgen05.mma takes them from uniform registers, and a lane's own have to be moved
    // there first (16 products of a tile: 1,750 clocks that way).
    auto issue_s = [&](int i) {  // S_g = K codes of tile i x Q_g
      constexpr uint32_t id = idesc_f16(128, kRows);
      const uint32_t odd = __shfl_sync(0xffffffffu, i & 1, 0);
      const uint32_t d = tmem + C::S + odd * GR * kRows, k0 = tmem + C::K + odd * GR * 32;
#pragma unroll
      for (int gr = 0; gr < GR; ++gr)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(leader, d + gr * kRows, k0 + gr * 32 + 8 * k, q_desc + (gr * L::Q_GROUP + 32 * k) / 16, id, k > 0);
      commit(leader, &ctl.s_done);
    };
    auto issue_pv = [&](int i, uint32_t c) {  // O += (P sv_g) x V codes, buffers c % 2
      constexpr uint32_t id = idesc_f16(128, D) | (1u << 15) | (1u << 16);  // both read across their rows
      const uint32_t odd = __shfl_sync(0xffffffffu, c & 1, 0), old = __shfl_sync(0xffffffffu, i > 0 ? 1 : 0, 0);
      const uint64_t v = v_desc + odd * (GR * L::V_GROUP / 16), p = p_desc + odd * (2 * L::P_GROUP / 16);
#pragma unroll
      for (int k = 0; k < 8; ++k) mma_ss(leader, tmem + C::O, p + k * 128, v + k * 128, id, k > 0 ? 1u : old);
      commit(leader, &ctl.pv_done[odd]);
    };

    // Threads that widen K: wg 0 and 3; V: 1 and 2, half a row each.
    const bool k_side = wg == 0 || wg == 3;
    auto widen_keys = [&](int i) {
      if (k_side) {
        widen_k<D>(stage_of(i) + key * At::CW, lanes + C::K + (i & 1) * GR * 32, wg == 3);
        tc::tmem_st_wait();
      }
    };
    if (nt > 0) {
      wait_tile(0);
      if (nt > 1) wait_tile(1);
      widen_keys(0);
    }
    tc::fence_proxy_async();  // (the queries)
    tc::fence_before_sync();
    if (__syncthreads_or(ctl.abort)) {
      ok = false;
      break;
    }
    if (warp == kIssueS && nt > 0) {
      tc::fence_after_sync();
      issue_s(0);
    }
    if (nt > 0) ++s_count;

    // a thread's rows: 8 of each half of the block, [32 h + 8 wg, 32 h + 8 wg + 8), so that a short block
    // leaves every fourth of the warps the same share
    const int halves = 8 * wg >= live ? 0 : kRows / 2 + 8 * wg >= live ? 1 : 2;
    for (int i = 0; i < nt; ++i) {
      const uint32_t cur = stage_of(i);
      const uint32_t buf = pv_count & 1;
      // Widen the next tile's K and this tile's V.  (That the tiles are here, and the buffers' last product
      // done, a warp has made sure of before the last barrier.)
      if (i + 1 < nt) widen_keys(i + 1);
      if (wg == 1 || wg == 2) widen_v<D>(cur + At::VC + key * At::CW, sm + L::V + buf * GR * L::V_GROUP, key, wg - 1);

      // this thread's key: scales (K's with log2(e) / sqrt(d), and 2^24 as codes are subnormals), position
      constexpr float kBack = kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f) * 16777216.f;
      const int pos = (first + i) * kTile + key;
      float sk[GR], mk[GR], sv[GR], mv[GR];
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) {
        const uint32_t uk = lds32(cur + At::KS + key * At::SW + 4 * gr), uv = lds32(cur + At::VS + key * At::SW + 4 * gr);
        sk[gr] = lo_bf16(uk) * kBack;
        mk[gr] = hi_bf16(uk) * kBack;
        sv[gr] = lo_bf16(uv);
        mv[gr] = fmaf(8.f, sv[gr], hi_bf16(uv));
      }
      const bool edge = (first + i + 1) * kTile > n0;  // some query position does not attend some key of the tile
      if (edge && pos >= keys) {  // (past the last key the bytes may be anything)
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) sk[gr] = mk[gr] = sv[gr] = mv[gr] = 0.f;
      }
      wait_for(&ctl.s_done, (s_count - 1) & 1u, &ctl.abort, a.err);
      tc::fence_after_sync();

      const uint32_t s_at = lanes + C::S + (i & 1) * GR * kRows + wg * 8;
      const uint32_t p_at = sm + L::P + buf * 2 * L::P_GROUP + key * 128;
      // Weights and the operand's rows.  Where some weight x scale x factor leaves fp16's range (the first tile of a
      // unit, as no reference is set yet, and rarely after it) references and factors move and it is done once more; a
      // thread whose own weights fit has added them to its sums by then, which move with the references.
      bool added = false;
      for (bool moved = false;;) {
        float big = 0.f, most = 0.f;
        f32x2 p[kShare / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h < halves) {
            uint32_t s[GR][8];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) tmem_ld_x8(s_at + gr * kRows + h * (kRows / 2), s[gr]);
            const float* at = tab + h * (kRows / 2) + wg * 8;
            f32x2 x[4];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {  // rows 2 k .. 2 k + 3
              const ulonglong2 q0 = *reinterpret_cast<const ulonglong2*>(at + 2 * k);
              x[k] = f2_mul(f2_make(mk[0], mk[0]), q0.x);
              x[k + 1] = f2_mul(f2_make(mk[0], mk[0]), q0.y);
              if constexpr (GR == 2) {
                const ulonglong2 q1 = *reinterpret_cast<const ulonglong2*>(at + kRows + 2 * k);
                x[k] = f2_fma(f2_make(mk[1], mk[1]), q1.x, x[k]);
                x[k + 1] = f2_fma(f2_make(mk[1], mk[1]), q1.y, x[k + 1]);
              }
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) tmem_ld_wait8(s[gr]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int gr = 0; gr < GR; ++gr)
                x[k] = f2_fma(f2_make(sk[gr], sk[gr]),
                              f2_make(__uint_as_float(s[gr][2 * k]), __uint_as_float(s[gr][2 * k + 1])), x[k]);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(at + 2 * kRows + 2 * k);
              const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(at + 5 * kRows + 2 * k);
              x[k] = f2_fma(x[k], b.x, m.x);
              x[k + 1] = f2_fma(x[k + 1], b.y, m.y);
            }
            if (edge) {
              const int* lim = reinterpret_cast<const int*>(at) + 4 * kRows;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float x0, x1;
                f2_split(x[k], x0, x1);
                x[k] = f2_make(pos < lim[2 * k] ? x0 : -INFINITY, pos < lim[2 * k + 1] ? x1 : -INFINITY);
              }
            }
            uint32_t pk[GR][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x0, x1;
              f2_split(x[k], x0, x1);
              x0 = ex2(x0);
              x1 = ex2(x1);
              most = max3f(most, x0, x1);
              p[4 * h + k] = f2_make(x0, x1);
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(at + (6 + gr) * kRows + 2 * k);
                const f32x2 s2 = f2_make(sv[gr], sv[gr]);
                float w0, w1;
                f2_split(f2_mul(f2_mul(p[4 * h + k], s2), f.x), w0, w1);
                big = max3f(big, w0, w1);
                pk[gr][k] = as_u32(__floats2half2_rn(w0, w1));
                f2_split(f2_mul(f2_mul(p[4 * h + k + 1], s2), f.y), w0, w1);
                big = max3f(big, w0, w1);
                pk[gr][k + 1] = as_u32(__floats2half2_rn(w0, w1));
              }
            const int chunk = 4 * h + wg;
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
              sts128(p_at + gr * L::P_GROUP + ((chunk ^ (key & 7)) << 4), pk[gr][0], pk[gr][1], pk[gr][2], pk[gr][3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[4 * h + k] = 0;
          }
        }
        const bool fits = big <= kLimit && most <= kMostWeight;
        if (!added && (fits || moved)) {
          added = true;
          if (edge && (mv[0] != mv[0] || mv[GR - 1] != mv[GR - 1])) {
            // a row that is not finite: query positions that do not attend it must not multiply by it
            const int* lim = reinterpret_cast<const int*>(tab) + 4 * kRows + wg * 8;
#pragma unroll
            for (int j = 0; j < kShare / 2; ++j) {
              float p0, p1;
              f2_split(p[j], p0, p1);
              const int row = (j >> 2) * (kRows / 2) + 2 * (j & 3);
#pragma unroll
              for (int gr = 0; gr < GR; ++gr)
                pm[gr][j] = f2_add(pm[gr][j], f2_make(pos < lim[row] ? p0 * mv[gr] : 0.f, pos < lim[row + 1] ? p1 * mv[gr] : 0.f));
            }
          } else {
#pragma unroll
            for (int j = 0; j < kShare / 2; ++j)
#pragma unroll
              for (int gr = 0; gr < GR; ++gr) pm[gr][j] = f2_fma(p[j], f2_make(mv[gr], mv[gr]), pm[gr][j]);
          }
#pragma unroll
          for (int j = 0; j < kShare / 2; ++j) l[j] = f2_add(l[j], p[j]);
        }
        if (warp == kThreads / 32 - 1) {  // what the next tile's start relies on
          if (i + 2 < nt) wait_tile(i + 2);
          if (pv_count > 0) wait_pv(pv_count - 1);
        }
        tc::fence_proxy_async();
        tc::fence_before_sync();
        if (!__syncthreads_or((!moved && !fits) || ctl.abort)) break;
        // References move, or a wait gave up.  (O is still: its last product has been waited for.)
        if (__syncthreads_or(ctl.abort)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        moved = true;
        auto each_logit = [&](auto f) {  // f(row, logit): the logits above, summed in the same order
#pragma unroll 1
          for (int r = 0; r < 8 * halves; r += 4) {
            const int row0 = (r >> 3) * (kRows / 2) + wg * 8 + (r & 4);
            uint32_t s[GR][4];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) tc::tmem_ld_x4(s_at - wg * 8 + gr * kRows + row0, s[gr]);
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) tc::tmem_ld_wait4(s[gr]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = row0 + k;
              float x = mk[0] * tab[row];
              if constexpr (GR == 2) x = fmaf(mk[1], tab[kRows + row], x);
#pragma unroll
              for (int gr = 0; gr < GR; ++gr) x = fmaf(sk[gr], __uint_as_float(s[gr][k]), x);
              f(row, x, pos < reinterpret_cast<const int*>(tab)[4 * kRows + row]);
            }
          }
        };
        auto over_warps = [&](int i) {
          return fmaxf(fmaxf(red[i], red[2 * kRows + i]), fmaxf(red[4 * kRows + i], red[6 * kRows + i]));
        };
        const bool mine = tid < kRows && (tid & ~7) < live;  // (rows behind the last share its eight)
        // every row's largest logit, first over the warps
        each_logit([&](int row, float x, bool seen) {
          const float z = warp_max_f32(seen ? x * tab[5 * kRows + row] : -INFINITY);
          if (lane == 0) red[2 * (qd * kRows + row)] = z;
        });
        __syncthreads();
        if (tid < kRows) {
          float f = 1.f, times[2] = {1.f, 1.f};
          const float m0 = -tab[2 * kRows + tid], z = mine ? over_warps(2 * tid) : m0;
          if (z - m0 > 14.9f) {
            const float m1 = z - kHeadroom, rise = ex2(m1 - m0);
            f = ex2(m0 - m1);
            tab[2 * kRows + tid] = -m1;
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {  // (what went to fp16 keeps its size)
              const float f0 = tab[(6 + gr) * kRows + tid], f1 = fminf(f0 * rise, kMostFactor);
              tab[(6 + gr) * kRows + tid] = f1;
              times[gr] = __fdividef(f * f1, f0);
            }
          }
          tab[3 * kRows + tid] = f;
          tab[8 * kRows + tid] = times[0];
          tab[9 * kRows + tid] = times[1];
        }
        __syncthreads();
        // every row's largest weight x scale in each group
        each_logit([&](int row, float x, bool seen) {
          const float w = seen ? ex2(fmaf(x, tab[5 * kRows + row], tab[2 * kRows + row])) : 0.f;
#pragma unroll
          for (int gr = 0; gr < GR; ++gr) {
            const float top = warp_max_f32(seen ? w * sv[gr] : 0.f);
            if (lane == 0) red[2 * (qd * kRows + row) + gr] = top;
          }
        });
        __syncthreads();
        if (mine) {
#pragma unroll
          for (int gr = 0; gr < GR; ++gr) {
            const float w = over_warps(2 * tid + gr), f0 = tab[(6 + gr) * kRows + tid];
            if (w * f0 > kLimit) {  // to [2^7, 2^8)
              const float f1 = __uint_as_float((261u - (__float_as_uint(w) >> 23)) << 23);
              tab[(6 + gr) * kRows + tid] = f1;
              tab[(8 + gr) * kRows + tid] *= __fdividef(f1, f0);
            }
          }
        }
        __syncthreads();
        const f32x2* f = reinterpret_cast<const f32x2*>(tab + 3 * kRows + wg * 8);
#pragma unroll
        for (int j = 0; j < kShare / 2; ++j) {
          const f32x2 fj = f[(j >> 2) * (kRows / 4) + (j & 3)];
          l[j] = f2_mul(l[j], fj);
#pragma unroll
          for (int gr = 0; gr < GR; ++gr) pm[gr][j] = f2_mul(pm[gr][j], fj);
        }
        if (pv_count > pv0) {
          // this thread's row (lane) of O, a quarter of its group's channels
          const float fr = tab[(8 + (key >> 6)) * kRows + (key & 63)];
          if (GR == 2 || key < 64) {
            const uint32_t o_at = lanes + C::O + (key < 64 ? 0 : 64) + wg * 16;
            uint32_t o[16];
            tc::tmem_ld_x16(o_at, o);
            tc::tmem_ld_wait16(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fr);
            tc::tmem_st_x16(o_at, o);
            tc::tmem_st_wait();
          }
        }
      }
      if (!ok) break;
      if (warp == kIssueS) {
        tc::fence_after_sync();
        if (i + 1 < nt) issue_s(i + 1);
      } else if (warp == kIssuePV) {
        tc::fence_after_sync();
        issue_pv(i, pv_count);
      } else if (tid == kFetcher) {
        fetch_tile<D, kStages>(a, &ctl.fetch, ctl.split, ctl.full, ring, end);  // into this tile's stage
      }
      if (i + 1 < nt) ++s_count;
      ++pv_count;
    }
    if (!ok) break;
    tiles_read += nt > 0 ? nt : 0;

    // Sums over the keys: the two half-warps, then 16 rows over 16 lanes (each step halves the rows a lane
    // holds), then the warps.
    if (nt > 0) wait_pv(pv_count - 1);
    tc::fence_after_sync();
    auto scatter = [&](const f32x2 (&pairs)[kShare / 2]) {
      float v[kShare];
#pragma unroll
      for (int k = 0; k < kShare; ++k) {
        float a0, a1;
        f2_split(pairs[k / 2], a0, a1);
        v[k] = k & 1 ? a1 : a0;
        v[k] += __shfl_xor_sync(0xffffffffu, v[k], 16);
      }
#pragma unroll
      for (int w = kShare / 2; w >= 1; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int k = 0; k < kShare / 2; ++k) {
          if (k < w) {
            const float give = up ? v[k] : v[k + w], keep = up ? v[k + w] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, w);
          }
        }
      }
      return v[0];
    };
    {
      float* mine = red + (qd * kRows + (lane & 8) * (kRows / 16) + wg * 8 + (lane & 7)) * 3;
      const float sl = scatter(l);
      if (lane < 16) mine[0] = sl;
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) {
        const float sp = scatter(pm[gr]);
        if (lane < 16) mine[1 + gr] = sp;
      }
    }
    if (__syncthreads_or(ctl.abort)) {
      ok = false;
      break;
    }
    {
      const bool whole = n == u.groups;
      float* slot = nullptr;
      if (!whole) slot = a.ws + (2 * (int64_t)blockIdx.x + (t == begin ? 0 : 1)) * slot_floats<D>(kRows);
      // this thread's row of O (the lanes of both groups' halves) and a quarter of the group's channels
      const int row = key & 63, gr = key >> 6, r = u.rb * kRows + row, c0 = 64 * gr + 16 * wg;
      uint32_t o[16];
      if (nt > 0) {
        tc::tmem_ld_x16(lanes + C::O + c0, o);
        tc::tmem_ld_wait16(o);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = 0;
      }
      if (r < a.rows && gr < GR) {
        float sl = 0.f, sp = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          sl += red[(w * kRows + row) * 3];
          sp += red[(w * kRows + row) * 3 + 1 + gr];
        }
        const float inv = sl == 0.f ? 0.f : 1.f / sl;  // a row that attends no key: zeros
        const float undo = __fdividef(1.f, tab[(6 + gr) * kRows + row]);
        float v[16];  // in the channels' order
#pragma unroll
        for (int j = 0; j < 16; ++j) v[(j & 8) + perm8(j & 7)] = fmaf(__uint_as_float(o[j]), undo, sp);
        if (whole) {
          const int64_t at = ((((int64_t)u.l * a.B + u.b) * a.Hq + u.h * a.G) * a.nq + r) * D + c0;
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + at;
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            store4(out + j, make_float4(v[j] * inv, v[j + 1] * inv, v[j + 2] * inv, v[j + 3] * inv));
        } else {
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<float4*>(slot + row * D + c0 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          if (c0 == 0) *reinterpret_cast<float2*>(slot + kRows * D + 2 * row) = make_float2(-tab[2 * kRows + row], sl);
        }
      }
    }
    tc::fence_before_sync();
    __syncthreads();  // tables and accumulators are free for the next unit
    tc::fence_after_sync();
    t += n;
  }

  if (!ok) {  // what is in flight lands in this CTA's memory: wait for it
    __syncthreads();
    if (tid == 0) {
      volatile int none = 0;
      for (int k = max(0, ctl.fetch.fills - kStages); k < ctl.fetch.fills; ++k)
        tc::mbar_wait(&ctl.full[k % kStages], (uint32_t)(k / kStages) & 1u, &none, a.err);
      if (pv_count > 0) tc::mbar_wait(&ctl.pv_done[(pv_count - 1) & 1], ((pv_count - 1) >> 1) & 1u, &none, a.err);
      if (s_count > 0) tc::mbar_wait(&ctl.s_done, (s_count - 1) & 1u, &none, a.err);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, C::N);
}

template <int D>
cudaError_t launch(const Kv4AttnArgs& a, cudaStream_t s) {
  auto* kern = kv4_attn_tc_kernel<D>;
  constexpr int bytes = Lay<D>::BYTES + 1024;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  e = launch_pdl(kern, dim3(a.ctas), dim3(kThreads), bytes, s, a);
  if (e != cudaSuccess) return e;
  return launch_kv4_merge<D, kRows, __nv_bfloat16>(a, s);
}

}  // namespace

int kv4_attn_tc_rows() { return kRows; }

cudaError_t launch_kv4_attn_tc(const Kv4AttnArgs& a, cudaStream_t s) {
  return a.d == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

}  // namespace stdb
