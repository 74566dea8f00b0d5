// Decode attention over a 4-bit K/V cache (format: kv4.cuh), for one query position (a draft
// step) up to gamma + 1 causal ones.
//
//   K_jc = mk_jg + sk_jg a_jc,  V_jc = mv_jg + sv_jg b_jc       codes a, b in 0..15, group g of channel c
//   x_rj = sum_g sk_jg (q_r . a_j)_g + mk_jg (sum q_r)_g                          scaled by log2(e) / sqrt(d)
//   o_rc = [ sum_j (p_rj sv_jg) (b_jc - 8) + sum_j p_rj (mv_jg + 8 sv_jg) ] / sum_j p_rj,   p = 2^(x - M_r)
//
// so the scales never touch the codes: K's multiply the two partial dot products of a key, V's
// multiply the weights (with a factor of the row's and group's own, undone at the end, which keeps the products in
// fp16's range).  A code enters the tensor cores as the fp16 number whose bits are the masked
// code: a subnormal, c 2^-24 (low nibble of a byte) or c 2^-20 (high), exact in the product and in the
// fp32 sum; powers of two in q and in the result undo it.  One mask for two codes is all that widening
// costs.  (The sum over keys has to be centred, b - 8, because sum p b grows without bound while the
// answer stays near the mean: at 140,000 keys the fp32 accumulator would lose it.  A product with a
// matrix of eights, one for sixteen, gathers 8 sum p sv, and is subtracted every few tiles.  What the
// accumulator's own rounding loses until then is 1e-4 of a bf16 result's last place but 5e-5 of the
// result over 2,000 keys: for fp32 queries all codes are centred before they are multiplied.)
//
// A byte of the cache feeds 2 G x rows multiply-adds, and a key's codes have to be widened
// before any of them: at d = 128 a (row, head) is 144 bytes, against 512 in bf16, with 256
// codes, and at full HBM rate an SM has some 400 issue slots for 16 keys, three for a code and lane.  So
// the widened codes go straight from registers into mma.sync (m16n8k16: 16 keys or 16 channels by 8
// query rows), with no shared-memory round trip: K is the A operand of S^T = K q^T,
// V^T the A operand of O^T = V^T P^T, and one movmatrix turns S^T's accumulator layout into
// P^T's operand layout.  A 5th-generation MMA would need the operand written to shared or
// tensor memory first, for 8 of its 128 columns.
//
// The 128-key tiles of all (layer, sequence, KV head, row block) units are split over the CTAs; bulk
// copies stream them through a shared-memory ring, and each of eight warps takes 16 keys of every tile
// with a softmax state of its own.  The states merge once for each unit a CTA touches; units that several
// CTAs touch merge in a second kernel.
//
// Measured: 28 layers x 4 heads x 143,616 keys, 7 rows, 495 to 538 us a call among many, where the power cap holds the
// clock at some 1,740 MHz (4.3 to 4.7 TB/s of 6.46), 460 us in a short sequence at 1,965.  16 keys are 312 instructions
// of a warp; with the 16 warps that 128 registers leave an SM, 59% of the issue slots and 53% of the integer pipe
// are used: four warps a scheduler do not hide their own latencies.
#include "kv4_attn.cuh"

#include <atomic>
#include <type_traits>

namespace stdb {
namespace {

constexpr int kWarps = kTile / 16;       // warps that compute, 16 keys each
constexpr int kThreads = 32 * kWarps;
// 2^70: a sum of weights above it moves the reference too, where scales are so small (0, for constant values) that
// weight x scale never does.  Minima are below 2^41 in magnitude (values up to 2^40), so that sum p (mv + 8 sv) of a
// lane stays below 2^111, and of all warps and CTAs below 2^122.
constexpr float kMostSum = 1.1805916e21f;

// ---------------------------------------------------------------- shared memory
template <int D, int NT, bool F32>
struct Layout {
  static constexpr int CW = TileAt<D>::CW, SW = TileAt<D>::SW, STAGE = TileAt<D>::BYTES;
  static constexpr int ROWS = 8 * NT;
  static constexpr int OSTR = D + 4;                    // row stride of the merge buffer, floats
  static constexpr int MERGE = kWarps * ROWS * OSTR * 4;
  static constexpr int QREGS = NT * (D / 16) * 2;       // a lane's query operands
  static constexpr int Q = QREGS * 128 * (F32 ? 2 : 1);
  static constexpr int BUDGET = NT == 1 && !F32 ? 110 * 1024 : 221 * 1024;
  static constexpr int FIT = (BUDGET - MERGE - Q) / STAGE;
  static constexpr int STAGES = FIT < 16 ? FIT : 16;
  static constexpr int AT_Q = STAGES * STAGE, AT_MERGE = AT_Q + Q;
  static constexpr int BYTES = AT_MERGE + MERGE;
};

constexpr int kMaxStages = 16;
struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  Fetch fetch;
  float m[kWarps][16], l[kWarps][16];
  Split split;
  volatile int abort;
};

// ---------------------------------------------------------------- instructions
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {  // d = a b
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {  // 16-bit elements, rows over lane / 4
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
constexpr uint32_t kEight0 = 0x00080008u, kEight4 = 0x00800080u;  // the code 8 in either place
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_f4(uint32_t a, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ void sts_f2(uint32_t a, float2 v) {
  asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ float column_sum(float v) {  // over the eight lanes of one accumulator column
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

__device__ __forceinline__ void arrive_if(bool on, uint32_t bar) {  // (a predicate, not a branch)
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n"
               ::"r"(bar), "r"((uint32_t)on)
               : "memory");
}

// ---------------------------------------------------------------- a warp's state for one unit
// Lane = 4 g + t.  Query rows are the n index of the matrix instructions: as an operand a lane
// holds row g of each 8-row block, in an accumulator rows 2 t and 2 t + 1.  Accumulator row
// m of S^T is key kappa(m) of the warp's 16: for m < 8 even m are keys m / 2 and odd m
// keys 4 + (m / 2 ^ 1), and likewise 8 higher.  So the four V rows that lane t multiplies
// (operand columns 2 t, 2 t + 1, 2 t + 8, 2 t + 9) are t, 4 + (t ^ 1), 8 + t and 12 + (t ^ 1): four
// neighbouring rows for the quad, and the K rows of neighbouring g lie in different banks.
template <int D, int NT, bool F32>
struct State {
  static constexpr int GR = D / kKv4Group;   // groups
  static constexpr int MT = D / 16;          // 16-channel tiles of O^T
  // The queries, each row scaled by a power of two, are B operands in shared memory, four registers of a lane
  // together: [NT][KS / 2][32 lanes][4], and for fp32 queries what is below fp16 behind them.
  float back[NT][2];                         // a row's power of two: undoes its scaling
  float qsum[NT][GR][2];                     // sum of the scaled q over a group
  float M[NT][2], l[NT][2], pm[NT][GR][2];   // reference, sum p, sum p (mv + 8 sv)
  // A group's weights x scales times this go to fp16.  It puts the row's largest in that group at 2^7 to 2^15, so
  // that they keep their 11 bits (or 2^-32 of the largest) whatever the sizes of the other group and of the minima.
  float factor[NT][GR][2];
  // sum (p sv factor) b, in units of 2^-24 (rows g) and 2^-20 (rows g + 8); fp32 queries: sum (p sv factor) (b - 8)
  float o[NT][MT][4];
  float eight[F32 ? 1 : NT][GR][4];          // sum (p sv factor) 8 of the same keys since the last settle(), same units
};

template <int D, int NT, bool F32>
__device__ __forceinline__ void load_queries(State<D, NT, F32>& st, const Kv4AttnArgs& a, const Unit& u, uint32_t qs,
                                             bool store, int lane) {
  using S = State<D, NT, F32>;
  const int g = lane >> 2, t = lane & 3;
  constexpr int WPL = D / 32;  // words of a row that lane t multiplies
  float x[NT][WPL][8];
  float mul[NT], back[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = u.rb * 8 * NT + nt * 8 + g;
    float top = 0.f;
#pragma unroll
    for (int w = 0; w < WPL; ++w) {
      const int ch = kv4_word_channel<D>(WPL * t + w);
      float(&y)[8] = x[nt][w];
      if (r < a.rows) {
        const int64_t at = ((((int64_t)u.l * a.B + u.b) * a.Hq + u.h * a.G) * a.nq + r) * D + ch;
        if constexpr (F32) {
          const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
          const float4 v0 = p[0], v1 = p[1];
          y[0] = v0.x; y[1] = v0.y; y[2] = v0.z; y[3] = v0.w;
          y[4] = v1.x; y[5] = v1.y; y[6] = v1.z; y[7] = v1.w;
        } else {
          const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at);
          y[0] = lo_bf16(v.x); y[1] = hi_bf16(v.x); y[2] = lo_bf16(v.y); y[3] = hi_bf16(v.y);
          y[4] = lo_bf16(v.z); y[5] = hi_bf16(v.z); y[6] = lo_bf16(v.w); y[7] = hi_bf16(v.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (fabsf(y[i]) < INFINITY) top = fmaxf(top, fabsf(y[i]));  // (a row with an infinity gives NaN by itself)
    }
    // Scale each row by a power of two of its own, so that it keeps its bits whatever the other rows of the
    // block hold: its largest entry lies in [2^14, 2^15), a sixteenth of that where it meets codes at 2^-20.
    // That is exact, and bf16 entries down to 2^-27 of it keep all their bits.  Products come out in units of
    // 2^(ex - 14).
    top = quad_max(top);
    int ex = (int)(__float_as_uint(top) >> 23) - 127;
    ex = ex < -100 ? -100 : ex;
    mul[nt] = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
    back[nt] = __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float sum[S::GR];
#pragma unroll
    for (int gr = 0; gr < S::GR; ++gr) sum[gr] = 0.f;
#pragma unroll
    for (int w = 0; w < WPL; ++w) {
      float(&y)[8] = x[nt][w];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] *= mul[nt];
        sum[S::GR == 2 ? (w & 1) : 0] += y[i];
      }
      if (store) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // channels i and i + 4 of the word: one register; odd i meet codes at 2^-20
          const float x0 = y[i] * (i & 1 && !F32 ? 0.0625f : 1.f), x1 = y[i + 4] * (i & 1 && !F32 ? 0.0625f : 1.f);
          const __half2 hv = __floats2half2_rn(x0, x1);
          const float2 f = __half22float2(hv);
          hi[i] = as_u32(hv);
          lo[i] = as_u32(__floats2half2_rn(x0 - f.x, x1 - f.y));
        }
        const uint32_t at = qs + ((nt * WPL + w) * 32 + lane) * 16;
        sts128(at, hi);
        if constexpr (F32) sts128(at + NT * WPL * 512, lo);
      }
    }
#pragma unroll
    for (int gr = 0; gr < S::GR; ++gr) sum[gr] = quad_sum(sum[gr]) * (F32 ? 1.f : 5.9604645e-8f);  // 2^-24
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int from = 4 * (2 * t + e);  // a lane that holds row 2 t + e
#pragma unroll
      for (int gr = 0; gr < S::GR; ++gr) st.qsum[nt][gr][e] = __shfl_sync(0xffffffffu, sum[gr], from);
      st.back[nt][e] = __shfl_sync(0xffffffffu, back[nt], from);
      st.M[nt][e] = -INFINITY;
      st.l[nt][e] = 0.f;
#pragma unroll
      for (int gr = 0; gr < S::GR; ++gr) {
        st.pm[nt][gr][e] = 0.f;
        st.factor[nt][gr][e] = kMostFactor;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int mt = 0; mt < S::MT; ++mt) st.o[nt][mt][i] = 0.f;
#pragma unroll
      for (int gr = 0; gr < S::GR; ++gr) st.eight[F32 ? 0 : nt][gr][i] = 0.f;
    }
  }
}

// Centre the sums gathered since the last call.
template <int D, int NT, bool F32>
__device__ __forceinline__ void settle(State<D, NT, F32>& st) {
  using S = State<D, NT, F32>;
  if constexpr (!F32) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int mt = 0; mt < S::MT; ++mt) st.o[nt][mt][i] -= st.eight[nt][mt / 4][i];
#pragma unroll
        for (int gr = 0; gr < S::GR; ++gr) st.eight[nt][gr][i] = 0.f;
      }
  }
}

// A lane's byte offsets into shared memory: everything it reads of a warp's 16 rows lies at one of
// them plus the stage's base plus a constant.
template <int D, int NT, bool F32>
struct LaneAt {
  uint32_t k, v, scale, w16, r16;
  __device__ __forceinline__ LaneAt(int warp, int lane) {
    using Lay = Layout<D, NT, F32>;
    const int g = lane >> 2, t = lane & 3;
    const int kap = (g & 1) ? 4 + ((g >> 1) ^ 1) : (g >> 1);
    k = (16 * warp + kap) * Lay::CW + t * (Lay::CW / 4);
    v = TileAt<D>::VC + (16 * warp + t) * Lay::CW + g * (Lay::CW / 8);
    scale = (lane < 16 ? TileAt<D>::KS : TileAt<D>::VS) + (16 * warp + (lane & 15)) * Lay::SW;
    w16 = Lay::AT_MERGE + warp * 512 + lane * (2 * Lay::SW);
    r16 = Lay::AT_MERGE + warp * 512 + kap * (2 * Lay::SW);
  }
};

// A warp's 16 keys of the tile at shared address `tile` (of the ring at `ring`); key0 = the first
// one's position.  MASK: some of the keys may lie past a row's limit, n0 for query position 0 (or past
// the cache, where the shared memory holds stale bytes: codes are finite whatever they are, scales
// are not).
template <int D, int NT, bool F32, bool MASK>
__device__ __forceinline__ void attend16(State<D, NT, F32>& st, const LaneAt<D, NT, F32>& at, uint32_t ring,
                                         uint32_t tile, int key0, int n0, int rb, int nq, int rows, int lane) {
  using S = State<D, NT, F32>;
  using Lay = Layout<D, NT, F32>;
  constexpr int GR = S::GR, WPL = D / 32;
  int lim[NT][2], kap = 0;  // keys a row attends; key of accumulator row lane / 4
  if constexpr (MASK) {
    const int g = lane >> 2, t = lane & 3;
    kap = (g & 1) ? 4 + ((g >> 1) ^ 1) : (g >> 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = (rb * NT + nt) * 8 + 2 * t + e;
        lim[nt][e] = n0 + (row < rows ? row % nq : 0);
      }
  }
  // The 16 keys' scales to fp32, one half-warp for K (with log2(e) / sqrt(d), and 2^24 where codes are
  // subnormals) and one for V, (s, m) of both groups: each lane needs two keys' of each, and four lanes the
  // same ones.
  {
    const float c = lane < 16 && !F32 ? 0.f : 8.f;
    const float f = lane < 16 ? kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f) * (F32 ? 1.f : 16777216.f) : 1.f;
    if constexpr (GR == 2) {
      const uint2 u = lds64(at.scale + tile);
      const float s0 = lo_bf16(u.x), s1 = lo_bf16(u.y);
      sts_f4(at.w16 + ring, make_float4(f * s0, f * s1, f * fmaf(c, s0, hi_bf16(u.x)), f * fmaf(c, s1, hi_bf16(u.y))));
    } else {
      const uint32_t u = lds32(at.scale + tile);
      const float s0 = lo_bf16(u);
      sts_f2(at.w16 + ring, make_float2(f * s0, f * fmaf(c, s0, hi_bf16(u))));
    }
  }

  // S^T: a partial product for each group
  float acc[NT][GR][4];
  uint32_t wa[WPL], wb[WPL];
  {
    const uint32_t ra = at.k + tile, rb = ra + 8 * Lay::CW;
    if constexpr (WPL == 4) {
      const uint4 x = lds128(ra), y = lds128(rb);
      wa[0] = x.x; wa[1] = x.y; wa[2] = x.z; wa[3] = x.w;
      wb[0] = y.x; wb[1] = y.y; wb[2] = y.z; wb[3] = y.w;
    } else {
      const uint2 x = lds64(ra), y = lds64(rb);
      wa[0] = x.x; wa[1] = x.y;
      wb[0] = y.x; wb[1] = y.y;
    }
  }
#pragma unroll
  for (int w = 0; w < WPL; ++w) {
    const int gr = GR == 2 ? (w & 1) : 0;
    uint4 qh[NT], ql[F32 ? NT : 1];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      qh[nt] = lds128(lane * 16 + (ring + Lay::AT_Q + (nt * WPL + w) * 512));
      if constexpr (F32) ql[nt] = lds128(lane * 16 + (ring + Lay::AT_Q + ((NT + nt) * WPL + w) * 512));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t x = k ? wa[w] >> 8 : wa[w], y = k ? wb[w] >> 8 : wb[w];
      const uint32_t a0 = F32 ? centre0(x) : widen0(x), a1 = F32 ? centre0(y) : widen0(y);
      const uint32_t a2 = F32 ? centre4(x) : widen4(x), a3 = F32 ? centre4(y) : widen4(y);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float(&c)[4] = acc[nt][gr];
        if (w < GR && k == 0)
          mma_f16_zero(c, a0, a1, a2, a3, k ? qh[nt].z : qh[nt].x, k ? qh[nt].w : qh[nt].y);
        else
          mma_f16(c, a0, a1, a2, a3, k ? qh[nt].z : qh[nt].x, k ? qh[nt].w : qh[nt].y);
        if constexpr (F32) mma_f16(c, a0, a1, a2, a3, k ? ql[nt].z : ql[nt].x, k ? ql[nt].w : ql[nt].y);
      }
    }
  }

  __syncwarp();
  float sk[2][GR], mk[2][GR], sv[2][GR], mv[2][GR];  // of keys kap and kap + 8
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    if constexpr (GR == 2) {
      const float4 x = lds_f4(at.r16 + (ring + 128 * hf)), y = lds_f4(at.r16 + (ring + 128 * hf + 256));
      sk[hf][0] = x.x; sk[hf][1] = x.y; mk[hf][0] = x.z; mk[hf][1] = x.w;
      sv[hf][0] = y.x; sv[hf][1] = y.y; mv[hf][0] = y.z; mv[hf][1] = y.w;
    } else {
      const float2 x = lds_f2(at.r16 + (ring + 64 * hf)), y = lds_f2(at.r16 + (ring + 64 * hf + 128));
      sk[hf][0] = x.x; mk[hf][0] = x.y; sv[hf][0] = y.x; mv[hf][0] = y.y;
    }
  }

  // Logits and weights against the running reference M.  Element i of an accumulator: key half
  // i / 2, row 2 t + i % 2.  w = p sv factor has to fit fp16 and the sum of p fp32; where they do not (or no
  // reference is set yet) this warp's references move up, factors move, and the weights are taken again.
  float p[NT][4], wt[NT][GR][4], l[NT][2];
  bool seen[NT][4];
  auto dot = [&](int nt, int i) {  // the logit but for the row's power of two
    float x = mk[i >> 1][0] * st.qsum[nt][0][i & 1];
    x = fmaf(sk[i >> 1][0], acc[nt][0][i], x);
    if constexpr (GR == 2) {
      x = fmaf(mk[i >> 1][1], st.qsum[nt][1][i & 1], x);
      x = fmaf(sk[i >> 1][1], acc[nt][1][i], x);
    }
    return x;
  };
  auto probabilities = [&](int nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[nt][i] = ex2(fmaf(dot(nt, i), st.back[nt][i & 1], -st.M[nt][i & 1]));
      if constexpr (MASK) {
        seen[nt][i] = key0 + kap + 8 * (i >> 1) < lim[nt][i & 1];
        if (!seen[nt][i]) p[nt][i] = 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) l[nt][e] = st.l[nt][e] + (p[nt][e] + p[nt][2 + e]);
  };
  auto times_scale = [&](int nt, int gr, int i) {  // (a scale past the limit may be anything)
    if constexpr (MASK) {
      if (!seen[nt][i]) return 0.f;
    }
    return p[nt][i] * sv[i >> 1][gr];
  };
  auto weigh = [&](int nt) {
#pragma unroll
    for (int gr = 0; gr < GR; ++gr)
#pragma unroll
      for (int i = 0; i < 4; ++i) wt[nt][gr][i] = times_scale(nt, gr, i) * st.factor[nt][gr][i & 1];
  };
  float big = 0.f, lbig = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    probabilities(nt);
    weigh(nt);
#pragma unroll
    for (int gr = 0; gr < GR; ++gr) {
      const float m0 = nt + gr == 0 ? wt[nt][gr][0] : fmaxf(big, wt[nt][gr][0]);
      big = max3f(max3f(m0, wt[nt][gr][1], wt[nt][gr][2]), wt[nt][gr][3], m0);
    }
    lbig = max3f(lbig, l[nt][0], l[nt][1]);
  }
  // (a NaN among others is the data's; where all weights are NaN, 0 x infinity, no reference is set)
  if (__any_sync(0xffffffffu, !(big <= kLimit) || !(lbig <= kMostSum))) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2], rise[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float z = -INFINITY;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          if (!MASK || seen[nt][2 * hf + e]) z = fmaxf(z, dot(nt, 2 * hf + e) * st.back[nt][e]);
        z = column_max(z);
        const float m0 = st.M[nt][e], m1 = z - m0 > 14.9f ? z - kHeadroom : m0;
        f[e] = m1 > m0 ? ex2(m0 - m1) : 1.f;
        rise[e] = m1 > m0 ? ex2(m1 - m0) : 1.f;
        st.M[nt][e] = m1;
        st.l[nt][e] *= f[e];
      }
      probabilities(nt);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          // What went to fp16 keeps its size as its reference moves, unless the new largest would not fit: that
          // goes to [2^7, 2^8).
          const float w = column_max(fmaxf(times_scale(nt, gr, e), times_scale(nt, gr, 2 + e)));
          float to = fminf(st.factor[nt][gr][e] * rise[e], kMostFactor);
          if (w * to > kLimit) to = __uint_as_float((261u - (__float_as_uint(w) >> 23)) << 23);
          const float times = __fdividef(f[e] * to, st.factor[nt][gr][e]);
          st.factor[nt][gr][e] = to;
          st.pm[nt][gr][e] *= f[e];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            st.o[nt][gr * 4 + i][e] *= times;
            st.o[nt][gr * 4 + i][2 + e] *= times;
          }
          if constexpr (!F32) {
            st.eight[nt][gr][e] *= times;
            st.eight[nt][gr][2 + e] *= times;
          }
        }
      weigh(nt);
    }
  }

  // P^T operands: rows of a key pack side by side, and an 8 x 8 transposition puts keys there
  uint32_t ph[NT][GR][2], pl[F32 ? NT : 1][F32 ? GR : 1][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    st.l[nt][0] = l[nt][0];
    st.l[nt][1] = l[nt][1];
#pragma unroll
    for (int gr = 0; gr < GR; ++gr)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float w0 = wt[nt][gr][2 * hf], w1 = wt[nt][gr][2 * hf + 1];
        if (!MASK || seen[nt][2 * hf]) st.pm[nt][gr][0] = fmaf(p[nt][2 * hf], mv[hf][gr], st.pm[nt][gr][0]);
        if (!MASK || seen[nt][2 * hf + 1]) st.pm[nt][gr][1] = fmaf(p[nt][2 * hf + 1], mv[hf][gr], st.pm[nt][gr][1]);
        const __half2 hv = __floats2half2_rn(w0, w1);
        ph[nt][gr][hf] = transpose8x8(as_u32(hv));
        if constexpr (F32) {
          const float2 f = __half22float2(hv);
          pl[nt][gr][hf] = transpose8x8(as_u32(__floats2half2_rn(w0 - f.x, w1 - f.y)));
        }
      }
    if constexpr (!F32) {
#pragma unroll
      for (int gr = 0; gr < GR; ++gr)
        mma_f16(st.eight[nt][gr], kEight0, kEight4, kEight0, kEight4, ph[nt][gr][0], ph[nt][gr][1]);
    }
  }

  // O^T += V^T P^T with lane t's values: four keys (t, 4 + (t ^ 1), ...), two words (d = 128: one of each group) of 8
  // channels at 8 g.  A row is CW bytes and the rows of a warp start at a multiple of 4 CW, so t ^ 1
  // is one bit of the address.
  uint32_t v[4][GR];
  {
    const uint32_t even = at.v + tile, odd = even ^ Lay::CW;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t row = ((i & 1) ? odd : even) + 4 * i * Lay::CW;
      if constexpr (GR == 2) {
        const uint2 y = lds64(row);
        v[i][0] = y.x; v[i][1] = y.y;
      } else {
        v[i][0] = lds32(row);
      }
    }
  }
#pragma unroll
  for (int gr = 0; gr < GR; ++gr)
#pragma unroll
    for (int hw = 0; hw < 2; ++hw) {  // low and high halves of the words: channels 0-3 and 4-7
      const uint32_t y01 = __byte_perm(v[0][gr], v[1][gr], hw ? 0x7632 : 0x5410);
      const uint32_t y23 = __byte_perm(v[2][gr], v[3][gr], hw ? 0x7632 : 0x5410);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t b01 = k ? y01 >> 8 : y01, b23 = k ? y23 >> 8 : y23;
        const uint32_t a0 = F32 ? centre0(b01) : widen0(b01), a1 = F32 ? centre4(b01) : widen4(b01);
        const uint32_t a2 = F32 ? centre0(b23) : widen0(b23), a3 = F32 ? centre4(b23) : widen4(b23);
        const int mt = gr * 4 + hw * 2 + k;  // rows g: channel 8 g + 2 (2 hw + k), rows g + 8: the next one
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(st.o[nt][mt], a0, a1, a2, a3, ph[nt][gr][0], ph[nt][gr][1]);
          if constexpr (F32) mma_f16(st.o[nt][mt], a0, a1, a2, a3, pl[nt][gr][0], pl[nt][gr][1]);
        }
      }
    }
}

// Merge the warps' states of one unit and write the output (`whole`) or the partial slot.  False,
// to every thread, once a wait has given up: nothing is written then.
template <int D, int NT, bool F32>
__device__ __forceinline__ bool finish_unit(State<D, NT, F32>& st, const Kv4AttnArgs& a, const Unit& u, Ctl* ctl,
                                            float* buf, bool whole, float* slot, int warp, int lane) {
  using S = State<D, NT, F32>;
  using Lay = Layout<D, NT, F32>;
  using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
  const int g = lane >> 2, t = lane & 3;
  settle(st);
  // (the merge buffer's first bytes were the loop's scratch)
  if (__syncthreads_or(ctl->abort)) return false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      st.l[nt][e] = column_sum(st.l[nt][e]);
#pragma unroll
      for (int gr = 0; gr < S::GR; ++gr) {
        const float c = column_sum(st.pm[nt][gr][e]), undo = __fdividef(1.f, st.factor[nt][gr][e]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          st.o[nt][gr * 4 + i][e] = fmaf(st.o[nt][gr * 4 + i][e], F32 ? undo : undo * 16777216.f, c);         // 2^24
          st.o[nt][gr * 4 + i][2 + e] = fmaf(st.o[nt][gr * 4 + i][2 + e], F32 ? undo : undo * 1048576.f, c);  // 2^20
        }
      }
      const int n = nt * 8 + 2 * t + e;
      if (g == 0) {
        ctl->m[warp][n] = st.M[nt][e];
        ctl->l[warp][n] = st.l[nt][e];
      }
      float* row = buf + (warp * Lay::ROWS + n) * Lay::OSTR;
#pragma unroll
      for (int gr = 0; gr < S::GR; ++gr)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float4*>(row + gr * 64 + 8 * g + 4 * i) =
              make_float4(st.o[nt][gr * 4 + 2 * i][e], st.o[nt][gr * 4 + 2 * i][2 + e], st.o[nt][gr * 4 + 2 * i + 1][e],
                          st.o[nt][gr * 4 + 2 * i + 1][2 + e]);
    }
  __syncthreads();
  for (int i = warp * 32 + lane; i < Lay::ROWS * (D / 4); i += kWarps * 32) {
    const int n = i / (D / 4), c = (i - n * (D / 4)) * 4;
    const int r = u.rb * Lay::ROWS + n;
    if (r >= a.rows) break;
    float top = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ctl->m[w][n]);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float m = ctl->m[w][n];
      const float f = m == -INFINITY ? 0.f : ex2(m - top);
      l = fmaf(f, ctl->l[w][n], l);
      const float4 v = *reinterpret_cast<const float4*>(buf + (w * Lay::ROWS + n) * Lay::OSTR + c);
      sum.x = fmaf(f, v.x, sum.x); sum.y = fmaf(f, v.y, sum.y);
      sum.z = fmaf(f, v.z, sum.z); sum.w = fmaf(f, v.w, sum.w);
    }
    if (whole) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that attends no key: zeros
      const int64_t at = ((((int64_t)u.l * a.B + u.b) * a.Hq + u.h * a.G) * a.nq + r) * D + c;
      store4(static_cast<T*>(a.o) + at, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
    } else {
      *reinterpret_cast<float4*>(slot + n * D + c) = sum;
      if (c == 0) *reinterpret_cast<float2*>(slot + Lay::ROWS * D + 2 * n) = make_float2(top, l);
    }
  }
  __syncthreads();  // the buffers are free for the next unit
  return true;
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kThreads, NT == 1 && !F32 ? 2 : 1) kv4_attn_kernel(const Kv4AttnArgs a) {
  using Lay = Layout<D, NT, F32>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Ctl ctl;
  constexpr int STAGES = Lay::STAGES;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be the same for the warp)
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(&ctl.full[s], 1);
      tc::mbar_init(&ctl.empty[s], kWarps);
    }
    ctl.abort = 0;
    ctl.fetch.fills = ctl.fetch.left = 0;
    tc::fence_mbar_init();
  }
  pdl_wait();  // memory of earlier kernels in the stream is visible from here on
  pdl_trigger();
  if (warp == 0) plan_split(a, &ctl.split, gridDim.x, lane, blockIdx.x == 0);
  __syncthreads();
  const int total = ctl.split.total, share = ctl.split.share;
  const int64_t begin64 = (int64_t)share * blockIdx.x;
  if (begin64 >= total) return;
  const int begin = (int)begin64, end = min(begin + share, total);
  const uint32_t ring = smem_u32(smem);
  if (tid == 0) {
    ctl.fetch.next = begin;
    for (int s = 0; s < STAGES; ++s) fetch_tile<D, STAGES>(a, &ctl.fetch, ctl.split, ctl.full, ring, end);
  }
  const LaneAt<D, NT, F32> at(warp, lane);
  const uint32_t full_at = smem_u32(ctl.full), empty_at = smem_u32(ctl.empty);
  int stage = 0, turn = -1;  // turn: tiles read before this one, mod kWarps (-1: none)
  uint32_t phase = 0;
  for (int t = begin; t < end;) {
    State<D, NT, F32> st;
    int key0, n0, left, rb;
    {
      const Unit u = locate(a, ctl.split, t);
      const int keys = keys_of(a, u.b), group = ctl.split.group, first = u.first * group;
      key0 = first * kTile;
      left = min(min(u.groups - u.first, end - t) * group, (keys + kTile - 1) / kTile - first);  // (may be none)
      n0 = keys - a.nq + 1;  // keys that query position 0 attends
      rb = u.rb;
      load_queries<D, NT, F32>(st, a, u, ring + Lay::AT_Q, warp == 0, lane);
    }
    __syncthreads();
    key0 += 16 * warp;
    for (; left > 0; --left, key0 += kTile) {
      if (!__all_sync(0xffffffffu, tc::mbar_try_wait(full_at + 8 * stage, phase)) &&
          !tc::mbar_wait_warp(&ctl.full[stage], phase, &ctl.abort, a.err))
        break;
      const uint32_t tile = ring + stage * Lay::STAGE;
      if (key0 + 16 <= n0) {
        attend16<D, NT, F32, false>(st, at, ring, tile, 0, 0, 0, 1, 0, lane);
      } else if (key0 < n0 + a.nq - 1) {
        attend16<D, NT, F32, true>(st, at, ring, tile, key0, n0, rb, a.nq, a.rows, lane);
      }
      // The warps take turns to fetch: into the stage of the tile before this one, which the others
      // have most likely left by now.  A fetch comes before its warp leaves this tile, so fetches
      // happen one at a time and in order.
      __syncwarp();
      if (turn == warp) {
        if (lane == 0) {
          const int before = stage == 0 ? STAGES - 1 : stage - 1;
          if (tc::mbar_wait(&ctl.empty[before], stage == 0 ? phase ^ 1 : phase, &ctl.abort, a.err))
            fetch_tile<D, STAGES>(a, &ctl.fetch, ctl.split, ctl.full, ring, end);
        }
        __syncwarp();
      }
      arrive_if(lane == 0, empty_at + 8 * stage);
      turn = (turn + 1) & (kWarps - 1);
      if (turn == 0) settle(st);
      const bool wrap = stage == STAGES - 1;
      phase ^= wrap;
      stage = wrap ? 0 : stage + 1;
    }
    const Unit u = locate(a, ctl.split, t);
    const int n = min(u.groups - u.first, end - t);
    const bool whole = n == u.groups;
    float* slot = nullptr;
    if (!whole) slot = a.ws + (2 * (int64_t)blockIdx.x + (t == begin ? 0 : 1)) * slot_floats<D>(Lay::ROWS);
    if (!finish_unit<D, NT, F32>(st, a, u, &ctl, reinterpret_cast<float*>(smem + Lay::AT_MERGE), whole, slot, warp,
                                 lane))
      break;
    t += n;
  }
  if (ctl.abort && tid == 0) {  // the copies in flight land in this CTA's shared memory: wait for them
    volatile int none = 0;
    for (int k = max(0, ctl.fetch.fills - STAGES); k < ctl.fetch.fills; ++k)
      tc::mbar_wait(&ctl.full[k % STAGES], (uint32_t)(k / STAGES) & 1u, &none, a.err);
  }
}

template <int D, int NT, bool F32>
cudaError_t launch(const Kv4AttnArgs& a, cudaStream_t s) {
  using Lay = Layout<D, NT, F32>;
  auto* kern = kv4_attn_kernel<D, NT, F32>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::BYTES);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  e = launch_pdl(kern, dim3(a.ctas), dim3(kThreads), Lay::BYTES, s, a);
  if (e != cudaSuccess) return e;
  return launch_kv4_merge<D, 8 * NT, typename std::conditional<F32, float, __nv_bfloat16>::type>(a, s);
}

}  // namespace

// More than 16 query rows share a widened code often enough for the tensor-memory kernel (bf16; fp32
// queries need their second fp16 term, and two weights for one, and stay here).  28 layers x 4 heads x
// 33,024 keys, there / here: 16 rows 301 / 198 us, 18 rows 310 / 380, 28 rows 353 / 383, 49 rows 393 / 748.
// (One layer of 16,512 keys: 18 rows 18.8 / 18.1, 28 rows 19.8 / 18.9, 49 rows 23.1 / 25.2.)
static bool on_tensor_memory(const Kv4AttnArgs& a) { return a.dtype == STD_BF16 && a.rows > 16; }

// Query rows of a block, and CTAs of an SM, by the kernel the call takes.
void plan_kv4_attn(Kv4AttnArgs* a, int sms) {
  const bool tm = on_tensor_memory(*a);
  const int block = tm ? kv4_attn_tc_rows() : a->rows <= 8 ? 8 : 16;
  a->row_blocks = (a->rows + block - 1) / block;
  const int64_t tiles = (int64_t)a->L * a->B * a->Hkv * a->row_blocks * ((a->cap + kTile - 1) / kTile);
  const int64_t most = (int64_t)sms * (block == 8 && a->dtype == STD_BF16 ? 2 : 1);
  a->ctas = (int)(tiles < most ? tiles : most);
  a->ws_floats = 2 * a->ctas * (int64_t)block * (a->d + 2);
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t s) {
  if (on_tensor_memory(a)) return launch_kv4_attn_tc(a, s);
  const bool one = a.rows <= 8, f32 = a.dtype == STD_F32;
  if (a.d == 128) {
    if (f32) return one ? launch<128, 1, true>(a, s) : launch<128, 2, true>(a, s);
    return one ? launch<128, 1, false>(a, s) : launch<128, 2, false>(a, s);
  }
  if (f32) return one ? launch<64, 1, true>(a, s) : launch<64, 2, true>(a, s);
  return one ? launch<64, 1, false>(a, s) : launch<64, 2, false>(a, s);
}

}  // namespace stdb
