// Gated feed-forward product over feature rows and its backward pass.
//
//   g = x W0 + b0, u = x W1 + b1, out = act(g) u
//   dg = dh u act'(g), du = dh act(g)
//   dx = dg W0^T + du W1^T, dW = x^T [dg du], db = column sums of [dg du]
//
// Four matrix products on one kernel, k_gated: a persistent cluster of two
// CTAs per pair of SMs issues tcgen05.mma.cta_group::2 (M = 256 rows over the
// pair, N = 128 or 256 columns, fp32 accumulators in tensor memory, two sets),
// fed by TMA through a ring of 64-deep stages.  The modes differ in which
// operands they load, and in the epilogue:
//
//   kPre     A = x rows (K = cin), B = W as it lies (hidden contiguous).  The
//            leader of the pair loads gate columns and its peer the up columns
//            of the same hidden units, so one accumulator row holds g and u of
//            the same units side by side, and act(g) u is formed in registers.
//   kPreBwd  the same products again (nothing is saved by the forward); the
//            epilogue reads dh and writes dg, du, and their sums over 32 rows.
//   kDx      A = [dg du] rows (K = 2 hidden), B = W as it lies (hidden is K).
//   kDw      A = [dg du]^T, B = x (K = rows): the sum over rows is cut into
//            equal shares, one per pair of SMs, whatever tile they fall in; a
//            tile that more than one pair worked on is joined by k_join_dw in
//            a fixed order.
//
// fp32 inputs run on the same tensor cores: each value is split exactly into
// three bf16 parts (8 + 8 + 8 bits), and the six products of parts that matter
// (all but those below 2^-24 of the largest) are accumulated.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "smc_internal.h"
#include "smc_ptx.cuh"
#include "smc_rows.cuh"

namespace smc {
namespace {

using namespace ptx;
using rows::add2;
using rows::dup2;
using rows::fma2;
using rows::mul2;

enum Mode { kPre, kPreBwd, kDx, kDw };

constexpr int kBK = 64;  // depth of a stage: one 128-byte row of 16-bit values
// Sixteen epilogue warps, four per quarter of the tensor-memory lanes: a warp's
// way through a chunk is a chain of latencies (accumulator load, exponential,
// division, staging, fence), so each scheduler gets four of them to interleave
// (55,100 rows, 512 -> 2048 bf16, SiLU: 201 us with eight, 180 us with
// sixteen; its backward's first product 325 and 287 us).
constexpr int kEpiWarp0 = 4, kEpiWarps = 16;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kSmemMax = 227 * 1024;
constexpr uint64_t kAbortDrainNs = 50000000ull;

// An accumulation in tensor memory cuts what falls below the sum's last bit
// instead of rounding it, so its error has one sign and grows with the number of
// steps (terms of one sign lose 6.8e-8 of the final sum per 16-deep step: 8.5e-4
// of a 16-bit dW over 200,000 rows, more than fp16's half step).  Long sums are
// therefore accumulated in pieces, which the epilogue's warps add up in
// registers, rounding: fp32 stage by stage (24 steps); 16-bit sums of more than 64
// stages (LONG) 64 at a time (256 steps, 1.7e-5 of a piece).  Shorter ones go
// without: the registers that the pieces take cost them time (26,214 rows 64 ->
// 256, backward: 45.1 us with pieces throughout, 40.6 us so; 55,100 rows 512 ->
// 2048, whose dW is long: 751 us, 750 us before there were pieces).
constexpr int kLongStages = 64;
template <int DT, bool LONG>
constexpr int piece_stages() {  // 0: the whole range
  return DT == SMC_F32 ? 1 : (LONG ? kLongStages : 0);
}

// fp32: the products of parts that are accumulated, smallest first.  A
// stage holds all three parts of its A and B, so that 96 KB of loads feed six
// products (with a stage per product it would be 192 KB: 26,214 rows, 128 -> 512:
// 36.7 us, 31.5 us so).
constexpr int kPartPairs = 6;
__host__ __device__ constexpr int part_a(int q) { return q == 0 ? 2 : (q == 2 || q == 3 ? 1 : 0); }
__host__ __device__ constexpr int part_b(int q) { return q == 1 ? 2 : (q == 2 || q == 4 ? 1 : 0); }

struct GemmArgs {
  int64_t n;
  int C, H, act;
  int m_tiles, n_tiles;  // kDw: tiles of hidden units per half, of channels
  int k_iters;           // stages of a whole tile
  int pairs;             // clusters launched
  bool early;            // launched while the kernel before runs out
  const void* bias;      // [2][H] of the element type, or null
  void* out;             // kPre out, kDx dx, kDw dW
  const void* dh;
  uint16_t* dgu;         // [n][2 parts][Hp]
  int Hp;
  int tma_out, tma_dh;   // rows are multiples of 16 bytes
  float* db_part;        // [8 m_tiles][2][H], or null
  float* slots;          // kDw: [2 pairs][BN][256] partial tiles
  int32_t* status;
  uint64_t wait_ns;
};

// One accumulation of a pair: a tile and its range of stages.
struct Seg {
  int m, n, s;  // tile row, tile column, half (kDw: 0 gate, 1 up)
  int k0, k1;
};

// The segments of one pair, in order: whole tiles dealt round-robin, or (kDw)
// the pair's equal share of all tiles' stages.
template <int MODE>
struct Walk {
  const GemmArgs& a;
  int64_t cur, end;   // kDw: stages
  int m, n, dm, dn;   // otherwise: the next tile, and the step from tile to tile
  __device__ __forceinline__ Walk(const GemmArgs& args, int pair) : a(args) {
    if constexpr (MODE == kDw) {
      const int64_t all = int64_t(2) * a.m_tiles * a.n_tiles * a.k_iters;
      cur = pair * all / a.pairs;
      end = (pair + 1) * all / a.pairs;
    } else {
      m = pair / a.n_tiles;
      n = pair % a.n_tiles;
      dm = a.pairs / a.n_tiles;
      dn = a.pairs % a.n_tiles;
    }
  }
  __device__ __forceinline__ bool next(Seg& g) {
    if constexpr (MODE == kDw) {
      if (cur >= end) return false;
      int tile = int(cur / a.k_iters);
      g.k0 = int(cur % a.k_iters);
      g.k1 = int(min(int64_t(a.k_iters), g.k0 + end - cur));
      cur += g.k1 - g.k0;
      // channel tiles outermost: pairs half the launch apart then read the
      // same rows of dg and du at the same time, from L2
      g.n = tile / (2 * a.m_tiles);
      tile -= g.n * 2 * a.m_tiles;
      g.s = tile / a.m_tiles;
      g.m = tile % a.m_tiles;
    } else {
      if (m >= a.m_tiles) return false;
      g = Seg{m, n, 0, 0, a.k_iters};
      m += dm;
      n += dn;
      if (n >= a.n_tiles) {
        n -= a.n_tiles;
        ++m;
      }
    }
    return true;
  }
};

// exp2 and 1 / x by the hardware's approximations (2 and 1 ulp).  Results below the
// normal range become 0: an exponential is only ever added to 1, and a sigmoid
// becomes 0 below -87, where SiLU is under 2e-36.
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e), e = exp(-v); e = inf gives the correct limit 0.
__device__ __forceinline__ float2 sigmoid2(float2 v, float2& e) {
  const float2 x = mul2(v, dup2(-kLog2e));
  e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
  const float2 d = add2(e, dup2(1.f));
  return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}

// For GELU and its slope: minus the lower tail of the normal distribution,
// -cdf(-|v|) = -t q(t) exp(-v^2 / 2), t = 1 / (1 + 0.3 |v|), as erfc(x) exp(x^2)
// falls like 1 / x and is smooth in such a t.  q, of degree 7, is fitted to least
// largest relative error (1.2e-7 for |v| up to 13.3, where the exponential leaves
// fp32's range), so that the tail keeps its bits however small it is: in fp32
// within (4 + v^2 / 2) 2^-23 of itself, the second term from the rounded argument
// of the exponential.  Also a = min(|v|, 14), beyond which the tail is 0, and
// e = exp(-v^2 / 2).
__device__ __forceinline__ float2 normal_tail2(float2 v, float2& a, float2& e) {
  const float2 x = mul2(mul2(v, v), dup2(-0.5f * kLog2e));
  e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
  a = make_float2(fminf(fabsf(v.x), 14.f), fminf(fabsf(v.y), 14.f));
  const float2 d = fma2(a, dup2(0.3f), dup2(1.f));
  const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
  float2 q = fma2(t, dup2(-0.0360362306f), dup2(0.158713311f));
  q = fma2(t, q, dup2(-0.20896408f));
  q = fma2(t, q, dup2(0.0560954437f));
  q = fma2(t, q, dup2(-0.129843205f));
  q = fma2(t, q, dup2(-0.0995231271f));
  q = fma2(t, q, dup2(-0.120816886f));
  q = fma2(t, q, dup2(-0.119625174f));
  return mul2(mul2(t, e), q);
}
// v cdf(v) = max(v, 0) - |v| cdf(-|v|)
__device__ __forceinline__ float2 gelu2(float2 v, float2 a, float2 tail) {
  return fma2(a, tail, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

// The activation's value, and its value and slope, of a pair.  Everything that
// can go in pairs does: the epilogue's instructions have to fit beside the
// products (see k_gated).
template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 v) {
  // a maximum with 0 would hide a NaN
  if constexpr (ACT == SMC_ACT_RELU) return make_float2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);
  if constexpr (ACT == SMC_ACT_SILU) {
    float2 e;
    return mul2(v, sigmoid2(v, e));
  }
  if constexpr (ACT == SMC_ACT_GELU) {
    float2 a, e;
    const float2 tail = normal_tail2(v, a, e);
    return gelu2(v, a, tail);
  }
  return v;
}
template <int ACT>
__device__ __forceinline__ void act_both2(float2 v, float2& value, float2& slope) {
  if constexpr (ACT == SMC_ACT_RELU) {
    value = act_value2<ACT>(v);
    slope = make_float2(v.x > 0.f ? 1.f : value.x, v.y > 0.f ? 1.f : value.y);  // 0, or the NaN
  } else if constexpr (ACT == SMC_ACT_SILU) {
    // s + v s (1 - s) with 1 - s = e s: a difference of s and 1, or of v s and
    // v s^2, would leave nothing of it for large v (s is 0 where e is infinite)
    float2 e;
    const float2 s = sigmoid2(v, e);
    value = mul2(v, s);
    constexpr float kMax = 3.402823466e38f;
    slope = fma2(value, mul2(make_float2(fminf(e.x, kMax), fminf(e.y, kMax)), s), s);
  } else if constexpr (ACT == SMC_ACT_GELU) {
    // cdf(v) + v exp(-v^2 / 2) / sqrt(2 pi)
    float2 a, e;
    const float2 tail = normal_tail2(v, a, e), rest = add2(tail, dup2(1.f));
    value = gelu2(v, a, tail);
    slope = fma2(mul2(v, dup2(0.3989422804014327f)), e,
                 make_float2(v.x < 0.f ? -tail.x : rest.x, v.y < 0.f ? -tail.y : rest.y));
  } else {
    value = v;
    slope = dup2(1.f);
  }
}

// x = p[0] + p[1] + p[2] exactly (to 24 bits), each part a bf16 value.  A value
// that rounds up to infinity is cut instead; infinities and NaN stay in p[0].
__device__ __forceinline__ void split3(float x, __nv_bfloat16 (&p)[3]) {
  __nv_bfloat16 h = __float2bfloat16_rn(x);
  if (isinf(__bfloat162float(h)) && !isinf(x)) h = __float2bfloat16_rz(x);
  float r = x - __bfloat162float(h);
  if (!isfinite(x)) r = 0.f;
  p[0] = h;
  p[1] = __float2bfloat16_rn(r);
  p[2] = __float2bfloat16_rn(r - __bfloat162float(p[1]));
}

template <int DT>
struct Elem;
template <>
struct Elem<SMC_F32> {
  using type = float;
};
template <>
struct Elem<SMC_F16> {
  using type = __half;
};
template <>
struct Elem<SMC_BF16> {
  using type = __nv_bfloat16;
};

// Shared memory of a configuration: the ring, the epilogue warps' staging, the
// tail.
template <int MODE, int BN, int DT>
struct Smem {
  static constexpr int kParts = DT == SMC_F32 ? 3 : 1;
  static constexpr int kA = 16384;         // this CTA's 128 rows of A, 64 deep, one part
  static constexpr int kB = BN / 2 * 128;  // its half of B
  static constexpr int kStage = kParts * (kA + kB);
  // A staged chunk is 32 rows of 64 bytes: 32 columns, or 16 of fp32.
  static constexpr int kChunkBytes = 2048;
  static constexpr int kCols = DT == SMC_F32 ? 16 : 32;
  // 32-column groups of a tile's outputs, dealt to four warps per lane quarter
  static constexpr int kTileChunks = MODE == kPre || MODE == kPreBwd ? BN / 64 : BN / 32;
  static constexpr int kChunks = (kTileChunks + 3) / 4;  // per warp
  // kPreBwd: dh of this tile (dg takes its place) and of the next, and du;
  // fp32, whose tiles take six times the products, reads dh and writes the
  // parts of dg and du directly.  kPre, kDx: two outgoing chunks in turn (fp32:
  // one).  kDw stores from registers.
  static constexpr int kSlots = MODE == kDw       ? 0
                                : MODE == kPreBwd ? (DT == SMC_F32 ? 0 : 3)
                                                  : (DT == SMC_F32 ? 1 : 2);
  static constexpr int kWarpStage = kSlots * kChunkBytes;
  static constexpr int kBias = 128;  // bias of a warp's chunk: of g, then of u
  static constexpr int kTailBytes = kEpiWarps * kBias + 512;  // and the barriers
  static constexpr int kStages0 = (kSmemMax - kTailBytes - kEpiWarps * kWarpStage) / kStage;
  static constexpr int kStages = kStages0 > 8 ? 8 : kStages0;
  static constexpr int kBytes = kStages * kStage + kEpiWarps * kWarpStage + kTailBytes;
  static_assert(kStages >= 2, "stages");
};

// Where 16-byte piece `j` of row `r` of a staged chunk lies (the TMA's 64-byte
// swizzle), and the value in column `col`.
__device__ __forceinline__ uint32_t piece(int r, int j) {
  return r * 64 + ((j ^ ((r >> 1) & 3)) << 4);
}
template <int DT>
__device__ __forceinline__ uint32_t value_at(int r, int col) {
  if constexpr (DT == SMC_F32)
    return piece(r, col >> 2) + (col & 3) * 4;
  else
    return piece(r, col >> 3) + (col & 7) * 2;
}

// Eight values of a row into the chunk's type: columns 8 g8 .. (fp32: of the
// chunk's 16).
template <int DT>
__device__ __forceinline__ void put8(uint8_t* chunk, int r, int g8, const float2 (&v)[4]) {
  if constexpr (DT == SMC_F32) {
    *reinterpret_cast<float4*>(chunk + piece(r, 2 * (g8 & 1))) =
        make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    *reinterpret_cast<float4*>(chunk + piece(r, 2 * (g8 & 1) + 1)) =
        make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack2<DT == SMC_BF16>(__float_as_uint(v[i].x), __float_as_uint(v[i].y));
    *reinterpret_cast<uint4*>(chunk + piece(r, g8)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <class T>
__device__ __forceinline__ void unpack8(uint4 x, float2 (&v)[4]) {
  v[0] = rows::unpack2<T>(x.x);
  v[1] = rows::unpack2<T>(x.y);
  v[2] = rows::unpack2<T>(x.z);
  v[3] = rows::unpack2<T>(x.w);
}

// Store a warp's staged chunk at (row0, col0) of a matrix whose rows hold `width`
// values: one TMA store where the rows are 16-byte multiples (it clips what lies
// outside), else row by row with a lane per column (words of two 16-bit values,
// two rows at a time, took longer: 26,213 rows 100 -> 387 fp16, 43 us against 30).
// Every lane calls it; the staging may be written again after bulk_wait_read of
// lane 0 and a __syncwarp.
template <int DT>
__device__ __forceinline__ void store_chunk(const CUtensorMap* map, bool tma, uint8_t* chunk,
                                            void* base, int64_t row0, int col0, int64_t n,
                                            int width, int lane) {
  using T = typename Elem<DT>::type;
  if (tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(map, smem_addr(chunk), col0, int(row0), 0);
      bulk_commit();
    }
  } else {
    constexpr int kCols = 64 / int(sizeof(T)), kStep = 32 / kCols;  // kStep rows at a time
    __syncwarp();
    const int r0 = lane / kCols, col = col0 + lane % kCols;
    const int rows_here = int(min(int64_t(32), n - row0));
    T* to = static_cast<T*>(base) + (row0 + r0) * width + col;
    if (col < width) {
#pragma unroll 8
      for (int r = 0; r < 32; r += kStep)
        if (r + r0 < rows_here)
          to[int64_t(r) * width] =
              *reinterpret_cast<const T*>(chunk + value_at<DT>(r + r0, lane % kCols));
    }
    __syncwarp();
  }
}

// Sums over the warp's lanes of eight values each; lane l ends with the sum of
// value l / 4 (exchanges that halve the values three times, then two plain steps).
__device__ __forceinline__ float sum8(const float (&v)[8], int lane) {
  float a[4], b[2], c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    const float send = up ? v[i] : v[i + 4], keep = up ? v[i + 4] : v[i];
    a[i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    const float send = up ? a[i] : a[i + 2], keep = up ? a[i + 2] : a[i];
    b[i] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
  }
  {
    const bool up = lane & 4;
    const float send = up ? b[0] : b[1], keep = up ? b[1] : b[0];
    c = keep + __shfl_xor_sync(0xffffffffu, send, 4);
  }
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// What one lane needs for its row of a 32 x 32 chunk of g and u.
struct GateRow {
  const uint8_t* bias;  // in shared memory, of g, then of u: 32 columns (fp32: the
                        // half's 16) of each; or null
  uint8_t *slot, *slot_u;
  int lane;
  // fp32, kPreBwd:
  const float* dh;  // the row's dh (dh_vec: 16-byte aligned)
  bool dh_vec, row_ok;
  uint16_t* dgu;  // where the row's dg parts go
  int Hp;
  // kPreBwd:
  int valid;     // columns of the chunk that exist
  float* db;     // the chunk's column sums of dg, or null
  int64_t db_u;  // from there to those of du
};

// Column sums of eight columns of dg (s = 0) or du before they are rounded.
__device__ __forceinline__ void sum_columns(const float (&v)[8], int s, int g8, const GateRow& c) {
  const float sum = sum8(v, c.lane);
  const int col = g8 * 8 + (c.lane >> 2);
  if ((c.lane & 3) == 0 && col < c.valid) c.db[s * c.db_u + col] = sum;
}

// Columns g8 * 8 .. + 7 of g and u: accumulators and bias.
template <int DT, bool BIAS>
__device__ __forceinline__ void biased8(const uint32_t* gv, const uint32_t* uv, int g8,
                                        const GateRow& c, float2 (&gg)[4], float2 (&uu)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    gg[i] = make_float2(__uint_as_float(gv[2 * i]), __uint_as_float(gv[2 * i + 1]));
    uu[i] = make_float2(__uint_as_float(uv[2 * i]), __uint_as_float(uv[2 * i + 1]));
  }
  if constexpr (BIAS) {
    using T = typename Elem<DT>::type;
    float2 b[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint8_t* from =
          c.bias + (DT == SMC_F32 ? 16 * k + (g8 & 1) * 8 : 32 * k + g8 * 8) * sizeof(T);
      if constexpr (DT == SMC_F32) {
        const float4 p = reinterpret_cast<const float4*>(from)[0];
        const float4 q = reinterpret_cast<const float4*>(from)[1];
        b[k][0] = make_float2(p.x, p.y), b[k][1] = make_float2(p.z, p.w);
        b[k][2] = make_float2(q.x, q.y), b[k][3] = make_float2(q.z, q.w);
      } else {
        unpack8<T>(*reinterpret_cast<const uint4*>(from), b[k]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      gg[i] = add2(gg[i], b[0][i]);
      uu[i] = add2(uu[i], b[1][i]);
    }
  }
}

// kPre: act(g) u into `slot`; kPreBwd, 16-bit: dh from `slot`, dg in its place
// and du into `slot_u`, rounded to the operands' type: the matrix unit multiplies
// them with 16-bit W and x.  That adds as much error to dx and dW as their own
// rounding does (55,100 rows 512 -> 2048 bf16: 2.3e-3 in place of 1.7e-3 of the
// values' size); a second 16-bit part of dg and du would take it away at twice
// the products of dx and dW, which are 333 of the call's 570 us of kernels.
template <int MODE, int DT, int ACT, bool BIAS>
__device__ __forceinline__ void gate8(const uint32_t* gv, const uint32_t* uv, int g8,
                                      const GateRow& c) {
  float2 gg[4], uu[4];
  biased8<DT, BIAS>(gv, uv, g8, c, gg, uu);
  if constexpr (MODE == kPre) {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(act_value2<ACT>(gg[i]), uu[i]);
    put8<DT>(c.slot, c.lane, g8, v);
  } else {
    using T = typename Elem<DT>::type;
    float2 dh[4], G[4], U[4];
    unpack8<T>(*reinterpret_cast<const uint4*>(c.slot + piece(c.lane, g8)), dh);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 value, slope;
      act_both2<ACT>(gg[i], value, slope);
      G[i] = mul2(mul2(dh[i], uu[i]), slope);  // dh is 0 in rows and columns that do not exist
      U[i] = mul2(dh[i], value);
    }
    put8<DT>(c.slot, c.lane, g8, G);
    put8<DT>(c.slot_u, c.lane, g8, U);
    if (c.db) {
      const float g[8] = {G[0].x, G[0].y, G[1].x, G[1].y, G[2].x, G[2].y, G[3].x, G[3].y};
      const float u[8] = {U[0].x, U[0].y, U[1].x, U[1].y, U[2].x, U[2].y, U[3].x, U[3].y};
      sum_columns(g, 0, g8, c);
      sum_columns(u, 1, g8, c);
    }
  }
}

// Eight words as one 32-byte store: a whole sector.
__device__ __forceinline__ void store_32(void* to, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// kPreBwd, fp32, sixteen columns: the parts of dg, then of du (the activation
// is taken twice rather than both held), 32 bytes of a row at a time, and the
// column sums.
template <int ACT, bool BIAS>
__device__ __forceinline__ void gate16_parts(const uint32_t* gv, const uint32_t* uv, int hf,
                                             const GateRow& c) {
  const int left = c.row_ok ? c.valid - hf * 16 : 0;
  float dh[16];
  if (c.dh_vec && left >= 16) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 p = *reinterpret_cast<const float4*>(c.dh + hf * 16 + i);
      dh[i] = p.x, dh[i + 1] = p.y, dh[i + 2] = p.z, dh[i + 3] = p.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) dh[i] = i < left ? c.dh[hf * 16 + i] : 0.f;
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint32_t parts[3][8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 gg[4], uu[4];
      float v[8];
      biased8<SMC_F32, BIAS>(gv + 8 * j, uv + 8 * j, j, c, gg, uu);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 value, slope;
        act_both2<ACT>(gg[i], value, slope);
        const float2 d = make_float2(dh[8 * j + 2 * i], dh[8 * j + 2 * i + 1]);
        const float2 r = s == 0 ? mul2(mul2(d, uu[i]), slope) : mul2(d, value);
        v[2 * i] = r.x;
        v[2 * i + 1] = r.y;
        __nv_bfloat16 lo[3], hi[3];
        split3(r.x, lo);
        split3(r.y, hi);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          parts[p][4 * j + i] = uint32_t(__bfloat16_as_ushort(lo[p])) |
                                uint32_t(__bfloat16_as_ushort(hi[p])) << 16;
      }
      if (c.db) sum_columns(v, s, 2 * hf + j, c);
    }
    if (left > 0) {
#pragma unroll
      for (int p = 0; p < 3; ++p) store_32(c.dgu + (p * 2 + s) * c.Hp + hf * 16, parts[p]);
    }
  }
}

// Sixteen columns (half `hf` of the chunk).  The activation and the presence of
// a bias are chosen once here, so that the code of a choice is straight.
template <int MODE, int DT>
__device__ __forceinline__ void gate16(const uint32_t (&gv)[16], const uint32_t (&uv)[16], int hf,
                                       int act, const GateRow& c) {
  auto go = [&](auto a, auto b) {
    if constexpr (MODE == kPreBwd && DT == SMC_F32) {
      gate16_parts<decltype(a)::value, decltype(b)::value>(gv, uv, hf, c);
    } else {
      gate8<MODE, DT, decltype(a)::value, decltype(b)::value>(gv, uv, 2 * hf, c);
      gate8<MODE, DT, decltype(a)::value, decltype(b)::value>(gv + 8, uv + 8, 2 * hf + 1, c);
    }
  };
  auto choose = [&](auto b) {
    switch (act) {
      case SMC_ACT_RELU:
        return go(std::integral_constant<int, SMC_ACT_RELU>(), b);
      case SMC_ACT_SILU:
        return go(std::integral_constant<int, SMC_ACT_SILU>(), b);
      case SMC_ACT_GELU:
        return go(std::integral_constant<int, SMC_ACT_GELU>(), b);
      default:
        return go(std::integral_constant<int, SMC_ACT_NONE>(), b);
    }
  };
  if (c.bias)
    choose(std::true_type());
  else
    choose(std::false_type());
}

template <int MODE, int BN, int DT, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
k_gated(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
        const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_dh,
        const GemmArgs a) {
  using L = Smem<MODE, BN, DT>;
  using T = typename Elem<DT>::type;
  constexpr int kStages = L::kStages;
  constexpr bool kPreMode = MODE == kPre || MODE == kPreBwd;
  constexpr uint32_t kTmemCols = 2 * BN;
  constexpr int kPiece = piece_stages<DT, LONG>();
  constexpr bool kStageSums = kPiece > 0;  // pieces are added up in registers
  constexpr int kSums = kStageSums ? (kPreMode ? 2 : L::kChunks) * 32 : 1;
  // M = 256 over the pair; A is MN-major in kDw, B in all modes but kDx
  constexpr uint32_t kIdesc = (1u << 4) | ((DT != SMC_F16 ? 1u : 0u) << 7) |
                              ((DT != SMC_F16 ? 1u : 0u) << 10) | ((MODE == kDw ? 1u : 0u) << 15) |
                              ((MODE != kDx ? 1u : 0u) << 16) | (uint32_t(BN >> 3) << 17) |
                              (16u << 24);

  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* staging = smem + kStages * L::kStage;
  uint8_t* bias_smem = staging + kEpiWarps * L::kWarpStage;  // [kEpiWarps][kBias]
  uint64_t* bars = reinterpret_cast<uint64_t*>(bias_smem + kEpiWarps * L::kBias);
  // full[kStages] empty[kStages] tfull[2] tempty[2] drain dh[kEpiWarps][2]
  constexpr int kBars = 2 * kStages + 5 + 2 * kEpiWarps;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  static_assert(kBars * 8 + 8 <= 512, "barriers");
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1;
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * kStages;
  const uint32_t tfull0 = empty0 + 8 * kStages, tempty0 = tfull0 + 16, drain = tempty0 + 16;
  const uint32_t dh0 = drain + 8;
  const uint32_t ring0 = smem_addr(ring);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);   // the leader's producer; both CTAs' bytes
      mbar_init(empty0 + 8 * s, 1);  // the leader's commit, in both CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull0 + 8 * i, 1);
      mbar_init(tempty0 + 8 * i, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    for (int w = 0; w < 2 * kEpiWarps; ++w) mbar_init(dh0 + 8 * w, 1);
    *abort_flag = 0;
    mbar_init_fence_cluster();
    // the 128-byte swizzle needs the ring 1024-byte aligned
    if ((ring0 & 1023u) != 0) {
      *abort_flag = 1;
      atomicOr(a.status, kDevLayout);
    }
  }
  if (warp == 2) tmem_alloc_pair(smem_addr(tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  rows::let_next_start();
  rows::after_previous();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const Waits waits{abort_flag, a.status, a.wait_ns};
  Walk<MODE> walk(a, pair);
  Seg g;

  if (warp == 0 && lane == 0) {
    // ---------------- producer: this CTA's rows of A, its half of B ----------
    const uint32_t lead_full0 = map_to_rank(full0, 0);
    int st = 0;
    uint32_t phase = 0;
    bool ok = *abort_flag == 0;
    while (ok && walk.next(g)) {
      for (int it = g.k0; it < g.k1; ++it) {
        if (!(ok = waits.wait(empty0 + 8 * st, phase ^ 1))) break;
        if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * st, 2 * L::kStage);
        const uint32_t bar = lead_full0 + 8 * st;
        const int k = it * kBK;
#pragma unroll
        for (int p = 0; p < L::kParts; ++p) {
          const uint32_t da = ring0 + st * L::kStage + p * L::kA;
          const uint32_t db = ring0 + st * L::kStage + L::kParts * L::kA + p * L::kB;
          if constexpr (kPreMode) {
            tma_load_3d_pair(da, &map_a, k, g.m * 256 + int(rank) * 128, p, bar);
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_load_3d_pair(db + j * 8192, &map_b, g.n * (BN / 2) + j * 64, k, p * 2 + int(rank),
                               bar);
          } else if constexpr (MODE == kDx) {
            const int half = a.k_iters >> 1, s = it >= half ? 1 : 0;
            const int h = (it - s * half) * kBK;
            tma_load_3d_pair(da, &map_a, h, p * 2 + s, g.m * 256 + int(rank) * 128, bar);
            tma_load_3d_pair(db, &map_b, h, g.n * BN + int(rank) * (BN / 2), p * 2 + s, bar);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_3d_pair(da + j * 8192, &map_a, g.m * 256 + int(rank) * 128 + j * 64,
                               p * 2 + g.s, k, bar);
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_load_3d_pair(db + j * 8192, &map_b, g.n * BN + int(rank) * (BN / 2) + j * 64, k,
                               p, bar);
          }
        }
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------- the pair's MMAs (leader only) ---------------------------
    int st = 0, seg = 0;
    uint32_t phase = 0;
    bool ok = *abort_flag == 0;
    while (ok && walk.next(g)) {
      int acc = 0;
      for (int it = g.k0; it < g.k1; ++it) {
        const int piece_it = kPiece > 0 ? (it - g.k0) % kPiece : it - g.k0;
        if (piece_it == 0) {  // a new accumulation
          acc = seg & 1;
          if (!(ok = waits.wait(tempty0 + 8 * acc, ((seg >> 1) & 1) ^ 1))) break;
          ++seg;
        }
        if (!(ok = waits.wait(full0 + 8 * st, phase))) break;
        tc_fence_after();
        const uint32_t stage = ring0 + st * L::kStage;
#pragma unroll
        for (int q = 0; q < (L::kParts == 1 ? 1 : kPartPairs); ++q) {
          const uint32_t sa = stage + (L::kParts == 1 ? 0 : part_a(q)) * L::kA;
          const uint32_t sb = stage + L::kParts * L::kA + (L::kParts == 1 ? 0 : part_b(q)) * L::kB;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k) {
            const uint64_t da = MODE == kDw ? desc_b_mnmajor(sa + k * 2048, 8192)
                                            : desc_a_kmajor(sa + k * 32);
            const uint64_t db = MODE != kDx ? desc_b_mnmajor(sb + k * 2048, 8192)
                                            : desc_a_kmajor(sb + k * 32);
            umma_f16_pair(tmem + acc * BN, da, db, kIdesc,
                          piece_it > 0 || q > 0 || k > 0);
          }
        }
        umma_commit_pair(empty0 + 8 * st);
        if (piece_it + 1 == kPiece || it + 1 == g.k1) umma_commit_pair(tfull0 + 8 * acc);
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {  // let what was issued finish before memory is released
      umma_commit_pair(drain);
      mbar_drain(drain, 0);
      for (int s = 0; s < kStages; ++s) {
        // loads of stages that were announced and not consumed
        const uint64_t t0 = global_ns();
        const uint32_t p = s >= st ? phase : phase ^ 1;
        while (!mbar_try_wait(full0 + 8 * s, p) && global_ns() - t0 < kAbortDrainNs) {
        }
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------- epilogue -------------------------------------------------
    const int quarter = warp & 3, group = (warp - kEpiWarp0) >> 2, w = warp - kEpiWarp0;
    uint8_t* mine = staging + w * L::kWarpStage;
    T* bias_w = reinterpret_cast<T*>(bias_smem + w * L::kBias);
    const uint32_t lead_tempty0 = map_to_rank(tempty0, 0);
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t dh_bar0 = dh0 + 16 * w;
    const int hc = group * 32;  // kPre, kPreBwd: the warp's chunk of every tile
    const int64_t my_rows = rank * 128 + quarter * 32;
    int seg = 0, stored = 0;  // stored: the slot of the next store
    uint32_t dh_phases = 0;  // the parity to wait for next, per slot
    bool ok = *abort_flag == 0;

    // What a tile's epilogue needs from memory, asked for one tile ahead: its bias
    // values, and dh into the staging.
    T next_bias[2] = {};
    auto live_of = [&](const Seg& t) {
      return hc < BN / 2 && int64_t(t.m) * 256 + my_rows < a.n && t.n * (BN / 2) + hc < a.H;
    };
    auto prefetch = [&](const Seg& t, int slot) {
      if (!kPreMode || !live_of(t)) return;
      const int h = t.n * (BN / 2) + hc;
      if (a.bias) {
        // 16-bit: of g and of u in column `lane`; fp32: of g (lanes 0-15) and u
        // (16-31) in the first 16 columns, and the second
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = h + (DT == SMC_F32 ? 16 * k + (lane & 15) : lane);
          const int row = DT == SMC_F32 ? lane >> 4 : k;
          if (col < a.H) next_bias[k] = static_cast<const T*>(a.bias)[row * a.H + col];
        }
      }
      if constexpr (MODE == kPreBwd && DT != SMC_F32) {
        const int64_t row0 = int64_t(t.m) * 256 + my_rows;
        uint8_t* to = mine + slot * L::kChunkBytes;
        if (a.tma_dh) {
          fence_proxy_async_smem();  // all lanes have read and written the slot
          __syncwarp();
          if (lane == 0) {
            bulk_wait_read<0>();
            mbar_arrive_expect_tx(dh_bar0 + 8 * slot, L::kChunkBytes);
            tma_load_3d(smem_addr(to), &map_dh, h, int(row0), 0, dh_bar0 + 8 * slot);
          }
        } else {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          const int rows_here = int(min(int64_t(32), a.n - row0));
          const T* from = static_cast<const T*>(a.dh) + row0 * a.H + h + lane;
#pragma unroll 8
          for (int r = 0; r < 32; ++r)
            *reinterpret_cast<T*>(to + value_at<DT>(r, lane)) =
                r < rows_here && h + lane < a.H ? from[int64_t(r) * a.H]
                                                : rows::from_float<T>(0.f);
        }
      }
    };
    Seg gn;
    bool more = ok && walk.next(g);
    if (more) prefetch(g, 0);
    for (int turn = 0; ok && more; g = gn, ++turn) {
      const int slot = turn & 1;
      const int64_t row0 = int64_t(g.m) * 256 + my_rows;
      // The accumulation that is next, from the warp's lanes of tensor memory.
      uint32_t d = 0;
      int acc = 0;
      auto next_sums = [&]() {
        acc = seg & 1;
        d = lanes + acc * BN;
        const bool got = waits.wait(tfull0 + 8 * acc, (seg >> 1) & 1);
        tc_fence_after();
        ++seg;
        return got;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8 * acc);
      };
      // The pieces' sums, added up.  Value i is column column_of(i / 32) + i % 32.
      float sums[kSums];
      auto add_pieces = [&](bool live, auto column_of) {
#pragma unroll
        for (int i = 0; i < kSums; ++i) sums[i] = 0.f;
        for (int it = g.k0; it < g.k1; it += kStageSums ? kPiece : 1) {
          if (!next_sums()) return false;
          if (live) {
#pragma unroll
            for (int i = 0; i < kSums; i += 16) {
              uint32_t v[16];
              tmem_ld_x16_async(d + column_of(i / 32) + i % 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) sums[i + j] += __uint_as_float(v[j]);
            }
          }
          release();
        }
        return true;
      };
      if constexpr (kPreMode) {
        // one chunk per warp: units h .. h + 31 of the rows row0 .. row0 + 31
        const int h = g.n * (BN / 2) + hc;
        const bool live = live_of(g);
        const T bias[2] = {next_bias[0], next_bias[1]};
        if constexpr (DT != SMC_F32) {
          bias_w[lane] = bias[0];
          bias_w[32 + lane] = bias[1];
        }
        __syncwarp();
        more = walk.next(gn);
        if (more) prefetch(gn, slot ^ 1);
        if constexpr (kStageSums) {
          ok = add_pieces(live, [&](int k) { return k * (BN / 2) + hc; });
          if (!ok) break;
        } else {
          if (!(ok = next_sums())) break;
        }
        if (!live) {
          if (!kStageSums) release();
          continue;
        }
        // kPre: act(g) u, in the slot of the store before last; kPreBwd: dh, then dg
        uint8_t* out = mine + (MODE == kPre && DT != SMC_F32 ? stored * L::kChunkBytes : 0);
        if constexpr (MODE == kPreBwd && DT != SMC_F32) {
          out += slot * L::kChunkBytes;
          if (a.tma_dh) {
            // a slot's barrier completes a phase for each live tile of it
            if (!(ok = waits.wait(dh_bar0 + 8 * slot, (dh_phases >> slot) & 1))) break;
            dh_phases ^= 1u << slot;
          }
          if (lane == 0) bulk_wait_read<0>();  // du of the last tile
        } else {
          if (lane == 0) bulk_wait_read<MODE == kPre && DT != SMC_F32 ? 1 : 0>();
          stored ^= 1;
        }
        __syncwarp();
        uint8_t* out_u = mine + 2 * L::kChunkBytes;  // kPreBwd, 16-bit
        const int64_t block = (int64_t(g.m) * 2 + rank) * 4 + quarter;
        float* db = MODE == kPreBwd && a.db_part ? a.db_part + block * 2 * a.H + h : nullptr;
        GateRow row{a.bias ? reinterpret_cast<const uint8_t*>(bias_w) : nullptr, out, out_u, lane};
        if constexpr (MODE == kPreBwd && DT == SMC_F32) {
          row.dh = static_cast<const float*>(a.dh) + (row0 + lane) * a.H + h;
          row.dh_vec = a.tma_dh != 0;
          row.row_ok = row0 + lane < a.n;
          row.dgu = a.dgu + (row0 + lane) * 6 * a.Hp + h;
          row.Hp = a.Hp;
        }
        if constexpr (MODE == kPreBwd) {
          row.valid = a.H - h;
          row.db = db;
          row.db_u = a.H;
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t gv[16], uv[16];
          if constexpr (kStageSums) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              gv[i] = __float_as_uint(sums[hf * 16 + i]);
              uv[i] = __float_as_uint(sums[32 + hf * 16 + i]);
            }
          } else {
            tmem_ld_x16_async(d + hc + hf * 16, gv);
            tmem_ld_x16_async(d + BN / 2 + hc + hf * 16, uv);
            tmem_ld_wait();
            if (hf == 1) release();
          }
          if constexpr (DT == SMC_F32) {
            __syncwarp();
            bias_w[lane] = bias[hf];
            if (hf == 1 && lane == 0) bulk_wait_read<0>();  // the first half's store
            __syncwarp();
          }
          gate16<MODE, DT>(gv, uv, hf, a.act, row);
          if constexpr (MODE == kPre && DT == SMC_F32)
            if (h + hf * 16 < a.H)
              store_chunk<DT>(&map_out, a.tma_out, out, a.out, row0, h + hf * 16, a.n, a.H,
                              lane);
        }
        if constexpr (MODE == kPre && DT != SMC_F32) {
          store_chunk<DT>(&map_out, a.tma_out, out, a.out, row0, h, a.n, a.H, lane);
        } else if constexpr (MODE == kPreBwd && DT != SMC_F32) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&map_out, smem_addr(out), h, 0, int(row0));
            tma_store_3d(&map_out, smem_addr(out_u), h, 1, int(row0));
            bulk_commit();
          }
        }
        __syncwarp();
      } else {
        more = walk.next(gn);
        if constexpr (kStageSums)
          ok = add_pieces(true, [&](int k) { return (group * L::kChunks + k) * 32; });
        else
          ok = next_sums();
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c) {
          const int cc = (group * L::kChunks + c) * 32, col = g.n * BN + cc;
          uint32_t v[32];
          if constexpr (kStageSums) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(sums[c * 32 + i]);
          } else {
            tmem_ld_x32_async(d + cc, v);
            tmem_ld_wait();
            if (c == L::kChunks - 1) release();
          }
          if (col >= a.C) continue;
          if constexpr (MODE == kDx) {
            if (row0 >= a.n) continue;
#pragma unroll
            for (int part = 0; part < 32 / L::kCols; ++part) {
              if (col + part * L::kCols >= a.C) continue;
              uint8_t* to = mine + (DT != SMC_F32 ? stored * L::kChunkBytes : 0);
              stored ^= 1;
              if (lane == 0) bulk_wait_read<DT != SMC_F32 ? 1 : 0>();
              __syncwarp();
#pragma unroll
              for (int g8 = 0; g8 < L::kCols / 8; ++g8) {
                const uint32_t* from = v + part * L::kCols + g8 * 8;
                float2 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  f[i] = make_float2(__uint_as_float(from[2 * i]), __uint_as_float(from[2 * i + 1]));
                put8<DT>(to, lane, g8, f);
              }
              store_chunk<DT>(&map_out, a.tma_out, to, a.out, row0, col + part * L::kCols, a.n,
                              a.C, lane);
            }
          } else {
            const int64_t h = row0 + lane;
            if (g.k0 == 0 && g.k1 == a.k_iters) {
              T* to = static_cast<T*>(a.out) + (int64_t(g.s) * a.C + col) * a.H + h;
              if (h < a.H) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (col + i < a.C)
                    to[int64_t(i) * a.H] = rows::from_float<T>(__uint_as_float(v[i]));
              }
            } else {
              float* to = a.slots + (int64_t(2 * pair + (g.k0 == 0 ? 1 : 0)) * BN + cc) * 256 +
                          rank * 128 + quarter * 32 + lane;
#pragma unroll
              for (int i = 0; i < 32; ++i) to[i * 256] = __uint_as_float(v[i]);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_read<0>();
    if (MODE == kPreBwd && DT != SMC_F32 && !ok && lane == 0) {  // dh copies may be in flight
      const uint64_t t0 = global_ns();
      for (int i = 0; i < 2; ++i)
        while (!mbar_try_wait(dh_bar0 + 8 * i, (dh_phases >> i) & 1) &&
               global_ns() - t0 < kAbortDrainNs) {
        }
    }
    tc_fence_before();
  }
  __syncthreads();
  __syncwarp();
  cluster_sync();  // both CTAs are done with each other's memory
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// dW of the tiles that several pairs worked on: their partial tiles in the
// order of the pairs.  A block takes COLS columns (input channels) of a tile; a
// thread has up to eight pairs' values of each in flight.  I: an integer that
// holds the tiles times their stages times the pairs (32 bits divide several
// times faster).
template <class T, class I, int COLS>
__global__ void __launch_bounds__(256)
k_join_dw(const float* __restrict__ slots, T* __restrict__ dW, int C, int H, int m_tiles,
          int n_tiles, int k_iters, int pairs, int bn) {
  rows::let_next_start();
  rows::after_previous();
  int tile = blockIdx.x;
  const int cl = blockIdx.y * COLS, c = tile / (2 * m_tiles) * bn + cl;
  if (c >= C) return;
  const I all = I(2) * m_tiles * n_tiles * k_iters;
  const I i0 = I(tile) * k_iters, i1 = i0 + k_iters;
  const int p0 = int(((i0 + 1) * pairs - 1) / all), p1 = int((i1 * pairs - 1) / all);
  if (p0 == p1) return;  // one pair stored it whole
  // the first pair has the tile's first stage, so its part is in its second slot
  const int64_t first = 2 * int64_t(p0) + 1;
  tile %= 2 * m_tiles;
  const int64_t s = tile / m_tiles, h = int64_t(tile % m_tiles) * 256 + threadIdx.x;
  if (h >= H) return;
  const float* from = slots + cl * 256 + threadIdx.x;
  const int64_t slot = int64_t(bn) * 256;
  float v[COLS];
#pragma unroll
  for (int i = 0; i < COLS; ++i) v[i] = from[first * slot + i * 256];
#pragma unroll 8
  for (int p = p0 + 1; p <= p1; ++p) {
#pragma unroll
    for (int i = 0; i < COLS; ++i) v[i] += from[2 * p * slot + i * 256];
  }
#pragma unroll
  for (int i = 0; i < COLS; ++i)
    if (c + i < C) dW[(s * C + c + i) * H + h] = rows::from_float<T>(v[i]);
}

// dbias: the sums over 32 rows, added up in a fixed order: a block takes 32
// columns, its 32 warps every 32nd sum, then the warps in order.
template <class T>
__global__ void __launch_bounds__(1024)
k_join_db(const float* __restrict__ part, T* __restrict__ dbias, int64_t blocks, int H2) {
  __shared__ float sums[32][33];
  rows::let_next_start();
  rows::after_previous();
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < H2) {
#pragma unroll 8
    for (int64_t b = w; b < blocks; b += 32) s += part[b * H2 + col];
  }
  sums[w][lane] = s;
  __syncthreads();
  if (w == 0 && col < H2) {
    for (int i = 1; i < 32; ++i) s += sums[i][lane];
    dbias[col] = rows::from_float<T>(s);
  }
}

// A matrix [rows][cols] and its 16-bit copy [parts][rows][cols_p].
struct Packing {
  const void* src;
  uint16_t* dst;
  int64_t rows;
  int cols, cols_p;
};

// Copies of up to two matrices: the three bf16 parts of fp32 values, or the
// values themselves, rows padded with zeros to a multiple of 16 bytes.
template <class T>
__global__ void __launch_bounds__(256) k_pack(const Packing one, const Packing two) {
  rows::let_next_start();
  rows::after_previous();
  const int64_t n1 = one.rows * (one.cols_p / 8), n2 = two.rows * (two.cols_p / 8);
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < n1 + n2;
       i += int64_t(gridDim.x) * 256) {
    const Packing& p = i < n1 ? one : two;
    const int64_t at = i < n1 ? i : i - n1;
    const int per_row = p.cols_p / 8;
    const int64_t r = at >> 32 ? at / per_row : uint32_t(at) / uint32_t(per_row);
    const int c = int(at - r * per_row) * 8;
    const T* from = static_cast<const T*>(p.src) + r * p.cols + c;
    alignas(16) uint16_t v[3][8] = {};
    alignas(16) T x[8];
    if (p.cols % 8 == 0) {
#pragma unroll
      for (int j = 0; j < int(sizeof(T)) / 2; ++j)
        reinterpret_cast<uint4*>(x)[j] = reinterpret_cast<const uint4*>(from)[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = c + j < p.cols ? from[j] : rows::from_float<T>(0.f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (sizeof(T) == 4) {
        __nv_bfloat16 q[3];
        split3(x[j], q);
#pragma unroll
        for (int k = 0; k < 3; ++k) v[k][j] = __bfloat16_as_ushort(q[k]);
      } else {
        v[0][j] = *reinterpret_cast<const uint16_t*>(&x[j]);
      }
    }
#pragma unroll
    for (int k = 0; k < (sizeof(T) == 4 ? 3 : 1); ++k)
      *reinterpret_cast<uint4*>(p.dst + (k * p.rows + r) * p.cols_p + c) =
          *reinterpret_cast<const uint4*>(v[k]);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    PFN_cuTensorMapEncodeTiled_v12000 f = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    cudaGetLastError();
    return f;
  }();
  return fn;
}

// A 3-D map: dims and box innermost first, strides in bytes of dims 1 and 2.
bool encode_3d(CUtensorMap* map, int dtype, const void* base, uint64_t d0, uint64_t d1,
               uint64_t d2, uint64_t s1, uint64_t s2, uint32_t b0, uint32_t b1, uint32_t b2) {
  auto encode = encode_fn();
  if (!encode) return false;
  const bool f32 = dtype == SMC_F32;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {s1, s2};
  cuuint32_t box[3] = {b0, b1, b2}, estr[3] = {1, 1, 1};
  const uint32_t row_bytes = b0 * (f32 ? 4 : 2);
  return encode(map,
                f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                    : (dtype == SMC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16),
                3, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_pairs() {
  constexpr int kMaxDev = 64;
  static int cache[kMaxDev] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < kMaxDev && cache[dev] > 0) return cache[dev];
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 2) {
    cudaGetLastError();
    sms = 148;
  }
  if (dev >= 0 && dev < kMaxDev) cache[dev] = sms / 2;
  return sms / 2;
}

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t parts_up(int64_t v, int64_t m) { return (v + m - 1) / m; }

// Where a call's operands lie: the caller's own buffers, or 16-bit copies in
// the workspace (parts of fp32 values; rows padded to 16 bytes).
struct Layout {
  int parts, Cp, Hp;
  bool pack_x, pack_w;
  int64_t x, w, dgu, db, slots, total;  // byte offsets
  Layout(int64_t n, int C, int H, int dtype, bool backward) {
    const bool f32 = dtype == SMC_F32;
    parts = f32 ? 3 : 1;
    Cp = int(up(C, 8));
    Hp = int(up(H, f32 ? 16 : 8));  // fp32: dg and du are written in 32-byte pieces
    pack_x = f32 || C % 8 != 0;
    pack_w = f32 || H % 8 != 0;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
      const int64_t here = at;
      at += up(bytes, 256);
      return here;
    };
    x = take(pack_x ? parts * n * Cp * 2 : 0);
    w = take(pack_w ? parts * int64_t(2) * C * Hp * 2 : 0);
    dgu = take(backward ? n * 2 * parts * Hp * 2 : 0);
    db = take(backward ? parts_up(n, 256) * 8 * 2 * H * 4 : 0);
    slots = take(backward ? int64_t(2) * sm_pairs() * bn_for(C) * 256 * 4 : 0);
    total = at > 0 ? at + 256 : 0;  // offsets are from a 256-byte boundary
  }
  // Columns of a dx or dW tile.
  static int bn_for(int C) { return C > 128 ? 256 : 128; }
};

template <int MODE, int BN, int DT, bool LONG>
int launch_mode(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
                const CUtensorMap& md, const GemmArgs& a, cudaStream_t s) {
  using L = Smem<MODE, BN, DT>;
  static_assert(L::kBytes <= kSmemMax, "shared memory");
  auto kern = k_gated<MODE, BN, DT, LONG>;
  constexpr int kMaxDev = 64;
  static bool attr_set[kMaxDev] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return SMC_ERR_CUDA;
  if (!(dev >= 0 && dev < kMaxDev && attr_set[dev])) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
        cudaSuccess)
      return SMC_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDev) attr_set[dev] = true;
  }
  return rows::launch_after(a.early, kern, dim3(2 * a.pairs), kThreads, L::kBytes, s, ma, mb, mo,
                            md, a);
}

template <int MODE, int DT>
int launch_bn(int bn, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
              const CUtensorMap& md, const GemmArgs& a, cudaStream_t s) {
  if constexpr (DT != SMC_F32) {
    // the longest accumulation: a tile's stages, or a pair's share of all of them
    int64_t most = a.k_iters;
    if (MODE == kDw)
      most = std::min(most, parts_up(int64_t(2) * a.m_tiles * a.n_tiles * a.k_iters, a.pairs));
    if (most > kLongStages)
      return bn == 256 ? launch_mode<MODE, 256, DT, true>(ma, mb, mo, md, a, s)
                       : launch_mode<MODE, 128, DT, true>(ma, mb, mo, md, a, s);
  }
  return bn == 256 ? launch_mode<MODE, 256, DT, false>(ma, mb, mo, md, a, s)
                   : launch_mode<MODE, 128, DT, false>(ma, mb, mo, md, a, s);
}

template <int DT>
struct Run {
  using T = typename Elem<DT>::type;
  static constexpr int kOp = DT == SMC_F32 ? SMC_BF16 : DT;  // the operands' type
  static constexpr int kE = DT == SMC_F32 ? 4 : 2;
  const GatedCall& g;
  const Layout lay;
  cudaStream_t s;
  uint8_t* work;
  const void *x, *W;
  GemmArgs a = {};

  Run(const GatedCall& call, bool backward, cudaStream_t stream)
      : g(call), lay(call.n, call.cin, call.hidden, call.dtype, backward), s(stream),
        work(reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(call.workspace) + 255) &
                                        ~uintptr_t(255))) {
    x = lay.pack_x ? work + lay.x : g.x;
    W = lay.pack_w ? work + lay.w : g.W;
    a.n = g.n;
    a.C = g.cin;
    a.H = g.hidden;
    a.act = g.act;
    a.Hp = lay.Hp;
    a.bias = g.bias;
    a.status = g.status;
    a.wait_ns = wait_limit_ns();
    // Short chains overlap their kernels' starts and ends (backward of 26,214
    // rows, 64 -> 256 fp16: 48 us without, 40 us with); on long ones, which run
    // at the power limit, it costs a little (55,100 rows, 512 -> 2048 bf16:
    // 657-711 us without, 687-735 us with, over the same seconds).
    a.early = parts_up(g.n, 256) * parts_up(g.hidden, 128) <= 8 * sm_pairs();
  }

  int pack() const {
    if (!lay.pack_x && !lay.pack_w) return SMC_OK;
    const Packing px{g.x, reinterpret_cast<uint16_t*>(work + lay.x), lay.pack_x ? g.n : 0, g.cin,
                     lay.Cp};
    const Packing pw{g.W, reinterpret_cast<uint16_t*>(work + lay.w),
                     lay.pack_w ? 2 * int64_t(g.cin) : 0, g.hidden, lay.Hp};
    const int64_t blocks = parts_up(px.rows * (px.cols_p / 8) + pw.rows * (pw.cols_p / 8), 256);
    const dim3 grid(unsigned(std::min<int64_t>(blocks, sm_pairs() * 32)));
    return rows::launch_after(a.early, k_pack<T>, grid, 256, 0, s, px, pw);
  }

  // x [parts][n][Cp], W [parts][2][C][Hp], dgu [n][parts][2][Hp]
  bool map_x(CUtensorMap* m, uint32_t b0, uint32_t b1) const {
    return encode_3d(m, kOp, x, g.cin, g.n, lay.parts, lay.Cp * 2ull, lay.Cp * 2ull * g.n, b0, b1,
                     1);
  }
  bool map_w(CUtensorMap* m, uint32_t b0, uint32_t b1) const {
    return encode_3d(m, kOp, W, g.hidden, g.cin, 2 * lay.parts, lay.Hp * 2ull,
                     lay.Hp * 2ull * g.cin, b0, b1, 1);
  }
  bool map_dgu(CUtensorMap* m, uint32_t b0, uint32_t b2) const {
    return encode_3d(m, kOp, work + lay.dgu, g.hidden, 2 * lay.parts, g.n, lay.Hp * 2ull,
                     lay.Hp * 4ull * lay.parts, b0, 1, b2);
  }
  // a caller's [n][width] matrix in chunks, if its rows allow it
  bool map_rows(CUtensorMap* m, const void* base, int width, int* usable) const {
    *usable = (int64_t(width) * kE) % 16 == 0;
    if (!*usable) return true;
    return encode_3d(m, DT, base, width, g.n, 1, uint64_t(width) * kE, uint64_t(width) * kE * g.n,
                     64 / kE, 32, 1);
  }

  // 256 columns a tile, or 128 where there are no more columns, or so few rows
  // that 256 would leave half of the SMs without a tile: a tile of 128 takes half
  // the time.  (11 rows, 896 -> 1600: bf16 forward 8.6 -> 7.3 us and
  // backward 35 -> 31, fp32 34 -> 23 and 141 -> 91; from 2,000 rows on both alike.)
  static int tile_columns(int m_tiles, int64_t columns) {
    return columns > 128 && 2 * m_tiles * parts_up(columns, 256) > sm_pairs() ? 256 : 128;
  }

  // out = act(g) u, or (dh given) dg and du into the workspace
  int pre(void* out, const void* dh, bool want_db) {
    CUtensorMap ma, mb, mo = {}, md = {};
    a.m_tiles = int(parts_up(g.n, 256));
    const int bn = tile_columns(a.m_tiles, 2 * int64_t(g.hidden));
    a.n_tiles = int(parts_up(g.hidden, bn / 2));
    a.k_iters = int(parts_up(g.cin, kBK));
    a.pairs = int(std::min<int64_t>(sm_pairs(), int64_t(a.m_tiles) * a.n_tiles));
    if (!map_x(&ma, kBK, 128) || !map_w(&mb, kBK, kBK)) return SMC_ERR_CUDA;
    if (!dh) {
      a.out = out;
      if (!map_rows(&mo, out, g.hidden, &a.tma_out)) return SMC_ERR_CUDA;
      return launch_bn<kPre, DT>(bn, ma, mb, mo, md, a, s);
    }
    a.dh = dh;
    a.dgu = reinterpret_cast<uint16_t*>(work + lay.dgu);
    a.db_part = want_db ? reinterpret_cast<float*>(work + lay.db) : nullptr;
    if (!map_dgu(&mo, 32, 32) || !map_rows(&md, dh, g.hidden, &a.tma_dh)) return SMC_ERR_CUDA;
    return launch_bn<kPreBwd, DT>(bn, ma, mb, mo, md, a, s);
  }

  int grad_x(void* dx) {
    CUtensorMap ma, mb, mo = {}, md = {};
    a.m_tiles = int(parts_up(g.n, 256));
    const int bn = tile_columns(a.m_tiles, g.cin);
    a.n_tiles = int(parts_up(g.cin, bn));
    a.k_iters = 2 * int(parts_up(g.hidden, kBK));
    a.pairs = int(std::min<int64_t>(sm_pairs(), int64_t(a.m_tiles) * a.n_tiles));
    a.out = dx;
    if (!map_dgu(&ma, kBK, 128) || !map_w(&mb, kBK, bn / 2) ||
        !map_rows(&mo, dx, g.cin, &a.tma_out))
      return SMC_ERR_CUDA;
    return launch_bn<kDx, DT>(bn, ma, mb, mo, md, a, s);
  }

  int grad_w(void* dW) {
    CUtensorMap ma, mb, mo = {}, md = {};
    const int bn = Layout::bn_for(g.cin);
    a.m_tiles = int(parts_up(g.hidden, 256));
    a.n_tiles = int(parts_up(g.cin, bn));
    a.k_iters = int(parts_up(g.n, kBK));
    a.pairs = int(std::min<int64_t>(sm_pairs(), int64_t(2) * a.m_tiles * a.n_tiles * a.k_iters));
    a.out = dW;
    a.slots = reinterpret_cast<float*>(work + lay.slots);
    if (!map_dgu(&ma, kBK, kBK) || !map_x(&mb, kBK, kBK)) return SMC_ERR_CUDA;
    return launch_bn<kDw, DT>(bn, ma, mb, mo, md, a, s);
  }

  // The joins behind grad_w (its arguments are still in `a`) and pre.
  int join(void* dW, void* dbias) {
    if (dW) {
      const int tiles = 2 * a.m_tiles * a.n_tiles, bn = Layout::bn_for(g.cin);
      const int64_t all = int64_t(tiles) * a.k_iters;
      bool split = false;  // a pair's share ends inside a tile
      for (int64_t p = 1; p < a.pairs; ++p) split |= p * all / a.pairs % a.k_iters != 0;
      if (split) {
        // one column per block while the blocks are few (two tiles of 37 parts
        // each: 5 us, with four 14.5), else four (32 tiles: 11 us, with one 28)
        const bool few = int64_t(tiles) * bn < 4096, small = (all + 1) * a.pairs < int64_t(1) << 32;
        auto kern = small ? (few ? k_join_dw<T, uint32_t, 1> : k_join_dw<T, uint32_t, 4>)
                          : (few ? k_join_dw<T, uint64_t, 1> : k_join_dw<T, uint64_t, 4>);
        const int rc = rows::launch_after(
            a.early, kern, dim3(tiles, few ? bn : bn / 4), 256, 0, s, a.slots, static_cast<T*>(dW),
            g.cin, g.hidden, a.m_tiles, a.n_tiles, a.k_iters, a.pairs, bn);
        if (rc != SMC_OK) return rc;
      }
    }
    if (!dbias) return SMC_OK;
    const int H2 = 2 * g.hidden;
    return rows::launch_after(a.early, k_join_db<T>, dim3(unsigned(parts_up(H2, 32))), 1024, 0, s,
                              reinterpret_cast<const float*>(work + lay.db),
                              static_cast<T*>(dbias), parts_up(g.n, 32), H2);
  }
};

template <class F>
int by_dtype(int dtype, F&& f) {
  switch (dtype) {
    case SMC_F32:
      return f(std::integral_constant<int, SMC_F32>());
    case SMC_F16:
      return f(std::integral_constant<int, SMC_F16>());
    default:
      return f(std::integral_constant<int, SMC_BF16>());
  }
}

}  // namespace

int64_t gated_workspace(int64_t n, int cin, int hidden, int dtype, bool backward) {
  return Layout(n, cin, hidden, dtype, backward).total;
}

int gated_forward(const GatedCall& g, void* out, cudaStream_t s) {
  return by_dtype(g.dtype, [&](auto dt) {
    Run<decltype(dt)::value> r(g, false, s);
    const int rc = r.pack();
    return rc != SMC_OK ? rc : r.pre(out, nullptr, false);
  });
}

int gated_backward(const GatedCall& g, const void* dh, void* dx, void* dW, void* dbias,
                   cudaStream_t s) {
  if (!dx && !dW && !dbias) return SMC_OK;
  return by_dtype(g.dtype, [&](auto dt) {
    Run<decltype(dt)::value> r(g, true, s);
    int rc = r.pack();
    if (rc == SMC_OK) rc = r.pre(nullptr, dh, dbias != nullptr);
    if (rc == SMC_OK && dx) rc = r.grad_x(dx);
    if (rc == SMC_OK && dW) rc = r.grad_w(dW);
    if (rc == SMC_OK && (dW || dbias)) rc = r.join(dW, dbias);
    return rc;
  });
}

}  // namespace smc
