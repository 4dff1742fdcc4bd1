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
#include <mutex>

#include "smc_internal.h"
#include "smc_ptx.cuh"
#include "smc_rows.cuh"

namespace smc {
namespace {

using namespace ptx;

enum Mode { kPre, kPreBwd, kDx, kDw };

constexpr int kBK = 64;  // depth of a stage: one 128-byte row of 16-bit values
constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;  // two per quarter of the tensor-memory lanes
constexpr int kSmemMax = 227 * 1024;
constexpr int kTailBytes = 4096;  // bias (2 KB) and barriers
constexpr uint64_t kAbortDrainNs = 50000000ull;

// The part products of fp32 inputs, smallest first: parts of A and of B.
constexpr int kPartPairs = 6;
__constant__ int8_t kPartA[kPartPairs] = {2, 0, 1, 1, 0, 0};
__constant__ int8_t kPartB[kPartPairs] = {0, 2, 1, 0, 1, 0};

struct GemmArgs {
  int64_t n;
  int C, H, act;
  int m_tiles, n_tiles;  // kDw: tiles of hidden units per half, of channels
  int k_chunks, k_iters;  // stages per part product, in all
  int pairs;             // clusters launched
  int f32;               // fp32 parts: kPartPairs products instead of one
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
  int64_t cur, end, step;
  const GemmArgs& a;
  __device__ __forceinline__ Walk(const GemmArgs& args, int pair) : a(args) {
    if (MODE == kDw) {
      const int64_t all = int64_t(2) * a.m_tiles * a.n_tiles * a.k_iters;
      cur = pair * all / a.pairs;
      end = (pair + 1) * all / a.pairs;
    } else {
      cur = pair;
      end = int64_t(a.m_tiles) * a.n_tiles;
    }
  }
  __device__ __forceinline__ bool next(Seg& g) {
    if (cur >= end) return false;
    int tile;
    if (MODE == kDw) {
      tile = int(cur / a.k_iters);
      g.k0 = int(cur % a.k_iters);
      g.k1 = int(min(int64_t(a.k_iters), g.k0 + end - cur));
      cur += g.k1 - g.k0;
      g.s = tile / (a.n_tiles * a.m_tiles);
      tile -= g.s * a.n_tiles * a.m_tiles;
    } else {
      tile = int(cur);
      g.k0 = 0;
      g.k1 = a.k_iters;
      g.s = 0;
      cur += a.pairs;
    }
    g.m = tile / a.n_tiles;
    g.n = tile % a.n_tiles;
    return true;
  }
};

// SiLU and its slope through one exponential and one division (both of the
// fast kind: together within 2^-21 of the value, far inside a 16-bit result's
// rounding; exp(-v) = inf gives the correct limit 0).
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

__device__ __forceinline__ float act_value(float v, int act) {
  switch (act) {
    case SMC_ACT_RELU:
      return fmaxf(v, 0.f);
    case SMC_ACT_SILU:
      return v * sigmoid(v);
    case SMC_ACT_GELU:
      return 0.5f * v * (1.f + erff(v * 0.7071067811865476f));
    default:
      return v;
  }
}
// The activation's value and slope.
__device__ __forceinline__ float2 act_both(float v, int act) {
  switch (act) {
    case SMC_ACT_RELU:
      return make_float2(fmaxf(v, 0.f), v > 0.f ? 1.f : 0.f);
    case SMC_ACT_SILU: {
      const float s = sigmoid(v);
      return make_float2(v * s, s * (1.f + v * (1.f - s)));
    }
    case SMC_ACT_GELU: {
      const float cdf = 0.5f * (1.f + erff(v * 0.7071067811865476f));
      return make_float2(v * cdf, cdf + v * __expf(-0.5f * v * v) * 0.3989422804014327f);
    }
    default:
      return make_float2(v, 1.f);
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
  static constexpr int kB = BN / 2 * 128;  // this CTA's half of B
  static constexpr int kStage = 16384 + kB;
  static constexpr int kChunkBytes = DT == SMC_F32 ? 4096 : 2048;  // 32 rows x 32 values
  static constexpr int kChunks = MODE == kPre || MODE == kPreBwd ? BN / 128 : BN / 64;
  // kPreBwd: dh of every chunk (dg takes its place) and du of every chunk (of
  // one for fp32, whose du is staged for its column sums only); kPre, kDx: two
  // slots in turn; kDw stores straight from registers.
  static constexpr int kWarpStage =
      MODE == kPreBwd ? (kChunks + (DT == SMC_F32 ? 1 : kChunks)) * kChunkBytes
                      : (MODE == kDw ? 0 : 2 * kChunkBytes);
  static constexpr int kStages0 = (kSmemMax - kTailBytes - kEpiWarps * kWarpStage) / kStage;
  static constexpr int kStages = kStages0 > 8 ? 8 : kStages0;
  static constexpr int kBytes = kStages * kStage + kEpiWarps * kWarpStage + kTailBytes;
  static_assert(kStages >= 3, "stages");
};

// Where 16-byte piece `j` of row `r` of a 32-row chunk lies: the TMA's 64-byte
// swizzle for 16-bit values (64-byte rows), its 128-byte one for fp32.
template <int DT>
__device__ __forceinline__ uint32_t piece(int r, int j) {
  if constexpr (DT == SMC_F32)
    return r * 128 + ((j ^ (r & 7)) << 4);
  else
    return r * 64 + ((j ^ ((r >> 1) & 3)) << 4);
}
template <int DT>
__device__ __forceinline__ uint32_t value_at(int r, int col) {
  if constexpr (DT == SMC_F32)
    return piece<DT>(r, col >> 2) + (col & 3) * 4;
  else
    return piece<DT>(r, col >> 3) + (col & 7) * 2;
}

// Eight values of a row in the chunk's type, and back.
template <int DT>
__device__ __forceinline__ void put8(uint8_t* chunk, int r, int g8, const float (&v)[8]) {
  if constexpr (DT == SMC_F32) {
    *reinterpret_cast<float4*>(chunk + piece<DT>(r, 2 * g8)) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(chunk + piece<DT>(r, 2 * g8 + 1)) =
        make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack2<DT == SMC_BF16>(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]));
    *reinterpret_cast<uint4*>(chunk + piece<DT>(r, g8)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <int DT>
__device__ __forceinline__ void get8(const uint8_t* chunk, int r, int g8, float (&v)[8]) {
  if constexpr (DT == SMC_F32) {
    const float4 x = *reinterpret_cast<const float4*>(chunk + piece<DT>(r, 2 * g8));
    const float4 y = *reinterpret_cast<const float4*>(chunk + piece<DT>(r, 2 * g8 + 1));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  } else {
    using T = typename Elem<DT>::type;
    uint4 x = *reinterpret_cast<const uint4*>(chunk + piece<DT>(r, g8));
    const T* t = reinterpret_cast<const T*>(&x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = rows::to_float(t[i]);
  }
}

// Store a warp's staged chunk (32 rows x 32 columns) at (row0, col0) of a
// matrix whose rows hold `width` values: one TMA store where the rows are
// 16-byte multiples (it clips what lies outside), else row by row with a lane
// per column.  Every lane calls it; the staging may be written again after
// bulk_wait_read of lane 0 and a __syncwarp.
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
    __syncwarp();
    const int col = col0 + lane;
    const int rows_here = int(min(int64_t(32), n - row0));
    if (col < width)
      for (int r = 0; r < rows_here; ++r)
        static_cast<T*>(base)[(row0 + r) * width + col] =
            *reinterpret_cast<const T*>(chunk + value_at<DT>(r, lane));
    __syncwarp();
  }
}

// Sum over a staged chunk's 32 rows, for column `lane`.
template <int DT>
__device__ __forceinline__ float column_sum(const uint8_t* chunk, int lane) {
  using T = typename Elem<DT>::type;
  float s = 0.f;
#pragma unroll 8
  for (int r = 0; r < 32; ++r)
    s += rows::to_float(*reinterpret_cast<const T*>(chunk + value_at<DT>(r, lane)));
  return s;
}

template <int MODE, int BN, int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
k_gated(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
        const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_dh,
        const GemmArgs a) {
  using L = Smem<MODE, BN, DT>;
  using T = typename Elem<DT>::type;
  constexpr int kStages = L::kStages;
  constexpr bool kPreMode = MODE == kPre || MODE == kPreBwd;
  constexpr uint32_t kTmemCols = 2 * BN;
  // M = 256 over the pair; A is MN-major in kDw, B in all modes but kDx
  constexpr uint32_t kIdesc = (1u << 4) | ((DT != SMC_F16 ? 1u : 0u) << 7) |
                              ((DT != SMC_F16 ? 1u : 0u) << 10) | ((MODE == kDw ? 1u : 0u) << 15) |
                              ((MODE != kDx ? 1u : 0u) << 16) | (uint32_t(BN >> 3) << 17) |
                              (16u << 24);

  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* staging = smem + kStages * L::kStage;
  float* bias_smem = reinterpret_cast<float*>(staging + kEpiWarps * L::kWarpStage);  // [8][64]
  uint64_t* bars = reinterpret_cast<uint64_t*>(bias_smem + kEpiWarps * 64);
  // full[kStages] empty[kStages] tfull[2] tempty[2] drain dh[8]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5 + kEpiWarps);
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
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(dh0 + 8 * w, 1);
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
      int q = g.k0 / a.k_chunks, kc = g.k0 % a.k_chunks;
      for (int it = g.k0; it < g.k1; ++it) {
        if (!(ok = waits.wait(empty0 + 8 * st, phase ^ 1))) break;
        if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * st, 2 * L::kStage);
        const uint32_t bar = lead_full0 + 8 * st;
        const uint32_t da = ring0 + st * L::kStage, db = da + 16384;
        const int pa = a.f32 ? kPartA[q] : 0, pb = a.f32 ? kPartB[q] : 0;
        const int k = kc * kBK;
        if constexpr (kPreMode) {
          tma_load_3d_pair(da, &map_a, k, g.m * 256 + int(rank) * 128, pa, bar);
#pragma unroll
          for (int j = 0; j < BN / 128; ++j)
            tma_load_3d_pair(db + j * 8192, &map_b, g.n * (BN / 2) + j * 64, k, pb * 2 + int(rank),
                             bar);
        } else if constexpr (MODE == kDx) {
          const int half = a.k_chunks >> 1, s = kc >= half ? 1 : 0;
          const int h = (kc - s * half) * kBK;
          tma_load_3d_pair(da, &map_a, h, pa * 2 + s, g.m * 256 + int(rank) * 128, bar);
          tma_load_3d_pair(db, &map_b, h, g.n * BN + int(rank) * (BN / 2), pb * 2 + s, bar);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            tma_load_3d_pair(da + j * 8192, &map_a, g.m * 256 + int(rank) * 128 + j * 64,
                             pa * 2 + g.s, k, bar);
#pragma unroll
          for (int j = 0; j < BN / 128; ++j)
            tma_load_3d_pair(db + j * 8192, &map_b, g.n * BN + int(rank) * (BN / 2) + j * 64, k, pb,
                             bar);
        }
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
        if (++kc == a.k_chunks) {
          kc = 0;
          ++q;
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------- the pair's MMAs (leader only) ---------------------------
    int st = 0, seg = 0;
    uint32_t phase = 0;
    bool ok = *abort_flag == 0;
    while (ok && walk.next(g)) {
      const int acc = seg & 1;
      if (!(ok = waits.wait(tempty0 + 8 * acc, ((seg >> 1) & 1) ^ 1))) break;
      tc_fence_after();
      for (int it = g.k0; it < g.k1; ++it) {
        if (!(ok = waits.wait(full0 + 8 * st, phase))) break;
        tc_fence_after();
        const uint32_t sa = ring0 + st * L::kStage, sb = sa + 16384;
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) {
          const uint64_t da = MODE == kDw ? desc_b_mnmajor(sa + k * 2048, 8192)
                                          : desc_a_kmajor(sa + k * 32);
          const uint64_t db = MODE != kDx ? desc_b_mnmajor(sb + k * 2048, 8192)
                                          : desc_a_kmajor(sb + k * 32);
          umma_f16_pair(tmem + acc * BN, da, db, kIdesc, it > g.k0 || k > 0);
        }
        umma_commit_pair(empty0 + 8 * st);
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      umma_commit_pair(tfull0 + 8 * acc);
      ++seg;
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
    const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2, w = warp - kEpiWarp0;
    uint8_t* mine = staging + w * L::kWarpStage;
    float* bias_w = bias_smem + w * 64;
    const uint32_t lead_tempty0 = map_to_rank(tempty0, 0);
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t dh_bar = dh0 + 8 * w;
    uint32_t dh_phase = 0;
    int seg = 0, turn = 0;  // turn: the staging slot of the next store
    bool ok = *abort_flag == 0;
    while (ok && walk.next(g)) {
      const int acc = seg & 1;
      const uint32_t parity = (seg >> 1) & 1;
      const uint32_t d = lanes + acc * BN;
      ++seg;
      if constexpr (kPreMode) {
        const int h0 = g.n * (BN / 2) + half * (BN / 4);
        const int64_t row0 = int64_t(g.m) * 256 + rank * 128 + quarter * 32;
        const int chunks = row0 < a.n ? min(L::kChunks, (a.H - h0 + 31) / 32) : 0;
        if constexpr (MODE == kPreBwd) {
          // dh of this tile, while the products run
          if (a.tma_dh) {
            fence_proxy_async_smem();  // the staging was read and written by all lanes
            __syncwarp();
            if (lane == 0 && chunks > 0) {
              bulk_wait_read<0>();
              mbar_arrive_expect_tx(dh_bar, chunks * L::kChunkBytes);
              for (int c = 0; c < chunks; ++c)
                tma_load_3d(smem_addr(mine + c * L::kChunkBytes), &map_dh, h0 + c * 32, int(row0),
                            0, dh_bar);
            }
          } else {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            const int rows_here = int(min(int64_t(32), a.n - row0));
            for (int c = 0; c < chunks; ++c) {
              const int h = h0 + c * 32 + lane;
              for (int r = 0; r < 32; ++r)
                *reinterpret_cast<T*>(mine + c * L::kChunkBytes + value_at<DT>(r, lane)) =
                    r < rows_here && h < a.H ? static_cast<const T*>(a.dh)[(row0 + r) * a.H + h]
                                             : rows::from_float<T>(0.f);
            }
            __syncwarp();
          }
        }
        if (!(ok = waits.wait(tfull0 + 8 * acc, parity))) break;
        tc_fence_after();
        if constexpr (MODE == kPreBwd) {
          if (a.tma_dh && chunks > 0) {
            if (!(ok = waits.wait(dh_bar, dh_phase))) break;
            dh_phase ^= 1;
          }
        }
#pragma unroll
        for (int c = 0; c < L::kChunks; ++c) {
          const int h = h0 + c * 32;
          uint32_t gv[32], uv[32];
          tmem_ld_x32_async(d + half * (BN / 4) + c * 32, gv);
          tmem_ld_x32_async(d + BN / 2 + half * (BN / 4) + c * 32, uv);
          tmem_ld_wait();
          if (c == L::kChunks - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8 * acc);
          }
          if (c >= chunks) continue;
          const bool biased = a.bias != nullptr;
          if (biased) {
            const T* b = static_cast<const T*>(a.bias);
            __syncwarp();
            bias_w[lane] = h + lane < a.H ? rows::to_float(b[h + lane]) : 0.f;
            bias_w[32 + lane] = h + lane < a.H ? rows::to_float(b[a.H + h + lane]) : 0.f;
            __syncwarp();
          }
          uint8_t* slot = mine + (MODE == kPreBwd ? c : turn) * L::kChunkBytes;
          uint8_t* slot_u =
              mine + (L::kChunks + (DT == SMC_F32 ? 0 : c)) * L::kChunkBytes;  // kPreBwd
          if constexpr (MODE == kPre) {
            turn ^= 1;
            if (lane == 0) bulk_wait_read<1>();  // the slot's last store, two stores back
            __syncwarp();
          }
#pragma unroll
          for (int g8 = 0; g8 < 4; ++g8) {
            float gg[8], uu[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              gg[i] = __uint_as_float(gv[g8 * 8 + i]);
              uu[i] = __uint_as_float(uv[g8 * 8 + i]);
            }
            if (biased) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                gg[i] += bias_w[g8 * 8 + i];
                uu[i] += bias_w[32 + g8 * 8 + i];
              }
            }
            if constexpr (MODE == kPre) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = act_value(gg[i], a.act) * uu[i];
              put8<DT>(slot, lane, g8, v);
            } else {
              float dh[8], G[8], U[8];
              get8<DT>(slot, lane, g8, dh);
              const bool row_ok = row0 + lane < a.n;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 f = act_both(gg[i], a.act);
                G[i] = row_ok ? dh[i] * uu[i] * f.y : 0.f;
                U[i] = row_ok ? dh[i] * f.x : 0.f;
              }
              put8<DT>(slot, lane, g8, G);
              put8<DT>(slot_u, lane, g8, U);
              if constexpr (DT == SMC_F32) {
                // three bf16 parts of each, straight to memory
                if (row_ok && h + g8 * 8 < a.H) {
                  uint16_t* to = a.dgu + (row0 + lane) * 6 * a.Hp + h + g8 * 8;
#pragma unroll
                  for (int s = 0; s < 2; ++s) {
                    uint32_t w3[3][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      __nv_bfloat16 lo[3], hi[3];
                      split3(s ? U[2 * i] : G[2 * i], lo);
                      split3(s ? U[2 * i + 1] : G[2 * i + 1], hi);
#pragma unroll
                      for (int p = 0; p < 3; ++p)
                        w3[p][i] = uint32_t(__bfloat16_as_ushort(lo[p])) |
                                   uint32_t(__bfloat16_as_ushort(hi[p])) << 16;
                    }
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                      *reinterpret_cast<uint4*>(to + (p * 2 + s) * a.Hp) =
                          make_uint4(w3[p][0], w3[p][1], w3[p][2], w3[p][3]);
                  }
                }
              }
            }
          }
          if constexpr (MODE == kPre) {
            store_chunk<DT>(&map_out, a.tma_out, slot, a.out, row0, h, a.n, a.H, lane);
          } else {
            if constexpr (DT != SMC_F32) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&map_out, smem_addr(slot), h, 0, int(row0));
                tma_store_3d(&map_out, smem_addr(slot_u), h, 1, int(row0));
                bulk_commit();
              }
            } else {
              __syncwarp();
            }
            if (a.db_part) {
              const int64_t block = (int64_t(g.m) * 2 + rank) * 4 + quarter;
              const float sg = column_sum<DT>(slot, lane), su = column_sum<DT>(slot_u, lane);
              if (h + lane < a.H) {
                a.db_part[(block * 2 + 0) * a.H + h + lane] = sg;
                a.db_part[(block * 2 + 1) * a.H + h + lane] = su;
              }
            }
            __syncwarp();
          }
        }
      } else {
        if (!(ok = waits.wait(tfull0 + 8 * acc, parity))) break;
        tc_fence_after();
        const int c0 = g.n * BN + half * (BN / 2);
        const int64_t row0 = int64_t(g.m) * 256 + rank * 128 + quarter * 32;
#pragma unroll 1
        for (int c = 0; c < L::kChunks; ++c) {
          const int col = c0 + c * 32;
          uint32_t v[32];
          tmem_ld_x32_async(d + half * (BN / 2) + c * 32, v);
          tmem_ld_wait();
          if (c == L::kChunks - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8 * acc);
          }
          if (col >= a.C) continue;
          if constexpr (MODE == kDx) {
            if (row0 >= a.n) continue;
            uint8_t* slot = mine + turn * L::kChunkBytes;
            turn ^= 1;
            if (lane == 0) bulk_wait_read<1>();
            __syncwarp();
#pragma unroll
            for (int g8 = 0; g8 < 4; ++g8) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[g8 * 8 + i]);
              put8<DT>(slot, lane, g8, f);
            }
            store_chunk<DT>(&map_out, a.tma_out, slot, a.out, row0, col, a.n, a.C, lane);
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
              float* to = a.slots + (int64_t(2 * pair + (g.k0 == 0 ? 1 : 0)) * BN + half * (BN / 2) +
                                     c * 32) * 256 + rank * 128 + quarter * 32 + lane;
#pragma unroll
              for (int i = 0; i < 32; ++i) to[i * 256] = __uint_as_float(v[i]);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_read<0>();
    if (MODE == kPreBwd && !ok && lane == 0) mbar_drain(dh_bar, dh_phase);
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
// order of the pairs.
template <class T>
__global__ void __launch_bounds__(256)
k_join_dw(const float* __restrict__ slots, T* __restrict__ dW, int C, int H, int m_tiles,
          int n_tiles, int k_iters, int pairs, int bn) {
  int tile = blockIdx.x;
  const int64_t all = int64_t(2) * m_tiles * n_tiles * k_iters;
  const int64_t i0 = int64_t(tile) * k_iters, i1 = i0 + k_iters;
  const int64_t p0 = ((i0 + 1) * pairs - 1) / all, p1 = (i1 * pairs - 1) / all;
  if (p0 == p1) return;  // one pair stored it whole
  const int s = tile / (n_tiles * m_tiles);
  tile -= s * n_tiles * m_tiles;
  const int64_t h = int64_t(tile / n_tiles) * 256 + threadIdx.x;
  if (h >= H) return;
  const int cl0 = blockIdx.y * 8, c0 = tile % n_tiles * bn + cl0;
  for (int i = 0; i < 8 && c0 + i < C; ++i) {
    float v = 0.f;
    for (int64_t p = p0; p <= p1; ++p) {
      const int64_t slot = 2 * p + (p * all / pairs > i0 ? 0 : 1);  // as the pair chose it
      v += slots[(slot * bn + cl0 + i) * 256 + threadIdx.x];
    }
    dW[(int64_t(s) * C + c0 + i) * H + h] = rows::from_float<T>(v);
  }
}

// dbias: the sums over 32 rows, added up in a fixed order.
template <class T>
__global__ void __launch_bounds__(1024)
k_join_db(const float* __restrict__ part, T* __restrict__ dbias, int64_t blocks, int H2) {
  __shared__ float sums[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
  float s = 0.f;
  if (col < H2)
    for (int64_t b = w; b < blocks; b += 32) s += part[b * H2 + col];
  sums[w][threadIdx.x % 32] = s;
  __syncthreads();
  if (w == 0 && col < H2) {
    for (int i = 1; i < 32; ++i) s += sums[i][threadIdx.x];
    dbias[col] = rows::from_float<T>(s);
  }
}

// src [rows][cols] -> dst [parts][rows][cols_p], 16-bit: the three bf16 parts of
// fp32 values, or the values themselves, rows padded with zeros to a multiple
// of 16 bytes.
template <class T>
__global__ void __launch_bounds__(256)
k_parts(const T* __restrict__ src, uint16_t* __restrict__ dst, int64_t nrows, int cols,
        int cols_p) {
  const int per_row = cols_p / 8;
  for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < nrows * per_row;
       i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / per_row;
    const int c = int(i % per_row) * 8;
    uint16_t v[3][8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) {
        if constexpr (sizeof(T) == 4) {
          __nv_bfloat16 p[3];
          split3(src[r * cols + c + j], p);
          for (int k = 0; k < 3; ++k) v[k][j] = __bfloat16_as_ushort(p[k]);
        } else {
          v[0][j] = *reinterpret_cast<const uint16_t*>(&src[r * cols + c + j]);
        }
      }
#pragma unroll
    for (int k = 0; k < (sizeof(T) == 4 ? 3 : 1); ++k)
      *reinterpret_cast<uint4*>(dst + (k * nrows + r) * cols_p + c) =
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
    Hp = int(up(H, 8));
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
    total = at;
  }
  // Columns of a dx or dW tile.
  static int bn_for(int C) { return C > 128 ? 256 : 128; }
};

template <int MODE, int BN, int DT>
int launch_mode(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
                const CUtensorMap& md, const GemmArgs& a, cudaStream_t s) {
  using L = Smem<MODE, BN, DT>;
  static_assert(L::kBytes <= kSmemMax, "shared memory");
  auto kern = k_gated<MODE, BN, DT>;
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
  kern<<<2 * a.pairs, kThreads, L::kBytes, s>>>(ma, mb, mo, md, a);
  return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
}

template <int MODE, int DT>
int launch_bn(int bn, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
              const CUtensorMap& md, const GemmArgs& a, cudaStream_t s) {
  return bn == 256 ? launch_mode<MODE, 256, DT>(ma, mb, mo, md, a, s)
                   : launch_mode<MODE, 128, DT>(ma, mb, mo, md, a, s);
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
        work(static_cast<uint8_t*>(call.workspace)) {
    x = lay.pack_x ? work + lay.x : g.x;
    W = lay.pack_w ? work + lay.w : g.W;
    a.n = g.n;
    a.C = g.cin;
    a.H = g.hidden;
    a.act = g.act;
    a.f32 = DT == SMC_F32;
    a.Hp = lay.Hp;
    a.bias = g.bias;
    a.status = g.status;
    a.wait_ns = wait_limit_ns();
  }

  int pack() const {
    auto one = [&](const void* src, int64_t off, int64_t nrows, int cols, int cols_p) {
      const int64_t blocks = parts_up(nrows * (cols_p / 8), 256);
      k_parts<T><<<unsigned(std::min<int64_t>(blocks, 148 * 16)), 256, 0, s>>>(
          static_cast<const T*>(src), reinterpret_cast<uint16_t*>(work + off), nrows, cols, cols_p);
    };
    if (lay.pack_x) one(g.x, lay.x, g.n, g.cin, lay.Cp);
    if (lay.pack_w) one(g.W, lay.w, 2 * int64_t(g.cin), g.hidden, lay.Hp);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
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
  // a caller's [n][width] matrix in 32 x 32 chunks, if its rows allow it
  bool map_rows(CUtensorMap* m, const void* base, int width, int* usable) const {
    *usable = (int64_t(width) * kE) % 16 == 0;
    if (!*usable) return true;
    return encode_3d(m, DT, base, width, g.n, 1, uint64_t(width) * kE, uint64_t(width) * kE * g.n,
                     32, 32, 1);
  }

  void stages(int chunks) {
    a.k_chunks = chunks;
    a.k_iters = chunks * (DT == SMC_F32 ? kPartPairs : 1);
  }

  // out = act(g) u, or (dh given) dg and du into the workspace
  int pre(void* out, const void* dh, bool want_db) {
    CUtensorMap ma, mb, mo = {}, md = {};
    const int bn = g.hidden > 64 ? 256 : 128;
    a.m_tiles = int(parts_up(g.n, 256));
    a.n_tiles = int(parts_up(g.hidden, bn / 2));
    stages(int(parts_up(g.cin, kBK)));
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
    const int bn = Layout::bn_for(g.cin);
    a.m_tiles = int(parts_up(g.n, 256));
    a.n_tiles = int(parts_up(g.cin, bn));
    stages(2 * int(parts_up(g.hidden, kBK)));
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
    stages(int(parts_up(g.n, kBK)));
    const int tiles = 2 * a.m_tiles * a.n_tiles;
    a.pairs = int(std::min<int64_t>(sm_pairs(), int64_t(tiles) * a.k_iters));
    a.out = dW;
    a.slots = reinterpret_cast<float*>(work + lay.slots);
    if (!map_dgu(&ma, kBK, kBK) || !map_x(&mb, kBK, kBK)) return SMC_ERR_CUDA;
    const int rc = launch_bn<kDw, DT>(bn, ma, mb, mo, md, a, s);
    if (rc != SMC_OK) return rc;
    k_join_dw<T><<<dim3(tiles, bn / 8), 256, 0, s>>>(a.slots, static_cast<T*>(dW), g.cin, g.hidden,
                                                     a.m_tiles, a.n_tiles, a.k_iters, a.pairs, bn);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
  }

  int grad_bias(void* dbias) {
    const int H2 = 2 * g.hidden;
    k_join_db<T><<<unsigned(parts_up(H2, 32)), 1024, 0, s>>>(
        reinterpret_cast<const float*>(work + lay.db), static_cast<T*>(dbias),
        parts_up(g.n, 32), H2);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
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
    if (rc == SMC_OK && dbias) rc = r.grad_bias(dbias);
    return rc;
  });
}

}  // namespace smc
