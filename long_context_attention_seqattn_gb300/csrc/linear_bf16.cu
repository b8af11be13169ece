// linear_bf16.cu -- the matrix products of a linear layer on the tensor cores
// (bf16 in, float32 accumulation), each with its epilogue in the same kernel:
//   forward   Y  = act(X W + b) + R      (and optionally Z = X W + b)
//   dgrad     dX = act'(Z) o (G W^T) + R
//   wgrad     dW += X^T G
// X [rows, k], G [rows, n], W [k, n] row-major.  One kernel serves the three:
// an operand whose contraction index is contiguous in memory is K-major, the
// other kind MN-major, and tcgen05 reads both from the 128-byte swizzled
// tiles that TMA writes, so nothing is ever transposed:
//             A (M index)          B (N index)         contraction
//   forward   X   rows, K-major    W   n,   MN-major   k
//   dgrad     G   rows, K-major    W   k,   K-major    n
//   wgrad     X^T k,    MN-major   G   n,   MN-major   rows
// Rows, columns and contraction tails past the tensors arrive as TMA zeros.
//
// Two shapes of the kernel:
//   pair   clusters of two CTAs, persistent.  A pair owns a 256 x N tile (N =
//          256, or a narrower one that fills the last wave better): one
//          thread issues M256 K16 MMAs for both SMs, each SM loads half of A
//          (its 128 rows) and half of B (N / 2 columns), at most 32 KB a
//          stage of 64, and keeps its 128 x N half of the result in TMEM.
//          Two result buffers (512 columns): the epilogue of a tile runs
//          under the products of the next.
//   split  clusters of 1 to 8 CTAs that share one 128 x 128 tile: CTA i sums
//          the i-th part of the contraction, the parts meet in distributed
//          shared memory and are added in order.  For results with few tiles
//          (few rows, down to a single token's, or a small weight gradient),
//          where the pairs would leave most SMs idle, and for the last tiles
//          of a larger one when they would keep the pairs for a whole wave.
// Warps of a CTA:
//   warp 0      TMA producer (A and B tile of a stage, 16 KB each)
//   warp 1      TMEM owner + MMA issuer (pair: the even CTA's thread for both)
//   warps 2..9  epilogue, two per TMEM lane quadrant, each half of the columns
//               of its 32 rows
//
// wgrad's result is float32, and a long running sum on the tensor core is not
// quite: its additions truncate (measured: 9.1e-6 relative over 8192 rows,
// against 9.5e-7 for a float32 library product).  So its products are summed
// in TMEM for at most kChunkStages stages (768 rows); the epilogue warps add
// these partial sums in registers, rounding to nearest, while the next are
// computed into the other buffer.  bf16 results need no such care.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace seqattn {
namespace {

constexpr int kTK = kLinearStageK;             // contraction per stage
constexpr int kOperandRows = 128;              // rows of an operand tile in one CTA
constexpr int kStages = 6;
constexpr int kOperandBytes = kOperandRows * kTK * 2;   // 16 KB, either operand
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kMnBlockBytes = kTK * 128;       // one 64-column block of an MN-major tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kBoxBytes = 32 * 128;            // a warp's staging box: 32 rows x 32 float32
constexpr int kOffBox = kStages * kStageBytes;
constexpr int kSmemAlloc = kOffBox + kEpiWarps * kBoxBytes + 1024;
constexpr int kChunkStages = 12;               // wgrad: stages summed on the tensor core
constexpr int kMaxSplit = 8;                   // CTAs of a split cluster (portable limit)
constexpr int kPartStride = 128 + 4;           // floats between rows of a split CTA's partial tile
// Cost model of the two shapes, in SM cycles (see plan_mode).  Measured with
// every SM busy: a pair's stage 0.32 us with a tile of 256 columns and 0.27
// with 128 (kPairStageCost, and kPairColumnCost for 128 columns more), so a
// narrow tile pays only where it saves a wave; a split CTA's 0.24, whatever
// A's rows (its four MMAs are issued in about 110 cycles each).  A join costs
// more for tiles of more rows.  The constants are fitted: over 100 shapes of 2
// to 2048 rows the geometric means of forward and dgrad are 6.61 and 6.57 us
// with these, 6.67 and 6.63 with joins that cost the same whatever the rows
// (4000 and 600; 512 x 1024 x 1024 then takes 9.8 us instead of 8.1).
// kSecondLaunchCost: what a second launch has to save before it is made (501 x
// 4104 x 10248 took 55 us with it and 62 without, see plan_mode).
constexpr int64_t kPairStageCost = 510, kPairColumnCost = 98, kPairFixedCost = 12300;
constexpr int64_t kSplitStageCost = 455, kSplitFixedCost = 8000;
constexpr int64_t kSplitFirstJoinCost = 3500, kSplitFirstJoinRowCost = 10;   // two CTAs, and for each row of the tile
constexpr int64_t kSplitJoinCost = 400, kSplitJoinRowCost = 5;               // each further CTA, and row
constexpr int64_t kSecondLaunchCost = 3000;
static_assert(128 * kPartStride * 4 <= kStages * kStageBytes, "the partial tile is kept in the ring");

template <bool kPair>
struct Shape {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTM = 128 * kCtas;      // tile rows
  static constexpr int kTN = 128 * kCtas;      // tile columns
  static constexpr uint32_t kTmemCols = 2 * kTN;   // two result buffers
  static constexpr int kColsPerWarp = kTN / 2;
};

struct LinearBarriers {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_final;
};

// ---- activations (z in float32) -------------------------------------------
// (fast exponential and quotient: a few 2^-22 of a value that is rounded to bf16)
__device__ __forceinline__ float sigmoidf(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
constexpr float kTanhA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

template <int kAct>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (kAct == kActRelu) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (kAct == kActSilu) return z * sigmoidf(z);
  if constexpr (kAct == kActGelu) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  // 0.5 (1 + tanh u) = sigmoid(2 u)
  if constexpr (kAct == kActGeluTanh) return z * sigmoidf(2.f * kTanhA * (z + kTanhB * z * z * z));
  return z;
}

// Past |z| = 128 every derivative is 0 or 1 in float32; taking the limit there
// keeps infinite intermediate products (0 * inf) out of the formulas.
// (relu's is not multiplied but chosen, as 0 * inf is not 0, see times_grad.)
template <int kAct>
__device__ __forceinline__ float act_grad(float z) {
  if (fabsf(z) > 128.f) return z > 0.f ? 1.f : 0.f;
  if constexpr (kAct == kActSilu) {
    const float s = sigmoidf(z);
    return s * (1.f + z * (1.f - s));
  }
  if constexpr (kAct == kActGelu)
    return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * 0.3989422804014327f * __expf(-0.5f * z * z);
  if constexpr (kAct == kActGeluTanh) {
    const float s = sigmoidf(2.f * kTanhA * (z + kTanhB * z * z * z));
    return s + z * s * (1.f - s) * 2.f * kTanhA * (1.f + 3.f * kTanhB * z * z);
  }
}

// v act'(z); a NaN of z passes relu, as it does in the forward.
template <int kAct>
__device__ __forceinline__ float times_grad(float v, float z) {
  if constexpr (kAct == kActRelu) return z > 0.f ? v : (z != z ? z : 0.f);
  else return v * act_grad<kAct>(z);
}

__device__ __forceinline__ void unpack8(const uint4& q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// What else eight consecutive columns of a result row need from memory, so
// that it can be loaded ahead of their sum.
struct Extra {
  uint4 a = {}, b = {};   // forward: bias, residual; dgrad: z, residual; wgrad: the old dw
  template <int kMode>
  __device__ __forceinline__ void load(const LinearParams& p, int64_t row, int col) {
    if constexpr (kMode == kLinearWgrad) {
      const uint4* o = reinterpret_cast<const uint4*>(static_cast<float*>(p.out) + row * p.ldo + col);
      a = o[0], b = o[1];
    } else {
      if constexpr (kMode == kLinearFwd) {
        if (p.bias != nullptr) a = __ldg(reinterpret_cast<const uint4*>(p.bias + col));
      } else {
        if (p.act != kActNone) a = *reinterpret_cast<const uint4*>(p.z + row * p.ldz + col);
      }
      if (p.residual != nullptr) b = *reinterpret_cast<const uint4*>(p.residual + row * p.ldr + col);
    }
  }
};

// Eight consecutive columns of one result row (an absent bias or residual is
// zeros: x + 0 is x).
template <int kMode, int kAct>
__device__ __forceinline__ void finish8(const LinearParams& p, int64_t row, int col, const Extra& extra, float (&v)[8]) {
  float t[8];
  if constexpr (kMode == kLinearWgrad) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * p.ldo + col);
    o[0] = make_float4(__uint_as_float(extra.a.x) + v[0], __uint_as_float(extra.a.y) + v[1],
                       __uint_as_float(extra.a.z) + v[2], __uint_as_float(extra.a.w) + v[3]);
    o[1] = make_float4(__uint_as_float(extra.b.x) + v[4], __uint_as_float(extra.b.y) + v[5],
                       __uint_as_float(extra.b.z) + v[6], __uint_as_float(extra.b.w) + v[7]);
    return;
  }
  unpack8(extra.a, t);
  if constexpr (kMode == kLinearFwd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
    if (p.z != nullptr) *reinterpret_cast<uint4*>(p.z + row * p.ldz + col) = pack8(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_value<kAct>(v[i]);
  } else if constexpr (kAct != kActNone) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = times_grad<kAct>(v[i], t[i]);
  }
  unpack8(extra.b, t);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += t[i];
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row * p.ldo + col) = pack8(v);
}

// 32 x 32 of the result: this lane's row of it in `acc`, rows from row0 and
// columns from col on, those below p.m and `end`.  The warp turns the block
// around in its shared-memory box (4 KB, 128-byte rows, 16-byte chunks XORed
// with the row), so that four lanes finish a row's 32 columns side by side:
// eight rows of 64 contiguous bytes an access instead of 32 rows of 16.
template <int kMode, int kAct>
__device__ __forceinline__ void finish_block(const LinearParams& p, uint8_t* box, int row0, int col, int end,
                                             const uint32_t (&acc)[32]) {
  const int lane = lane_id();
  __syncwarp();                                  // the previous block has been read
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
  __syncwarp();
  const int q = lane & 3, c = col + 8 * q;
  if (c >= end) return;
  float bias[8] = {};
  if (kMode == kLinearFwd && p.bias != nullptr) unpack8(__ldg(reinterpret_cast<const uint4*>(p.bias + c)), bias);
  constexpr int kAhead = 2;                      // rows whose z and residual are loaded together
#pragma unroll 1
  for (int i0 = 0; i0 < 4; i0 += kAhead) {
    uint4 zin[kAhead], res[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t row = row0 + 8 * (i0 + i) + (lane >> 2);
      if (row >= p.m) break;
      if constexpr (kMode == kLinearDgrad && kAct != kActNone)
        zin[i] = *reinterpret_cast<const uint4*>(p.z + row * p.ldz + c);
      if (p.residual != nullptr) res[i] = *reinterpret_cast<const uint4*>(p.residual + row * p.ldr + c);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = 8 * (i0 + i) + (lane >> 2);
      const int64_t row = row0 + r;
      if (row >= p.m) break;
      float v[8], t[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 x = *reinterpret_cast<const float4*>(box + r * 128 + (((2 * q + h) ^ (r & 7)) << 4));
        v[4 * h] = x.x, v[4 * h + 1] = x.y, v[4 * h + 2] = x.z, v[4 * h + 3] = x.w;
      }
      if constexpr (kMode == kLinearFwd) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += bias[k];
        if (p.z != nullptr) *reinterpret_cast<uint4*>(p.z + row * p.ldz + c) = pack8(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = act_value<kAct>(v[k]);
      } else if constexpr (kAct != kActNone) {
        unpack8(zin[i], t);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = times_grad<kAct>(v[k], t[k]);
      }
      if (p.residual != nullptr) {
        unpack8(res[i], t);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += t[k];
      }
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row * p.ldo + c) = pack8(v);
    }
  }
}

// f with the activation as a constant.  Kernels without one (kActs false) do
// not carry the others' code: a short call's time is partly that of fetching
// its instructions.
template <bool kActs, typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if constexpr (!kActs) {
    f(std::integral_constant<int, kActNone>());
  } else {
    switch (act) {
      case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
      case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
      case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
      case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
      default: f(std::integral_constant<int, kActNone>()); break;
    }
  }
}

// v += the eight floats at shared address `at` of every CTA of the cluster, in
// rank order, four CTAs' loads in flight.
__device__ __forceinline__ void add_parts(uint32_t at, int ctas, float (&v)[8]) {
  for (int i0 = 0; i0 < ctas; i0 += 4) {
    float4 x[4] = {}, y[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i0 + i < ctas) {
        const uint32_t from = cluster_map(at, static_cast<uint32_t>(i0 + i));
        x[i] = ld_cluster_v4(from);
        y[i] = ld_cluster_v4(from + 16);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[0] += x[i].x, v[1] += x[i].y, v[2] += x[i].z, v[3] += x[i].w;
      v[4] += y[i].x, v[5] += y[i].y, v[6] += y[i].z, v[7] += y[i].w;
    }
  }
}

__device__ __forceinline__ bool warp_wait(Watchdog& wd, uint64_t* bar, uint32_t parity) {
  const bool ok = wd.wait(bar, parity);
  return __all_sync(0xffffffffu, ok);
}

// Start of K-step ks (16 of the contraction) within an operand tile, in
// 16-byte descriptor units.
template <bool kMn>
__host__ __device__ constexpr uint32_t kstep_off(int ks) {
  return static_cast<uint32_t>((kMn ? ks * 2048 : ks * 32) >> 4);
}

// One operand tile (16 KB): 128 of its M/N index from `mn` on, 64 of the
// contraction from `k` on.  One copy where the tensor map allows: the issuing
// thread's time goes by the copy (halves issued by four lanes side by side
// were slower, 280 against 247 us for 8192 x 4096 x 6144).  An MN-major tile is
// two 64-column blocks; when the row length is a multiple of 64 the map has
// the block as a dimension of its own and one box takes both.
template <bool kMn, bool kPair>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, bool blocked, uint32_t bar, int mn,
                                          int k) {
  if (kMn && blocked) {
    tma_load_3d_at<kPair>(dst, map, bar, 0, k, mn >> 6);
  } else if (kMn) {
    tma_load_2d_at<kPair>(dst, map, bar, mn, k);
    tma_load_2d_at<kPair>(dst + kMnBlockBytes, map, bar, mn + 64, k);
  } else {
    tma_load_2d_at<kPair>(dst, map, bar, k, mn);
  }
}

// Tile t of the result.  Bands of 8 tile rows, rows fastest within a band:
// the tiles in flight form a block of the result, whose operands L2 serves.
// With `quarters`, t counts the 128 x 128 quarters of the 256 x 256 tiles from
// `base` on (the pairs' last tiles, left to split clusters).
struct Tiles {
  int m, n;
  bool quarters;
  int base;
  __device__ __forceinline__ void at(int t, int* tm, int* tn) const {
    if (quarters) {
      whole(base + t / 4, tm, tn);
      *tm = 2 * *tm + (t & 1);
      *tn = 2 * *tn + ((t >> 1) & 1);
    } else {
      whole(t, tm, tn);
    }
  }
  __device__ __forceinline__ void whole(int t, int* tm, int* tn) const {
    const int band = 8 * n;
    const int b = t / band, r = t - b * band;
    const int rows = min(8, m - 8 * b);
    *tm = 8 * b + r % rows;
    *tn = r / rows;
  }
};

template <int kMode, bool kPair, bool kActs>
__global__ void __launch_bounds__(kThreads, 1)
    linear_bf16_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_out, const __grid_constant__ LinearParams p) {
  using S = Shape<kPair>;
  constexpr bool kAMn = kMode == kLinearWgrad;
  constexpr bool kBMn = kMode != kLinearDgrad;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ LinearBarriers bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  Watchdog wd(&abort_flag, p.err, p.wait_cycles);

  const uint32_t rank = cluster_rank();
  const int warp = warp_id();
  const int lane = lane_id();
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kEpiWarps * S::kCtas);
    }
    mbar_init(&bars.mma_final, 1);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
    if (kMode == kLinearWgrad) prefetch_tensormap(&map_out);
  }
  grid_launch_dependents();
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(&tmem_base_sh, S::kTmemCols);
    } else {
      tmem_alloc(&tmem_base_sh, S::kTmemCols);
      tmem_relinquish();
    }
  }
  // barriers and TMEM are ready, for a pair those of both CTAs; the CTAs of a
  // split cluster work by themselves until their parts meet
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_base_sh;
  const int ctas = kPair ? 2 : p.split;
  const bool join = !kPair && ctas > 1;   // parts of a tile's sum meet at the end
  grid_wait();             // operands, outputs and the error word belong to earlier kernels until here

  // ---- this cluster's tiles and this CTA's part of the contraction
  const int tile_n = kPair ? p.tile_n : S::kTN;
  const bool quarters = !kPair && p.tail_base >= 0;
  const int grain_m = quarters ? 256 : S::kTM, grain_n = quarters ? 256 : tile_n;
  const Tiles tiles = {(p.m + grain_m - 1) / grain_m, (p.n + grain_n - 1) / grain_n, quarters, p.tail_base};
  const int all_stages = (p.k + kTK - 1) / kTK;
  const int first_tile = blockIdx.x / ctas;
  const int tile_step = gridDim.x / ctas;
  const int n_tiles = p.tiles;
  // split: parts of the contraction as even as whole stages allow
  const int s_begin = kPair ? 0 : static_cast<int>(static_cast<int64_t>(all_stages) * rank / ctas);
  const int s_end = kPair ? all_stages : static_cast<int>(static_cast<int64_t>(all_stages) * (rank + 1) / ctas);
  const int n_st = s_end - s_begin;
  const int chunk = kMode == kLinearWgrad ? kChunkStages : n_st;   // stages of one result buffer
  int n_issued = 0;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = first_tile; ok && t < n_tiles; t += tile_step) {
        int tm, tn;
        tiles.at(t, &tm, &tn);
        const int m0 = tm * S::kTM + (kPair ? 128 * static_cast<int>(rank) : 0);
        const int n0 = tn * tile_n + (kPair ? tile_n / 2 * static_cast<int>(rank) : 0);
        for (int s = s_begin; s < s_end; ++s, ++it) {
          const int st = it % kStages;
          if (!(ok = wd.wait(&bars.empty[st], ((it / kStages) & 1) ^ 1))) break;
          uint8_t* stage = smem + st * kStageBytes;
          // both CTAs' copies of a pair count on the even CTA's barrier, which
          // its producer arms with the bytes of both
          uint32_t bar = smem_u32(&bars.full[st]);
          if constexpr (kPair) bar = cluster_map(bar, 0);
          if (!kPair || rank == 0)
            mbar_arrive_expect_tx(&bars.full[st], kPair ? 2 * kStageBytes : p.a_bytes + kOperandBytes);
          load_tile<kAMn, kPair>(stage, &map_a, p.a_blocked, bar, m0, s * kTK);
          load_tile<kBMn, kPair>(stage + kOperandBytes, &map_b, p.b_blocked, bar, n0, s * kTK);
          n_issued = it + 1;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && (!kPair || rank == 0)) {
      const uint32_t idesc = make_idesc_bf16(S::kTM, tile_n, kAMn, kBMn);
      const uint64_t a0 = make_desc_sw128(smem_u32(smem), kAMn ? kMnBlockBytes : 16, 1024);
      const uint64_t b0 = make_desc_sw128(smem_u32(smem) + kOperandBytes, kBMn ? kMnBlockBytes : 16, 1024);
      int it = 0, c = 0;       // stages and result buffers issued so far
      bool ok = true;
      for (int t = first_tile; ok && t < n_tiles; t += tile_step) {
        for (int s = 0; ok && s < n_st; ++c) {
          if (!(ok = wd.wait(&bars.acc_empty[c & 1], ((c >> 1) & 1) ^ 1))) break;
          tc_fence_after_sync();
          const uint32_t d = tmem + static_cast<uint32_t>((c & 1) * S::kTN);
          const int s_chunk = min(n_st, s + chunk);
          for (bool first = true; s < s_chunk; ++s, ++it) {
            const int st = it % kStages;
            if (!(ok = wd.wait(&bars.full[st], (it / kStages) & 1))) break;
            tc_fence_after_sync();
            const uint64_t off = static_cast<uint64_t>(st * (kStageBytes >> 4));
#pragma unroll
            for (int ks = 0; ks < kTK / 16; ++ks) {
              const uint64_t a = a0 + off + kstep_off<kAMn>(ks), b = b0 + off + kstep_off<kBMn>(ks);
              const uint32_t add = (first && ks == 0) ? 0u : 1u;
              if constexpr (kPair) umma_bf16_ss_pair(d, a, b, idesc, add);
              else umma_bf16_ss(d, a, b, idesc, add);
            }
            first = false;
            if constexpr (kPair) umma_commit_pair(&bars.empty[st]);
            else umma_commit(&bars.empty[st]);
          }
          if (!ok) break;
          if constexpr (kPair) umma_commit_pair(&bars.acc_full[c & 1]);
          else umma_commit(&bars.acc_full[c & 1]);
        }
      }
      if constexpr (kPair) umma_commit_pair(&bars.mma_final);
      else umma_commit(&bars.mma_final);
      wd.drain(&bars.mma_final, 0, 4000000);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const int warp_cols = tile_n / 2;
    const uint32_t my_cols = tmem + lane_base + static_cast<uint32_t>(half * warp_cols);
    const int tile_row = (kPair ? 128 * static_cast<int>(rank) : 0) + quad * 32 + lane;
    const uint32_t leader_empty[2] = {cluster_map(smem_u32(&bars.acc_empty[0]), kPair ? 0 : rank),
                                      cluster_map(smem_u32(&bars.acc_empty[1]), kPair ? 0 : rank)};
    uint8_t* box = smem + kOffBox + (warp - 2) * kBoxBytes;    // this warp's 4 KB
    // sums of several result buffers or CTAs pass through registers, bf16
    // results of a whole contraction go straight out
    const bool direct = kMode != kLinearWgrad && !join;
    int c = 0;
    // After an earlier error nothing is written, and the CTA gives up.  Asked
    // here, under the first loads: before them it would cost their start 0.5 us.
    bool ok = !error_already_set(p.err);
    if (!ok) *wd.abort_flag = 1;
    for (int t = first_tile; ok && t < n_tiles; t += tile_step) {
      int tm, tn;
      tiles.at(t, &tm, &tn);
      const int64_t row = static_cast<int64_t>(tm) * S::kTM + tile_row;
      const int col = tn * tile_n + half * warp_cols;
      if (!direct) {
        float acc[S::kColsPerWarp];
        for (int s = 0; ok && s < n_st; s += chunk, ++c) {
          if (!(ok = warp_wait(wd, &bars.acc_full[c & 1], (c >> 1) & 1))) break;
          tc_fence_after_sync();
#pragma unroll
          for (int c0 = 0; c0 < S::kColsPerWarp; c0 += 32) {
            uint32_t r[32];
            tmem_ld32(my_cols + static_cast<uint32_t>((c & 1) * S::kTN + c0), r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              acc[c0 + j] = s == 0 ? __uint_as_float(r[j]) : acc[c0 + j] + __uint_as_float(r[j]);
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(leader_empty[c & 1]);
        }
        if (!ok) break;
        if (!join) {
          // dw += the tile, 32 x 32 at a time through this warp's box: TMA adds
          // it in L2 (float32, one addition an element), clipped at dw's edges
          const int row0 = static_cast<int>(row) - lane;
#pragma unroll
          for (int c0 = 0; c0 < S::kColsPerWarp; c0 += 32) {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                  make_float4(acc[c0 + 4 * j], acc[c0 + 4 * j + 1], acc[c0 + 4 * j + 2], acc[c0 + 4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && row0 < p.m && col + c0 < p.n) {
              tma_reduce_add_2d(&map_out, box, col + c0, row0);
              bulk_commit_group();
            }
          }
        } else if (row < p.m) {
          // this CTA's part of the sum, into its own ring (idle: every stage
          // it issued has been consumed)
          float* part = reinterpret_cast<float*>(smem) + tile_row * kPartStride + half * S::kColsPerWarp;
#pragma unroll
          for (int j = 0; j < S::kColsPerWarp; j += 4)
            *reinterpret_cast<float4*>(part + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        }
      } else {
        if (!(ok = warp_wait(wd, &bars.acc_full[c & 1], (c >> 1) & 1))) break;
        tc_fence_after_sync();
        with_act<kActs>(p.act, [&](auto act) {
#pragma unroll 1
          for (int c0 = 0; c0 < warp_cols; c0 += 32) {
            uint32_t r[32];
            tmem_ld32(my_cols + static_cast<uint32_t>((c & 1) * S::kTN + c0), r);
            tmem_ld_wait();
            finish_block<kMode, decltype(act)::value>(p, box, static_cast<int>(row) - lane, col + c0,
                                                      min(p.n, col + warp_cols), r);
          }
        });
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(leader_empty[c & 1]);
        ++c;
      }
    }
    if (kMode == kLinearWgrad && lane == 0) bulk_wait_group<0>();   // every addition has been made
  }

  tc_fence_before_sync();
  __syncthreads();
  if (wd.aborted()) {
    // a wait ran out: let the copies already in flight land first.  The odd
    // CTA of a pair has them counted on the even one's barrier, whose phases
    // it cannot rely on now: it gives them 100 us instead.
    if (kPair && rank != 0) {
      const long long t0 = clock64();
      while (warp == 0 && lane == 0 && n_issued > 0 && clock64() - t0 < 200000) {
      }
    } else if (warp == 0 && lane == 0) {
      for (int st = 0; st < kStages && st < n_issued; ++st) {
        const int last = st + kStages * ((n_issued - 1 - st) / kStages);
        wd.drain(&bars.full[st], (last / kStages) & 1, 1000000);
      }
    }
    __syncthreads();
  }
  if constexpr (!kPair)
    if (warp == 1) {
      tc_fence_after_sync();
      tmem_dealloc(tmem, S::kTmemCols);
    }
  // ---- the split's join: units of eight columns of a row, dealt over the
  // cluster's threads.  What a thread's first unit needs from memory is loaded
  // while the other CTAs' parts are waited for.
  int join_row = 0, join_col = 0, groups = 1, units = 0, unit = 0;
  Extra extra;
  if (join) {
    int tm, tn;
    tiles.at(first_tile, &tm, &tn);
    join_row = 128 * tm, join_col = 128 * tn;
    groups = max(1, min(128, p.n - join_col) / 8);
    units = max(0, min(128, p.m - join_row)) * max(0, min(128, p.n - join_col) / 8);   // (a quarter may lie past the edge)
    unit = static_cast<int>(rank) * kThreads + threadIdx.x;
    if (unit < units) extra.load<kMode>(p, join_row + unit / groups, join_col + 8 * (unit % groups));
  }
  // nothing of this cluster touches another CTA's shared memory or TMEM from
  // here, but the split's reads of the partial tiles below
  if (ctas > 1) cluster_sync();
  if (join) {
    // an aborted CTA's part is missing: every CTA then leaves its share out
    uint32_t lost = 0;
#pragma unroll
    for (int i = 0; i < kMaxSplit; ++i)
      if (i < ctas) lost |= ld_cluster_u32(cluster_map(smem_u32(const_cast<int*>(&abort_flag)), i));
    with_act<kActs>(p.act, [&](auto act) {
      for (; unit < units; unit += ctas * kThreads) {
        const int r = unit / groups, g = unit - r * groups;
        float v[8] = {};
        add_parts(smem_u32(smem) + static_cast<uint32_t>((r * kPartStride + 8 * g) * 4), ctas, v);
        if (lost != 0u) break;
        finish8<kMode, decltype(act)::value>(p, join_row + r, join_col + 8 * g, extra, v);
        const int next = unit + ctas * kThreads;
        if (next < units) extra.load<kMode>(p, join_row + next / groups, join_col + 8 * (next % groups));
      }
    });
    cluster_sync();        // the parts have been read
  }
  if constexpr (kPair)
    if (warp == 1) {
      tc_fence_after_sync();
      tmem_dealloc_pair(tmem, S::kTmemCols);
    }
}

// How many clusters of each size a kernel's launch has on the device at once,
// looked up once per device and kernel.  The SMs of a group that a whole
// cluster does not fill stay out (48 clusters of 3 CTAs do not fit on 152 SMs at
// one CTA per SM), and a grid that passes the number by one takes twice as long.
constexpr int kMaxDevices = 64;
struct Residency {
  std::atomic<int> ready{0};
  std::atomic<int> fit[kMaxSplit + 1] = {};
  int operator[](int c) const { return fit[c].load(std::memory_order_relaxed); }
};

template <typename... Params>
cudaError_t look_up(void (*kernel)(Params...), unsigned threads, size_t smem, Residency (&table)[kMaxDevices],
                    const Residency** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  Residency& r = table[dev];
  *out = &r;
  if (r.ready.load(std::memory_order_acquire)) return cudaSuccess;
  if (smem > 0 && (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(smem))) != cudaSuccess)
    return e;
  for (int c = 1; c <= kMaxSplit; ++c) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(c) * 256u);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(c);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
    r.fit[c].store(n, std::memory_order_relaxed);
  }
  r.ready.store(1, std::memory_order_release);
  return cudaSuccess;
}

// The largest cluster, up to `most`, with which `count` clusters run at once (1 if none).
int widest_cluster(const Residency& r, int count, int64_t most) {
  int c = most < kMaxSplit ? static_cast<int>(most) : kMaxSplit;
  while (c > 1 && r[c] < count) --c;
  return c < 1 ? 1 : c;
}

// Chooses the shape for p.m x p.n with contraction p.k: the one, and the tile
// width or split, whose waves of tiles take the least time in the cost model;
// or pairs for the whole waves and split clusters for the quarters of the
// tiles that are left (501 x 4104 x 10248: 82 tiles on 76 pairs).
template <int kMode, bool kActs>
cudaError_t plan_mode(LinearParams& p) {
  static Residency pair_table[kMaxDevices], split_table[kMaxDevices];
  const Residency *pair_fit = nullptr, *split_fit = nullptr;
  cudaError_t e = look_up(linear_bf16_kernel<kMode, true, kActs>, kThreads, kSmemAlloc, pair_table, &pair_fit);
  if (e != cudaSuccess) return e;
  if ((e = look_up(linear_bf16_kernel<kMode, false, kActs>, kThreads, kSmemAlloc, split_table, &split_fit)) != cudaSuccess)
    return e;
  const int pairs = (*pair_fit)[2];
  if (pairs < 1 || (*split_fit)[1] < 1) return cudaErrorLaunchOutOfResources;
  const int64_t stages = (static_cast<int64_t>(p.k) + kTK - 1) / kTK;
  p.a_bytes = kMode == kLinearWgrad ? kOperandBytes : static_cast<uint32_t>(linear_a_rows(p.m) * kTK * 2);
  const int64_t rows = p.m < 128 ? p.m : 128;      // of a small tile
  const int64_t first_join = kSplitFirstJoinCost + kSplitFirstJoinRowCost * rows;
  const int64_t further_join = kSplitJoinCost + kSplitJoinRowCost * rows;
  // least time of `count` small tiles, and its split
  auto split_cost = [&](int64_t count, int* split) {
    int64_t least = INT64_MAX;
    for (int c = 1; c <= kMaxSplit && c <= stages; ++c) {
      const int fit = (*split_fit)[c];
      if (fit < 1 || count > INT32_MAX / kMaxSplit) continue;
      const int64_t cost = ((count + fit - 1) / fit) * ((stages + c - 1) / c * kSplitStageCost + kSplitFixedCost) +
                           (c > 1 ? first_join + (c - 2) * further_join : 0);
      if (cost < least) {
        least = cost;
        *split = c;
      }
    }
    return least;
  };
  int split = 1;
  const int64_t small = static_cast<int64_t>((p.m + 127) / 128) * ((p.n + 127) / 128);
  int64_t best = split_cost(small, &split);
  p.pair_tiles = 0;
  p.split = split;
  p.split_tiles = static_cast<int>(small < INT32_MAX ? small : INT32_MAX);
  p.tile_n = 256;
  // a pair copies whole tiles of A, so a result of fewer rows is left to the split shape
  if (p.a_bytes != kOperandBytes) return cudaSuccess;
  // widths: wgrad's epilogue adds 32-column boxes of a half; a forward whose
  // W comes in whole blocks (see load_tile) would lose that with halves that
  // are not (2048 x 4096 x 4096 with 240 columns: 62 us, 50 with 256)
  const int step = kMode == kLinearDgrad || (kMode == kLinearFwd && p.n % 64 != 0) ? 16 : 128;
  for (int tn = 256; tn >= (kMode == kLinearWgrad ? 256 : 128); tn -= step) {
    const int64_t tiles = static_cast<int64_t>((p.m + 255) / 256) * ((p.n + tn - 1) / tn);
    const int64_t wave = stages * (kPairStageCost + kPairColumnCost * (tn - 128) / 128);
    int64_t cost = (tiles + pairs - 1) / pairs * wave + kPairFixedCost;
    if (cost < best) {
      best = cost;
      p.pair_tiles = static_cast<int>(tiles);
      p.tile_n = tn;
      p.split_tiles = 0;
    }
    const int64_t rest = tiles % pairs;
    if (tn == 256 && tiles > pairs && rest > 0) {
      cost = tiles / pairs * wave + kPairFixedCost + split_cost(4 * rest, &split) + kSecondLaunchCost;
      if (cost < best) {
        best = cost;
        p.pair_tiles = static_cast<int>(tiles - rest);
        p.tile_n = tn;
        p.split_tiles = static_cast<int>(4 * rest);
        p.split = split;
      }
    }
  }
  p.pairs = pairs;
  return cudaSuccess;
}

template <int kMode, bool kActs>
cudaError_t launch_mode(const LinearMaps& maps, LinearParams p, cudaStream_t s) {
  if (p.pair_tiles > 0) {
    p.tiles = p.pair_tiles;
    const unsigned clusters = static_cast<unsigned>(p.tiles < p.pairs ? p.tiles : p.pairs);
    const cudaError_t e = launch_overlapped(linear_bf16_kernel<kMode, true, kActs>, 2u * clusters, kThreads, kSmemAlloc, 2, s,
                                            maps.a, maps.b, maps.out, p);
    if (e != cudaSuccess || p.split_tiles == 0) return e;
  }
  p.tail_base = p.pair_tiles > 0 ? p.pair_tiles : -1;
  p.tiles = p.split_tiles;
  return launch_overlapped(linear_bf16_kernel<kMode, false, kActs>, static_cast<unsigned>(p.tiles) * p.split, kThreads,
                           kSmemAlloc, static_cast<unsigned>(p.split), s, maps.a, maps.b, maps.out, p);
}

// ---------------------------------------------------------------------------
// forward of a few rows (a token, or one of each of a few sequences)
//
// Bound by reading W once.  Tensor-core tiles would multiply mostly zeros, and
// their pipeline's start costs more than these products: here a warp reads 16
// bytes a lane, 512 bytes of W in rows of kCols columns, straight into float32
// FMAs for all R rows of x.  A block of 8 warps and a cluster of up to 8
// blocks split the contraction of one strip of kCols columns; partial sums
// meet in shared and distributed shared memory and are added in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kGvThreads = 256;
constexpr int kGvSlab = 1024;       // rows of W per x slab in shared memory
constexpr int kGvLoads = 8;         // loads in flight per lane

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int R, int kCols>
__global__ void __launch_bounds__(kGvThreads)
    linear_gemv_kernel(const __grid_constant__ LinearParams p, const __nv_bfloat16* __restrict__ x, int64_t ldx,
                       const __nv_bfloat16* __restrict__ w) {
  __shared__ __align__(16) float xs[kGvSlab][R];
  __shared__ __align__(16) float part[kGvThreads / 32][R][kCols];
  constexpr int kLanes = kCols / 8, kRows = 32 / kLanes;    // lanes across a strip, rows of W a warp reads at once
  const int lane = lane_id(), warp = warp_id();
  const int cs = p.split, rank = static_cast<int>(cluster_rank());
  const int strip = blockIdx.x / cs;
  const int col = strip * kCols + 8 * (lane % kLanes);
  const bool in = col < p.n;
  const int sub = lane / kLanes;          // which of the warp's rows of W
  // this block's contraction rows
  const int k0 = static_cast<int>(static_cast<int64_t>(p.k) * rank / cs);
  const int k1 = static_cast<int>(static_cast<int64_t>(p.k) * (rank + 1) / cs);
  uint64_t acc[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[r][i] = 0ull;
  grid_launch_dependents();
  grid_wait();
  for (int s0 = k0; s0 < k1; s0 += kGvSlab) {
    const int len = min(kGvSlab, k1 - s0);
    // the slab's W rows of this lane: every kStep-th
    uint4 q[kGvLoads];
    const __nv_bfloat16* wp = w + static_cast<int64_t>(s0 + kRows * warp + sub) * p.n + col;
    constexpr int kStep = kRows * (kGvThreads / 32);
    int k = kRows * warp + sub;
#pragma unroll
    for (int j = 0; j < kGvLoads; ++j)
      q[j] = in && k + j * kStep < len ? ld_stream(wp + static_cast<int64_t>(j) * kStep * p.n) : make_uint4(0, 0, 0, 0);
    __syncthreads();                       // the previous slab of x has been used
    for (int i = threadIdx.x; i < len * R; i += kGvThreads) {
      const int r = i / len, kk = i - r * len;
      xs[kk][r] = r < p.m ? __bfloat162float(x[r * ldx + s0 + kk]) : 0.f;
    }
    __syncthreads();
    while (k < len) {
      const __nv_bfloat16* next = wp + static_cast<int64_t>(kGvLoads) * kStep * p.n;
#pragma unroll
      for (int j = 0; j < kGvLoads; ++j) {
        const int kk = k + j * kStep;
        const uint4 v = q[j];
        // the load that takes this one's place, one round ahead
        q[j] = in && kk + kGvLoads * kStep < len ? ld_stream(next + static_cast<int64_t>(j) * kStep * p.n)
                                                 : make_uint4(0, 0, 0, 0);
        if (kk < len) {
          const uint32_t word[4] = {v.x, v.y, v.z, v.w};
          uint64_t f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[i] = f2_pack(__uint_as_float(word[i] << 16), __uint_as_float(word[i] & 0xffff0000u));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float xv = xs[kk][r];
            const uint64_t x2 = f2_pack(xv, xv);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][i] = f2_fma(f[i], x2, acc[r][i]);
          }
        }
      }
      k += kGvLoads * kStep;
      wp = next;
    }
  }
  // ---- sums of the warp's rows, of the block's warps, of the cluster
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(acc[r][i], v[2 * i], v[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (sub == 0) {
      float4* o = reinterpret_cast<float4*>(&part[warp][r][8 * lane]);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < R * kCols; i += kGvThreads) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < kGvThreads / 32; ++g) t += part[g][i / kCols][i % kCols];
    part[0][i / kCols][i % kCols] = t;
  }
  // 8-column groups of the R rows, the first threads of the cluster's first block
  static_assert(R * (kCols / 8) <= kGvThreads, "a group a thread");
  const int out_row = threadIdx.x / (kCols / 8), out_col = strip * kCols + 8 * (threadIdx.x % (kCols / 8));
  const bool writes = rank == 0 && out_row < R && out_row < p.m && out_col < p.n;
  Extra extra;
  if (writes) extra.load<kLinearFwd>(p, out_row, out_col);
  cluster_sync();
  if (writes)
    with_act<true>(p.act, [&](auto act) {
      float v[8] = {};
      add_parts(smem_u32(&part[0][out_row][out_col - strip * kCols]), cs, v);
      finish8<kLinearFwd, decltype(act)::value>(p, out_row, out_col, extra, v);
    });
  cluster_sync();                          // the other blocks have read this one's part
}

template <int R, int kCols>
cudaError_t gemv_strips(LinearParams p, const void* x, int64_t ldx, const void* w, cudaStream_t s) {
  static Residency table[kMaxDevices];
  const Residency* fit = nullptr;
  const cudaError_t e = look_up(linear_gemv_kernel<R, kCols>, kGvThreads, 0, table, &fit);
  if (e != cudaSuccess) return e;
  const int strips = (p.n + kCols - 1) / kCols;
  p.split = widest_cluster(*fit, strips, p.k / 64);      // each block at least 64 rows of W
  return launch_overlapped(linear_gemv_kernel<R, kCols>, static_cast<unsigned>(strips) * p.split, kGvThreads, 0,
                           static_cast<unsigned>(p.split), s, p, static_cast<const __nv_bfloat16*>(x), ldx,
                           static_cast<const __nv_bfloat16*>(w));
}

// Wide strips read 256 consecutive bytes of W a row; a result of few columns
// takes narrow ones (64 bytes), so that 8 blocks a strip still fill the SMs.
template <int R>
cudaError_t gemv_rows(const LinearParams& p, const void* x, int64_t ldx, const void* w, cudaStream_t s) {
  return p.n >= 2048 ? gemv_strips<R, 128>(p, x, ldx, w, s) : gemv_strips<R, 32>(p, x, ldx, w, s);
}

// ---------------------------------------------------------------------------
// column sums of a bf16 matrix, dbias[j] += sum_r g[r, j], in a fixed order
//
// Bound by reading g once.  A warp reads two rows of a strip of 128 columns, 16
// bytes a lane; a block of 8 warps, and a cluster of up to 8 blocks when there
// are rows for them, share the strip's rows.  A lane keeps four sums per column;
// they, the warps and the blocks are added as trees.  Three blocks an SM, so
// that the clusters all run at once: with 100 registers a thread 46 clusters
// of 6 fit where 8192 x 6144 needs 48, and the call took 55 us.
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 256;
constexpr int kSumCols = 128;
constexpr int kSumLoads = 8;        // loads in flight per lane
constexpr int kSumAccs = 4;         // sums per lane and column
constexpr int kSumSplit = kMaxSplit;

__global__ void __launch_bounds__(kSumThreads, 3)
    colsum_bf16_kernel(const __nv_bfloat16* __restrict__ g, int64_t ldg, int rows, int n, int split,
                       float* __restrict__ dbias) {
  __shared__ __align__(16) float part[kSumThreads / 32][kSumCols];
  const int lane = lane_id(), warp = warp_id(), sub = lane >> 4;
  const int rank = static_cast<int>(cluster_rank());
  const int strip = blockIdx.x / split;
  const int col = strip * kSumCols + 8 * (lane & 15);
  const int r0 = static_cast<int>(static_cast<int64_t>(rows) * rank / split);
  const int r1 = static_cast<int>(static_cast<int64_t>(rows) * (rank + 1) / split);
  grid_launch_dependents();
  grid_wait();
  uint64_t acc[kSumAccs][4] = {};
  constexpr int kStep = 2 * (kSumThreads / 32);
  if (col < n) {
    for (int64_t r = r0 + 2 * warp + sub; r < r1; r += kSumLoads * kStep) {
      uint4 q[kSumLoads];
#pragma unroll
      for (int j = 0; j < kSumLoads; ++j)
        q[j] = r + j * kStep < r1 ? ld_stream(g + (r + j * kStep) * ldg + col) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kSumLoads; ++j) {
        const uint32_t word[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[j % kSumAccs][i] = f2_add(acc[j % kSumAccs][i],
                                       f2_pack(__uint_as_float(word[i] << 16), __uint_as_float(word[i] & 0xffff0000u)));
      }
    }
  }
#pragma unroll
  for (int half = kSumAccs / 2; half > 0; half >>= 1)
#pragma unroll
    for (int j = 0; j < half; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = f2_add(acc[j][i], acc[j + half][i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f2_unpack(acc[0][i], a, b);
    a += __shfl_xor_sync(0xffffffffu, a, 16);
    b += __shfl_xor_sync(0xffffffffu, b, 16);
    if (sub == 0) {
      part[warp][8 * lane + 2 * i] = a;
      part[warp][8 * lane + 2 * i + 1] = b;
    }
  }
  for (int half = kSumThreads / 64; half > 0; half >>= 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < half * kSumCols; i += kSumThreads)
      part[i / kSumCols][i % kSumCols] += part[i / kSumCols + half][i % kSumCols];
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x < kSumCols && strip * kSumCols + static_cast<int>(threadIdx.x) < n) {
    float v[kSumSplit];
    const uint32_t at = smem_u32(&part[0][threadIdx.x]);
#pragma unroll
    for (int i = 0; i < kSumSplit; ++i) v[i] = i < split ? __uint_as_float(ld_cluster_u32(cluster_map(at, i))) : 0.f;
#pragma unroll
    for (int half = kSumSplit / 2; half > 0; half >>= 1)
#pragma unroll
      for (int i = 0; i < half; ++i) v[i] += v[i + half];
    dbias[strip * kSumCols + threadIdx.x] += v[0];
  }
  cluster_sync();                          // the other blocks' sums have been read
}

}  // namespace

// f with the mode and whether there is an activation as constants.
template <typename F>
static cudaError_t with_mode(int mode, int act, F&& f) {
  if (mode == kLinearWgrad) return f(std::integral_constant<int, kLinearWgrad>(), std::false_type());
  if (mode == kLinearFwd)
    return act == kActNone ? f(std::integral_constant<int, kLinearFwd>(), std::false_type())
                           : f(std::integral_constant<int, kLinearFwd>(), std::true_type());
  return act == kActNone ? f(std::integral_constant<int, kLinearDgrad>(), std::false_type())
                         : f(std::integral_constant<int, kLinearDgrad>(), std::true_type());
}

cudaError_t plan_linear_bf16(int mode, LinearParams& p) {
  return with_mode(mode, p.act, [&](auto m, auto acts) { return plan_mode<decltype(m)::value, decltype(acts)::value>(p); });
}

cudaError_t launch_linear_bf16(int mode, const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  return with_mode(mode, p.act, [&](auto m, auto acts) {
    return launch_mode<decltype(m)::value, decltype(acts)::value>(maps, p, s);
  });
}

cudaError_t launch_linear_gemv(const LinearParams& p, const void* x, int64_t ldx, const void* w, cudaStream_t s) {
  return p.m <= 1 ? gemv_rows<1>(p, x, ldx, w, s) : gemv_rows<2>(p, x, ldx, w, s);
}

cudaError_t launch_colsum_bf16(const void* g, int64_t ldg, int rows, int n, float* dbias, cudaStream_t s) {
  static Residency table[kMaxDevices];
  const Residency* fit = nullptr;
  const cudaError_t e = look_up(colsum_bf16_kernel, kSumThreads, 0, table, &fit);
  if (e != cudaSuccess) return e;
  const int strips = (n + kSumCols - 1) / kSumCols;
  const int split = widest_cluster(*fit, strips, rows / (kSumLoads * 16));     // rows for every load of a block
  return launch_overlapped(colsum_bf16_kernel, static_cast<unsigned>(strips * split),
                           kSumThreads, 0, static_cast<unsigned>(split), s, static_cast<const __nv_bfloat16*>(g), ldg,
                           rows, n, split, dbias);
}

}  // namespace seqattn
