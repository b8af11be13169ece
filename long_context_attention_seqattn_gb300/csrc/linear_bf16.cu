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
// One CTA owns a 128 x 128 tile of the result and streams the contraction in
// stages of 64 through a shared-memory ring:
//   warp 0      TMA producer (A and B tile of a stage, 16 KB each)
//   warp 1      TMEM owner + MMA issuer (4 MMAs M128 N128 K16 per stage)
//   warps 2..5  epilogue, one TMEM lane quadrant each: a thread owns one row
#include <cuda_bf16.h>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace seqattn {
namespace {

constexpr int kTM = 128;                       // result rows per CTA
constexpr int kTN = 128;                       // result columns per CTA
constexpr int kTK = kLinearStageK;             // contraction per stage
constexpr int kStages = 6;
constexpr int kOperandBytes = kTM * kTK * 2;   // 16 KB, either operand
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kMnBlockBytes = kTK * 128;       // one 64-column block of an MN-major tile
constexpr int kThreads = 192;
constexpr int kSmemAlloc = kStages * kStageBytes + 1024;
constexpr uint32_t kTmemCols = 128;

struct LinearBarriers {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full;
  uint64_t mma_final;
};

// ---- activations (z in float32) -------------------------------------------
__device__ __forceinline__ float sigmoidf(float z) { return 1.f / (1.f + __expf(-z)); }
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
template <int kAct>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (kAct != kActNone && kAct != kActRelu)
    if (fabsf(z) > 128.f) return z > 0.f ? 1.f : 0.f;
  if constexpr (kAct == kActRelu) return z > 0.f ? 1.f : 0.f;
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
  return 1.f;
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

// Eight consecutive columns of one result row, forward or dgrad.
template <int kMode, int kAct>
__device__ __forceinline__ void finish8(const LinearParams& p, int64_t row, int col, float (&v)[8]) {
  float t[8];
  if constexpr (kMode == kLinearFwd) {
    if (p.bias != nullptr) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(p.bias + col)), t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
    if (p.z != nullptr) *reinterpret_cast<uint4*>(p.z + row * p.ldz + col) = pack8(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_value<kAct>(v[i]);
  } else if constexpr (kAct != kActNone) {
    unpack8(*reinterpret_cast<const uint4*>(p.z + row * p.ldz + col), t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= act_grad<kAct>(t[i]);
  }
  if (p.residual != nullptr) {
    unpack8(*reinterpret_cast<const uint4*>(p.residual + row * p.ldr + col), t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
  }
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row * p.ldo + col) = pack8(v);
}

template <int kMode, int kAct>
__device__ __forceinline__ void finish32(const LinearParams& p, int64_t row, int col, const uint32_t (&r)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    if (col + j >= p.n) break;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[j + i]);
    finish8<kMode, kAct>(p, row, col + j, v);
  }
}

__device__ __forceinline__ bool warp_wait(Watchdog& wd, uint64_t* bar, uint32_t parity) {
  const bool ok = wd.wait_sleep(bar, parity);
  return __all_sync(0xffffffffu, ok);
}

// Start of K-step ks (16 of the contraction) within an operand tile, in
// 16-byte descriptor units.
template <bool kMn>
__host__ __device__ constexpr uint32_t kstep_off(int ks) {
  return static_cast<uint32_t>((kMn ? ks * 2048 : ks * 32) >> 4);
}

// One operand tile: 128 of its M/N index at `mn`, 64 of the contraction at `k`.
template <bool kMn>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int mn, int k) {
  if constexpr (kMn) {
    tma_load_2d(dst, map, bar, mn, k);
    tma_load_2d(dst + kMnBlockBytes, map, bar, mn + 64, k);
  } else {
    tma_load_2d(dst, map, bar, k, mn);
  }
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    linear_bf16_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ LinearParams p) {
  constexpr bool kAMn = kMode == kLinearWgrad;
  constexpr bool kBMn = kMode != kLinearDgrad;
  if (error_already_set(p.err)) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ LinearBarriers bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  Watchdog wd(&abort_flag, p.err, p.wait_cycles);

  const int m_tiles = (p.m + kTM - 1) / kTM;
  const int m0 = (blockIdx.x % m_tiles) * kTM;
  const int n0 = (blockIdx.x / m_tiles) * kTN;
  const int n_st = (p.k + kTK - 1) / kTK;

  const int warp = warp_id();
  const int lane = lane_id();
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    mbar_init(&bars.acc_full, 1);
    mbar_init(&bars.mma_final, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_base_sh;
  int n_issued = 0;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_tensormap(&map_a);
      prefetch_tensormap(&map_b);
      for (int s = 0; s < n_st; ++s) {
        const int st = s % kStages;
        if (!wd.wait_sleep(&bars.empty[st], ((s / kStages) & 1) ^ 1)) break;
        uint8_t* stage = smem + st * kStageBytes;
        mbar_arrive_expect_tx(&bars.full[st], kStageBytes);
        load_tile<kAMn>(stage, &map_a, &bars.full[st], m0, s * kTK);
        load_tile<kBMn>(stage + kOperandBytes, &map_b, &bars.full[st], n0, s * kTK);
        n_issued = s + 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_bf16(kTM, kTN, kAMn, kBMn);
      const uint64_t a0 = make_desc_sw128(smem_u32(smem), kAMn ? kMnBlockBytes : 16, 1024);
      const uint64_t b0 = make_desc_sw128(smem_u32(smem) + kOperandBytes, kBMn ? kMnBlockBytes : 16, 1024);
      bool ok = true;
      for (int s = 0; s < n_st; ++s) {
        const int st = s % kStages;
        if (!(ok = wd.wait_sleep(&bars.full[st], (s / kStages) & 1))) break;
        tc_fence_after_sync();
        const uint64_t off = static_cast<uint64_t>(st * (kStageBytes >> 4));
#pragma unroll
        for (int ks = 0; ks < kTK / 16; ++ks)
          umma_bf16_ss(tmem, a0 + off + kstep_off<kAMn>(ks), b0 + off + kstep_off<kBMn>(ks), idesc,
                       (s > 0 || ks > 0) ? 1u : 0u);
        umma_commit(&bars.empty[st]);
      }
      if (ok) umma_commit(&bars.acc_full);
      umma_commit(&bars.mma_final);
      wd.drain(&bars.mma_final, 0, 4000000);
    }
  } else {
    const int quad = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const int64_t row = m0 + quad * 32 + lane;
    if (warp_wait(wd, &bars.acc_full, 0)) {
      tc_fence_after_sync();
#pragma unroll 1
      for (int c0 = 0; c0 < kTN && n0 + c0 < p.n; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + lane_base + c0, r);
        tmem_ld_wait();
        if (row >= p.m) continue;
        if constexpr (kMode == kLinearWgrad) {
          float* o = static_cast<float*>(p.out) + row * p.ldo + n0 + c0;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            if (n0 + c0 + j >= p.n) break;
            float4 v = *reinterpret_cast<float4*>(o + j);
            v.x += __uint_as_float(r[j]);
            v.y += __uint_as_float(r[j + 1]);
            v.z += __uint_as_float(r[j + 2]);
            v.w += __uint_as_float(r[j + 3]);
            *reinterpret_cast<float4*>(o + j) = v;
          }
        } else {
          switch (p.act) {
            case kActRelu: finish32<kMode, kActRelu>(p, row, n0 + c0, r); break;
            case kActSilu: finish32<kMode, kActSilu>(p, row, n0 + c0, r); break;
            case kActGelu: finish32<kMode, kActGelu>(p, row, n0 + c0, r); break;
            case kActGeluTanh: finish32<kMode, kActGeluTanh>(p, row, n0 + c0, r); break;
            default: finish32<kMode, kActNone>(p, row, n0 + c0, r); break;
          }
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (wd.aborted()) {
    // a wait ran out: let the copies already in flight land first
    if (warp == 0 && lane == 0) {
      for (int st = 0; st < kStages && st < n_issued; ++st) {
        const int last = st + kStages * ((n_issued - 1 - st) / kStages);
        wd.drain(&bars.full[st], (last / kStages) & 1, 1000000);
      }
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int kMode>
cudaError_t launch_mode(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(linear_bf16_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemAlloc);
  if (e != cudaSuccess) return e;
  const int64_t grid = static_cast<int64_t>((p.m + kTM - 1) / kTM) * ((p.n + kTN - 1) / kTN);
  linear_bf16_kernel<kMode><<<static_cast<unsigned>(grid), kThreads, kSmemAlloc, s>>>(maps.a, maps.b, p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// column sums of a bf16 matrix, dbias[j] += sum_r g[r, j], in a fixed order:
// one block owns 32 columns and every row; thread (y, x) sums rows y, y + 64,
// ... of eight columns, then the block adds its 64 partial rows in a tree.
// ---------------------------------------------------------------------------
constexpr int kSumCols = 32;
constexpr int kSumRows = 128;

__global__ void __launch_bounds__(kSumRows * kSumCols / 8)
    colsum_bf16_kernel(const __nv_bfloat16* __restrict__ g, int64_t ldg, int rows, int n, float* __restrict__ dbias) {
  __shared__ float part[kSumRows][kSumCols + 1];
  const int x = threadIdx.x % (kSumCols / 8), y = threadIdx.x / (kSumCols / 8);
  const int col = blockIdx.x * kSumCols + 8 * x;
  float acc[8] = {};
  if (col < n) {
#pragma unroll 4
    for (int64_t r = y; r < rows; r += kSumRows) {
      float v[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(g + r * ldg + col)), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[y][8 * x + i] = acc[i];
  for (int half = kSumRows / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (y < half)
#pragma unroll
      for (int i = 0; i < 8; ++i) part[y][8 * x + i] += part[y + half][8 * x + i];
  }
  if (y == 0 && col < n)
#pragma unroll
    for (int i = 0; i < 8; ++i) dbias[col + i] += part[0][8 * x + i];
}

}  // namespace

cudaError_t launch_linear_bf16(int mode, const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  switch (mode) {
    case kLinearFwd: return launch_mode<kLinearFwd>(maps, p, s);
    case kLinearDgrad: return launch_mode<kLinearDgrad>(maps, p, s);
    default: return launch_mode<kLinearWgrad>(maps, p, s);
  }
}

cudaError_t launch_colsum_bf16(const void* g, int64_t ldg, int rows, int n, float* dbias, cudaStream_t s) {
  colsum_bf16_kernel<<<(n + kSumCols - 1) / kSumCols, kSumRows * kSumCols / 8, 0, s>>>(
      static_cast<const __nv_bfloat16*>(g), ldg, rows, n, dbias);
  return cudaGetLastError();
}

}  // namespace seqattn
